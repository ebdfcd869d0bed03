"""Measured cases of the operators around the 8-bit key/value cache.

Four operators that run next to the attention of this library in a serving loop:

* ``rope``    rotary positions applied to q and k (half or interleaved pairs, part of
              the head, frequencies scaled for long contexts), or their transpose, which
              is the gradient;
* ``append``  new keys and values quantised into a cache of 8-bit codes with one fp32
              scale per block of tokens and head; the touched blocks are read back;
* ``decode``  split-KV attention over that cache with a log2 LSE per row, adding each
              key's attention weight to a running sum;
* ``evict``   the cache cut down to a budget: the first tokens, the last ones, and the
              heaviest of the rest, compacted in order.

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits
(angles in 64); with ``own`` true it calls the library.  ``exact`` restates each in 64
bits.
"""
import math

import numpy as np
import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
TINY = 2.0 ** -126  # a block's scale below this is stored as 0
LOG2E = 1.4426950408889634


# ---------------------------------------------------------------- cases

def rope(name=None, B=1, S=1, Hq=32, Hkv=8, D=128, R=128, layout="HND", pairs="half", scaling="none", factor=1.0,
         far=0, inverse=False, dtype="bf16"):
    c = {"op": "rope", "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R, "layout": layout, "pairs": pairs,
         "scaling": scaling, "factor": factor, "far": far, "inverse": inverse, "dtype": dtype}
    return dict(c, name=name) if name else c


def append(name=None, B=1, S=1, Hkv=8, D=128, capacity=4096, filled=0, ragged=False, layout="HND", block=64,
           codes="int8", dtype="bf16"):
    c = {"op": "append", "B": B, "S": S, "Hkv": Hkv, "D": D, "capacity": capacity, "filled": filled,
         "ragged": ragged, "layout": layout, "block": block, "codes": codes, "dtype": dtype}
    return dict(c, name=name) if name else c


def decode(name=None, B=1, Lq=1, Hq=32, Hkv=8, D=128, capacity=4096, ragged=False, causal=False, weights=False,
           block=64, codes="int8", dtype="bf16"):
    c = {"op": "decode", "B": B, "Lq": Lq, "Hq": Hq, "Hkv": Hkv, "D": D, "capacity": capacity, "ragged": ragged,
         "causal": causal, "weights": weights, "block": block, "codes": codes, "dtype": dtype}
    return dict(c, name=name) if name else c


def evict(name=None, B=1, Hkv=8, D=128, capacity=4096, budget=1024, sink=4, recent=256, ragged=False, block=64,
          codes="int8"):
    c = {"op": "evict", "B": B, "Hkv": Hkv, "D": D, "capacity": capacity, "budget": budget, "sink": sink,
         "recent": recent, "ragged": ragged, "block": block, "codes": codes}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the new token of each of eight sequences, between projection and cache: latency only
        rope("rope 8 new tokens", B=8),
        # a long prompt as the projections leave it (token-major), frequencies stretched fourfold
        rope("rope long prompt", S=16384, layout="NHD", scaling="yarn", factor=4.0),
        # gradient of a packed batch, half of the head rotated in adjacent pairs, positions near a million
        rope("rope packed gradient", S=7001, Hq=24, Hkv=24, R=64, layout="TND", pairs="interleaved", far=1000000,
             inverse=True, dtype="fp16"),
        # one decode step of a batch: each sequence's token goes into its own part-filled block
        append("append one token", B=32, capacity=4096, filled=4000, ragged=True),
        # a prompt quantised into an empty cache
        append("append prompt", S=16384, capacity=16384, layout="NHD", block=32, codes="e4m3"),
        # the next chunk of a padded batch, each sequence with its own length, behind tokens that are there
        append("append padded chunk", B=6, S=1001, Hkv=4, D=256, capacity=8192, filled=6000, ragged=True, block=128,
               dtype="fp16"),
        # one sequence, short cache: launch latency
        decode("decode 4096"),
        # four draft tokens each over two long sequences, with the keys' weights kept for eviction
        decode("decode 32768 weights", B=2, Lq=4, capacity=32768, causal=True, weights=True),
        # a batch whose lengths differ
        decode("decode ragged batch", B=16, Hq=16, Hkv=16, D=64, capacity=16384, ragged=True, weights=True, block=32,
               codes="e4m3", dtype="fp16"),
        # wide heads over a very long cache
        decode("decode wide heads", B=1, Hq=16, Hkv=4, D=256, capacity=131072, block=128, codes="e4m3"),
        # one sequence cut to a quarter
        evict("evict 4096 to 1024"),
        # a batch of long sequences cut to a quarter, coarse blocks
        evict("evict batch to 8192", B=8, capacity=32768, budget=8192, recent=1024, ragged=True, block=32,
              codes="e4m3"),
    ]


def _size(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "evict"])
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    block = rng.choice([16, 32, 64, 128])
    codes, dtype = rng.choice(["int8", "e4m3"]), rng.choice(["bf16", "fp16"])
    if op == "rope":
        layout = rng.choice(["HND", "NHD", "TND"])
        Hq = Hkv * rng.choice([1, 2, 4])
        tokens = _size(rng, 1, max(1, 16384 * 40 * 128 // ((Hq + Hkv) * D) // 2))
        B = 1 if layout == "TND" else min(tokens, _size(rng, 1, 16))
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return rope(B=B, S=max(1, tokens // B), Hq=Hq, Hkv=Hkv, D=D, R=rng.choice([D, D // 2, 32]), layout=layout,
                    pairs=rng.choice(["half", "interleaved"]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                    far=rng.choice([0, 100000, 1000000]), inverse=rng.random() < 0.4, dtype=dtype)
    if op == "append":
        B = _size(rng, 1, 16)
        S = _size(rng, 1, max(1, 16384 * 8 * 128 // (Hkv * D * B) // 2))
        filled = rng.choice([0, _size(rng, 1, 4000)])
        capacity = -(-(filled + S) // 128) * 128
        return append(B=B, S=S, Hkv=Hkv, D=D, capacity=capacity, filled=filled, ragged=B > 1 and rng.random() < 0.6,
                      layout=rng.choice(["HND", "NHD"]), block=block, codes=codes, dtype=dtype)
    if op == "decode":
        B = _size(rng, 1, 16)
        Lq, G = rng.choice([1, 1, 2, 4, 5]), rng.choice([1, 2, 4, 8])
        capacity = -(-_size(rng, 16, max(16, 131072 * 4 * 256 // (B * Hkv * D) // 4)) // 128) * 128
        return decode(B=B, Lq=Lq, Hq=G * Hkv, Hkv=Hkv, D=D, capacity=capacity, ragged=rng.random() < 0.6,
                      causal=rng.random() < 0.4, weights=rng.random() < 0.5, block=block, codes=codes, dtype=dtype)
    B = _size(rng, 1, 8)
    capacity = -(-_size(rng, 128, max(128, 8 * 8 * 32768 * 128 // (B * Hkv * D) // 4)) // 128) * 128
    budget = max(16, int(capacity * rng.uniform(0.1, 0.9)))
    return evict(B=B, Hkv=Hkv, D=D, capacity=capacity, budget=budget, sink=rng.choice([0, 4, 8]),
                 recent=rng.randrange(0, budget // 2), ragged=rng.random() < 0.6, block=block, codes=codes)


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["B"] * c["S"] * (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": 4.0 * n + 4.0 * c["B"] * c["S"], "flops": 3.0 * n}
    if c["op"] == "append":
        # each new value is read in 16 bits and written in 8 (a ragged batch has 3/4 of them); the
        # touched blocks are read back: 8 bits in, 16 out
        per = 2 * c["B"] * c["Hkv"] * c["D"]
        n = per * c["S"] * (0.75 if c["ragged"] and c["S"] > 1 else 1.0)
        window = min(-(-(c["S"] + c["block"] - 1) // c["block"]) * c["block"], c["capacity"])
        return {"bytes": 3.0 * n + 3.0 * per * window, "flops": 3.0 * n + per * window}
    if c["op"] == "decode":
        n = c["B"] * c["Hkv"] * c["capacity"] * (0.625 if c["ragged"] else 1.0)
        rows = c["B"] * c["Hq"] * c["Lq"]
        per_key = 2 * c["D"] + 8.0 / c["block"] + (8.0 if c["weights"] else 0.0)
        return {"bytes": n * per_key + rows * (4.0 * c["D"] + 4.0), "flops": 4.0 * c["D"] * n * c["Hq"] // c["Hkv"] * c["Lq"]}
    n = c["B"] * c["Hkv"] * c["capacity"] * (0.875 if c["ragged"] else 1.0)
    kept = c["B"] * c["Hkv"] * min(c["budget"], c["capacity"])
    # weights once; each kept token's codes in and out, its weight and index out, and the read-back
    return {"bytes": 4.0 * n + kept * (2 * 2.0 * c["D"] + 2 * 3.0 * c["D"] + 8.0), "flops": 4.0 * kept * c["D"]}


# ---------------------------------------------------------------- inputs

class State(dict):
    __getattr__ = dict.__getitem__


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 64 + salt)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _lengths(g, B, lo, hi):
    return torch.randint(lo, hi + 1, (B,), generator=g, device="cuda", dtype=torch.int32)


def _channels(g, Hkv, D):
    """Per-channel sizes of keys: most near one, a few channels several times larger."""
    return 0.5 + torch.rand(Hkv, 1, D, generator=g, device="cuda") + 6.0 * (
        torch.rand(Hkv, 1, D, generator=g, device="cuda") < 0.03)


def _filled_cache(c, g):
    """A cache whose every block is full: codes and scales of normal keys and values."""
    shape = (c["B"], c["Hkv"], c["capacity"], c["D"])
    got = {}
    for name, size in (("k", _channels(g, c["Hkv"], c["D"])), ("v", torch.ones(1, device="cuda"))):
        codes = torch.empty(shape, dtype=torch.int8, device="cuda")
        scale = torch.empty(shape[0], shape[1], shape[2] // c["block"], device="cuda")
        for b in range(c["B"]):  # one sequence at a time: 32-bit values of the whole cache need not fit
            x = _randn(g, *shape[1:]) * size
            x = x.view(shape[1], -1, c["block"], shape[3])
            s = x.abs().amax((-1, -2)) / QMAX[c["codes"]]
            scale[b] = s
            codes[b] = _to_codes(x / s[..., None, None], c["codes"]).view(shape[1:])
        got[name], got[name + "_scale"] = codes if c["codes"] == "int8" else codes.view(torch.float8_e4m3fn), scale
    return got


def frequencies(R, scaling, factor, base=10000.0, original=4096):
    """Radians per position of each pair, and the factor on the rotated values."""
    i = np.arange(R // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (R / (R - 2.0))
    f = base ** (-2.0 * i / R)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        turns = lambda n: R * math.log(original / (n * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(turns(32.0)), 0), min(math.ceil(turns(1.0)), R // 2 - 1)
        g = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        f = f * (1.0 - g) + f / factor * g
    return f, 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0


def prepare(case, seed):
    c, st = case, State(c=dict(case))
    g = _gen(seed, 1)
    if c["op"] == "rope":
        t = DT[c["dtype"]]
        lead = lambda H: {"HND": (c["B"], H, c["S"]), "NHD": (c["B"], c["S"], H), "TND": (c["S"], H)}[c["layout"]] + (c["D"],)  # noqa: E731
        st["q"], st["k"] = (_randn(g, *lead(H)).to(t) for H in (c["Hq"], c["Hkv"]))
        f, st["factor"] = frequencies(c["R"], c["scaling"], c["factor"])
        st["inv_freq"] = torch.from_numpy(f).cuda()
        first = torch.randint(0, c["far"] + 4096, (c["B"], 1), generator=g, device="cuda")
        pos = (first + torch.arange(c["S"], device="cuda")).to(torch.int32)
        st["pos"] = pos[0].contiguous() if c["layout"] == "TND" else pos
        return st
    if c["op"] == "append":
        st.update(_filled_cache(c, g))
        B, S, lead = c["B"], c["S"], (c["B"], c["Hkv"], c["S"], c["D"])
        size = _channels(g, c["Hkv"], c["D"])
        new = [_randn(g, *lead) * size * 1.25, _randn(g, *lead) * 1.25]
        if c["layout"] == "NHD":
            new = [x.permute(0, 2, 1, 3) for x in new]
        st["k_new"], st["v_new"] = (x.to(DT[c["dtype"]]).contiguous() for x in new)
        st["start"] = _lengths(g, B, c["filled"] // 2, c["filled"]) if c["ragged"] else torch.full(
            (B,), c["filled"], dtype=torch.int32, device="cuda")
        st["num_new"] = _lengths(g, B, S // 2, S) if c["ragged"] and S > 1 else None
        # the touched blocks, read back in 16 bits
        st["first"] = (st["start"] // c["block"] * c["block"]).to(torch.int32)
        st["window"] = min(-(-(S + c["block"] - 1) // c["block"]) * c["block"], c["capacity"])
        st["end"] = torch.clamp(st["start"] + (S if st["num_new"] is None else st["num_new"]), max=c["capacity"]).to(torch.int32)
        return st
    st.update(_filled_cache(c, g))
    if c["op"] == "decode":
        st["q"] = (_randn(g, c["B"], c["Hq"], c["Lq"], c["D"]) * 0.8).to(DT[c["dtype"]])
        st["len"] = _lengths(g, c["B"], c["capacity"] // 4, c["capacity"]) if c["ragged"] else None
        st["weights"] = torch.rand(c["B"], c["Hkv"], c["capacity"], generator=g, device="cuda") if c["weights"] else None
        return st
    # weights as attention leaves them: heavy tails, many alike, many zero
    shape = (c["B"], c["Hkv"], c["capacity"])
    w = torch.exp(2.0 * _randn(g, *shape)) / 64.0
    w = torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.05, torch.round(w * 16.0) / 16.0, w)
    st["weights"] = torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.05, 0.0, w)
    st["len"] = _lengths(g, c["B"], max(1, c["capacity"] * 3 // 4), c["capacity"]) if c["ragged"] else torch.full(
        (c["B"],), c["capacity"], dtype=torch.int32, device="cuda")
    room = -(-c["budget"] // c["block"]) * c["block"]
    for name in ("k", "v"):
        st["to_" + name] = torch.zeros(c["B"], c["Hkv"], room, c["D"], dtype=torch.int8, device="cuda").view(st[name].dtype)
        st["to_" + name + "_scale"] = torch.zeros(c["B"], c["Hkv"], room // c["block"], device="cuda")
    st["to_weights"] = torch.zeros(c["B"], c["Hkv"], room, device="cuda")
    st["room"] = room
    return st


# ---------------------------------------------------------------- the library's calls

def _own(st):
    import split_kv_merge_attn_b200 as skv
    c = st.c
    if c["op"] == "rope":
        q, k = skv.rope_apply(st.q, st.k, st.pos, st.inv_freq, layout=c["layout"],
                              interleaved=c["pairs"] == "interleaved", factor=st.factor, inverse=c["inverse"])
        return {"q": q, "k": k}
    cache = skv.KV8Cache(st.k, st.v, st.k_scale, st.v_scale)
    if c["op"] == "append":
        skv.kv8_append(cache, st.k_new, st.v_new, st.start, num_new=st.num_new, layout=c["layout"])
        k, v = skv.kv8_fetch(cache, st.window, DT[c["dtype"]], start=st.first, kv_len=st.end)
        return {"k": k, "v": v}
    if c["op"] == "decode":
        out, lse = skv.attn_splitkv_decode_kv8(st.q, cache, kv_len=st.len, causal=c["causal"], weights=st.weights)
        return {"out": out, "lse": lse, "weights": st.weights} if c["weights"] else {"out": out, "lse": lse}
    to = skv.KV8Cache(st.to_k, st.to_v, st.to_k_scale, st.to_v_scale)
    kept, length = skv.kv8_evict(cache, to, st.weights, st.to_weights, st.len, c["budget"], sink=c["sink"],
                                 recent=c["recent"])
    k, v = skv.kv8_fetch(to, st.room, torch.bfloat16, kv_len=length)
    return {"kept": kept, "len": length, "weights": st.to_weights, "k": k, "v": v}


# ---------------------------------------------------------------- plain forms

def _to_codes(x, codes):
    """The 8-bit codes nearest to x (ties to even), as bytes."""
    if codes == "int8":
        return torch.round(x).clamp(-127.0, 127.0).to(torch.int8)
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.int8)


def _from_codes(x):
    return x.float()


def _inverse(s):
    return torch.where((s > 0) & torch.isfinite(s), 1.0 / s, 0.0)


def _turned(x, cos, sin, R, pairs):
    y = x.clone()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if pairs == "interleaved" else (x[..., : R // 2], x[..., R // 2: R])
    first, second = a * cos - b * sin, a * sin + b * cos
    if pairs == "interleaved":
        y[..., 0:R:2], y[..., 1:R:2] = first, second
    else:
        y[..., : R // 2], y[..., R // 2: R] = first, second
    return y


def _plain_rope(st):
    c = st.c
    t = st.pos.double()[..., None] * st.inv_freq * (-1.0 if c["inverse"] else 1.0)
    cos, sin = (f.float() * st.factor for f in (torch.cos(t), torch.sin(t)))
    at = {"HND": 1, "NHD": 2, "TND": 1}[c["layout"]]  # the heads' place
    cos, sin = cos.unsqueeze(at), sin.unsqueeze(at)
    q, k = (_turned(x.float(), cos, sin, c["R"], c["pairs"]).to(x.dtype) for x in (st.q, st.k))
    return {"q": q, "k": k}


def _window(st):
    """Positions of the touched blocks, [B, W], and which of them the cache has."""
    pos = st.first[:, None].long() + torch.arange(st.window, device="cuda")
    return pos.clamp(max=st.c["capacity"] - 1), pos < st.c["capacity"]


def _read(codes, scale, pos, block):
    """Values of the cache at positions [B, W]: [B, H, W, D] in 32 bits."""
    B, H, _, D = codes.shape
    at = pos[:, None, :].expand(B, H, -1)
    got = codes.view(torch.int8).gather(2, at[..., None].expand(-1, -1, -1, D)).view(codes.dtype)
    return _from_codes(got) * scale.gather(2, at // block)[..., None]


def _plain_append_one(st, codes, scale, x, pos, inside):
    c = st.c
    B, H, D, blk = c["B"], c["Hkv"], c["D"], c["block"]
    if c["layout"] == "NHD":
        x = x.permute(0, 2, 1, 3)
    W = -(-pos.shape[1] // blk) * blk
    start, end = st.start[:, None].long(), st.end[:, None].long()
    old, new = inside & (pos < start), inside & (pos >= start) & (pos < end)
    at = (pos - start).clamp(0, c["S"] - 1)[:, None, :, None].expand(B, H, -1, D)
    fresh = x.float().gather(2, at)
    held = _read(codes, scale, pos, blk)
    per = lambda m: m.view(B, 1, W // blk, blk)  # noqa: E731
    amax = torch.where(new[:, None, :, None], fresh, 0.0).abs().amax(-1).view(B, H, W // blk, blk).amax(-1)
    blocks = pos.view(B, W // blk, blk)[..., 0][:, None, :].expand(B, H, -1) // blk
    before = scale.gather(2, blocks)
    s_old = torch.where(per(old).any(-1), before, 0.0)
    s = torch.maximum(amax / torch.full_like(amax, QMAX[c["codes"]]), s_old)  # a quotient, not a product by 1 / qmax
    s = torch.where(s < TINY, 0.0, s)
    touched = per(new).any(-1)
    scale.scatter_(2, blocks, torch.where(touched, s, before))
    inv = _inverse(s).repeat_interleave(blk, 2)[..., None]
    wider = (touched & (s > s_old)).repeat_interleave(blk, 2)[..., None]
    raw = codes.view(torch.int8)
    place = pos[:, None, :, None].expand(B, H, -1, D)
    was = raw.gather(2, place)
    now = torch.where(new[:, None, :, None], _to_codes(fresh * inv, c["codes"]),
                      torch.where(old[:, None, :, None] & wider, _to_codes(held * inv, c["codes"]), was))
    raw.scatter_(2, place, now)


def _plain_fetch(codes, scale, pos, live, block, dtype):
    return torch.where(live[:, None, :, None], _read(codes, scale, pos, block), 0.0).to(dtype)


def _plain_append(st):
    c = st.c
    pos, inside = _window(st)
    _plain_append_one(st, st.k, st.k_scale, st.k_new, pos, inside)
    _plain_append_one(st, st.v, st.v_scale, st.v_new, pos, inside)
    live = inside & (pos < st.end[:, None])
    k, v = (_plain_fetch(x, s, pos, live, c["block"], DT[c["dtype"]]) for x, s in ((st.k, st.k_scale), (st.v, st.v_scale)))
    return {"k": k, "v": v}


def _plain_decode(st):
    c = st.c
    B, Hkv, n, D, Lq = c["B"], c["Hkv"], c["capacity"], c["D"], c["Lq"]
    G = c["Hq"] // Hkv
    spread = lambda s: s.repeat_interleave(c["block"], 2)  # noqa: E731
    q = st.q.float().view(B, Hkv, G * Lq, D)
    x = (q @ _from_codes(st.k).transpose(2, 3)) * (spread(st.k_scale)[:, :, None, :] * D ** -0.5)
    length = torch.full((B,), n, device="cuda") if st.len is None else st.len
    last = length[:, None].expand(B, Lq)
    if c["causal"]:
        last = last - Lq + 1 + torch.arange(Lq, device="cuda")
    seen = torch.arange(n, device="cuda") < last.repeat(1, G)[..., None]  # [B, G * Lq, n]
    x = torch.where(seen[:, None], x, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    out = p @ (_from_codes(st.v) * spread(st.v_scale)[..., None])
    lse = (top + torch.log(total)) * LOG2E
    got = {"out": out.view(B, c["Hq"], Lq, D).to(st.q.dtype), "lse": lse.view(B, c["Hq"], Lq)}
    if c["weights"]:
        st.weights.add_(p.sum(2))
        got["weights"] = st.weights
    return got


def _kept(weights, length, c):
    """Kept positions in order, [B, H, budget] with -1 behind the last, and how many."""
    n = weights.shape[-1]
    j = torch.arange(n, device="cuda")
    L = length[:, None, None].long()
    keep = torch.clamp(L, max=c["budget"])
    always = (j < c["sink"]) | (j >= L - c["recent"])
    rank_by = torch.where(always, math.inf, weights)
    rank_by = torch.where(j < L, rank_by, -math.inf)
    order = torch.sort(rank_by, dim=-1, descending=True, stable=True)[1]
    picked = torch.zeros_like(weights, dtype=torch.bool).scatter_(2, order, (j < keep).expand_as(weights))
    width = min(c["budget"], n)
    place = torch.sort(torch.where(picked, j, n + j), dim=-1)[0][..., :width]
    kept = torch.full((*weights.shape[:2], c["budget"]), -1, dtype=torch.int32, device="cuda")
    kept[..., :width] = torch.where(place < n, place, -1).to(torch.int32)
    return kept, keep[:, 0, 0].to(torch.int32)


def _plain_evict(st):
    c = st.c
    B, H, D, blk, room = c["B"], c["Hkv"], c["D"], c["block"], st.room
    kept, length = _kept(st.weights, st.len, c)
    live = torch.zeros(B, H, room, dtype=torch.bool, device="cuda")
    live[..., : c["budget"]] = kept >= 0
    at = torch.zeros(B, H, room, dtype=torch.int64, device="cuda")
    at[..., : c["budget"]] = kept.clamp(min=0)
    got = {"kept": kept, "len": length}
    for name in ("k", "v"):
        codes, scale = st[name], st[name + "_scale"]
        raw = codes.view(torch.int8).gather(2, at[..., None].expand(-1, -1, -1, D)).view(codes.dtype)
        s_tok = torch.where(live, scale.gather(2, at // blk), 0.0)
        s = s_tok.view(B, H, room // blk, blk).amax(-1)
        s = torch.where(s < TINY, 0.0, s)
        inv = _inverse(s).repeat_interleave(blk, 2)[..., None]
        now = _to_codes(_from_codes(raw) * s_tok[..., None] * inv, c["codes"])
        to, to_s = st["to_" + name].view(torch.int8), st["to_" + name + "_scale"]
        to.copy_(torch.where(live[..., None], now, to))
        to_s.copy_(torch.where(live.view(B, H, room // blk, blk).any(-1), s, to_s))
        everywhere = torch.arange(room, device="cuda")[None].expand(B, -1)
        got[name] = _plain_fetch(st["to_" + name], to_s, everywhere, live[:, 0], blk, torch.bfloat16)
    st.to_weights.copy_(torch.where(live, st.weights.gather(2, at), st.to_weights))
    got["weights"] = st.to_weights
    return got


PLAIN = {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode, "evict": _plain_evict}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state.c["op"]](state)


# ---------------------------------------------------------------- 64 bits

def _exact_rope(st):
    c = st.c
    f, m = frequencies(c["R"], c["scaling"], c["factor"])
    pos = st.pos.cpu().numpy().astype(np.float64)
    angle = torch.from_numpy(pos[..., None] * f).cuda()
    turn = torch.polar(torch.full_like(angle, m), -angle if c["inverse"] else angle)
    got = {}
    for name in ("q", "k"):
        x = st[name].double()
        part = x[..., : c["R"]]
        z = torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) if c["pairs"] == "interleaved" else \
            torch.complex(*part.chunk(2, -1))
        z = z * (turn[:, None] if c["layout"] != "NHD" else turn[:, :, None])
        y = torch.view_as_real(z).flatten(-2) if c["pairs"] == "interleaved" else torch.cat((z.real, z.imag), -1)
        got[name] = torch.cat((y, x[..., c["R"]:]), -1)
    return got


def _exact_codes(x, s, codes):
    """Codes of x by the scale s; s, its reciprocal and the scaled value are 32-bit numbers by definition."""
    y = (x * _held(1.0 / s.clamp(min=TINY))).float().double()
    if codes == "int8":
        return torch.round(y)
    # e4m3: steps of 2^-3 of the value's power of two, of 2^-9 below 2^-6
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _held(x):
    return x.float().double()


def _exact_append(st):
    c = st.c
    got, blk, W = {}, c["block"], st.window
    start, end = st.start.tolist(), st.end.tolist()
    for name in ("k", "v"):
        codes, scale, new = st[name].float().double(), st[name + "_scale"].double(), st[name + "_new"].double()
        if c["layout"] == "NHD":
            new = new.transpose(1, 2)
        out = torch.zeros(c["B"], c["Hkv"], W, c["D"], dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            base = start[b] // blk * blk
            count = end[b] - base
            if end[b] == start[b]:  # nothing new: the tokens before stay as they are
                out[b, :, :count] = codes[b, :, base:end[b]] * scale[b, :, base // blk, None, None]
                continue
            head = start[b] - base  # older tokens of the first block
            x = torch.cat((codes[b, :, base:start[b]] * scale[b, :, base // blk, None, None], new[b, :, : end[b] - start[b]]), 1)
            pad = -count % blk
            x = torch.nn.functional.pad(x, (0, 0, 0, pad)).view(c["Hkv"], -1, blk, c["D"])
            fresh = x.clone()
            fresh[:, 0, :head] = 0.0
            s = fresh.abs().amax((-1, -2)) / QMAX[c["codes"]]
            if head:
                s[:, 0] = torch.maximum(s[:, 0], scale[b, :, base // blk])
            s = _held(s)[..., None, None]
            y = _exact_codes(_held(x), s, c["codes"]) * s
            out[b, :, :count] = y.view(c["Hkv"], -1, c["D"])[:, :count]
        got[name] = out
    return got


def _exact_decode(st):
    c = st.c
    B, Hkv, D, Lq, blk = c["B"], c["Hkv"], c["D"], c["Lq"], c["block"]
    G = c["Hq"] // Hkv
    out = torch.zeros(B, c["Hq"], Lq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, c["Hq"], Lq), -math.inf, dtype=torch.float64, device="cuda")
    weights = st.weights.double() if c["weights"] else None
    lengths = [c["capacity"]] * B if st.len is None else st.len.tolist()
    for b, n in enumerate(lengths):
        for h in range(Hkv):
            k, v = (st[x][b, h, :n].float().double() * st[x + "_scale"][b, h].double().repeat_interleave(blk)[:n, None]
                    for x in ("k", "v"))
            for i in range(Lq):
                m = n - Lq + 1 + i if c["causal"] else n
                if m <= 0:
                    continue
                heads = slice(h * G, (h + 1) * G)
                logits = (st.q[b, heads, i].double() @ k[:m].T) / math.sqrt(D)
                total = torch.logsumexp(logits, -1)
                p = torch.exp(logits - total[:, None])
                out[b, heads, i] = p @ v[:m]
                lse[b, heads, i] = total / math.log(2.0)
                if weights is not None:
                    weights[b, h, :m] += p.sum(0)
    got = {"out": out, "lse": lse}
    if weights is not None:
        got["weights"] = weights
    return got


def _exact_evict(st):
    c = st.c
    B, H, D, blk, room = c["B"], c["Hkv"], c["D"], c["block"], st.room
    got = {"kept": None, "len": None, "weights": torch.zeros(B, H, room, dtype=torch.float64, device="cuda")}
    for name in ("k", "v"):
        got[name] = torch.zeros(B, H, room, D, dtype=torch.float64, device="cuda")
    weights, lengths = st.weights.cpu().numpy(), st.len.tolist()
    for b, n in enumerate(lengths):
        for h in range(H):
            w = weights[b, h, :n]
            if n <= c["budget"]:
                at = np.arange(n)
            else:
                middle = np.arange(c["sink"], n - c["recent"])
                best = middle[np.lexsort((middle, -w[middle]))][: c["budget"] - c["sink"] - c["recent"]]
                at = np.sort(np.concatenate((np.arange(c["sink"]), best, np.arange(n - c["recent"], n))))
            at = torch.from_numpy(at).cuda()
            got["weights"][b, h, : len(at)] = st.weights[b, h, at].double()
            for name in ("k", "v"):
                s_tok = st[name + "_scale"][b, h].double()[at // blk]
                x = _held(st[name][b, h].float().double()[at] * s_tok[:, None])
                s = torch.nn.functional.pad(s_tok, (0, -len(at) % blk)).view(-1, blk).amax(-1)
                s = s.repeat_interleave(blk)[: len(at), None]
                got[name][b, h, : len(at)] = _exact_codes(x, s, c["codes"]) * s
    return got


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "decode": _exact_decode, "evict": _exact_evict}[case["op"]](st)
