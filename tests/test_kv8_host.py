"""Host-only checks of rotary positions and the 8-bit cache (no GPU needed):
refusals of the C ABI and of the Python wrappers (only invalid calls are made,
so none reaches a launch), the frequency tables, the planner, and the oracle's
own pieces against independent statements."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as O
import split_kv_merge_attn_b200 as skv

INVALID, UNSUPPORTED, WS_SMALL = skv.SKV_ERR_INVALID_ARG, skv.SKV_ERR_UNSUPPORTED, skv.SKV_ERR_WORKSPACE_TOO_SMALL
P = 0x10000000  # aligned addresses that are never read: every call below is refused first
STEP = 0x10000000


def addr(i):
    return P + i * STEP


# ---------------------------------------------------------------- C ABI

def rope(**kw):
    a = dict(q=addr(0), k=addr(1), qo=addr(2), ko=addr(3), pos=addr(4), f=addr(5), B=1, Hq=4, Hkv=2, S=8, D=128, R=64,
             m=1.0, dt=0, layout=0, inter=0, inv=0)
    a.update(kw)
    return skv.lib().rope_apply(*a.values(), None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(q=None)), (INVALID, dict(qo=None)), (INVALID, dict(pos=None)), (INVALID, dict(f=None)),
    (INVALID, dict(q=P + 2)), (INVALID, dict(pos=addr(4) + 2)), (INVALID, dict(f=addr(5) + 4)),
    (INVALID, dict(k=None)), (INVALID, dict(ko=None)), (INVALID, dict(k=None, ko=None)),  # Hkv without k
    (INVALID, dict(Hkv=0)), (INVALID, dict(B=0)), (INVALID, dict(Hq=0)), (INVALID, dict(S=-1)), (INVALID, dict(D=0)),
    (INVALID, dict(layout=3)), (INVALID, dict(layout=2, B=2)), (INVALID, dict(R=0)), (INVALID, dict(R=63)),
    (INVALID, dict(R=144)), (INVALID, dict(m=math.inf)), (INVALID, dict(inter=2)), (INVALID, dict(inv=-1)),
    (INVALID, dict(dt=5)), (UNSUPPORTED, dict(dt=2)), (UNSUPPORTED, dict(D=72, R=16)), (UNSUPPORTED, dict(R=40)),
    (INVALID, dict(qo=P + 16)), (INVALID, dict(ko=addr(2))), (INVALID, dict(ko=P)), (INVALID, dict(qo=addr(1))),
])
def test_rope_refusals(status, kw):
    assert rope(**kw) == status


def freq(R=64, base=1e4, scaling=0, factor=1.0, L=4096, fast=32.0, slow=1.0):
    out, m = (ctypes.c_double * 256)(), ctypes.c_double()
    return skv.lib().rope_inv_freq(R, base, scaling, factor, L, fast, slow, out, ctypes.byref(m))


@pytest.mark.parametrize("kw", [dict(R=0), dict(R=7), dict(base=1.0), dict(base=math.nan), dict(scaling=4),
                                dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=2, factor=2.0, R=2),
                                dict(scaling=3, factor=2.0, L=0), dict(scaling=3, factor=2.0, slow=0.0),
                                dict(scaling=3, factor=2.0, fast=0.5), dict(scaling=3, factor=math.inf)])
def test_inv_freq_refusals(kw):
    assert freq(**kw) == INVALID


CACHE = dict(k=addr(0), v=addr(1), ks=addr(2), vs=addr(3))


def append(**kw):
    a = dict(kn=addr(8), vn=addr(9), **CACHE, start=addr(4), num=None, cu=None, B=2, Hkv=2, S=4, T=0, cap=128, D=128,
             block=32, dt=0, codes=0, layout=0)
    a.update(kw)
    return skv.lib().kv8_append(*a.values(), None)


def fetch(**kw):
    a = dict(**CACHE, ko=addr(8), vo=addr(9), start=None, kv_len=None, B=2, Hkv=2, n=4, cap=128, D=128, block=32, dt=0,
             codes=0, layout=0)
    a.update(kw)
    return skv.lib().kv8_fetch(*a.values(), None)


def decode(**kw):
    a = dict(q=addr(8), **CACHE, out=addr(9), lse=None, w=None, B=2, Hq=4, Hkv=2, Lq=1, cap=128, D=128, block=32,
             scale=0.1, dt=0, codes=0, kv_len=None, causal=0, ctas=1, ws=None, wsb=0)
    a.update(kw)
    return skv.lib().attn_splitkv_decode_kv8(*a.values(), None)


def evict(**kw):
    a = dict(**CACHE, w=addr(4), kv_len=addr(5), tk=addr(6), tv=addr(7), tks=addr(8), tvs=addr(9), tw=addr(10),
             kept=addr(11), new=addr(12), B=2, Hkv=2, cap=128, tcap=64, D=128, block=32, codes=0, budget=50, sink=4,
             recent=8)
    a.update(kw)
    return skv.lib().kv8_evict(*a.values(), None)


@pytest.mark.parametrize("call", [append, fetch, decode, evict])
@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(ks=None)), (INVALID, dict(vs=None)),
    (INVALID, dict(k=P + 8)), (INVALID, dict(vs=addr(3) + 2)), (INVALID, dict(B=0)), (INVALID, dict(Hkv=0)),
    (INVALID, dict(cap=0)), (INVALID, dict(cap=100)), (INVALID, dict(codes=2)), (INVALID, dict(block=0)),
    (INVALID, dict(D=0)), (UNSUPPORTED, dict(D=96)), (UNSUPPORTED, dict(block=8)), (UNSUPPORTED, dict(block=1)),
    (UNSUPPORTED, dict(B=40000, Hq=4)), (UNSUPPORTED, dict(B=1024, Hkv=16, Hq=16, cap=1 << 20)),
])
def test_cache_refusals(call, status, kw):
    if "Hq" in kw and call is not decode:
        kw = {k: v for k, v in kw.items() if k != "Hq"}
    if call is evict and kw.get("block") == 1:
        kw = dict(kw, tcap=64)
    assert call(**kw) == status


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(kn=None)), (INVALID, dict(vn=addr(9) + 4)), (INVALID, dict(start=None)), (INVALID, dict(S=-1)),
    (INVALID, dict(num=2)), (INVALID, dict(cu=addr(5))), (INVALID, dict(layout=2)), (INVALID, dict(layout=9)),
    (INVALID, dict(layout=2, cu=addr(5), num=addr(6), T=8)), (INVALID, dict(layout=2, cu=addr(5), T=3)),
    (INVALID, dict(layout=2, cu=addr(5), T=-1)), (INVALID, dict(dt=7)), (UNSUPPORTED, dict(dt=2)),
])
def test_append_refusals(status, kw):
    assert append(**kw) == status


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(ko=None)), (INVALID, dict(vo=addr(9) + 8)), (INVALID, dict(n=-1)), (INVALID, dict(layout=2)),
    (INVALID, dict(start=addr(4) + 1)), (INVALID, dict(kv_len=addr(4) + 1)), (UNSUPPORTED, dict(dt=2)),
])
def test_fetch_refusals(status, kw):
    assert fetch(**kw) == status


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(q=None)), (INVALID, dict(out=None)), (INVALID, dict(lse=addr(5) + 2)), (INVALID, dict(w=addr(5) + 4)),
    (INVALID, dict(kv_len=addr(5) + 2)), (INVALID, dict(Hq=3)), (INVALID, dict(Hq=0)), (INVALID, dict(Lq=0)),
    (INVALID, dict(scale=0.0)), (INVALID, dict(scale=math.nan)), (INVALID, dict(causal=2)), (INVALID, dict(ctas=-1)),
    (INVALID, dict(ctas=1025)), (UNSUPPORTED, dict(dt=2)), (INVALID, dict(dt=-1)),
    (UNSUPPORTED, dict(Hq=1 << 29, Lq=8)), (WS_SMALL, dict(ctas=2, cap=512)), (WS_SMALL, dict(w=addr(5))),
    (INVALID, dict(w=addr(5), wsb=1 << 30)), (INVALID, dict(ctas=2, cap=512, ws=P + 16, wsb=1 << 30)),
])
def test_decode_refusals(status, kw):
    assert decode(**kw) == status


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(w=None)), (INVALID, dict(tw=None)), (INVALID, dict(kept=None)), (INVALID, dict(new=None)),
    (INVALID, dict(kv_len=addr(5) + 2)), (INVALID, dict(tk=None)), (INVALID, dict(tcap=50)), (INVALID, dict(tcap=32)),
    (INVALID, dict(budget=0)), (INVALID, dict(sink=-1)), (INVALID, dict(recent=-1)), (INVALID, dict(sink=43)),
    (INVALID, dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1)),
    (INVALID, dict(tk=P)), (INVALID, dict(tv=addr(6))), (INVALID, dict(tw=addr(4))), (INVALID, dict(new=addr(5))),
    (INVALID, dict(kept=addr(4) + 64)), (INVALID, dict(tks=addr(2) + 16)),
])
def test_evict_refusals(status, kw):
    assert evict(**kw) == status


def test_workspace_and_plan():
    a = lambda x: (x + 255) // 256 * 256  # noqa: E731
    for B, Hq, Hkv, Lq, cap, D, c, w in [(1, 32, 8, 1, 4096, 128, 16, 0), (2, 8, 2, 3, 320, 64, 1, 1),
                                         (1, 4, 4, 1, 64, 256, 3, 0), (3, 6, 1, 5, 1024, 256, 5, 1),
                                         (2, 4, 2, 1, 256, 128, 4, 0)]:
        rows, units = B * Hq * Lq, B * Hkv * -(-Hq // Hkv * Lq // 16)
        slots = 16 * (units + c)
        divided = c > 1 and cap > (64 if D == 256 else 256)
        want = a(4 * (B + 1)) + a(4 * slots) + a(4 * slots * D) if divided else 0
        want += a(4 * rows) + a(4 * rows * cap) if w else 0
        assert skv.attn_splitkv_kv8_workspace(B, Hq, Hkv, Lq, cap, D, c, bool(w)) == want
    assert skv.attn_splitkv_kv8_workspace(1, 4, 4, 1, 64, 128, 0) == 0
    assert skv.attn_splitkv_kv8_plan(1, 32, 8, 1, 4096) == 8 * 17   # a place for each tile of 256 keys and one more
    assert skv.attn_splitkv_kv8_plan(1, 32, 8, 1, 32768) == 296
    assert skv.attn_splitkv_kv8_plan(1, 16, 4, 1, 4096, 256) == 4 * 65
    assert skv.attn_splitkv_kv8_plan(1, 32, 8, 1, 4096, requested_ctas=7) == 7
    for bad in [dict(B=0), dict(Hq=5, Hkv=2), dict(capacity=0), dict(num_sms=0), dict(requested_ctas=1025)]:
        with pytest.raises(skv.SkvError):
            skv.attn_splitkv_kv8_plan(**{**dict(B=1, Hq=4, Hkv=2, Lq=1, capacity=64), **bad})


# ---------------------------------------------------------------- wrappers

def test_wrapper_refusals():
    """What the library cannot see is refused in Python, before any launch (host tensors)."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    f, _ = skv.rope_inv_freq(64, device="cpu")
    q, k, pos = bf(2, 4, 8, 64), bf(2, 2, 8, 64), i32(2, 8)
    bad_rope = [dict(layout="XYZ"), dict(q=bf(4, 8, 64)), dict(k=bf(2, 2, 9, 64)), dict(k=k.half()), dict(positions=i32(8)),
                dict(positions=pos.long()), dict(inv_freq=f.float()), dict(inv_freq=f.view(2, -1)), dict(q_out=bf(2, 4, 8, 32)),
                dict(q_out=q.half()), dict(k=None, k_out=k), dict()]
    for kw in bad_rope:  # the last: host tensors
        with pytest.raises(ValueError):
            skv.rope_apply(**{**dict(q=q, k=k, positions=pos, inv_freq=f), **kw})
    with pytest.raises(ValueError):
        skv.rope_inv_freq(64, scaling="stretch", device="cpu")
    with pytest.raises(ValueError):
        skv.kv8_cache(1, 1, 100, 64, 16, device="cpu")
    with pytest.raises(ValueError):
        skv.kv8_cache(1, 1, 128, 64, 8, device="cpu")
    with pytest.raises(ValueError):
        skv.kv8_cache(1, 1, 128, 64, 16, codes="int4", device="cpu")
    c = skv.kv8_cache(2, 2, 64, 64, 16, device="cpu")
    bad_caches = [c._replace(k=c.k[0]), c._replace(k=c.k.float()), c._replace(v=c.v[:, :, :32]),
                  c._replace(v=c.v.view(torch.float8_e4m3fn)), c._replace(k_scale=c.k_scale.double()),
                  c._replace(v_scale=c.v_scale[:, :1]), c._replace(k_scale=c.k_scale[..., :3], v_scale=c.v_scale[..., :3]), c]
    for x in bad_caches:  # the last: host tensors
        for call in (lambda: skv.kv8_append(x, bf(2, 2, 1, 64), bf(2, 2, 1, 64), i32(2)),
                     lambda: skv.kv8_fetch(x, 4), lambda: skv.attn_splitkv_decode_kv8(bf(2, 4, 1, 64), x)):
            with pytest.raises(ValueError):
                call()
    assert repr(c).startswith("KV8Cache(")


def test_transposed_tensors_are_refused_on_the_host():
    c = skv.kv8_cache(2, 2, 64, 64, 16, device="cpu")
    x = c._replace(k=c.k.transpose(0, 1))
    with pytest.raises(ValueError):
        skv.kv8_fetch(x, 4)


# ---------------------------------------------------------------- frequencies, oracle pieces

def test_inv_freq_values():
    R, base, s = 64, 10000.0, 4.0
    i = np.arange(R // 2)
    plain = base ** (-2.0 * i / R)
    got = {n: skv.rope_inv_freq(R, base, n, s, original_len=2048, device="cpu") for n in skv.ROPE_SCALINGS}
    np.testing.assert_allclose(got["none"][0], plain, rtol=1e-14)
    np.testing.assert_allclose(got["linear"][0], plain / s, rtol=1e-14)
    ntk = got["ntk"][0].numpy()
    np.testing.assert_allclose(ntk[0], 1.0, rtol=1e-14)            # the fastest pair keeps its frequency
    np.testing.assert_allclose(ntk[-1], plain[-1] / s, rtol=1e-12)  # the slowest is interpolated
    yarn, m = got["yarn"]
    ratio = yarn.numpy() / plain
    turns = 2048 * plain / (2 * np.pi)  # turns over the original length
    # the ramp's ends are rounded outwards to whole pairs, base^(2 / R) = 1.34 apart in turns
    np.testing.assert_allclose(ratio[turns > 32 * 1.34], 1.0, rtol=1e-14)
    np.testing.assert_allclose(ratio[turns < 1 / 1.34], 1 / s, rtol=1e-14)
    assert 0 < np.sum((ratio < 0.999) & (ratio > 1.001 / s))
    assert np.all(np.diff(ratio) <= 1e-15) and m == 0.1 * math.log(s) + 1.0
    assert got["none"][1] == got["linear"][1] == got["ntk"][1] == 1.0


def test_round_e4m3_is_the_types_rounding():
    x = torch.cat((torch.randn(20000, generator=torch.Generator().manual_seed(0)) * 100,
                   torch.linspace(-448, 448, 7169), 2.0 ** torch.linspace(-12, -4, 4001)))
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(O.round_e4m3(x.double().numpy()), want)


def test_append_oracle_against_a_plain_statement():
    """Values read back are within half a step of the new tokens, and an old
    token's within half a step more."""
    rng = np.random.default_rng(1)
    codes, scale = np.zeros((64, 8)), np.zeros(4, dtype=np.float32)
    first, second = rng.standard_normal((20, 8)), 3 * rng.standard_normal((10, 8))
    O.kv8_append(codes, scale, first, 0, 20, 16, "int8")
    one = scale.copy()
    O.kv8_append(codes, scale, second, 20, 10, 16, "int8")
    held = codes * np.repeat(scale, 16)[:, None]
    step = np.repeat(scale, 16)[:, None] / 2 * (1 + 1e-4)
    assert np.all(np.abs(held[20:30] - second) <= step[20:30])
    old = np.repeat(one, 16)[:, None] / 2
    assert np.all(np.abs(held[:20] - first) <= step[:20] + old[:20])
    assert scale[0] == one[0] and scale[1] >= one[1] and np.all(scale[2:] == 0)
    assert np.all(np.abs(codes[:30]).reshape(-1) <= 127)


def test_key_weights_sum_to_the_rows():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 6, 3, 8)), rng.standard_normal((2, 2, 20, 8))
    w = O.key_weights(q, k, 0.3, [20, 2], causal=True)
    np.testing.assert_allclose(w.sum(-1), [[9, 9], [6, 6]], rtol=1e-12)  # the first row of entry 1 sees no key
    assert np.all(w[1, :, 2:] == 0)
    _, lse = O.decode(q, k, k, 0.3, kv_len=[20, 2], causal=True)
    x = 0.3 * np.log2(np.e) * np.einsum("hid,hjd->hij", q[0], np.repeat(k[0], 3, 0))
    p = np.where(np.arange(20) < 20 - 3 + 1 + np.arange(3)[:, None], 2.0 ** (x - lse[0][..., None]), 0.0)
    np.testing.assert_allclose(p.reshape(2, 9, 20).sum(1), w[0], rtol=1e-10)


def test_kept_by_hand():
    w = np.array([5.0, 1, 1, 9, np.nan, 1, 0, 2, 2, 3])
    assert O.kv8_kept(w, 10, 6, 1, 2).tolist() == [0, 1, 3, 7, 8, 9]
    assert O.kv8_kept(w, 10, 4, 0, 0).tolist() == [0, 3, 7, 9]
    assert O.kv8_kept(w, 10, 9, 0, 0).tolist() == [0, 1, 2, 3, 5, 6, 7, 8, 9]
    assert O.kv8_kept(w, 3, 3, 1, 1).tolist() == [0, 1, 2]


# ---------------------------------------------------------------- memory written twice, or written and read

@pytest.mark.parametrize("call,kw", [
    (append, dict(v=addr(0))), (append, dict(v=addr(0) + 2 * 2 * 128 * 128 - 16)), (append, dict(vs=addr(2))),
    (append, dict(kn=addr(0))), (append, dict(vn=addr(1) - 16)), (append, dict(start=addr(2))),
    (append, dict(num=addr(3) + 2 * 2 * 4 * 4 - 4)), (append, dict(kn=addr(8), k=addr(8) + 2 * 2 * 4 * 128 * 2 - 16)),
    (append, dict(layout=2, cu=addr(3) - 8, T=8)),
    (fetch, dict(vo=addr(8))), (fetch, dict(ko=addr(0))), (fetch, dict(vo=addr(3) - 16)), (fetch, dict(kv_len=addr(8))),
    (fetch, dict(start=addr(9) + 2 * 2 * 4 * 128 * 2 - 4)),
    (decode, dict(out=addr(8))), (decode, dict(out=addr(1))), (decode, dict(lse=addr(9))), (decode, dict(kv_len=addr(9))),
    (decode, dict(w=addr(2), ws=addr(20), wsb=1 << 20)), (decode, dict(w=addr(5), ws=addr(5), wsb=1 << 20)),
    (decode, dict(ctas=2, cap=512, ws=addr(9), wsb=1 << 20)), (decode, dict(ctas=2, cap=512, ws=addr(0), wsb=1 << 20)),
    (evict, dict(tv=addr(6))), (evict, dict(tk=addr(1))), (evict, dict(new=addr(5))), (evict, dict(tw=addr(4))),
])
def test_overlaps_are_refused(call, kw):
    assert call(**kw) == INVALID
