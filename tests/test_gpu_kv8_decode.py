"""attn_splitkv_decode_kv8 against the fp64 oracle on the cache's values.

Tolerances, with y = |scale| log2(e) max_j (max_d |q_d|) sum_d |k_jd| per row:
  logits   the fp16 q differs from q by at most 2^-25 of its row's largest
           value, and the fp32 sums of at most 16 MMA steps by 16 * 2^-23 of
           sum |q k|: together below 2^-18 y;
  LSE      2^-18 y, plus 2^-17 for ex2, log2 and the merge (2^-22 relative each
           of values up to a few tens);
  weights  relative 2 ln 2 times the LSE's error, plus 2^-20;
  O        half a rounding step of the output type relative to |O|, plus
           (2^-11 + the weights' relative error + 2^-16) of sum p |v|, plus
           2^-25 u sum |c_d| with u = max_j p_j vs_j: p vs / u' is rounded to
           fp16 once (u' <= u: the largest so far), by 2^-11 relative in fp16's
           normal range and by half its smallest step, 2^-25 of u', below it, and
           each error meets one code c_d; sums and merges are fp32."""
import numpy as np
import pytest
import torch

import oracle as O
import split_kv_merge_attn_b200 as skv
from tests._gpu_helpers import nan_empty
from tests._kv8_helpers import DT, HALF_STEP, code_values, filled_cache, gen, i32, values

pytestmark = pytest.mark.gpu


def row_sizes(q, k, scale, lengths):
    """y of the module's note: [B, Hq, Lq]."""
    q, a = np.abs(O.to_f64(q)), np.abs(k).sum(-1)
    B, Hq, Lq, _ = q.shape
    G = Hq // k.shape[1]
    top = np.array([[a[b, h // G, : lengths[b]].max(initial=0.0) for h in range(Hq)] for b in range(B)])
    return scale * np.log2(np.e) * q.max(-1) * top[..., None]


def subnormal_bound(q, cache, k, lengths, scale, causal):
    """2^-25 max_j(p_j vs_j) sum_j |c_jd| of the module's note: [B, Hq, Lq, D]."""
    q, vs, c = O.to_f64(q), cache.v_scale.cpu().double().numpy(), np.abs(code_values(cache.v))
    B, Hq, Lq, D = q.shape
    G, block = Hq // k.shape[1], k.shape[2] // vs.shape[2]
    out = np.zeros((B, Hq, Lq, D))
    for b in range(B):
        for h in range(Hq):
            for i in range(Lq):
                n = max(lengths[b] - Lq + 1 + i, 0) if causal else lengths[b]
                if n:
                    x = scale * (k[b, h // G, :n] @ q[b, h, i])
                    p = np.exp(x - x.max())
                    u = np.max(p / p.sum() * np.repeat(vs[b, h // G], block)[:n])
                    out[b, h, i] = 2.0 ** -25 * u * c[b, h // G, :n].sum(0)
    return out


def check(q, cache, out, lse, lengths, scale, causal, dtype, added=None):
    k, v = values(cache.k, cache.k_scale, lengths), values(cache.v, cache.v_scale, lengths)
    o_ref, l_ref = O.decode(q, k, v, scale, kv_len=lengths, causal=causal)
    size, _ = O.decode(q, k, np.abs(v), scale, kv_len=lengths, causal=causal)
    l_tol = 2.0 ** -18 * row_sizes(q, k, scale, lengths) + 2.0 ** -17
    o, l = O.to_f64(out), O.to_f64(lse)
    empty = np.isneginf(l_ref)
    assert np.all(np.isneginf(l[empty])) and np.all(o[empty] == 0)
    off = np.abs(l[~empty] - l_ref[~empty]) - l_tol[~empty]
    assert np.all(off <= 0), off.max()
    rel = 2 * np.log(2.0) * l_tol + 2.0 ** -20
    o_tol = HALF_STEP[dtype] * np.abs(o_ref) + (2.0 ** -11 + rel + 2.0 ** -16)[..., None] * size
    o_tol += subnormal_bound(q, cache, k, lengths, scale, causal) + (2.0 ** -25 if dtype == "fp16" else 0.0)
    worst = np.max(np.abs(o - o_ref) - o_tol)
    assert worst <= 0
    if added is not None:
        w_ref = O.key_weights(q, k, scale, lengths, causal)
        G = q.shape[1] // k.shape[1]
        top = rel.reshape(rel.shape[0], -1, G * rel.shape[2]).max(-1)[..., None]
        worst = np.max(np.abs(added - w_ref) - (top * w_ref + 2.0 ** -24 * (1 + w_ref)))
        assert worst <= 0


def run(B, Hq, Hkv, Lq, D, capacity, block, codes, dtype, lengths, causal=False, weights=False, ctas=0, seed=0,
        q_mult=1.0, scale_span=1.0, full=False):
    cache = filled_cache(B, Hkv, capacity, D, block, codes, lengths, seed, scale_span)
    q = (torch.randn(B, Hq, Lq, D, generator=gen(seed + 1)) * q_mult).to(DT[dtype]).cuda()
    scale = D ** -0.5
    nc = skv.attn_splitkv_kv8_plan(B, Hq, Hkv, Lq, capacity, D, 148, ctas)
    ws = torch.full((skv.attn_splitkv_kv8_workspace(B, Hq, Hkv, Lq, capacity, D, nc, weights) + 1,), 0xFF, dtype=torch.uint8,
                    device="cuda")  # NaN bit patterns
    out, lse = nan_empty(q.shape, q.dtype), nan_empty(q.shape[:3], torch.float32)
    w = torch.zeros(B, Hkv, capacity, device="cuda") if weights else None
    skv.attn_splitkv_decode_kv8(q, cache, scale, kv_len=None if full else i32(lengths), causal=causal, weights=w,
                                num_ctas=nc, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert skv.device_error() == 0
    check(q, cache, out, lse, lengths, scale, causal, dtype, None if w is None else O.to_f64(w))
    return q, cache, out, lse, w


CASES = [
    # B, Hq, Hkv, Lq, D, capacity, block, codes, dtype, lengths, causal, weights, ctas
    (1, 1, 1, 1, 64, 16, 16, "int8", "bf16", [1], False, True, 1),
    (1, 4, 4, 1, 128, 64, 64, "e4m3", "fp16", [17], False, True, 0),
    (2, 8, 2, 1, 128, 1024, 64, "int8", "bf16", [1000, 65], False, True, 0),
    (2, 8, 2, 4, 128, 512, 32, "e4m3", "bf16", [512, 3], True, True, 5),       # rows that see no key
    (1, 6, 1, 5, 64, 640, 16, "int8", "fp16", [639], True, True, 0),           # 30 rows: two row groups
    (3, 4, 2, 1, 64, 384, 128, "e4m3", "bf16", [0, 384, 129], False, True, 3),
    (1, 16, 4, 4, 256, 1152, 128, "int8", "bf16", [1151], False, False, 0),
    (2, 5, 1, 2, 256, 336, 16, "e4m3", "fp16", [336, 31], True, True, 2),
    (1, 16, 1, 1, 256, 128, 32, "int8", "fp16", [128], False, True, 1),
    (1, 32, 1, 1, 128, 256, 16, "int8", "bf16", [250], False, False, 4),       # 32 rows a kv head
    (4, 2, 2, 1, 128, 4096, 64, "int8", "fp16", [4096, 2049, 1, 4000], False, True, 0),
    # the division among CTAs: shares that end inside units, hold several, or are empty
    (5, 4, 2, 1, 64, 1536, 32, "int8", "bf16", [1536, 0, 257, 1, 900], False, True, 7),
    (5, 4, 2, 1, 128, 1536, 32, "e4m3", "fp16", [0, 300, 0, 1200, 0], False, False, 5),
    (2, 4, 4, 3, 256, 512, 64, "int8", "bf16", [512, 100], True, True, 37),
    (130, 2, 1, 1, 64, 512, 16, "e4m3", "bf16", [(i * 37) % 513 for i in range(130)], False, False, 11),
    (300, 1, 1, 1, 128, 272, 16, "int8", "fp16", [(i * 53) % 273 for i in range(300)], False, True, 0),
    (2, 2, 1, 1, 64, 512, 16, "int8", "bf16", [0, 0], False, True, 4),
    (1, 2, 1, 1, 128, 32768, 64, "e4m3", "bf16", [32768], False, False, 1024),
    (1, 40, 1, 2, 128, 768, 64, "int8", "bf16", [700], True, True, 9),         # 80 rows: five row groups
]


@pytest.mark.parametrize("B,Hq,Hkv,Lq,D,capacity,block,codes,dtype,lengths,causal,weights,ctas", CASES)
def test_against_oracle(B, Hq, Hkv, Lq, D, capacity, block, codes, dtype, lengths, causal, weights, ctas):
    run(B, Hq, Hkv, Lq, D, capacity, block, codes, dtype, lengths, causal, weights, ctas, seed=capacity + D)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("codes", ["int8", "e4m3"])
def test_no_kv_len_and_uneven_scales(D, codes):
    """The whole capacity, scales spread over 2^12, peaked attention."""
    run(1, 8, 2, 1, D, 768, 16, codes, "bf16", [768], weights=True, q_mult=4.0, scale_span=12.0, seed=D, full=True)


def test_workload_sizes():
    """The decode workloads' sizes over the 8-bit cache."""
    run(1, 32, 8, 4, 128, 32768, 64, "int8", "bf16", [32768], causal=True, weights=True, seed=1)
    run(1, 16, 4, 1, 256, 16384, 128, "e4m3", "bf16", [16001], seed=2)


@pytest.mark.parametrize("D", [64, 128])
def test_silent_values_under_strong_logits(D):
    """A block of zero values (scale 0) with logits hundreds of log2 units above
    the rest, before and behind blocks with values: the output is 0, not NaN."""
    B, Hkv, capacity, block = 1, 1, 512, 16
    for strong in (0, 8, 15, 31):
        cache = filled_cache(B, Hkv, capacity, D, block, "int8", [capacity], seed=3)
        q = torch.ones(B, 2, 1, D, dtype=torch.bfloat16, device="cuda")
        cache.k.fill_(-100)
        cache.k_scale.fill_(1.0)
        cache.k[:, :, strong * 16: strong * 16 + 16] = 100
        cache.v[:, :, strong * 16: strong * 16 + 16] = 0
        cache.v_scale[:, :, strong] = 0.0
        for ctas in (1, 2):
            out, lse = skv.attn_splitkv_decode_kv8(q, cache, 1.0, num_ctas=ctas)
            want = D * 100.0 * np.log2(np.e) + 4.0
            assert torch.all(out == 0), out.abs().max()
            assert np.all(np.abs(O.to_f64(lse) - want) <= 2.0 ** -22 * want + 2.0 ** -17)


@pytest.mark.parametrize("where", ["k_scale", "v_scale"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_scales_reach_only_rows_that_see_them(where, bad):
    """A non-finite scale (codes 0, as the append leaves them) makes the rows that
    see its block NaN; rows of other heads, and causal rows that end before the
    block, keep their values."""
    B, Hq, Hkv, Lq, D, capacity, block, n = 1, 4, 2, 4, 128, 512, 16, 323
    cache = filled_cache(B, Hkv, capacity, D, block, "int8", [n], seed=9)
    q = torch.randn(B, Hq, Lq, D, generator=gen(2)).bfloat16().cuda()
    ref, lref = skv.attn_splitkv_decode_kv8(q, cache, kv_len=i32([n]), causal=True)
    getattr(cache, where)[0, 0, 20] = bad            # keys 320..322 of head 0: rows 1..3 see some of them
    (cache.k if where == "k_scale" else cache.v)[0, 0, 320:336] = 0
    for ctas in (1, 2):
        out, lse = skv.attn_splitkv_decode_kv8(q, cache, kv_len=i32([n]), causal=True, num_ctas=ctas)
        assert torch.isnan(out[:, :2, 1:]).all()
        assert torch.isnan(lse[:, :2, 1:]).all() or where == "v_scale"
        assert torch.isfinite(out[:, :2, 0]).all() and torch.isfinite(out[:, 2:]).all()
        assert (out[:, 2:].float() - ref[:, 2:].float()).abs().max() <= 2.0 ** -6 * ref.float().abs().max()
        assert (out[:, :2, 0].float() - ref[:, :2, 0].float()).abs().max() <= 2.0 ** -6 * ref.float().abs().max()


def test_bad_queries_give_nan():
    cache = filled_cache(1, 1, 512, 64, 16, "int8", [512], seed=1)
    q = torch.ones(1, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[0, 1, 0, 5] = float("nan")
    for ctas in (1, 2):
        out, lse = skv.attn_splitkv_decode_kv8(q, cache, num_ctas=ctas)
        assert torch.isfinite(out[0, 0]).all() and torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1]).all()


@pytest.mark.parametrize("mult", [2.0 ** -100, 2.0 ** -14, 2.0 ** 10, 2.0 ** 60])
def test_query_size_is_immaterial_to_the_products(mult):
    """q scaled by a power of two against the logit scale's inverse gives the same logits."""
    cache = filled_cache(1, 2, 512, 128, 64, "int8", [500], seed=5)
    q = torch.randn(1, 4, 1, 128, generator=gen(6)).bfloat16().cuda()
    base, bl = skv.attn_splitkv_decode_kv8(q, cache, 0.1, kv_len=i32([500]))
    out, lse = skv.attn_splitkv_decode_kv8(q * mult, cache, 0.1 / mult, kv_len=i32([500]))
    # the two products that scale a logit round once more or less: 2^-22 of its size
    assert (lse - bl).abs().max() <= 2.0 ** -17 * (1 + bl.abs().max())
    assert (out.float() - base.float()).abs().max() <= 2.0 ** -7 * base.float().abs().max()


def test_weights_are_added_and_the_rest_left():
    """Two calls add twice; entries behind kv_len keep their bits; the LSE is not
    needed by the caller; two runs are bit-equal."""
    B, Hq, Hkv, D, capacity, lengths = 2, 4, 2, 64, 192, [100, 0]
    cache = filled_cache(B, Hkv, capacity, D, 32, "e4m3", lengths, seed=4)
    q = torch.randn(B, Hq, 3, D, generator=gen(7)).half().cuda()
    w = torch.full((B, Hkv, capacity), float("nan"), device="cuda")
    w[0, :, :100] = 0.25
    for _ in range(2):
        out, lse = skv.attn_splitkv_decode_kv8(q, cache, kv_len=i32(lengths), weights=w, return_lse=False)
        assert lse is None
    once = torch.zeros_like(w)
    _, lse = skv.attn_splitkv_decode_kv8(q, cache, kv_len=i32(lengths), weights=once)
    again = torch.zeros_like(w)
    out2, lse2 = skv.attn_splitkv_decode_kv8(q, cache, kv_len=i32(lengths), weights=again)
    assert torch.equal(once, again) and torch.equal(lse, lse2) and torch.equal(out, out2)
    assert torch.isnan(w[0, :, 100:]).all() and torch.isnan(w[1]).all()
    assert torch.equal(w[0, :, :100], 0.25 + once[0, :, :100] + once[0, :, :100])
    # each row's weights sum to 1: 2 rows of heads x 3 queries a kv head, 100 terms of 2^-20 relative
    assert (once[0].double().sum(-1) - 6.0).abs().max() <= 6 * 2.0 ** -16
    assert torch.all(once[0, :, 100:] == 0) and torch.all(once[1] == 0)


def test_graphs_follow_kv_len_and_contents():
    """Two captured decodes with workspaces of their own over one cache, replayed
    in turn with a new q and kv_len."""
    B, Hq, Hkv, D, capacity = 2, 8, 2, 128, 1024
    cache = filled_cache(B, Hkv, capacity, D, 64, "int8", [capacity] * B, seed=8)
    q = torch.zeros(B, Hq, 1, D, dtype=torch.bfloat16, device="cuda")
    kv_len = i32([5, 5])
    nc = skv.attn_splitkv_kv8_plan(B, Hq, Hkv, 1, capacity, D)
    nbytes = skv.attn_splitkv_kv8_workspace(B, Hq, Hkv, 1, capacity, D, nc, True)
    sets = []
    for _ in range(2):
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        w = torch.zeros(B, Hkv, capacity, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(B, Hq, 1, device="cuda")
        call = lambda ws=ws, w=w, out=out, lse=lse: skv.attn_splitkv_decode_kv8(  # noqa: E731
            q, cache, kv_len=kv_len, weights=w, out=out, lse=lse, workspace=ws, num_ctas=nc)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        sets.append((graph, w, out, lse))
    for i, lengths in enumerate([[1024, 1], [300, 777]]):
        q.copy_(torch.randn(B, Hq, 1, D, generator=gen(20 + i)))
        kv_len.copy_(i32(lengths))
        for graph, w, out, lse in sets:
            w.zero_()
        for graph, *_ in sets:
            graph.replay()
        torch.cuda.synchronize()
        for _, w, out, lse in sets:
            check(q, cache, out, lse, lengths, D ** -0.5, False, "bf16", O.to_f64(w))
    assert skv.device_error() == 0


def test_inputs_written_just_before():
    """q, the cache and kv_len written by kernels right before the call, on a side
    stream (the call's kernels may start early but wait before they read)."""
    B, Hq, Hkv, D, capacity, lengths = 1, 8, 2, 128, 2048, [2000]
    src = filled_cache(B, Hkv, capacity, D, 64, "int8", lengths, seed=11)
    dst = skv.kv8_cache(B, Hkv, capacity, D, 64, "int8")
    q0 = torch.randn(B, Hq, 1, D, generator=gen(1)).bfloat16().cuda()
    q, kl, w = torch.empty_like(q0), i32([0]), torch.empty(B, Hkv, capacity, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(3):
            for a, b in zip(dst, src):
                a.view(torch.uint8 if a.dtype != torch.float32 else torch.float32).copy_(
                    b.view(torch.uint8 if b.dtype != torch.float32 else torch.float32))
            q.copy_(q0)
            kl.fill_(2000)
            w.zero_()
            out, lse = skv.attn_splitkv_decode_kv8(q, dst, kv_len=kl, weights=w)
    s.synchronize()
    check(q, src, out, lse, lengths, D ** -0.5, False, "bf16", O.to_f64(w))


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
@pytest.mark.parametrize("G,Lq,D,n,causal,q_mult", [(1, 1, 64, 5000, False, 1.0), (4, 4, 128, 2000, True, 1.0),
                                                    (1, 1, 128, 3001, False, 4.0), (8, 3, 64, 1000, False, 0.2),
                                                    (4, 1, 256, 1500, False, 1.0)])
def test_fp16_output_is_as_exact_as_its_rounding(codes, G, Lq, D, n, causal, q_mult):
    """The rms error of an fp16 output is at most 1.1 times that of the oracle's O
    rounded to fp16.  Rounding alone gives at least 2^-11 / sqrt(12) = 1.4e-4 of
    |O|, so what the kernel may add to it is sqrt(1.1^2 - 1) * 1.4e-4 = 6.4e-5.  It
    adds the weights' own error, 2^-22, and that of their exponents: fp32 sums of
    D / 16 MMA steps are off by (D / 16) 2^-23 scale log2(e) sum |q k| ln 2 at
    most, where |q| is 0.8 q_mult and |k| at most 1 (127 / 2 / 64) on average: 3e-6
    at D = 64, 9e-6 at D = 128 (3.5e-5 with q_mult = 4), 2.4e-5 at D = 256.  Weights
    rounded to fp16 once add 1.4e-4 or more."""
    B, Hkv = 4, 8
    capacity = -(-n // 64) * 64
    cache = filled_cache(B, Hkv, capacity, D, 64, codes, [n] * B, seed=7, scale_span=0.0)
    q = (q_mult * torch.randn(B, G * Hkv, Lq, D, generator=gen(8))).half().cuda()
    out, _ = skv.attn_splitkv_decode_kv8(q, cache, kv_len=i32([n] * B), causal=causal)
    k, v = values(cache.k, cache.k_scale, [n] * B), values(cache.v, cache.v_scale, [n] * B)
    ref, _ = O.decode(q, k, v, D ** -0.5, kv_len=[n] * B, causal=causal)
    rounded = torch.from_numpy(ref).half().double().numpy()
    rms = lambda x: np.sqrt(np.mean(x * x))  # noqa: E731
    assert rms(O.to_f64(out) - ref) <= 1.1 * rms(rounded - ref)
