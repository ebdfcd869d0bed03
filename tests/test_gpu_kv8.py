"""kv8_append and kv8_fetch: codes and scales bit-equal to the fp32 definition
(oracle.kv8_append), and every byte that a call has no business with unchanged."""
import numpy as np
import pytest
import torch

import oracle as O
import split_kv_merge_attn_b200 as skv
from tests._kv8_helpers import DT, code_values, filled_cache, gen, i32, poisoned_cache

pytestmark = pytest.mark.gpu


def new_tokens(layout, B, S, H, D, dtype, seed, mult=1.0):
    g = gen(seed)
    x = [torch.randn(B, H, S, D, generator=g) * mult * (1 + torch.rand(B, H, S, 1, generator=g) * 3) for _ in range(2)]
    return [t.to(DT[dtype]) for t in x]


def laid_out(x, layout):
    return (x if layout == "HND" else x.permute(0, 2, 1, 3)).contiguous().cuda()


def expect_append(cache_before, new, starts, counts, block, codes):
    """The cache's codes (values) and scales after the append, by the oracle."""
    out = []
    for codes_t, scale_t, x in zip(cache_before[:2], cache_before[2:], new):
        c, s = codes_t.copy(), scale_t.copy()
        for b in range(c.shape[0]):
            for h in range(c.shape[1]):
                O.kv8_append(c[b, h], s[b, h], x[b, h], starts[b], counts[b], block, codes)
        out.append((c, s))
    return out


def snapshot(cache):
    return [code_values(cache.k), code_values(cache.v), cache.k_scale.cpu().numpy(), cache.v_scale.cpu().numpy()]


def assert_cache(cache, want):
    got = snapshot(cache)
    for c, s, (wc, wsc) in zip(got[:2], got[2:], want):
        np.testing.assert_array_equal(s, wsc)
        np.testing.assert_array_equal(c, wc)


CASES = [
    # codes, dtype, layout, B, H, D, block, capacity, S, starts, counts
    ("int8", "bf16", "HND", 1, 1, 64, 16, 16, 1, [0], [1]),
    ("int8", "bf16", "HND", 3, 2, 128, 64, 256, 1, [0, 63, 100], [1, 1, 1]),
    ("e4m3", "fp16", "NHD", 2, 3, 128, 32, 384, 130, [0, 17], [130, 130]),
    ("int8", "fp16", "NHD", 4, 2, 256, 128, 512, 200, [0, 5, 128, 400], [200, 0, 131, 200]),   # the last overruns
    ("e4m3", "bf16", "HND", 2, 1, 64, 16, 304, 77, [300, 11], [77, 76]),
    ("int8", "bf16", "HND", 2, 2, 64, 128, 1280, 1001, [1, 127], [1001, 999]),
    ("e4m3", "bf16", "NHD", 1, 2, 256, 64, 640, 513, [64], [513]),
]


@pytest.mark.parametrize("codes,dtype,layout,B,H,D,block,capacity,S,starts,counts", CASES)
def test_append_bit_exact(codes, dtype, layout, B, H, D, block, capacity, S, starts, counts):
    cache = filled_cache(B, H, capacity, D, block, codes, starts, seed=S + D, scale_span=4.0)
    new = new_tokens(layout, B, S, H, D, dtype, seed=S)
    want = expect_append(snapshot(cache), new, starts, counts, block, codes)
    k, v = (laid_out(x, layout) for x in new)
    num = None if all(c == S for c in counts) else i32(counts)
    got = skv.kv8_append(cache, k, v, i32(starts), num_new=num, layout=layout)
    assert got is cache
    assert_cache(cache, want)
    # once more: the same tokens leave the same bytes
    skv.kv8_append(cache, k, v, i32(starts), num_new=num, layout=layout)
    assert_cache(cache, want)


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
def test_append_token_by_token(codes):
    """Forty tokens one at a time, their sizes growing and shrinking: every step
    re-scales its block as the definition says."""
    B, H, D, block = 2, 2, 64, 16
    cache = poisoned_cache(B, H, 64, D, block, codes)
    want = snapshot(cache)
    want = list(zip(want[:2], want[2:]))
    start = i32([0, 7])
    for i in range(40):
        new = new_tokens("HND", B, 1, H, D, "bf16", seed=i, mult=2.0 ** ((i * 7) % 9 - 4))
        skv.kv8_append(cache, new[0].cuda(), new[1].cuda(), start)
        before = [c for c, _ in want] + [s for _, s in want]
        want = expect_append(before, new, [i, 7 + i], [1, 1], block, codes)
        start += 1
    assert_cache(cache, want)


def test_append_packed():
    """TND rows with cu_seqlens, one sequence empty."""
    B, H, D, block, capacity = 4, 2, 128, 32, 192
    lens, starts = [3, 0, 100, 50], [0, 9, 40, 180]
    g = gen(3)
    rows = [torch.randn(sum(lens), H, D, generator=g).bfloat16() for _ in range(2)]
    cu = np.concatenate(([0], np.cumsum(lens)))
    cache = filled_cache(B, H, capacity, D, block, "int8", starts, seed=4)
    padded = []
    for x in rows:
        p = torch.zeros(B, H, max(lens), D, dtype=x.dtype)
        for b in range(B):
            p[b, :, : lens[b]] = x[cu[b]: cu[b + 1]].permute(1, 0, 2)
        padded.append(p)
    want = expect_append(snapshot(cache), padded, starts, lens, block, "int8")
    skv.kv8_append(cache, rows[0].cuda(), rows[1].cuda(), i32(starts), layout="TND", cu_seqlens=i32(cu.tolist()),
                   max_seqlen=max(lens))
    assert_cache(cache, want)


def test_append_clamps_what_the_device_reads():
    """Positions and counts outside their ranges touch nothing out of range: a
    negative start is 0, a start behind the capacity appends nothing, a negative
    count appends nothing, a count above S is S."""
    B, H, D, block, capacity, S = 4, 1, 64, 16, 64, 20
    cache = filled_cache(B, H, capacity, D, block, "int8", [0, 0, 8, 8], seed=1)
    new = new_tokens("HND", B, S, H, D, "bf16", seed=2)
    want = expect_append(snapshot(cache), new, [0, capacity, 8, 8], [S, S, 0, S], block, "int8")
    skv.kv8_append(cache, new[0].cuda(), new[1].cuda(), i32([-3, 1000, 8, 8]), num_new=i32([S, S, -1, 99]))
    assert_cache(cache, want)


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_extreme_values(codes, dtype):
    """Zeros, the type's largest and smallest values, and infinities or NaN, each
    in a block of its own: only the last two blocks lose their values."""
    D, block = 64, 16
    big, small = torch.finfo(DT[dtype]).max, torch.finfo(DT[dtype]).smallest_normal
    x = torch.randn(1, 1, 7 * block, D, generator=gen(0))
    x = x.to(DT[dtype])
    x[:, :, :16] = 0
    x[:, :, 16:32] = 0
    x[:, :, 20, 3] = small
    x[:, :, 33, 5] = big
    x[:, :, 50, 7] = -big
    x[:, :, 70, 1] = float("inf")
    x[:, :, 90, 63] = float("nan")
    cache = poisoned_cache(1, 1, 7 * block, D, block, codes)
    want = expect_append(snapshot(cache), [x, -x], [0], [7 * block], block, codes)
    skv.kv8_append(cache, x.cuda(), (-x).cuda(), i32([0]))
    assert_cache(cache, want)
    k, v = skv.kv8_fetch(cache, 7 * block, DT[dtype])
    bad = torch.isnan(k.cpu()).all(-1)[0, 0]
    assert bad.tolist() == [64 <= j < 96 for j in range(7 * block)]
    assert torch.equal(torch.isnan(v), torch.isnan(k))
    # a bad value behind good ones takes its block's older tokens along, and only them
    y = torch.ones(1, 1, 1, D, dtype=DT[dtype])
    y[..., 0] = float("nan")
    skv.kv8_append(cache, y.cuda(), y.cuda(), i32([40]))
    k, _ = skv.kv8_fetch(cache, 7 * block, DT[dtype])
    bad = torch.isnan(k.cpu()).all(-1)[0, 0]
    assert bad.tolist() == [32 <= j < 48 or 64 <= j < 96 for j in range(7 * block)]


@pytest.mark.parametrize("codes,dtype,layout,D", [("int8", "bf16", "HND", 64), ("e4m3", "fp16", "NHD", 128),
                                                  ("int8", "fp16", "NHD", 256), ("e4m3", "bf16", "HND", 256)])
def test_fetch_bit_exact(codes, dtype, layout, D):
    B, H, block, capacity, n = 3, 2, 32, 160, 45
    lengths = [160, 33, 0]
    cache = filled_cache(B, H, capacity, D, block, codes, lengths, seed=D)
    start = [130, 0, 5]
    shape = (B, H, n, D) if layout == "HND" else (B, n, H, D)
    ko, vo = (torch.full(shape, float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
    k, v = skv.kv8_fetch(cache, n, start=i32(start), kv_len=i32(lengths), layout=layout, k_out=ko, v_out=vo)
    assert k is ko and v is vo
    for got, codes_t, scale_t in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        got = got.cpu() if layout == "HND" else got.cpu().permute(0, 2, 1, 3)
        x = codes_t.cpu().float() * scale_t.cpu().repeat_interleave(block, 2)[..., None]
        for b in range(B):
            live = max(0, min(start[b] + n, lengths[b]) - start[b])
            assert torch.equal(got[b, :, :live], x[b, :, start[b]: start[b] + live].to(DT[dtype]))
            assert torch.all(got[b, :, live:] == 0)


def test_fetch_outside_the_cache():
    cache = filled_cache(2, 1, 32, 64, 16, "int8", [32, 32], seed=0)
    k, _ = skv.kv8_fetch(cache, 8, torch.bfloat16, start=i32([-4, 2 ** 31 - 4]))
    assert torch.all(k[0, :, :4] == 0) and torch.all(k[0, :, 4:].abs().sum(-1) > 0) and torch.all(k[1] == 0)
    k, v = skv.kv8_fetch(cache, 0, torch.bfloat16)
    assert k.shape == (2, 1, 0, 64) and v.shape == k.shape


def test_append_in_a_graph_follows_its_start():
    """A captured one-token append, replayed with new contents and a start the
    graph reads on the device."""
    B, H, D, block = 2, 2, 128, 32
    cache = poisoned_cache(B, H, 96, D, block, "int8")
    want = snapshot(cache)
    want = list(zip(want[:2], want[2:]))
    k, v = (torch.zeros(B, H, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    start = i32([0, 30])
    skv.kv8_append(poisoned_cache(B, H, 96, D, block, "int8"), k, v, start)  # warm-up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        skv.kv8_append(cache, k, v, start)
    for i in range(5):
        new = new_tokens("HND", B, 1, H, D, "bf16", seed=100 + i)
        k.copy_(new[0])
        v.copy_(new[1])
        start.copy_(i32([i, 30 + i]))
        graph.replay()
        before = [c for c, _ in want] + [s for _, s in want]
        want = expect_append(before, new, [i, 30 + i], [1, 1], block, "int8")
    torch.cuda.synchronize()
    assert_cache(cache, want)
