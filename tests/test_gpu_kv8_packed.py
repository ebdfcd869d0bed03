"""kv8_append of packed (TND) rows as a captured step makes it: a fixed number of rows
and a fixed bound of the lengths, cu_seqlens changing from replay to replay."""
import numpy as np
import pytest
import torch

import split_kv_merge_attn_b200 as skv
from tests._kv8_helpers import filled_cache, gen, i32
from tests.test_gpu_kv8 import assert_cache, expect_append, snapshot

pytestmark = pytest.mark.gpu

B, H, D, BLOCK, CAP, T = 3, 2, 64, 32, 160, 40


def padded(rows, lens):
    cu = np.concatenate(([0], np.cumsum(lens)))
    out = []
    for x in rows:
        p = torch.zeros(B, H, max(max(lens), 1), D, dtype=x.dtype)
        for b in range(B):
            p[b, :, : lens[b]] = x[cu[b]: cu[b + 1]].cpu().permute(1, 0, 2)
        out.append(p)
    return out, cu.tolist()


@pytest.mark.parametrize("bound", [T, T + 1, 1000, 2 ** 31 - 1])
def test_any_bound_of_the_lengths(bound):
    """A bound above the number of rows is a bound all the same; rows behind the last
    sequence are not appended."""
    lens, starts = [7, 0, 30], [0, 9, 140]
    rows = [torch.randn(T, H, D, generator=gen(s)).bfloat16().cuda() for s in (1, 2)]
    cache = filled_cache(B, H, CAP, D, BLOCK, "int8", starts, seed=4)
    new, cu = padded(rows, lens)
    want = expect_append(snapshot(cache), new, starts, lens, BLOCK, "int8")
    skv.kv8_append(cache, *rows, i32(starts), layout="TND", cu_seqlens=i32(cu), max_seqlen=bound)
    assert_cache(cache, want)


def test_captured_with_a_bound():
    cache = filled_cache(B, H, CAP, D, BLOCK, "e4m3", [CAP] * B, seed=4)
    rows = [torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    start, cu = i32([0] * B), i32([0] * (B + 1))
    call = lambda: skv.kv8_append(cache, *rows, start, layout="TND", cu_seqlens=cu, max_seqlen=128)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed, (lens, starts) in enumerate([([40, 0, 0], [5, 5, 5]), ([1, 1, 38], [45, 0, 3]), ([0, 0, 0], [1, 2, 3])]):
        for r, x in enumerate(rows):
            x.copy_(torch.randn(T, H, D, generator=gen(10 * seed + r)))
        new, c = padded(rows, lens)
        cu.copy_(i32(c))
        start.copy_(i32(starts))
        want = expect_append(snapshot(cache), new, starts, lens, BLOCK, "e4m3")
        graph.replay()
        torch.cuda.synchronize()
        assert_cache(cache, want)


def test_refused_bounds():
    rows = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    cache = skv.kv8_cache(B, H, CAP, D, BLOCK)
    cu = i32([0, 1, 2, 3])
    for bad in (-1, 2 ** 31):
        with pytest.raises((ValueError, skv.SkvError)):
            skv.kv8_append(cache, rows, rows, i32([0] * B), layout="TND", cu_seqlens=cu, max_seqlen=bad)
