"""kv8_evict bit-equal to its definition: kept positions, lengths, weights,
codes and scales; nothing else of the receiving cache touched."""
import numpy as np
import pytest
import torch

import oracle as O
import split_kv_merge_attn_b200 as skv
from tests._kv8_helpers import code_values, filled_cache, gen, i32, poisoned_cache

pytestmark = pytest.mark.gpu


def check(cache, weights, lengths, to_capacity, budget, sink, recent, kv_len="given"):
    B, H, capacity, D = cache.k.shape
    block = capacity // cache.k_scale.shape[2]
    codes = "int8" if cache.k.dtype == torch.int8 else "e4m3"
    to = poisoned_cache(B, H, to_capacity, D, block, codes)
    before = [code_values(to.k), code_values(to.v)]
    to_w = torch.full((B, H, to_capacity), -7.0, device="cuda")
    kept, new_len = skv.kv8_evict(cache, to, weights, to_w, i32(lengths) if kv_len == "given" else None, budget, sink,
                                  recent)
    torch.cuda.synchronize()
    assert new_len.tolist() == [min(n, budget) for n in lengths]
    w = weights.cpu()
    for b in range(B):
        for h in range(H):
            at = O.kv8_kept(w[b, h], lengths[b], budget, sink, recent)
            m = len(at)
            assert kept[b, h].tolist() == at.tolist() + [-1] * (budget - m)
            np.testing.assert_array_equal(to_w[b, h, :m].cpu().numpy(), w[b, h].numpy()[at])
            assert torch.all(to_w[b, h, m:] == -7.0)
            for src, s_src, dst, s_dst, old in ((cache.k, cache.k_scale, to.k, to.k_scale, before[0]),
                                                (cache.v, cache.v_scale, to.v, to.v_scale, before[1])):
                c, s = O.kv8_move(code_values(src[b, h]), s_src[b, h].cpu().numpy(), at, block, codes)
                np.testing.assert_array_equal(code_values(dst[b, h])[:m], c)
                np.testing.assert_array_equal(code_values(dst[b, h])[m:], old[b, h, m:])
                np.testing.assert_array_equal(s_dst[b, h].cpu().numpy()[: len(s)], s)
                assert torch.isnan(s_dst[b, h, len(s):]).all()
    return to, kept, new_len


def random_weights(B, H, capacity, seed):
    return torch.exp(2 * torch.randn(B, H, capacity, generator=gen(seed))).cuda()


CASES = [
    # B, H, D, block, codes, capacity, lengths, to_capacity, budget, sink, recent
    (1, 1, 64, 16, "int8", 32, [32], 16, 1, 0, 0),
    (1, 2, 128, 64, "e4m3", 256, [256], 128, 100, 4, 31),
    (4, 2, 128, 32, "int8", 512, [512, 100, 0, 101], 128, 100, 4, 32),      # at, below and above the budget
    (2, 1, 256, 128, "e4m3", 1024, [1000, 777], 512, 513 - 128, 0, 129),
    (2, 2, 64, 16, "int8", 2048, [2047, 64], 1024, 1000, 16, 0),
    (1, 1, 128, 64, "int8", 512, [500], 64, 64, 0, 64),                     # only the last ones
    (1, 1, 128, 64, "int8", 512, [500], 64, 64, 64, 0),                     # only the first ones
    (1, 1, 128, 64, "int8", 512, [500], 512, 499, 100, 100),                # one goes
    (1, 2, 64, 128, "e4m3", 9984, [9983, ], 1280, 1279, 5, 7),              # a cluster of four
]


@pytest.mark.parametrize("B,H,D,block,codes,capacity,lengths,to_capacity,budget,sink,recent", CASES)
def test_bit_exact(B, H, D, block, codes, capacity, lengths, to_capacity, budget, sink, recent):
    cache = filled_cache(B, H, capacity, D, block, codes, lengths, seed=budget, scale_span=4.0)
    check(cache, random_weights(B, H, capacity, budget), lengths, to_capacity, budget, sink, recent)


def test_long_head_and_no_kv_len():
    """A cluster of eight; kv_len None is the whole capacity."""
    cache = filled_cache(1, 1, 40960, 64, 64, "int8", [40960], seed=1, scale_span=2.0)
    check(cache, random_weights(1, 1, 40960, 3), [40960], 4096, 4001, 4, 256, kv_len=None)


@pytest.mark.parametrize("capacity", [256, 20480])
def test_ties_go_to_the_lowest_position(capacity):
    cache = filled_cache(1, 2, capacity, 64, 16, "int8", [capacity], seed=2)
    w = torch.randint(0, 3, (1, 2, capacity), generator=gen(1)).float().cuda()
    w[0, 1] = 1.0  # all equal
    check(cache, w, [capacity], 128, 100, 3, 5)


def test_special_weights():
    """-0 equals +0, infinities order, NaN comes last, negative weights order."""
    capacity = 256
    cache = filled_cache(1, 1, capacity, 64, 16, "int8", [capacity], seed=3)
    w = torch.randn(1, 1, capacity, generator=gen(4))
    w[..., ::7], w[..., 1::7], w[..., 2::14], w[..., 3::21] = 0.0, -0.0, float("nan"), float("-inf")
    w[..., 5::50] = float("inf")
    for budget in (3, 60, 110, 150, 250):
        check(cache, w.cuda(), [capacity], 256, budget, 0, 0)
    check(cache, torch.full_like(w, float("nan")).cuda(), [capacity], 256, 100, 10, 10)


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
def test_bad_and_empty_scales(codes):
    """Blocks with scale 0 join others; a non-finite scale makes its new block
    non-finite with codes 0 and no other."""
    capacity, block = 256, 16
    cache = filled_cache(1, 1, capacity, 64, block, codes, [capacity], seed=6)
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        for blk, value in ((1, 0.0), (5, float("nan")), (9, float("inf"))):
            s[..., blk] = value
            t.view(torch.int8)[:, :, blk * block: blk * block + block] = 0
    check(cache, random_weights(1, 1, capacity, 8), [capacity], 128, 128, 20, 30)


def test_graph_follows_kv_len():
    cache = filled_cache(2, 2, 512, 128, 64, "int8", [512, 512], seed=7)
    to = poisoned_cache(2, 2, 128, 128, 64, "int8")
    w, to_w, kv_len = random_weights(2, 2, 512, 1), torch.zeros(2, 2, 128, device="cuda"), i32([512, 512])
    kept, new_len = torch.zeros(2, 2, 100, dtype=torch.int32, device="cuda"), i32([0, 0])
    call = lambda: skv.kv8_evict(cache, to, w, to_w, kv_len, 100, 2, 10, kept=kept, new_len=new_len)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lengths in ([300, 99], [101, 512]):
        kv_len.copy_(i32(lengths))
        w.copy_(random_weights(2, 2, 512, lengths[0]))
        graph.replay()
        torch.cuda.synchronize()
        assert new_len.tolist() == [min(n, 100) for n in lengths]
        for b in range(2):
            for h in range(2):
                at = O.kv8_kept(w[b, h].cpu(), lengths[b], 100, 2, 10).tolist()
                assert kept[b, h].tolist() == at + [-1] * (100 - len(at))
