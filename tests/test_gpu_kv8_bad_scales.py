"""Non-finite scales in a cache whose codes the append did not write."""
import pytest
import torch

import split_kv_merge_attn_b200 as skv
from tests._kv8_helpers import DT, filled_cache, gen, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("where", ["k_scale", "v_scale"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D,G,Lq,dtype,codes", [(64, 2, 1, "bf16", "int8"), (128, 4, 4, "bf16", "e4m3"),
                                                (256, 1, 1, "fp16", "int8"), (64, 4, 4, "fp16", "e4m3")])
def test_rows_that_see_the_block_are_nan(where, bad, sign, D, G, Lq, dtype, codes):
    """All codes of the block are 3 or all -3, q is positive: the block's logits would
    be +inf or -inf, not only NaN.  Rows of the other heads and sequences keep their bits,
    and so do their weights.  Causal rows that end before the block may round elsewhere
    (a reference of the softmax moves for all rows of a unit at once): two values within
    a step of each other, LSEs within 2^-10 (twice 2^-18 y + 2^-17, y < 60)."""
    B, Hkv, capacity, block, n = 2, 2, 512, 16, 321
    cache = filled_cache(B, Hkv, capacity, D, block, codes, [n] * B, seed=9)
    q = (torch.rand(B, G * Hkv, Lq, D, generator=gen(2)) + 0.1).to(DT[dtype]).cuda()
    w = [torch.zeros(B, Hkv, capacity, device="cuda") for _ in range(2)]
    ref, lref = skv.attn_splitkv_decode_kv8(q, cache, kv_len=i32([n] * B), causal=True, weights=w[0], num_ctas=2)
    codes_t = cache.k if where == "k_scale" else cache.v
    codes_t[0, 0, 320:336] = torch.full((16, D), 3.0 * sign).to(codes_t.dtype).cuda()  # key 320: the last row's only
    getattr(cache, where)[0, 0, 20] = bad
    out, lse = skv.attn_splitkv_decode_kv8(q, cache, kv_len=i32([n] * B), causal=True, weights=w[1], num_ctas=2)
    seen = torch.zeros(B, G * Hkv, Lq, dtype=torch.bool)
    seen[0, :G, -1] = True
    assert torch.isnan(out[seen.cuda()]).all()
    for t, r in ((out, ref), (lse, lref)):
        assert torch.equal(t[0, G:], r[0, G:]) and torch.equal(t[1], r[1])
    before = (slice(0, 1), slice(0, G), slice(0, Lq - 1))
    assert ((out[before].float() - ref[before].float()).abs() <= 2.0 ** -6 * ref.float().abs().max()).all()
    assert ((lse[before] - lref[before]).abs() <= 2.0 ** -10).all()
    if where == "k_scale":
        assert torch.isnan(lse[seen.cuda()]).all() and torch.isnan(w[1][0, 0, :n]).all()
    assert torch.equal(w[1][0, 1], w[0][0, 1]) and torch.equal(w[1][1], w[0][1])
