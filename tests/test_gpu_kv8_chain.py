"""The operators together, as a serving loop uses them: rotary positions, a
prompt appended to the 8-bit cache, decode steps that gather weights, eviction,
and decoding on; then attention over the cached prefix through attn_fwd_lse."""
import os

import numpy as np
import pytest
import torch

import oracle as O
import split_kv_merge_attn_b200 as skv
from tests._gpu_helpers import check_lse, check_o, vmax
from tests._kv8_helpers import gen, i32, values
from tests.test_gpu_kv8_decode import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
def test_serving_loop(codes):
    B, Hq, Hkv, D, block, capacity, budget = 2, 8, 2, 128, 32, 512, 128
    g = gen(1)
    prompt = [200, 77]
    S = max(prompt)
    inv_freq, factor = skv.rope_inv_freq(64, scaling="yarn", factor=4.0, original_len=128)
    cache = skv.kv8_cache(B, Hkv, capacity, D, block, codes)
    small = skv.kv8_cache(B, Hkv, budget, D, block, codes)
    weights, small_w = torch.zeros(B, Hkv, capacity, device="cuda"), torch.zeros(B, Hkv, budget, device="cuda")
    length = i32([0, 0])

    # ---- the prompt, token-major as projections leave it
    q, k, v = (torch.randn(B, S, H, D, generator=g).bfloat16().cuda() for H in (Hq, Hkv, Hkv))
    pos = torch.arange(S, dtype=torch.int32, device="cuda").expand(B, S).contiguous()
    q, k = skv.rope_apply(q, k, pos, inv_freq, layout="NHD", factor=factor, q_out=q, k_out=k)
    skv.kv8_append(cache, k, v, length, num_new=i32(prompt), layout="NHD")
    length += i32(prompt)
    # the cache holds the keys to half a code step of their block's scale (e4m3:
    # 2^-4 of the value, or half of 2^-9 scales).  The scaled value that is rounded
    # to a code carries three fp32 roundings (s, 1 / s, the product): of at most
    # 127 codes, 127 * 3 * 2^-24 < 2^-15 codes, i.e. 2^-14 of the half step.
    for b in range(B):
        n = prompt[b]
        held = values(cache.k, cache.k_scale, prompt)[b, :, :n]
        want = O.to_f64(k)[b, :n].transpose(1, 0, 2)
        s = np.repeat(cache.k_scale[b].cpu().double().numpy(), block, -1)[:, :n, None]
        step = 0.5 * s if codes == "int8" else np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s)
        assert np.all(np.abs(held - want) <= step * (1 + 2.0 ** -14))

    # ---- decode steps
    def step(cache, weights, length, at):
        q, k, v = (torch.randn(B, H, 1, D, generator=g).bfloat16().cuda() for H in (Hq, Hkv, Hkv))
        q, k = skv.rope_apply(q, k, at.view(B, 1), inv_freq, factor=factor)
        skv.kv8_append(cache, k, v, length)
        length += 1
        before = weights.clone()
        out, lse = skv.attn_splitkv_decode_kv8(q, cache, kv_len=length, weights=weights)
        n = length.tolist()
        check(q, cache, out, lse, n, D ** -0.5, False, "bf16")
        for b in range(B):  # what this step added is each key's weight
            added = (weights - before)[b, :, : n[b]].double().sum(-1).cpu().numpy()
            assert np.all(np.abs(added - Hq // Hkv) <= 2.0 ** -14)
            assert torch.equal(weights[b, :, n[b]:], before[b, :, n[b]:])
        return out

    position = i32(prompt)
    for _ in range(5):
        step(cache, weights, length, position)
        position = position + 1

    # ---- eviction: 4 sinks, the last 32, the heaviest between; one sequence is short enough to stay
    n = length.tolist()
    kept, length = skv.kv8_evict(cache, small, weights, small_w, length, budget - 32, sink=4, recent=32)
    assert length.tolist() == [min(x, budget - 32) for x in n]
    for b in range(B):
        for h in range(Hkv):
            at = O.kv8_kept(weights[b, h].cpu(), n[b], budget - 32, 4, 32)
            assert kept[b, h, : len(at)].tolist() == at.tolist()
    # decoding goes on at the old positions over the smaller cache
    for _ in range(5):
        step(small, small_w, length, position)
        position = position + 1
    torch.cuda.synchronize()
    assert skv.device_error() == 0


def test_prefill_over_a_cached_prefix():
    """A prefix read back from the cache in 16 bits joins new keys by merge_state."""
    B, Hq, Hkv, D, n, S = 1, 4, 2, 128, 300, 96
    g = gen(2)
    cache = skv.kv8_cache(B, Hkv, 384, D, 64, "int8")
    k0, v0 = (torch.randn(B, Hkv, n, D, generator=g).bfloat16().cuda() for _ in range(2))
    skv.kv8_append(cache, k0, v0, i32([0]))
    q = torch.randn(B, Hq, S, D, generator=g).bfloat16().cuda()
    k1, v1 = (torch.randn(B, Hkv, S, D, generator=g).bfloat16().cuda() for _ in range(2))
    k, v = skv.kv8_fetch(cache, n, torch.bfloat16, kv_len=i32([n]))
    parts = [skv.attn_fwd_lse(q, k, v), skv.attn_fwd_lse(q, k1, v1, causal=True)]
    out, lse = skv.merge_state(torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]))
    o_ref, l_ref = O.dense(q, torch.cat((k, k1), 2), torch.cat((v, v1), 2), D ** -0.5, causal=True)
    check_o(out, o_ref, vmax(torch.cat((v, v1), 2)))
    check_lse(lse, l_ref)


def test_readme_step_runs():
    """The step of a serving loop shown in README.md, as it stands there."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    code = open(path).read().split("```python\n")[1].split("```")[0]
    env = {}
    exec(code, env)
    g = torch.Generator().manual_seed(3)
    for i in range(40):
        q, k, v = (torch.randn(4, h, 1, 128, generator=g).bfloat16().cuda() for h in (32, 8, 8))
        out, lse = env["step"](q, k, v)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        if i == 29:
            env["shrink"](280)  # nothing to cut yet: all 30 move
            assert env["length"].tolist() == [30] * 4
    # every row's weights sum to 1: 4 rows a kv head, 40 steps, none lost with all tokens
    # kept.  Relative error 2 ln 2 (2^-18 y + 2^-17), y <= 128^-0.5 log2(e) max|q| sum|k|
    # with max|q| < 5 and |k| 0.8 on average: y < 66, 3.6e-4
    total = env["weights"].sum(-1)
    assert torch.allclose(total, torch.full_like(total, 160.0), rtol=3.6e-4)


def test_a_cache_beyond_32_bit_offsets():
    """Three heads of 2^23 tokens of 256 codes: byte offsets above 2^32, within and
    between heads.  K scales of 0 make every logit 0, so LSE = log2 n, O the mean of V
    and each weight G / n; V scales are 0 but for the last block.  An O is off by half a
    bf16 step and 2^-10 of sum p |v| (2^-11 of a weight's fp16 rounding, as much again
    for fp32 sums and the merge); LSE by 2^-17, weights by twice that (relative)."""
    H, G, n, D, block = 3, 2, 1 << 23, 256, 64
    cache = skv.kv8_cache(1, H, n, D, block)  # int8: any byte is a finite code
    cache.k_scale.zero_()
    cache.v_scale.zero_()
    g = gen(2)
    k, v = (torch.randn(1, H, 100, D, generator=g).bfloat16().cuda() for _ in range(2))
    small = skv.kv8_cache(1, H, 128, D, block)
    small.k_scale.zero_()
    small.v_scale.zero_()
    skv.kv8_append(cache, k, v, i32([n - 100]))
    skv.kv8_append(small, k, v, i32([28]))
    for t, s in zip(cache, small):  # the same blocks, seen from the end
        assert torch.equal(t[:, :, t.shape[2] - (100 if t.dtype == torch.int8 else 2):],
                           s[:, :, 28 if t.dtype == torch.int8 else 0:])
    far, near = (skv.kv8_fetch(c, 100, start=i32([at])) for c, at in ((cache, n - 100), (small, 28)))
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])

    cache.k_scale.zero_()
    cache.v_scale[:, :, :-1] = 0
    cache.v_scale[:, :, -1] = n / 1024
    q = torch.randn(1, G * H, 1, D, generator=g).bfloat16().cuda()
    weights = torch.zeros(1, H, n, device="cuda")
    out, lse = skv.attn_splitkv_decode_kv8(q, cache, weights=weights)
    want = cache.v[:, :, -block:].double().sum(2) / 1024
    size = cache.v[:, :, -block:].double().abs().sum(2) / 1024
    off = (out[:, :, 0].view(1, H, G, D).double() - want[:, :, None]).abs()
    assert (off <= 2.0 ** -8 * want.abs()[:, :, None] + 2.0 ** -10 * size[:, :, None]).all()
    assert (lse - 23).abs().max() <= 2.0 ** -17
    assert (weights * (n / G) - 1).abs().max() <= 2.0 ** -16

    cache.k_scale.fill_(0.5)
    cache.v_scale.fill_(0.25)
    weights.zero_()
    weights[:, :, n - 600 : n - 100] = 1 + torch.rand(1, H, 500, generator=g).cuda()
    to, to_weights = skv.kv8_cache(1, H, 512, D, block), torch.zeros(1, H, 512, device="cuda")
    kept, new_len = skv.kv8_evict(cache, to, weights, to_weights, None, 500, sink=3, recent=100)
    assert new_len.tolist() == [500]
    for h in range(H):
        w = weights[0, h, n - 600 : n - 100].tolist()
        order = sorted(range(500), key=lambda j: (-w[j], j))[:397]
        at = [0, 1, 2] + sorted(n - 600 + j for j in order) + list(range(n - 100, n))
        assert kept[0, h].tolist() == at
        at = torch.tensor(at, device="cuda")
        assert torch.equal(to.k[0, h, :500], cache.k[0, h, at]) and torch.equal(to.v[0, h, :500], cache.v[0, h, at])
        assert torch.equal(to_weights[0, h, :500], weights[0, h, at])
