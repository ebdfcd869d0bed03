"""Keys far into a cache: decode and eviction that read the right codes and the right
scales behind 32-bit offsets, where blocks all differ."""
import numpy as np
import pytest
import torch

import oracle as O
import split_kv_merge_attn_b200 as skv
from tests._kv8_helpers import code_values, gen

pytestmark = pytest.mark.gpu

H, G, N, D, BLOCK = 3, 2, 1 << 23, 256, 64  # heads of 2^31 bytes of codes each


@pytest.fixture(scope="module")
def cache():
    c = skv.kv8_cache(1, H, N, D, BLOCK)
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (c.k, c.v):
        t.random_(-127, 128, generator=g)
    yield c
    del c
    torch.cuda.empty_cache()


def blocks_of(h):
    """Blocks with scales: another three of every head, near its start, its middle and its end."""
    last = N // BLOCK - 1
    return [7 + h, last // 2 + 11 * h, last - 1 + (h == 0)]


def test_decode_takes_each_heads_own_far_blocks(cache):
    """Three blocks a head have scales, the others 0: their keys have logit 0 and value 0,
    so a row's softmax is over 192 keys it can be read from and N - 192 ones of e^0.
    Logits of about 8 (rms; y below 800) outweigh those.  Tolerances of the note in
    test_gpu_kv8_decode.py with y = 800: r = 2 ln 2 (2^-18 y + 2^-17) + 2^-20, the LSE
    2^-14 more for sums of 2^23 terms (443 additions of a lane, 2^-24 each, and its merge)."""
    g = gen(2)
    q = torch.randn(1, G * H, 1, D, generator=g).bfloat16().cuda()
    cache.k_scale.zero_()
    cache.v_scale.zero_()
    for h in range(H):
        for i, blk in enumerate(blocks_of(h)):
            cache.k_scale[0, h, blk] = 2.0 ** -7 * (1 + 0.25 * i)
            cache.v_scale[0, h, blk] = 2.0 ** -7 * (2 - 0.25 * i + 0.5 * h)
    scale = 8.0 / (D ** 0.5 * 73.0 * 2.0 ** -7 * 1.25)
    weights = torch.zeros(1, H, N, device="cuda")
    out, lse = skv.attn_splitkv_decode_kv8(q, cache, scale, weights=weights)
    y = 800.0
    l_tol = 2.0 ** -18 * y + 2.0 ** -17 + 2.0 ** -14
    rel = 2 * np.log(2.0) * l_tol + 2.0 ** -20
    for h in range(H):
        at = torch.cat([torch.arange(b * BLOCK, (b + 1) * BLOCK) for b in blocks_of(h)])
        scales = lambda t: np.repeat(t[0, h].cpu().double().numpy()[blocks_of(h)], BLOCK)[:, None]  # noqa: E731
        k, v = (code_values(c[0, h, at.cuda()]) * scales(s) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        w_ref = np.zeros(len(at))
        for r in range(G):
            row = O.to_f64(q)[0, h * G + r, 0]
            assert scale * np.log2(np.e) * np.abs(row).max() * np.abs(k).sum(-1).max() < y
            x = scale * (k @ row)
            total = np.exp(x).sum() + (N - len(at))
            p = np.exp(x) / total
            assert p.sum() > 0.5  # what is read from the blocks decides
            got = O.to_f64(out)[0, h * G + r, 0]
            size = p @ np.abs(v)
            assert np.all(np.abs(got - p @ v) <= 2.0 ** -8 * np.abs(p @ v) + (2.0 ** -11 + rel + 2.0 ** -16) * size)
            assert abs(lse[0, h * G + r, 0].item() - np.log2(total)) <= l_tol
            w_ref += p
        w = O.to_f64(weights[0, h, at.cuda()])
        assert np.all(np.abs(w - w_ref) <= rel * w_ref + 2.0 ** -24)
        rest = weights[0, h].double()
        rest[at.cuda()] = 0
        assert (rest > 0).sum().item() == N - len(at)


def test_evict_takes_each_tokens_own_scale(cache):
    """Every block has scales of its own; the kept tokens come from all over the head.
    Codes and scales are those of the definition, bit for bit."""
    g = torch.Generator(device="cuda").manual_seed(3)
    for t in (cache.k_scale, cache.v_scale):
        t.uniform_(0.5, 2.0, generator=g)
    budget, sink, recent = 500, 3, 100
    weights = torch.zeros(1, H, N, device="cuda")
    chosen = []
    for h in range(H):
        at = torch.randperm(N - sink - recent, generator=torch.Generator().manual_seed(h))[: budget - sink - recent] + sink
        chosen.append(sorted([0, 1, 2] + at.tolist() + list(range(N - recent, N))))
        weights[0, h, at.cuda()] = 1 + torch.rand(len(at), generator=gen(h)).cuda()
    to, to_w = skv.kv8_cache(1, H, 512, D, BLOCK), torch.zeros(1, H, 512, device="cuda")
    kept, new_len = skv.kv8_evict(cache, to, weights, to_w, None, budget, sink=sink, recent=recent)
    assert new_len.tolist() == [budget]
    for h in range(H):
        assert kept[0, h].tolist() == chosen[h]
        at = torch.tensor(chosen[h], device="cuda")
        assert torch.equal(to_w[0, h, :budget], weights[0, h, at])
        for codes, scale, to_codes, to_scale in ((cache.k, cache.k_scale, to.k, to.k_scale), (cache.v, cache.v_scale, to.v, to.v_scale)):
            # the tokens' codes and scales in a head of their own, a block each
            c = np.repeat(code_values(codes[0, h, at]), BLOCK, 0)
            s = scale[0, h, at // BLOCK].cpu().numpy()
            want, want_s = O.kv8_move(c, s, np.arange(budget) * BLOCK, BLOCK, "int8")
            assert np.array_equal(code_values(to_codes[0, h, :budget]), want)
            assert np.array_equal(to_scale[0, h, : len(want_s)].cpu().numpy(), want_s)
