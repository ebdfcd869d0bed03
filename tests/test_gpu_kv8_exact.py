"""How exact the 8-bit decode's outputs are, beyond the tolerances of
test_gpu_kv8_decode.py: what its weights may add to the output's own rounding."""
import numpy as np
import pytest
import torch

import oracle as O
import split_kv_merge_attn_b200 as skv
from tests._kv8_helpers import DT, filled_cache, gen, i32, values
from tests.test_gpu_kv8_decode import row_sizes

pytestmark = pytest.mark.gpu

DIGITS = {"bf16": 8, "fp16": 11}  # of the significand


def half_step(x, dtype):
    """Half a rounding step of the output type at x."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -14))) - DIGITS[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("codes", ["int8", "e4m3"])
@pytest.mark.parametrize("G,Lq,D", [(1, 1, 64), (4, 1, 128), (4, 2, 128), (2, 1, 256)])
def test_outputs_of_few_rows_are_those_of_the_exact_weights(G, Lq, D, codes, dtype):
    """With at most 8 rows a kv head an output is the exact O rounded once, but for what
    fp32 sums leave: half a step of the output type, plus (2^-21 + r + 2^-16) of sum p |v|,
    where a weight in two fp16 numbers is off by 2^-22, V's scale in it by as much, r = 2
    ln 2 (2^-18 y + 2^-17) + 2^-20 bounds its exponent's error (the note of
    test_gpu_kv8_decode.py), 2^-16 the fp32 sums and merge, and 2^-25 of each code for
    what lies below fp16's range.  Few keys and small logits, so that a weight rounded
    to fp16 once (2^-12 of it and more) shows: y < 2, r < 2^-15."""
    B, Hkv, n, capacity = 16, 8, 5, 64
    cache = filled_cache(B, Hkv, capacity, D, 16, codes, [n] * B, seed=G + D, scale_span=0.0)
    q = (0.02 * 128 ** 0.5 / D ** 0.5 * torch.randn(B, G * Hkv, Lq, D, generator=gen(Lq))).to(DT[dtype]).cuda()
    out, _ = skv.attn_splitkv_decode_kv8(q, cache, kv_len=i32([n] * B))
    k, v = values(cache.k, cache.k_scale, [n] * B), values(cache.v, cache.v_scale, [n] * B)
    ref, _ = O.decode(q, k, v, D ** -0.5, kv_len=[n] * B)
    size, _ = O.decode(q, k, np.abs(v), D ** -0.5, kv_len=[n] * B)
    y = row_sizes(q, k, D ** -0.5, [n] * B)
    assert y.max() < 2
    rel = 2 * np.log(2.0) * (2.0 ** -18 * y + 2.0 ** -17) + 2.0 ** -20
    codes_max = 127.0 if codes == "int8" else 448.0
    small = 2.0 ** -25 * n * codes_max * float(cache.v_scale[:, :, 0].max())
    off = np.abs(O.to_f64(out) - ref) - half_step(ref, dtype) - (2.0 ** -21 + rel + 2.0 ** -16)[..., None] * size - small
    assert off.max() <= 0, off.max()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,rows", [(64, 1), (128, 1), (64, 16)])
def test_many_light_keys_beside_a_heavy_one(D, rows, dtype):
    """2^20 keys in one CTA, 2^-26 of a heavy one each, whose value is 0: O is what the
    light ones leave, 2^-6 of their value.  An fp16 weight is off by half its smallest
    step, 2^-25, of a reference 2^7 below the heaviest: n 2^-32 |v| in all.  A lane's sum
    rounds once a tile of a warp (64 keys of every 256): n / 256 additions, 2^-24 each.
    The rest as in the module's other test, a weight rounded once being off by 2^-11, and
    y = 26 for every row."""
    n, c0, vs = 1 << 20, 100, 2.0 ** -7
    cache = skv.kv8_cache(1, 1, n, D, 128)
    cache.k.zero_()
    cache.k[:, :, 0] = c0
    cache.v.fill_(100)
    cache.v[:, :, 0] = 0
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(vs)
    scale = float(np.float32(26 * np.log(2.0) / (D * c0)))
    q = torch.ones(1, rows, 1, D, dtype=DT[dtype], device="cuda")
    out, lse = skv.attn_splitkv_decode_kv8(q, cache, scale, num_ctas=1)
    heavy = 2.0 ** (scale * np.log2(np.e) * D * c0)
    want, l_want = 100 * vs * (n - 1) / (n - 1 + heavy), np.log2(n - 1 + heavy)
    sums = n / 256 * 2.0 ** -24
    l_tol = 2.0 ** -18 * 26 + 2.0 ** -17 + 1.5 * sums
    assert np.abs(O.to_f64(lse) - l_want).max() <= l_tol
    tol = half_step(np.float64(want), dtype) + (2.0 ** -11 + 2 * np.log(2.0) * l_tol + 2.0 ** -16) * want + n * 2.0 ** -32 * 100 * vs
    assert tol < want / 30
    assert np.abs(O.to_f64(out) - want).max() <= tol


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [1, 16])
@pytest.mark.parametrize("power,unit", [(12, 1), (14, 1), (15, 1), (17, 1), (17, 2), (17, 4)])
def test_logits_of_millions_stay_finite(power, unit, rows, dtype):
    """Logits near 100 unit 2^power, where fp32 holds them to quarters at best and to
    whole steps of 4 at worst, and the exponents of the weights are off by as much as
    that: weights a few such steps above fp16's largest value must not become infinite.
    O is a value of V times what the exponents are off by, at most 2^6 either way; the
    LSE is right to 2^-20 of itself (the fp32 product of scale, K's scale and the sum),
    plus log2 n and a step."""
    n = 2048
    for step in range(1, 10):
        for frac in (0.0, 0.3, 0.5, 0.8):
            cache = skv.kv8_cache(1, 1, n, 64, 16)
            cache.k.zero_()
            cache.k[..., 0] = 100
            cache.k[0, 0, :, 1] = (torch.arange(n, device="cuda") // 256 * step).clamp(max=100).to(torch.int8)
            cache.v.fill_(100)
            cache.k_scale.fill_(1.0)
            cache.v_scale.fill_(2.0 ** (frac - 7))
            q = torch.zeros(1, rows, 1, 64, dtype=DT[dtype], device="cuda")
            q[..., 0], q[..., 1] = 2.0 ** (power - 2), 0.25  # (fp16 ends below 2^16)
            out, lse = skv.attn_splitkv_decode_kv8(q, cache, float(4 * unit * np.log(2.0)), num_ctas=1)
            want = 100 * 2.0 ** (frac - 7)
            assert torch.isfinite(out).all() and (out.float() <= 64 * want).all() and (out.float() >= want / 64).all(), (step, frac)
            x = unit * (100.0 * 2 ** power + 7 * step)
            assert ((lse.double() - x).abs() <= 2.0 ** -20 * x + 11 + 4).all()


@pytest.mark.parametrize("rows", [1, 16])
@pytest.mark.parametrize("dtype,logit", [("bf16", s * 2.0 ** e) for e in (10, 14, 17, 20, 24, 30, 60, 110, 120) for s in (1, -1)] +
                         [("fp16", s * 2.0 ** e) for e in (10, 14, 17, 20) for s in (1, -1)])
@pytest.mark.parametrize("n,ctas", [(1, 1), (48, 1), (1024, 5)])
def test_values_do_not_depend_on_the_logits_size(n, ctas, rows, dtype, logit):
    """All keys alike, logits of any size: O is the mean of the values, whose blocks have
    scales 2^-9 to 2^-3 apart, and LSE = logit + log2 n (parts of equal length: the LSE of a
    part holds log2 n to its own rounding only).  The softmax weights are 1 / n but
    for ex2 (2^-22) and log2 of V's scale (2^-21), and where rounded once for fp16's 2^-11;
    2^-16 for fp32 sums and the merge (the module's other notes)."""
    cache = skv.kv8_cache(1, 1, 1024, 64, 16)
    cache.k.zero_()
    cache.k[..., 0] = 100
    cache.k_scale.fill_(1.0)
    cache.v.random_(-127, 128, generator=torch.Generator(device="cuda").manual_seed(n))
    cache.v_scale.copy_(2.0 ** (-9 + 6 * torch.rand(cache.v_scale.shape, generator=gen(n))))
    q = torch.zeros(1, rows, 1, 64, dtype=DT[dtype], device="cuda")
    q[..., 0] = (1.0 if logit > 0 else -1.0) * (2.0 ** 9 if dtype == "fp16" else abs(logit) / 2.0 ** 5)
    scale = float(np.float32(logit / (float(q[0, 0, 0, 0]) * 100.0) * np.log(2.0)))
    out, lse = skv.attn_splitkv_decode_kv8(q, cache, scale, kv_len=i32([n]), num_ctas=ctas)
    v = values(cache.v, cache.v_scale, [n])[0, 0, :n]
    want, size = v.mean(0), np.abs(v).mean(0)
    weight = 2.0 ** -11 if dtype == "bf16" and rows > 8 else 0.0
    tol = half_step(want, dtype) + (2.0 ** -20 + 2.0 ** -16 + weight) * size
    assert np.all(np.abs(O.to_f64(out)[0, :, 0] - want) <= tol)
    x = float(q[0, 0, 0, 0]) * 100.0 * scale * np.log2(np.e)
    assert np.all(np.abs(O.to_f64(lse) - (x + np.log2(n))) <= 2.0 ** -21 * abs(x) + 2.0 ** -17)
