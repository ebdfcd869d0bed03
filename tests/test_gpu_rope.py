"""rope_apply against the fp64 oracle.

Tolerance per value: half a rounding step of the output type, plus 2^-19 of the
pair's size (factor * (|x| + |y|)): the angle is exact to 2^-24 half turns
(pi * 2^-24 rad) plus, at positions up to 2^31, three fp64 roundings of at most
3.4e8 turns (7e-7 rad, and 2.4e-7 rad of the oracle's own), sincospif and the
factor add 2^-22, the two products and the sum 3 * 2^-24: together below
2^-19.5.  fp16 results below 2^-14 are off by half of 2^-24 at most."""
import numpy as np
import pytest
import torch

import oracle as O
import split_kv_merge_attn_b200 as skv
from tests._kv8_helpers import DT, HALF_STEP, gen, i32

pytestmark = pytest.mark.gpu


def lead(layout, B, S, H, D):
    return {"HND": (B, H, S, D), "NHD": (B, S, H, D), "TND": (S, H, D)}[layout]


def pair_sizes(x, R, interleaved):
    a = np.abs(O.to_f64(x))
    out = np.zeros_like(a)
    first, second = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    out[..., first] = out[..., second] = a[..., first] + a[..., second]
    return out


def check(y, x, pos, f, layout, interleaved, factor, inverse, dtype):
    R = 2 * f.numel()
    ref = O.rope(x, pos, f, layout, interleaved, factor, inverse)
    tol = HALF_STEP[dtype] * np.abs(ref) + 2.0 ** -19 * abs(factor) * pair_sizes(x, R, interleaved)
    tol += 2.0 ** -25 if dtype == "fp16" else 0.0
    got = O.to_f64(y)
    assert got.shape == ref.shape
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) - tol)
    # copied dimensions are bit-equal
    assert torch.equal(y[..., R:].cpu(), x[..., R:].cpu())


CASES = [
    # layout, B, S, Hq, Hkv, D, R, interleaved, factor, inverse, dtype, first position, scaling
    ("HND", 1, 1, 1, 1, 64, 64, False, 1.0, False, "bf16", 0, "none"),
    ("HND", 8, 1, 32, 8, 128, 128, False, 1.0, False, "bf16", 4095, "none"),
    ("NHD", 2, 37, 6, 2, 128, 64, True, 1.0, True, "fp16", 1000000, "linear"),
    ("TND", 1, 301, 5, 5, 256, 256, False, 1.1386, False, "bf16", 31000, "yarn"),
    ("HND", 3, 130, 4, 1, 256, 32, True, 1.0, False, "fp16", 123456, "ntk"),
    ("NHD", 1, 700, 16, 4, 64, 16, False, 0.5, True, "bf16", 7, "none"),
    ("TND", 1, 1, 3, 1, 96, 48, True, 1.0, False, "bf16", 2 ** 31 - 2, "none"),   # any D, R multiples of 16
    ("HND", 1, 2, 2, 1, 16, 16, False, 1.0, False, "fp16", -5, "none"),           # negative positions turn back
]


@pytest.mark.parametrize("layout,B,S,Hq,Hkv,D,R,inter,factor,inverse,dtype,first,scaling", CASES)
def test_against_oracle(layout, B, S, Hq, Hkv, D, R, inter, factor, inverse, dtype, first, scaling):
    g = gen(S * D + R)
    q, k = (torch.randn(*lead(layout, B, S, H, D), generator=g).to(DT[dtype]).cuda() for H in (Hq, Hkv))
    f, m = skv.rope_inv_freq(R, scaling=scaling, factor=4.0)
    pos = (first + torch.arange(B * S, dtype=torch.int64)).clamp(max=2 ** 31 - 1).to(torch.int32).cuda()
    pos = pos if layout == "TND" else pos.view(B, S)
    qo, ko = skv.rope_apply(q, k, pos, f, layout, inter, factor * m, inverse)
    check(qo, q, pos, f, layout, inter, factor * m, inverse, dtype)
    check(ko, k, pos, f, layout, inter, factor * m, inverse, dtype)
    # in place, and q alone, are the same bits
    q2, k2 = q.clone(), k.clone()
    a, b = skv.rope_apply(q2, k2, pos, f, layout, inter, factor * m, inverse, q_out=q2, k_out=k2)
    assert a is q2 and b is k2 and torch.equal(q2, qo) and torch.equal(k2, ko)
    a, b = skv.rope_apply(q, None, pos, f, layout, inter, factor * m, inverse)
    assert b is None and torch.equal(a, qo)


def test_inverse_is_the_gradient():
    """The inverse is the transpose: <turn(x), g> = <x, inverse(g)>, and a central
    difference of <turn(x), g> gives its entries.  Values are multiples of 2^-3
    with |.| <= 2 and positions multiples that keep fp64 sums exact enough; each
    bf16 result is off by 2^-8 of itself, so the products of 128 * S * H values
    differ by at most 2 * 2^-8 * sum |turn(x)| |g|."""
    g = gen(5)
    x = (torch.randint(-16, 17, (1, 3, 11, 128), generator=g) / 8).bfloat16().cuda()
    d = (torch.randint(-16, 17, (1, 3, 11, 128), generator=g) / 8).bfloat16().cuda()
    f, m = skv.rope_inv_freq(64, scaling="yarn", factor=8.0)
    pos = torch.arange(100, 111, dtype=torch.int32, device="cuda").view(1, 11)
    y, _ = skv.rope_apply(x, None, pos, f, factor=m)
    dx, _ = skv.rope_apply(d, None, pos, f, factor=m, inverse=True)
    left, right = (y.double() * d.double()), (x.double() * dx.double())
    bound = 2.0 ** -8 * (left.abs().sum() + right.abs().sum()) + 2.0 ** -18 * m * (x.abs().double().sum() * 4)
    assert abs(left.sum() - right.sum()) <= bound
    # differences of the formula (the oracle is linear: any step is exact up to fp64)
    probe = np.zeros(tuple(x.shape))
    for at in [(0, 0, 0, 0), (0, 1, 5, 33), (0, 2, 10, 63), (0, 2, 3, 100)]:
        probe[at] = 1.0
        up, down = (np.sum(O.rope(O.to_f64(x) + s * probe, pos, f, factor=m) * O.to_f64(d)) for s in (0.5, -0.5))
        probe[at] = 0.0
        want = up - down
        assert abs(float(dx[at]) - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -19 * m * 4


def test_side_stream_and_graph():
    """Inputs written on a side stream just before; a captured call follows new
    contents and positions."""
    f, _ = skv.rope_inv_freq(128)
    q = torch.empty(2, 4, 9, 128, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(2, 2, 9, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(2, 9, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        skv.rope_apply(q, k, pos, f, q_out=qo, k_out=ko)
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            skv.rope_apply(q, k, pos, f, q_out=qo, k_out=ko)
        for seed in (1, 2):
            g = gen(seed)
            q.copy_(torch.randn(2, 4, 9, 128, generator=g))
            k.copy_(torch.randn(2, 2, 9, 128, generator=g))
            pos.copy_(torch.randint(0, 100000, (2, 9), generator=g))
            graph.replay()
            s.synchronize()
            check(qo, q, pos, f, "HND", False, 1.0, False, "bf16")
            check(ko, k, pos, f, "HND", False, 1.0, False, "bf16")


def test_no_tokens():
    f, _ = skv.rope_inv_freq(64)
    q = torch.empty(1, 4, 0, 64, dtype=torch.bfloat16, device="cuda")
    a, b = skv.rope_apply(q, None, torch.empty(1, 0, dtype=torch.int32, device="cuda"), f)
    assert a.shape == q.shape and b is None
