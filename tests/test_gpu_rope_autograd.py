"""rope_apply under autograd: its gradient is the transpose."""
import pytest
import torch

import split_kv_merge_attn_b200 as skv
from tests._kv8_helpers import DT, HALF_STEP, gen
from tests.test_gpu_rope import check, lead

pytestmark = pytest.mark.gpu

CASES = [("HND", 2, 33, 4, 2, 128, 64, False, False, "bf16"), ("NHD", 1, 130, 3, 1, 64, 64, True, False, "fp16"),
         ("TND", 1, 70, 5, 5, 96, 48, False, True, "bf16")]


def inputs(layout, B, S, Hq, Hkv, D, R, dtype, seed=0):
    g = gen(seed + S)
    q, k, gq, gk = (torch.randn(*lead(layout, B, S, H, D), generator=g).to(DT[dtype]).cuda() for H in (Hq, Hkv, Hq, Hkv))
    f, _ = skv.rope_inv_freq(R)
    pos = torch.randint(0, 10000, (S,) if layout == "TND" else (B, S), generator=g, dtype=torch.int32).cuda()
    return q, k, gq, gk, pos, f


@pytest.mark.parametrize("layout,B,S,Hq,Hkv,D,R,inter,inverse,dtype", CASES)
def test_gradients_are_the_transpose(layout, B, S, Hq, Hkv, D, R, inter, inverse, dtype):
    q, k, gq, gk, pos, f = inputs(layout, B, S, Hq, Hkv, D, R, dtype)
    turn = lambda q, k, inv=inverse: skv.rope_apply(q, k, pos, f, layout, inter, 0.5, inv)  # noqa: E731
    want = turn(q, k)
    q.requires_grad_()
    k.requires_grad_()
    y, z = turn(q, k)
    assert torch.equal(y, want[0]) and torch.equal(z, want[1]) and y.requires_grad and z.requires_grad
    dq, dk = torch.autograd.grad((y, z), (q, k), (gq, gk), create_graph=True)
    for d, g in ((dq, gq), (dk, gk)):
        check(d.detach(), g, pos, f, layout, inter, 0.5, not inverse, dtype)  # the formula, in fp64
    # gradients of gradients: the transpose of the transpose
    gq.requires_grad_()
    y, z = turn(q, k)
    dq, = torch.autograd.grad(y, q, gq, create_graph=True)
    twice, = torch.autograd.grad(dq, gq, q.detach())
    assert torch.equal(twice, want[0])


@pytest.mark.parametrize("layout,B,S,Hq,Hkv,D,R,inter,inverse,dtype", CASES)
def test_gradients_against_differences(layout, B, S, Hq, Hkv, D, R, inter, inverse, dtype):
    """L(x) = <turn(x), g> is linear: (L(x + d) - L(x - d)) / 2 = <grad, d> for any d.  Each
    value of turn() and of the gradient is off by half a step of the type and 2^-18 of
    its pair's size (at most that of |g|, |x| + |d| of a whole head, times 1.5)."""
    q, k, gq, gk, pos, f = inputs(layout, B, S, Hq, Hkv, D, R, dtype, seed=5)
    x = torch.round(q.float() * 8).clamp(-16, 16) / 8  # sums with d are exact
    d = torch.round(torch.randn(q.shape, generator=gen(9)).cuda() * 8).clamp(-16, 16) / 8
    half = DT[dtype]
    loss = lambda t: (skv.rope_apply(t.to(half), None, pos, f, layout, inter, 1.0, inverse)[0].double() * gq.double())  # noqa: E731
    up, down = loss(x + d), loss(x - d)
    leaf = x.to(half).requires_grad_()
    y, none = skv.rope_apply(leaf, None, pos, f, layout, inter, 1.0, inverse)
    assert none is None
    (y.double() * gq.double()).sum().backward()
    along = leaf.grad.double() * d.double()
    sizes = up.abs().sum() / 2 + down.abs().sum() / 2 + along.abs().sum()
    pairs = 2.0 ** -18 * 1.5 * 2 * (gq.double().abs().amax() * ((x + d).abs() + (x - d).abs() + 2 * d.abs()).double().sum())
    assert ((up - down).sum() / 2 - along.sum()).abs() <= HALF_STEP[dtype] * sizes + pairs


def test_only_what_requires_a_gradient():
    q, k, gq, gk, pos, f = inputs("HND", 1, 40, 4, 2, 64, 64, "bf16")
    want, _ = skv.rope_apply(gk, None, pos, f, inverse=True)
    k.requires_grad_()
    y, z = skv.rope_apply(q, k, pos, f)
    assert not y.requires_grad and z.requires_grad
    z.backward(gk)
    assert torch.equal(k.grad, want) and q.grad is None
    # an output that nothing follows; k alone behind it
    q.requires_grad_()
    k.grad = None
    y, z = skv.rope_apply(q, k, pos, f)
    z.backward(gk)
    assert torch.equal(k.grad, want) and q.grad is None
    # strided, broadcast and misaligned gradients
    y, z = skv.rope_apply(q, k, pos, f)
    k.grad = None
    z.sum().backward()
    assert torch.equal(k.grad, skv.rope_apply(torch.ones_like(gk), None, pos, f, inverse=True)[0])
    y, z = skv.rope_apply(q, k, pos, f)
    wide = torch.zeros(gk.numel() + 1, dtype=gk.dtype, device="cuda")
    wide[1:] = gk.reshape(-1)
    got, = torch.autograd.grad(z, k, wide[1:].view(gk.shape))
    assert torch.equal(got, want)
    y, z = skv.rope_apply(q, k, pos, f)
    got, = torch.autograd.grad(z, k, gk.transpose(1, 2).contiguous().transpose(1, 2))
    assert torch.equal(got, want)


def test_a_stream_of_its_own():
    q, k, gq, gk, pos, f = inputs("HND", 1, 40, 4, 2, 64, 64, "bf16")
    want = skv.rope_apply(q, k, pos, f)
    back, _ = skv.rope_apply(gq, None, pos, f, inverse=True)
    q.requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, z = skv.rope_apply(q, k, pos, f, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want[0]) and torch.equal(z, want[1])
    y.backward(gq)
    assert torch.equal(q.grad, back)


def test_without_gradients_nothing_is_recorded():
    q, k, gq, gk, pos, f = inputs("HND", 1, 40, 4, 2, 64, 64, "bf16")
    want = skv.rope_apply(q, k, pos, f)
    q.requires_grad_()
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            y, z = skv.rope_apply(q, k, pos, f)
            assert torch.equal(y, want[0]) and torch.equal(z, want[1]) and not y.requires_grad
            out = torch.empty_like(q)
            assert skv.rope_apply(q, None, pos, f, q_out=out)[0] is out and torch.equal(out, want[0])


def test_writing_in_place_is_seen_by_autograd():
    """A tensor that a recorded operation needs, turned in place: the backward pass
    refuses it.  Outputs over anything that autograd records are refused at once."""
    q, k, gq, gk, pos, f = inputs("HND", 1, 40, 4, 2, 64, 64, "bf16")
    leaf = torch.ones_like(q, requires_grad=True)
    y = (leaf * q).sum()
    skv.rope_apply(q, None, pos, f, q_out=q)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    before = skv.launch_count()
    for kw in (dict(q=leaf, k=None, q_out=leaf), dict(q=leaf, k=k, k_out=torch.empty_like(k)), dict(q=q, k=None, q_out=leaf)):
        with pytest.raises(ValueError):
            skv.rope_apply(**kw, positions=pos, inv_freq=f)
    with pytest.raises(ValueError):
        skv.rope_apply(q, None, pos, f.clone().requires_grad_())
    assert skv.launch_count() == before
    # memory made in inference mode keeps no versions
    with torch.inference_mode():
        x = q.clone()
    assert skv.rope_apply(x, None, pos, f, q_out=x)[0] is x


def test_forward_and_backward_captured():
    """Both passes in one graph, replayed with new inputs, gradients and positions."""
    q, k, gq, gk, pos, f = inputs("HND", 2, 40, 4, 2, 64, 64, "bf16")
    q.requires_grad_()
    k.requires_grad_()

    def both():
        y, z = skv.rope_apply(q, k, pos, f)
        return (y.detach(), z.detach(), *torch.autograd.grad((y, z), (q, k), (gq, gk)))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for seed in (1, 2):
        new = inputs("HND", 2, 40, 4, 2, 64, 64, "bf16", seed=seed)
        with torch.no_grad():
            for t, x in zip((q, k, gq, gk, pos), new):
                t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            want = (*skv.rope_apply(q, k, pos, f), *skv.rope_apply(gq, gk, pos, f, inverse=True))
        for a, b in zip(got, want):
            assert torch.equal(a, b)
