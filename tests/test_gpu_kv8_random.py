"""Seeded sweeps of small irregular problems of the rotary and 8-bit cache calls
against the oracle (the checks and tolerances of their own test files), and the
calls a serving program makes that the other files do not: captures that allocate
for themselves, two streams at once, misaligned and strided tensors."""
import random

import pytest
import torch

import oracle as O
import split_kv_merge_attn_b200 as skv
from tests import test_gpu_kv8 as A, test_gpu_kv8_decode as Dec, test_gpu_kv8_evict as E, test_gpu_rope as R
from tests._kv8_helpers import DT, filled_cache, gen, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(24))
def test_decode(seed):
    r = random.Random(seed)
    D, block = r.choice([64, 128, 256]), r.choice([16, 32, 64, 128])
    B, Hkv, G, Lq = r.choice([1, 2, 3, 9]), r.choice([1, 2, 3]), r.choice([1, 2, 4, 7]), r.choice([1, 1, 2, 5])
    capacity = block * r.randint(1, max(1, 1600 // block))
    lengths = [r.choice([0, 1, capacity, r.randint(0, capacity)]) for _ in range(B)]
    Dec.run(B, G * Hkv, Hkv, Lq, D, capacity, block, r.choice(["int8", "e4m3"]), r.choice(["bf16", "fp16"]), lengths,
            causal=r.random() < 0.5, weights=r.random() < 0.6, ctas=r.choice([0, 0, 1, 2, 3, 10, 77]), seed=seed,
            q_mult=r.choice([0.5, 1.0, 6.0]), scale_span=r.choice([0.0, 3.0, 10.0]))


@pytest.mark.parametrize("seed", range(16))
def test_append(seed):
    r = random.Random(1000 + seed)
    D, block = r.choice([64, 128, 256]), r.choice([16, 32, 64, 128])
    B, H, S = r.choice([1, 2, 5]), r.choice([1, 2, 3]), r.choice([1, 2, 17, 128, 129, 300])
    capacity = block * r.randint(1, max(1, 900 // block))
    starts = [r.choice([0, r.randint(0, capacity), capacity]) for _ in range(B)]
    counts = [r.choice([S, r.randint(0, S)]) for _ in range(B)]
    codes, dtype, layout = r.choice(["int8", "e4m3"]), r.choice(["bf16", "fp16"]), r.choice(["HND", "NHD"])
    cache = filled_cache(B, H, capacity, D, block, codes, starts, seed=seed, scale_span=r.choice([0.0, 4.0]))
    new = A.new_tokens(layout, B, S, H, D, dtype, seed=seed, mult=r.choice([0.01, 1.0, 30.0]))
    want = A.expect_append(A.snapshot(cache), new, starts, counts, block, codes)
    k, v = (A.laid_out(x, layout) for x in new)
    skv.kv8_append(cache, k, v, i32(starts), num_new=i32(counts), layout=layout)
    A.assert_cache(cache, want)


@pytest.mark.parametrize("seed", range(16))
def test_evict(seed):
    r = random.Random(2000 + seed)
    D, block = r.choice([64, 128, 256]), r.choice([16, 32, 64, 128])
    B, H = r.choice([1, 2, 3]), r.choice([1, 2])
    capacity = block * r.randint(1, max(1, 2000 // block))
    budget = r.randint(1, capacity)
    sink = r.randint(0, min(budget, 20))
    recent = r.randint(0, budget - sink)
    to_capacity = block * (-(-budget // block) + r.randint(0, 2))
    lengths = [r.choice([0, capacity, r.randint(0, capacity), min(budget, capacity)]) for _ in range(B)]
    cache = filled_cache(B, H, capacity, D, block, r.choice(["int8", "e4m3"]), lengths, seed=seed, scale_span=3.0)
    w = E.random_weights(B, H, capacity, seed)
    if r.random() < 0.5:
        w = torch.round(w * 2) / 2  # many ties, many zeros
    E.check(cache, w, lengths, to_capacity, budget, sink, recent)


@pytest.mark.parametrize("seed", range(16))
def test_rope(seed):
    r = random.Random(3000 + seed)
    D = 16 * r.randint(1, 24)
    rot = 16 * r.randint(1, D // 16)
    layout = r.choice(["HND", "NHD", "TND"])
    B, S = (1 if layout == "TND" else r.choice([1, 2, 7])), r.choice([1, 2, 33, 200, 1300])
    Hq, Hkv = r.choice([1, 3, 8, 50]), r.choice([1, 2, 5])
    inter, inverse, dtype = r.random() < 0.5, r.random() < 0.5, r.choice(["bf16", "fp16"])
    g = gen(seed)
    q, k = (torch.randn(*R.lead(layout, B, S, H, D), generator=g).to(DT[dtype]).cuda() for H in (Hq, Hkv))
    f, m = skv.rope_inv_freq(rot, base=r.choice([1e4, 5e5]), scaling=r.choice(sorted(skv.ROPE_SCALINGS)), factor=4.0)
    pos = torch.randint(0, 2 ** 20, (S,) if layout == "TND" else (B, S), generator=g, dtype=torch.int32).cuda()
    qo, ko = skv.rope_apply(q, k, pos, f, layout, inter, m, inverse)
    R.check(qo, q, pos, f, layout, inter, m, inverse, dtype)
    R.check(ko, k, pos, f, layout, inter, m, inverse, dtype)


def test_heads_wider_than_a_cta():
    """More heads x units than a CTA has threads: heads in groups."""
    for H, D in ((70, 256), (513, 16), (1, 8192)):
        q = torch.randn(1, H, 3, D, generator=gen(H)).bfloat16().cuda()
        f, _ = skv.rope_inv_freq(min(D, 4096))
        pos = torch.arange(5, 8, dtype=torch.int32, device="cuda").view(1, 3)
        y, _ = skv.rope_apply(q, None, pos, f)
        R.check(y, q, pos, f, "HND", False, 1.0, False, "bf16")


def test_captured_step_allocates_for_itself():
    """rope, append, decode with weights and evict captured together with their own
    outputs and workspaces, replayed with new inputs."""
    B, Hq, Hkv, D, capacity = 2, 4, 2, 64, 8192 + 64
    cache, small = (skv.kv8_cache(B, Hkv, n, D, 16) for n in (capacity, 64))
    for t in (cache.k, cache.v):
        t.view(torch.int8).random_(-127, 128)
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(0.01)
    f, _ = skv.rope_inv_freq(64)
    q = torch.zeros(B, Hq, 1, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(B, Hkv, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    length, w = i32([8000, 5000]), torch.zeros(B, Hkv, capacity, device="cuda")
    sw = torch.zeros(B, Hkv, 64, device="cuda")

    def step():
        qr, kr = skv.rope_apply(q, k, length.view(B, 1), f)
        skv.kv8_append(cache, kr, v, length)
        n = length + 1
        out, lse = skv.attn_splitkv_decode_kv8(qr, cache, kv_len=n, weights=w)
        kept, new_len = skv.kv8_evict(cache, small, w, sw, n, 50, sink=2, recent=10)
        return qr, out, lse, kept, new_len, n

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i, lengths in enumerate(([8000, 5000], [3, 8255])):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen(i)))
        length.copy_(i32(lengths))
        w.zero_()
        graph.replay()
        torch.cuda.synchronize()
        qr, out, lse, kept, new_len, n = got
        now = [x + 1 for x in lengths]
        assert n.tolist() == now
        Dec.check(qr, cache, out, lse, now, D ** -0.5, False, "bf16", O.to_f64(w))
        assert new_len.tolist() == [min(x, 50) for x in now]
        for b in range(B):
            for h in range(Hkv):
                at = O.kv8_kept(w[b, h].cpu(), now[b], 50, 2, 10).tolist()
                assert kept[b, h].tolist() == at + [-1] * (50 - len(at))


def test_two_streams_at_once():
    """Calls on two streams over the same cache, each with outputs and workspace of its own."""
    B, Hq, Hkv, D, capacity = 1, 8, 2, 128, 16384
    cache = filled_cache(B, Hkv, capacity, D, 64, "int8", [capacity], seed=1)
    qs = [torch.randn(B, Hq, 1, D, generator=gen(s)).bfloat16().cuda() for s in (1, 2)]
    want = [skv.attn_splitkv_decode_kv8(q, cache) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for s, q, g in zip(streams, qs, got):
            g.append(skv.attn_splitkv_decode_kv8(q, cache, stream=s,
                                                 workspace=torch.empty(1 << 22, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for g, (out, lse) in zip(got, want):
        for o, l in g:
            assert torch.equal(o, out) and torch.equal(l, lse)


def test_refusals_of_device_tensors():
    """Strided, misaligned and mistyped device tensors, before any launch."""
    before = skv.launch_count()
    cache = skv.kv8_cache(1, 2, 64, 64, 16)
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16, device="cuda")
    f, _ = skv.rope_inv_freq(64)
    pos = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    off = torch.zeros(1 + k.numel(), dtype=torch.bfloat16, device="cuda")[1:].view(k.shape)  # 2 bytes past alignment
    strided = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    calls = [lambda: skv.rope_apply(strided, None, pos, f), lambda: skv.rope_apply(off, None, pos, f),
             lambda: skv.rope_apply(k, None, pos.cpu(), f), lambda: skv.rope_apply(k, None, pos, f, q_out=off),
             lambda: skv.kv8_append(cache, strided, strided, i32([0])), lambda: skv.kv8_append(cache, off, k, i32([0])),
             lambda: skv.kv8_append(cache, k, k, torch.zeros(1, dtype=torch.int64, device="cuda")),
             lambda: skv.kv8_append(cache, k, k, i32([0]), max_seqlen=3),
             lambda: skv.kv8_append(cache, k.float(), k.float(), i32([0])),
             lambda: skv.kv8_fetch(cache, 4, torch.float32), lambda: skv.kv8_fetch(cache, -1),
             lambda: skv.attn_splitkv_decode_kv8(q, cache, workspace=torch.empty(8, dtype=torch.uint8)),
             lambda: skv.attn_splitkv_decode_kv8(q, cache, weights=torch.zeros(1, 2, 63, device="cuda")),
             lambda: skv.attn_splitkv_decode_kv8(q, cache, scale=-1.0),
             lambda: skv.attn_splitkv_decode_kv8(q[:, :3].contiguous(), cache),
             lambda: skv.kv8_evict(cache, cache, *[torch.zeros(1, 2, 64, device="cuda")] * 2, None, 4),
             lambda: skv.kv8_evict(cache, skv.kv8_cache(1, 2, 64, 64, 32), *[torch.zeros(1, 2, 64, device="cuda")] * 2, None, 4)]
    for call in calls:
        with pytest.raises((ValueError, skv.SkvError)):
            call()
    for bad in (lambda: skv.rope_apply(None, None, pos, f), lambda: skv.kv8_fetch((1, 2, 3, 4), 4),
                lambda: skv.attn_splitkv_decode_kv8(q, (cache.k, cache.v))):
        with pytest.raises(TypeError):
            bad()
    assert skv.launch_count() == before


def test_memory_of_a_call_belongs_to_its_stream():
    """A call given a stream allocates its workspace and outputs there: the current
    stream, which goes on at once, must not get that memory before the call has run."""
    B, Hq, Hkv, D, capacity = 1, 8, 2, 128, 16384
    cache = filled_cache(B, Hkv, capacity, D, 64, "int8", [capacity], seed=1)
    q = torch.randn(B, Hq, 1, D, generator=gen(1)).bfloat16().cuda()
    w = torch.zeros(B, Hkv, capacity, device="cuda")
    want = skv.attn_splitkv_decode_kv8(q, cache, weights=w)
    again, s = torch.zeros_like(w), torch.cuda.Stream()
    nbytes = skv.attn_splitkv_kv8_workspace(B, Hq, Hkv, 1, capacity, D, 296, True)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # the call waits about 10 ms behind this
    out, lse = skv.attn_splitkv_decode_kv8(q, cache, weights=again, stream=s)
    fills = [torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert len(fills) == 4
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(again, w)
