"""Calls around the 8-bit cache that are given a stream of their own: memory the
caller lets go of, outputs read elsewhere, two calls at once."""
import pytest
import torch

import split_kv_merge_attn_b200 as skv
from tests._kv8_helpers import filled_cache, gen, i32

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, CAP, BLOCK, N = 2, 8, 2, 128, 2048, 64, 1500
SLEEP = 100_000_000  # about 50 ms: the host makes its calls meanwhile


def rows(H, S, seed):
    return torch.randn(B, H, S, D, generator=gen(seed)).bfloat16().cuda()


def rope_case():
    f, _ = skv.rope_inv_freq(D)
    pos = torch.arange(300, dtype=torch.int32, device="cuda").repeat(B, 1)
    return [rows(HQ, 300, 1), rows(HKV, 300, 2), pos, f], lambda q, k, pos, f, s: skv.rope_apply(q, k, pos, f, stream=s)


def append_case():
    cache = skv.kv8_cache(B, HKV, CAP, D, BLOCK)

    def call(k, v, start, num, s):
        for t in cache:
            t.zero_()
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        skv.kv8_append(cache, k, v, start, num_new=num, stream=s)
        return cache
    return [rows(HKV, 200, 3), rows(HKV, 200, 4), i32([5, 1000]), i32([200, 77])], call


def fetch_case():
    return [*filled_cache(B, HKV, CAP, D, BLOCK, "int8", [N] * B, seed=5), i32([3, 500]), i32([N, 700])], \
        lambda a, b, c, d, start, n, s: skv.kv8_fetch(skv.KV8Cache(a, b, c, d), 400, start=start, kv_len=n, stream=s)


def decode_case():
    nbytes = skv.attn_splitkv_kv8_workspace(B, HQ, HKV, 1, CAP, D, 296, False)
    return [rows(HQ, 1, 6), *filled_cache(B, HKV, CAP, D, BLOCK, "e4m3", [N] * B, seed=7), i32([N, 900]),
            torch.empty(nbytes, dtype=torch.uint8, device="cuda")], \
        lambda q, a, b, c, d, n, ws, s: skv.attn_splitkv_decode_kv8(q, skv.KV8Cache(a, b, c, d), kv_len=n, workspace=ws,
                                                                    stream=s)


def evict_case():
    def call(a, b, c, d, w, n, s):
        to, to_w = skv.kv8_cache(B, HKV, 512, D, BLOCK), torch.zeros(B, HKV, 512, device="cuda")
        for t in to:
            t.zero_()
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        return (*skv.kv8_evict(skv.KV8Cache(a, b, c, d), to, w, to_w, n, 500, sink=4, recent=30, stream=s), *to, to_w)
    w = torch.rand(B, HKV, CAP, generator=gen(9)).cuda()
    return [*filled_cache(B, HKV, CAP, D, BLOCK, "int8", [N] * B, seed=8), w, i32([N, 300])], call


@pytest.mark.parametrize("case", [rope_case, append_case, fetch_case, decode_case, evict_case])
def test_what_a_call_is_given_is_kept_until_it_has_run(case):
    """Every input is let go of when the call returns, while the call waits on its
    stream, and the current stream fills memory of the same sizes at once (with bytes that
    are harmless as lengths and positions)."""
    inputs, call = case()
    fill = lambda count: [torch.full((t.nbytes,), 255, dtype=torch.uint8, device="cuda") for t in inputs  # noqa: E731
                          for _ in range(count)]
    fill(4)  # the fill's kernel is loaded, and the allocator has memory, before the stream is busy
    want = [t.clone() for t in call(*[t.clone() for t in inputs], None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    given = [t.clone() for t in inputs]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP)
    got = call(*given, s)
    del given
    fills = fill(6)
    assert not s.query()  # it has not run yet
    torch.cuda.synchronize()
    assert len(fills) == 6 * len(inputs)
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


def test_outputs_stay_until_the_current_stream_has_read_them():
    """An output read on the current stream and let go of before that read has run; the
    next call on the same stream writes an output of the same size at once."""
    cache = filled_cache(B, HKV, CAP, D, BLOCK, "int8", [N] * B, seed=1)
    q = [rows(HQ, 1, i) for i in (1, 2)]
    n = i32([N, N])
    want = skv.attn_splitkv_decode_kv8(q[0], cache, kv_len=n)[0].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, _ = skv.attn_splitkv_decode_kv8(q[0], cache, kv_len=n, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(SLEEP)
    read = out.clone()
    del out, _
    others = [skv.attn_splitkv_decode_kv8(q[1], cache, kv_len=n, stream=s) for _ in range(4)]
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert len(others) == 4 and torch.equal(read, want)


def test_two_calls_at_once_with_workspaces_of_their_own():
    """Calls on two streams over one cache that wait for the same event and so run at
    once; each stream has one workspace, kept until all have run."""
    cache = filled_cache(B, HKV, CAP, D, BLOCK, "int8", [N] * B, seed=1)
    qs = [rows(HQ, 1, i) for i in (1, 2)]
    lens = [i32([N, 700]), i32([33, N])]
    want = [skv.attn_splitkv_decode_kv8(q, cache, kv_len=n) for q, n in zip(qs, lens)]
    nbytes = skv.attn_splitkv_kv8_workspace(B, HQ, HKV, 1, CAP, D, 296, False)
    spaces = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert spaces[0].data_ptr() != spaces[1].data_ptr()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(16):
        for s, q, n, ws, g in zip(streams, qs, lens, spaces, got):
            g.append(skv.attn_splitkv_decode_kv8(q, cache, kv_len=n, stream=s, workspace=ws))
    assert not streams[0].query() and not streams[1].query()
    torch.cuda.synchronize()
    for g, (out, lse) in zip(got, want):
        for o, l in g:
            assert torch.equal(o, out) and torch.equal(l, lse)


def test_a_captured_call_on_a_side_stream():
    """Captured on the capturing stream's fork, with memory of its own, and replayed."""
    cache = filled_cache(B, HKV, CAP, D, BLOCK, "int8", [N] * B, seed=1)
    q, n = rows(HQ, 1, 1), i32([N, N])
    side = torch.cuda.Stream()
    skv.attn_splitkv_decode_kv8(q, cache, kv_len=n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out, lse = skv.attn_splitkv_decode_kv8(q * 1, cache, kv_len=n, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        doubled = out * 2
    for seed, lengths in ((3, [N, 5]), (4, [77, N])):
        q.copy_(rows(HQ, 1, seed))
        n.copy_(i32(lengths))
        graph.replay()
        torch.cuda.synchronize()
        want, l_want = skv.attn_splitkv_decode_kv8(q, cache, kv_len=n)
        assert torch.equal(out, want) and torch.equal(lse, l_want) and torch.equal(doubled, want * 2)
