"""Calls on a stream that is not the current one: the memory that they allocate.

A block that a temporary of the current stream gave back is handed out again to that stream's
next allocation, whose work the stream itself puts behind the temporary's.  Another stream
does not wait for it, so a call there has to take its results and scratch from elsewhere.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _inputs(*shapes):
    g = torch.Generator().manual_seed(5)
    return [torch.nn.functional.normalize(torch.randn(*s, generator=g), dim=-1).to(BF).cuda() for s in shapes]


def _kda():
    q, k, v = _inputs(*[(2, 200, 2, 128)] * 3)
    la = (-torch.rand(2, 200, 2, 128, generator=torch.Generator().manual_seed(6))).to(BF).cuda()
    return q, k, v, la, torch.full((2, 200, 2), 0.5, dtype=BF, device="cuda")


def _lin():
    q, k, v = _inputs(*[(2, 200, 2, 128)] * 3)
    return q, k, v, (-torch.rand(2, 200, 2, generator=torch.Generator().manual_seed(7))).to(BF).cuda()


def _calls():
    import kimi_delta_attention_30_b200 as kda
    x, y = _kda(), _lin()
    tok, ltok = tuple(t[:, 0].contiguous() for t in x), tuple(t[:, 0].contiguous() for t in y)
    state = iter([torch.zeros(2, 2, 128, 128, device="cuda") for _ in range(16)])   # one a call
    M, F = kda.segment_map(*x)
    w = torch.ones(128, dtype=BF, device="cuda")
    ones = (w, w, None, None)
    return dict(
        chunk_fwd=lambda s: kda.chunk_fwd(*x, stream=s),
        chunk_fwd_noalloc=lambda s: kda.chunk_fwd_noalloc(*x, stream=s),
        chunk_bwd=lambda s: kda.chunk_bwd(*x, x[2], stream=s),
        segment_map=lambda s: kda.segment_map(*x, stream=s),
        compose_states=lambda s: (kda.compose_states(M[None], F[None], stream=s),),
        decode_step=lambda s: (kda.decode_step(*tok, next(state), stream=s),),
        linear_chunk_fwd=lambda s: kda.linear_chunk_fwd(*y, stream=s),
        linear_chunk_bwd=lambda s: kda.linear_chunk_bwd(*y, y[2], stream=s),
        linear_decode_step=lambda s: (kda.linear_decode_step(*ltok, next(state), stream=s),),
        qk_norm_rope=lambda s: kda.qk_norm_rope(y[0], y[1], *ones, stream=s),
        qk_norm_rope_bwd=lambda s: kda.qk_norm_rope_bwd(y[0], y[1], *ones, y[2], y[2], stream=s),
    )


NAMES = ["chunk_fwd", "chunk_fwd_noalloc", "chunk_bwd", "segment_map", "compose_states", "decode_step",
         "linear_chunk_fwd", "linear_chunk_bwd", "linear_decode_step", "qk_norm_rope", "qk_norm_rope_bwd"]


def same(name, got, want):
    """The same bits; the KDA gradients that add with atomics may differ by a last bit."""
    if name != "chunk_bwd":
        return all(torch.equal(a, b) for a, b in zip(got, want))
    near = lambda a, b: bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-3 * b.square().mean().sqrt()).all())
    return all(near(a.float(), b.float()) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_memory_in_use_on_the_current_stream_is_not_taken(cuda_ok, name):
    call = _calls()[name]
    want = [t.clone() for t in call(None) if t is not None]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    call(side)                           # (the side stream has memory of its own from here on)
    torch.cuda.synchronize()
    # blocks of the results' sizes and larger ones, given back while work that uses them is queued
    held = [torch.full_like(t, 3) for t in want] + [torch.full((n,), 3, dtype=torch.uint8, device="cuda")
                                                    for n in (256, 5000, 300 << 10, 3 << 20, 9 << 20, 40 << 20)]
    kept = [torch.empty_like(t) for t in held]
    torch.cuda.synchronize()
    taken = [(t.untyped_storage().data_ptr(), t.untyped_storage().nbytes()) for t in held]
    torch.cuda._sleep(200_000_000)       # ~0.1 s of spinning on the current stream
    for a, b in zip(kept, held):
        a.copy_(b)
        b.fill_(5)
    del a, b, held
    got = [t for t in call(side) if t is not None]
    running = not torch.cuda.current_stream().query()
    side.synchronize()
    torch.cuda.synchronize()
    assert running, "the current stream was to be busy during the call"
    for t in got:
        at = t.untyped_storage().data_ptr()
        assert not any(p <= at < p + max(n, 1) for p, n in taken), "a result stands in memory that was in use"
    assert same(name, got, want)
    assert all((t == 3).all() for t in kept), "the call wrote into memory that was in use"


@pytest.mark.parametrize("name", NAMES)
def test_results_outlive_work_queued_on_the_current_stream(cuda_ok, name):
    """A result dropped while work queued on the current stream still reads it: the call after
    it on the side stream gets other memory."""
    call = _calls()[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    first = [t for t in call(side) if t is not None]
    side.synchronize()
    want = [t.clone() for t in first]
    kept = [torch.empty_like(t) for t in first]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for a, b in zip(kept, first):
        a.copy_(b)
    del a, b, first
    for _ in range(3):
        call(side)
    with torch.cuda.stream(side):
        junk = [torch.full_like(t, 9) for t in want]
    running = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    del junk
    assert running
    assert all(torch.equal(a, b) for a, b in zip(kept, want))


@pytest.mark.parametrize("name", [n for n in NAMES if not n.endswith("decode_step")])
def test_side_stream_inside_a_captured_graph(cuda_ok, name):
    """A call on a stream that was forked off inside a capture: its memory is the graph's."""
    call = _calls()[name]
    want = [t.clone() for t in call(None) if t is not None]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        got = [t for t in call(side) if t is not None]
        cur.wait_stream(side)
        copies = [t + 0 for t in got]
    for _ in range(3):
        for t in got + copies:
            t.fill_(9)
        graph.replay()
        junk = [torch.full_like(t, 7) for t in want]      # eager memory beside the graph's
        torch.cuda.synchronize()
        assert same(name, got, want) and same(name, copies, want)
        del junk


@pytest.mark.parametrize("name", NAMES)
def test_streams_of_other_libraries(cuda_ok, name):
    """A stream that torch did not make, by its handle."""
    call = _calls()[name]
    want = [t.clone() for t in call(None) if t is not None]
    own = torch.cuda.Stream()
    other = torch.cuda.ExternalStream(own.cuda_stream, device=torch.device("cuda", torch.cuda.current_device()))
    torch.cuda.synchronize()
    got = [t for t in call(other) if t is not None]
    own.synchronize()
    assert same(name, got, want)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def test_threads_with_streams_of_their_own(cuda_ok):
    import threading
    want = {n: [t.clone() for t in c(None) if t is not None] for n, c in _calls().items()}
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        calls = _calls()
        torch.cuda.current_stream().synchronize()
        for n in NAMES[i:] + NAMES[:i]:
            if n == "chunk_fwd_noalloc":
                continue                 # (one scratch for all calls: callers take turns)
            got = [t for t in calls[n](s) if t is not None]
            s.synchronize()
            if not same(n, got, want[n]):
                bad.append((i, n))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
