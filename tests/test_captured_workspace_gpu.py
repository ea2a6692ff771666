"""Calls captured into a CUDA graph with the library's own workspace: what comes between the
capture and a replay must not take that workspace away."""
import pytest
import torch

import hda_ref
from test_pages_gpu import Book, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def warm(stream, b):
    """One call of each kind on the stream (that changes nothing)."""
    from chunkwise_recurrent_prefill_gb300 import pages_fork, pages_free
    g, none = b.gpu, i32([-1, -1])
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        pages_fork(g["pool"], g["table"], g["free"], g["count"], none, none)
        pages_free(g["table"], g["free"], g["count"], none)
    torch.cuda.synchronize()


def capture(stream, b, parents, children):
    from chunkwise_recurrent_prefill_gb300 import pages_compact, pages_fork, pages_free
    g, graph = b.gpu, torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pages_fork(g["pool"], g["table"], g["free"], g["count"], parents, children)
        pages_free(g["table"], g["free"], g["count"], parents)
        pages_compact(g["pool"], g["table"], g["free"], g["count"])
    return graph


def replay(graph, b, parents, children):
    p, c = b.live()[:2], b.empty()[:2]
    parents.copy_(i32(p))
    children.copy_(i32(c))
    graph.replay()
    torch.cuda.synchronize()
    b.fork(p, c)
    b.release(p)
    b.compact()
    b.same()


def long_call(stream, T=4096):
    """A call that needs more workspace than the first allocation of 1 MB."""
    from chunkwise_recurrent_prefill_gb300 import hda_fwd, hda_workspace_size
    g = {n: hda_ref.to_gpu(t) for n, t in hda_ref.inputs(1, T, 4, 4, 4, 4, 128, 128, "bf16").items()}
    a = (g["q"], g["k"], g["v"], g["decay"])
    assert hda_workspace_size(*a) > 2 << 20
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        hda_fwd(*a, 0.1, return_state=True)
    torch.cuda.synchronize()


def test_a_larger_call_between_capture_and_replay():
    b = Book(30, 10, 2, 4, seed=6)
    parents, children = i32([0, 0]), i32([0, 0])
    s = torch.cuda.Stream()
    warm(s, b)
    graph = capture(s, b, parents, children)
    replay(graph, b, parents, children)
    long_call(s)
    torch.cuda.empty_cache()
    mine = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for _ in range(2):
        replay(graph, b, parents, children)
    assert all((t == 7).all() for t in mine)


def test_more_streams_than_the_library_keeps():
    b, other = Book(30, 10, 2, 4, seed=7), Book(30, 10, 2, 4, seed=8)
    parents, children = i32([0, 0]), i32([0, 0])
    s = torch.cuda.Stream()
    warm(s, b)
    graph = capture(s, b, parents, children)
    streams = [torch.cuda.Stream() for _ in range(24)]
    for t in streams:
        warm(t, other)
    replay(graph, b, parents, children)


def test_calls_outside_of_the_graph_have_their_own():
    """At most one allocation for the stream's next call (streams come from a pool, and this one may have
    been captured before), none after that, and none for further captures."""
    from chunkwise_recurrent_prefill_gb300.gla import workspace_allocations
    b = Book(30, 10, 2, 4, seed=9)
    parents, children = i32([0, 0]), i32([0, 0])
    s = torch.cuda.Stream()
    warm(s, b)
    graph = capture(s, b, parents, children)
    n = workspace_allocations()
    warm(s, b)
    m = workspace_allocations()
    assert m <= n + 1
    warm(s, b)
    again = capture(s, b, parents, children)
    warm(s, b)
    assert workspace_allocations() == m
    replay(graph, b, parents, children)
    replay(again, b, parents, children)


def test_a_capture_that_needs_more_than_there_is():
    """The call (3 GB of fp32 gradients of shared heads) is refused, the capture goes on."""
    from chunkwise_recurrent_prefill_gb300 import GLAError, hda_bwd, pages_free
    T, H = 1 << 18, 8
    one = torch.zeros(1, T, 1, 128, device="cuda", dtype=torch.bfloat16)
    do = torch.zeros(1, T, H, 128, device="cuda", dtype=torch.bfloat16)
    decay = torch.zeros(H, device="cuda")
    b = Book(30, 10, 2, 4, seed=10)
    rows, flag = i32([0, 0]), torch.zeros(1, device="cuda")
    known, unknown = torch.cuda.Stream(), torch.cuda.Stream()
    warm(known, b)
    for stream in (known, unknown):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            with pytest.raises(GLAError, match="WORKSPACE.*captured"):
                hda_bwd(do, one, one, one, decay, 0.1)
            if stream is known:
                pages_free(b.gpu["table"], b.gpu["free"], b.gpu["count"], rows)
            flag += 1
        r = b.live()[0]
        rows.copy_(i32([r, -1]))
        graph.replay()
        torch.cuda.synchronize()
        if stream is known:
            b.release([r])
        b.same()
    assert flag.item() == 2


def test_attention_replayed_after_a_larger_call():
    from chunkwise_recurrent_prefill_gb300 import hda_fwd
    g = {n: hda_ref.to_gpu(t) for n, t in hda_ref.inputs(1, 2048, 2, 2, 2, 2, 128, 128, "bf16", seed=3).items()}
    a = (g["q"], g["k"], g["v"], g["decay"], 0.1)
    want, want_h = hda_fwd(*a, return_state=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        hda_fwd(*a, return_state=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o, hT = hda_fwd(*a, return_state=True)
    long_call(s, T=16384)
    torch.cuda.empty_cache()
    mine = [torch.full((1 << 22,), 7, dtype=torch.uint8, device="cuda") for _ in range(32)]
    o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(hT, want_h)
    assert all((t == 7).all() for t in mine)
