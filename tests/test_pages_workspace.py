"""The page calls with a workspace of the caller's: refusals on the host (fake device addresses), and
on the GPU, graphs that are replayed at the same time, each with its own."""
import ctypes

import pytest
import torch


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("host-only checks on fake device addresses: run where no GPU is visible")
    from chunkwise_recurrent_prefill_gb300 import build_ext
    from chunkwise_recurrent_prefill_gb300.gla import load_library
    build_ext.build()
    return load_library()


def test_sizes_and_refusals(lib):
    pool, tab, st, cnt, a, c, w = (i << 36 for i in range(1, 8))
    size = lib.gla_pages_workspace_size
    assert size(8, 4, 2, 0) > 0 and size(8, 4, 2, 100) >= 100 * 2 * 8 + 4 * 4
    assert size(-1, 4, 2, 1) == 0 and size(8, 4, 2, -1) == 0 and size(8, 4, 1 << 40, 1) == 0
    need = size(8, 4, 2, 2)

    def fork(ws=w, n=need):
        return lib.gla_pages_fork_ex(vp(pool), 8, 64, vp(tab), 4, 2, vp(st), vp(cnt), vp(a), vp(c), 2,
                                     vp(ws), n, None)

    def free(ws=w, n=need):
        return lib.gla_pages_free_ex(8, vp(tab), 4, 2, vp(st), vp(cnt), vp(a), 2, vp(ws), n, None)

    def compact(ws=w, n=need):
        return lib.gla_pages_compact_ex(vp(pool), 8, 64, vp(tab), 4, 2, vp(st), vp(cnt), vp(ws), n, None)

    for call in (fork, free, compact):
        # a bad workspace is told before the device where there is one; here there is none
        assert call() in (6, 8) and call(ws=None, n=0) in (6, 8)
        assert call(n=8) in (6, 8, 9) and call(ws=w + 4) in (6, 8, 9)


def test_names():
    import chunkwise_recurrent_prefill_gb300 as pkg
    assert callable(pkg.pages_workspace_size)
    table, free = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    assert pkg.pages_workspace_size(table, free, 5) >= 5 * 2 * 8
    with pytest.raises(ValueError):
        pkg.pages_workspace_size(table.view(-1), free)


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.gpu
def test_refusals_of_a_workspace(built):
    from chunkwise_recurrent_prefill_gb300 import GLAError, pages_compact, pages_fork, pages_free
    from test_pages_gpu import Book, i32
    g = Book(8, 4, 1, 2).gpu
    one, book = i32([-1]), (g["table"], g["free"], g["count"])
    big = torch.empty(4096, dtype=torch.uint8, device="cuda")
    calls = (lambda w: pages_fork(g["pool"], *book, one, one, workspace=w),
             lambda w: pages_free(*book, one, workspace=w),
             lambda w: pages_compact(g["pool"], *book, workspace=w))
    for call in calls:
        call(big)
        for bad in (big[:8], big[4:]):
            with pytest.raises(GLAError, match="WORKSPACE"):
                call(bad)
        with pytest.raises(ValueError):
            call(big.cpu())
        with pytest.raises(ValueError):
            call(big[::2])


@pytest.mark.gpu
def test_graphs_of_one_stream_at_the_same_time(built):
    """Two pools' graphs, captured from one stream, replayed on two others without any order."""
    from chunkwise_recurrent_prefill_gb300 import pages_compact, pages_fork, pages_free, pages_workspace_size
    from test_pages_gpu import Book, i32
    s, graphs, books = torch.cuda.Stream(), [], [Book(600, 100, 2, 40, page=4096, seed=i) for i in (1, 2)]
    lists = [(i32([0] * 20), i32([0] * 20)) for _ in books]
    s.wait_stream(torch.cuda.current_stream())
    for b, (parents, children) in zip(books, lists):
        g = b.gpu
        book = (g["table"], g["free"], g["count"])
        ws = torch.empty(pages_workspace_size(g["table"], g["free"], 20), dtype=torch.uint8, device="cuda")
        none = i32([-1] * 20)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            pages_fork(g["pool"], *book, none, none, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            pages_fork(g["pool"], *book, parents, children, workspace=ws)
            pages_free(*book, parents, workspace=ws)
            pages_compact(g["pool"], *book, workspace=ws)
        graphs.append((graph, ws))
    sides = [torch.cuda.Stream() for _ in books]
    for _ in range(5):
        picks = [(b.live()[:20], b.empty()[:20]) for b in books]
        for (p, c), (parents, children) in zip(picks, lists):
            parents.copy_(i32(p))
            children.copy_(i32(c))
        torch.cuda.synchronize()
        for side, (graph, _) in zip(sides, graphs):
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for b, (p, c) in zip(books, picks):
            b.fork(p, c)
            b.release(p)
            b.compact()
            b.same()
