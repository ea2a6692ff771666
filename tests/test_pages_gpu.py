"""Pages of a state pool against a sequential walk on the host (all results are exact)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Book:
    """Pool, table, free stack and count on the host, and the same on the GPU."""

    def __init__(self, P, R, M, live_rows, page=16, seed=0, holes=False):
        g = torch.Generator("cpu").manual_seed(seed)
        self.P, self.R, self.M = P, R, M
        perm = torch.randperm(P, generator=g).tolist()
        self.table = [[-1] * M for _ in range(R)]
        for r in torch.randperm(R, generator=g).tolist()[:live_rows]:
            for m in range(M):
                if not (holes and m % 3 == 1):
                    self.table[r][m] = perm.pop()
        self.free = perm
        self.pool = torch.randn(P, page, generator=g)
        self.gpu = dict(
            pool=self.pool.cuda(), table=torch.tensor(self.table, dtype=torch.int32).view(R, M).cuda(),
            free=torch.tensor(perm + [-7] * (P - len(perm)), dtype=torch.int32).cuda(),
            count=torch.tensor([len(perm)], dtype=torch.int32).cuda())

    def live(self):
        return [r for r in range(self.R) if any(p >= 0 for p in self.table[r])]

    def empty(self):
        return [r for r in range(self.R) if all(p < 0 for p in self.table[r])]

    def fork(self, parents, children):
        before = [list(r) for r in self.table]
        bad, named = False, set()
        for a, c in zip(parents, children):
            if a < 0 or c < 0:
                continue
            if a >= self.R or c >= self.R:
                bad = True
                continue
            if c in named or any(p >= 0 for p in before[c]):
                bad = True
                named.add(c)
                continue
            named.add(c)
            for m in range(self.M):
                if before[a][m] >= 0:
                    if not self.free:
                        bad = True
                        continue
                    self.table[c][m] = self.free.pop()
                    self.pool[self.table[c][m]] = self.pool[before[a][m]]
        return bad

    def release(self, rows):
        out, bad = [], False
        for r in rows:
            if r >= self.R:
                bad = True
            elif r >= 0:
                out += [p for p in self.table[r] if p >= 0]
                self.table[r] = [-1] * self.M
        self.free += out[::-1]
        return bad

    def compact(self):
        used = sorted(p for row in self.table for p in row if p >= 0)
        holes = sorted(set(range(len(used))) - set(used))
        to = dict(zip([p for p in used if p >= len(used)], holes))
        for a, c in to.items():
            self.pool[c] = self.pool[a]
        self.table = [[to.get(p, p) if p >= 0 else -1 for p in row] for row in self.table]
        self.free = list(range(self.P - 1, len(used) - 1, -1))

    def same(self, status=0):
        from chunkwise_recurrent_prefill_gb300 import last_device_status
        assert last_device_status() == status
        assert self.gpu["table"].tolist() == self.table
        assert self.gpu["count"].item() == len(self.free)
        assert self.gpu["free"].tolist()[:len(self.free)] == self.free
        assert torch.equal(self.gpu["pool"].cpu(), self.pool)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def do_fork(b, parents, children):
    from chunkwise_recurrent_prefill_gb300 import pages_fork
    g = b.gpu
    pages_fork(g["pool"], g["table"], g["free"], g["count"], i32(parents), i32(children))
    return 12 if b.fork(parents, children) else 0


def do_free(b, rows):
    from chunkwise_recurrent_prefill_gb300 import pages_free
    g = b.gpu
    pages_free(g["table"], g["free"], g["count"], i32(rows))
    return 12 if b.release(rows) else 0


def do_compact(b):
    from chunkwise_recurrent_prefill_gb300 import pages_compact
    g = b.gpu
    pages_compact(g["pool"], g["table"], g["free"], g["count"])
    b.compact()


@pytest.mark.parametrize("P,R,M,live,page", [(1, 1, 1, 1, 4), (9, 4, 1, 3, 16), (40, 8, 3, 5, 20),
                                             (2500, 300, 4, 150, 8), (64, 20, 1, 10, 9000),
                                             (30, 6, 2, 6, 8196)])
def test_a_life_of_forks_frees_and_compactions(P, R, M, live, page):
    b = Book(P, R, M, live, page, seed=P, holes=M > 2)
    g = torch.Generator("cpu").manual_seed(R)
    for _ in range(4):
        rows, empty = b.live(), b.empty()
        if rows:
            n = int(torch.randint(1, R + 1, (1,), generator=g))
            pick = [rows[i] for i in torch.randint(0, len(rows), (n,), generator=g).tolist()]
            b.same(do_fork(b, pick, (empty + [-1] * n)[:n]))
        some = torch.randperm(R, generator=g).tolist()[:R // 2]
        b.same(do_free(b, some))
        do_compact(b)
        b.same()


def test_freeing_a_fork_restores_the_stack():
    b = Book(60, 10, 3, 4, seed=1)
    before = list(b.free)
    kids = b.empty()[:5]
    do_fork(b, (b.live() * 2)[:5], kids)
    assert len(b.free) == len(before) - 15
    do_free(b, kids)
    b.same()
    assert b.free == before


def test_fork_requests_that_cannot_be_met():
    b = Book(20, 10, 2, 4, seed=2)
    a, e = b.live(), b.empty()
    # skipped, out of range (both ways), a child with pages, a child listed twice, a parent that
    # is empty and is the child of another request
    b.same(do_fork(b, [-1, a[0], 10, a[1], a[0], a[1], e[0], a[2]],
                   [e[3], -1, e[1], 99, a[2], e[0], e[2], e[0]]))
    # the stack runs out half way through
    b = Book(11, 10, 2, 4, seed=3)
    b.same(do_fork(b, b.live()[:3], b.empty()[:3]))
    assert not b.free
    b.same(do_fork(b, b.live()[:1], b.empty()[:1]))


def test_free_rows_listed_twice_and_out_of_range():
    b = Book(20, 6, 3, 5, seed=4)
    r = b.live()
    b.same(do_free(b, [r[0], -1, r[1], r[0], b.empty()[0], 6, 1 << 30]))


def test_copy():
    from chunkwise_recurrent_prefill_gb300 import last_device_status, pages_copy
    pool = torch.randn(9, 3, 20, device="cuda")
    want = pool.clone()
    want[[7, 2]] = want[[0, 0]]
    pages_copy(pool, i32([0, 0, -1, 4, 5]), i32([7, 2, 3, -1, 5]))
    assert last_device_status() == 0 and torch.equal(pool, want)
    pages_copy(pool, i32([1, 9, 3]), i32([8, 1, 9]))
    want[8] = want[1]
    assert last_device_status() == 12 and torch.equal(pool, want)
    half = torch.randn(5, 24, device="cuda", dtype=torch.bfloat16)
    pages_copy(half, i32([1]), i32([4]))
    assert torch.equal(half[4], half[1])
    pages_copy(half, i32([]), i32([]))


def test_in_a_graph():
    """The bookkeeping never visits the host: a fork and a free replay with what the buffers hold."""
    from chunkwise_recurrent_prefill_gb300 import pages_fork, pages_free
    b = Book(30, 10, 2, 4, seed=5)
    g = b.gpu
    parents, children = i32([0, 0]), i32([0, 0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):      # the stream's workspace is made before the capture
        pages_fork(g["pool"], g["table"], g["free"], g["count"], i32([-1, -1]), i32([-1, -1]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pages_fork(g["pool"], g["table"], g["free"], g["count"], parents, children)
        pages_free(g["table"], g["free"], g["count"], parents)
    for _ in range(2):
        p, c = b.live()[:2], b.empty()[:2]
        parents.copy_(i32(p))
        children.copy_(i32(c))
        graph.replay()
        torch.cuda.synchronize()
        b.fork(p, c)
        b.release(p)
        b.same()


def test_refusals():
    from chunkwise_recurrent_prefill_gb300 import (GLAError, pages_compact, pages_copy, pages_fork,
                                                   pages_free)
    g = Book(8, 4, 1, 2).gpu
    one = i32([0])
    with pytest.raises(ValueError):
        pages_copy(g["pool"].cpu(), one, one)
    with pytest.raises(ValueError):
        pages_copy(g["pool"].t(), one, one)
    with pytest.raises(TypeError):
        pages_copy(g["pool"], one.long(), one)
    with pytest.raises(ValueError):
        pages_copy(g["pool"], one, i32([0, 1]))
    with pytest.raises(GLAError, match="MISALIGNED"):
        pages_copy(torch.zeros(4, 3, device="cuda"), one, one)     # pages of 12 bytes
    with pytest.raises(ValueError):
        pages_fork(g["pool"], g["table"].view(-1), g["free"], g["count"], one, one)
    with pytest.raises(ValueError):
        pages_fork(g["pool"], g["table"], g["free"][:4], g["count"], one, one)
    with pytest.raises(GLAError, match="ALIAS"):
        pages_free(g["table"], g["free"], g["count"], g["free"])
    with pytest.raises(TypeError):
        pages_compact(g["pool"], g["table"].long(), g["free"], g["count"])
