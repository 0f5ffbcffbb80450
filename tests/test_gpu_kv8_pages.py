"""GPU parity of the page book against the oracle: tables, counts and moves are whole numbers and equal, copied pages
equal byte for byte."""
import numpy as np
import pytest

from oracle import kv8_pages as pages
from quantized_linear_layers_packed_amd import qlin
from tests.gpu_util import say, torch_cuda

pytestmark = pytest.mark.gpu


def up(x, dtype=np.int32):
    return torch_cuda().from_numpy(np.ascontiguousarray(np.asarray(x, dtype))).cuda()


class Book:
    """A book on host and device; every call runs on both and compares all that it may change."""

    def __init__(self, num_pages, rows, stride, page_size=16):
        self.page_size = page_size
        self.refs, self.table = np.zeros(num_pages, np.int32), np.full((rows, stride), -1, np.int32)
        self.upload()

    def upload(self):
        self.d_refs, self.d_table = up(self.refs), up(self.table)
        self.book = qlin.Kv8Book(self.d_refs, self.d_table, self.page_size)

    def deal(self, rng, held):
        """Random pages to the first held[b] entries of each row."""
        order, at = rng.permutation(len(self.refs)), 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            self.refs[order[at:at + n]] = 1
            at += n
        self.upload()

    def check(self, want=None, moves=None):
        torch_cuda().cuda.synchronize()
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        assert np.array_equal(self.d_refs.cpu().numpy(), self.refs)
        if want is not None:
            assert np.array_equal(moves.cpu().numpy(), np.array(want, np.int32))

    def moves(self, n):
        return up(np.full((1 + n, 2), 77))

    def grow(self, lens):
        m = self.moves(0)
        qlin.qlin_kv8_grow(self.book, up(lens), m)
        want = pages.grow(self.refs, self.table, self.page_size, lens)
        self.check(want, m)
        return want[0]

    def fork(self, parents, children, lens):
        m = self.moves(len(parents))
        qlin.qlin_kv8_fork(self.book, up(parents), up(children), up(lens), m)
        want = pages.fork(self.refs, self.table, self.page_size, parents, children, lens)
        self.check(want, m)
        return want[0]

    def free(self, rows, begin=None, end=None):
        qlin.qlin_kv8_free(self.book, up(rows), None if begin is None else up(begin), None if end is None else up(end))
        pages.free(self.refs, self.table, self.page_size, rows, begin, end)
        self.check()

    def compact(self, most):
        m = self.moves(most)
        qlin.qlin_kv8_compact(self.book, m)
        want = pages.compact(self.refs, self.table, most)
        self.check(want, m)
        return want[0]


@pytest.mark.parametrize("num_pages,rows,stride,page_size,steps", [(300, 7, 40, 16, 60), (5000, 40, 70, 64, 25), (37, 3, 9, 128, 60)])
def test_a_serving_history_matches_the_oracle(num_pages, rows, stride, page_size, steps):
    say(f"kv8 pages: history on {num_pages} pages, {rows} x {stride}")
    r = np.random.default_rng(num_pages)
    b = Book(num_pages, rows, stride, page_size)
    lens = np.zeros(rows, np.int64)
    for step in range(steps):
        what = r.integers(0, 6)
        if what <= 1:                                    # tokens for some rows, single ones and prompts
            more = lens + r.integers(0, 2, rows) * r.choice([1, page_size, 5 * page_size + 3], rows)
            more = np.minimum(more, stride * page_size)
            if b.grow(more)[1] == 0:
                lens = more
        elif what == 2 and rows > 1:
            kids = r.permutation(rows)[:r.integers(1, rows)]
            others = [p for p in range(rows) if p not in kids]
            parents = r.choice(others, len(kids))
            part = (lens[parents] * r.uniform(0, 1, len(kids))).astype(np.int64)
            part = np.where(r.uniform(size=len(kids)) < 0.5, lens[parents], part)
            if b.fork(parents, kids, part)[1] == 0:
                lens[kids] = part
        elif what == 3:
            gone = r.permutation(rows)[:r.integers(1, rows + 1)]
            b.free(gone)
            lens[gone] = 0
        elif what == 4:                                  # behind a window
            b.free(np.arange(rows), np.full(rows, 4), np.maximum(lens - 3 * page_size, 0))
        else:
            b.compact(int(r.integers(1, num_pages // 2)))
    held = b.table[(b.table >= 0)]
    assert np.array_equal(np.bincount(held, minlength=num_pages), b.refs)


@pytest.mark.parametrize("num_pages", [16384, 16385, 16383, 40001, 70000])
def test_pools_of_several_steps(num_pages):
    """The only free pages at the end, in the middle and spread; more are wanted than one step of the search holds."""
    r = np.random.default_rng(num_pages)
    stride = 9000
    b = Book(num_pages, 5, stride)
    b.refs[:] = 1
    free = np.sort(r.permutation(num_pages)[:9])
    b.refs[free] = 0
    b.upload()
    assert b.grow([16 * 4, 0, 5, 16, 17]) == (8, 0)
    assert b.grow([16 * 4, 0, 5, 16, 49]) == (0, 1)
    b.refs[num_pages - 300:] = 0
    b.upload()
    assert b.fork([0, 0, 3], [1, 2, 4], [64, 17, 3]) == (3, 0)
    b = Book(num_pages, 5, stride)
    assert b.grow([16 * n for n in (3000, 1, 5000, 0, 4000)]) == (12001, 0)
    assert b.grow([16 * n for n in (3000, 9000, 9000, 9000, 9000)])[1] == max(0, 12001 + 8999 + 4000 + 9000 + 5000 - num_pages)
    b.free([0, 3, 2], [0, 0, 160], [16 * 2900, 999, 16 * 1000])
    for most in (7, 3000, num_pages // 2):
        b.compact(most)


def test_long_rows_are_searched_back_from_the_end():
    """Rows whose last held entry lies far before the wanted ones, at the borders of the search's steps, or nowhere."""
    b = Book(40000, 20, 2100)
    r = np.random.default_rng(3)
    b.deal(r, [1, 2, 63, 64, 65, 511, 512, 513, 1023, 1024, 1025, 1600, 0, 0, 2099, 2100, 2098, 88, 1587, 1588])
    b.table[17, 5:80] = -1                               # a hole before the last held entry
    b.refs[:] = np.bincount(b.table[b.table >= 0], minlength=40000)
    b.upload()
    assert b.grow([16 * 2100 - 5] * 12 + [0, 16 * 2100] + [16 * 2100] * 5 + [16 * 1589 + 1])[1] == 0


@pytest.mark.parametrize("per_row", [200, 600])
@pytest.mark.parametrize("rows", [31, 32, 33, 71, 600])
def test_many_rows_with_much_to_find(rows, per_row):
    """Rows of every kind side by side: nothing held, a few entries, holes before the last held one, nothing wanted; lengths
    around the number of entries that are looked at first, and at the borders of the search's steps.  The smaller pool
    does not hold all that is wanted."""
    r = np.random.default_rng(rows)
    b = Book(per_row * rows, rows, 1100)
    held = r.choice([0, 0, 1, 2, 3, 4, 5, 60, 64, 65, 255, 256, 257, 300], rows)
    b.deal(r, held)
    for row in range(0, rows, 3):
        b.table[row, :max(held[row] - 2, 0)] = -1
    b.refs[:] = np.bincount(b.table[b.table >= 0], minlength=len(b.refs))
    b.upload()
    for more in ([0, 1, 2, 3, 4, 5, 6], [0, 100, 256, 255, 257], [1, 3, 4, 5]):
        want = np.minimum(held + r.choice(more, rows), 1100)
        lens = want * 16 - r.integers(0, 16, rows)
        lens[r.uniform(size=rows) < 0.1] = r.choice([0, -5, 1])
        assert b.grow(lens)[1] == 0 or per_row == 200
        held = np.array([max([e + 1 for e in range(1100) if b.table[row, e] >= 0], default=0) for row in range(rows)])


def test_many_rows_and_forks():
    r = np.random.default_rng(9)
    b = Book(60000, 32767, 3)
    lens = r.integers(0, 20, 32767)
    lens[16384:] = 0
    b.grow(lens)
    n = 16383
    parents, kids = r.integers(0, 16384, n), 16384 + r.permutation(n)
    assert b.fork(parents, kids, lens[parents]) == (n, 0)
    b.free(r.permutation(32767)[:30000])
    b.compact(20000)


def test_fork_refuses_what_does_not_fit_and_skips_padding():
    b = Book(64, 6, 8)
    b.deal(np.random.default_rng(4), [8, 3, 0, 0, 2, 0])
    for bad in (([0, 0], [2, 2], [5, 5]), ([0, 2], [2, 3], [5, 5]), ([0, 1], [0, 3], [5, 5]), ([6, 1], [2, 3], [5, 5]),
                ([0, 1], [2, 6], [5, 5]), ([0, 1], [2, 3], [129, 5]), ([0, 1], [2, 3], [5, -1])):
        assert b.fork(*bad) == (0, -1)
    assert b.fork([-1, 0, 0, 1], [2, -5, 3, 4], [3, 4, 100, 33]) == (4, 0)       # row 4 held pages: back in the pool
    assert b.fork([0, 0], [2, 5], [128, 0]) == (2, 0)                            # nothing to copy; a child of no tokens
    b.table[0, 2] = -1                                                           # given back behind a window
    b.refs[:] = np.bincount(b.table[b.table >= 0], minlength=64)
    b.upload()
    assert b.fork([0, 0], [2, 3], [35, 50]) == (2, 0)                            # the page to be copied is not there; it is
    b.grow([128, 128, 0, 0, 0, 128])
    b.grow([0, 0, 128, 128, 128, 0])
    assert b.fork([0, 0], [4, 5], [20, 33])[1] == 0
    b.refs[b.refs == 0] = 1                                                      # held by something outside the table
    b.upload()
    assert b.fork([0, 0], [4, 5], [20, 100]) == (0, 2)


def test_free_twice_and_out_of_range():
    b = Book(64, 4, 8)
    b.deal(np.random.default_rng(5), [8, 8, 8, 8])
    b.table[3, 5] = 9999                                                         # not a page: given back as nothing
    b.refs[:] = np.bincount(b.table[(b.table >= 0) & (b.table < 64)], minlength=64)
    b.upload()
    b.free([1, 1, 1, -1, 4, 3], [0, 16, 40, 0, 0, 70], [64, 100, 128, 999, 999, (1 << 31) - 1])
    b.free([0, 0, 0])
    b.free([2], [-50], [-3])
    b.free([2], [50], [20])
    b.free([2], None, [33])
    b.free([2], [33], None)


def layers(r, count, pages_, H, P, D):
    torch = torch_cuda()
    out = []
    for _ in range(count):
        k, v = (r.integers(-127, 128, s).astype(np.int8) for s in ((pages_, H, P, D), (pages_, H, D, P)))
        out.append([torch.from_numpy(x).cuda() for x in (k, v, r.uniform(0.1, 1, (pages_, H, 2)).astype(np.float32))])
    return out


@pytest.mark.parametrize("H,P,D,count,most", [(8, 64, 128, 2, 40), (1, 16, 64, 3, 7), (3, 32, 256, 1, 9), (5, 128, 64, 33, 4), (65, 16, 64, 70, 3)])
def test_copy_pages(H, P, D, count, most):
    torch = torch_cuda()
    r = np.random.default_rng(H)
    say(f"kv8 copy_pages H={H} P={P} D={D} layers={count}")
    n = 2 * most + 3
    a, b = layers(r, count, n, H, P, D), layers(r, count, n + 5, H, P, D)
    make = lambda x: qlin.Kv8Caches([qlin.Kv8Cache(*t) for t in x])                              # noqa: E731
    order = r.permutation(n)
    pairs = np.stack([order[:most], order[most:2 * most]], 1)
    pairs[0] = (-1, -1)
    if most > 5:
        pairs[3], pairs[4] = (n, order[1]), (order[2], n + 5)      # outside their pools
    for source, to, limit in ((a, a, n), (a, b, n + 5)):
        want = [[x.clone() for x in t] for t in to]
        for s, d in pairs[:-1]:
            if 0 <= s < n and 0 <= d < limit:
                for w, x in zip(want, source):
                    for p, q in zip(w, x):
                        p[d] = q[s]
        moves = up(np.concatenate([[[most - 1, 0]], pairs]))        # the last pair is not counted
        qlin.qlin_kv8_copy_pages(make(to), make(source), moves)
        torch.cuda.synchronize()
        for w, x in zip(want, to):
            for p, q in zip(w, x):
                assert torch.equal(p, q)


def test_copy_pages_takes_one_cache_and_no_more_pairs_than_listed():
    torch = torch_cuda()
    [t] = layers(np.random.default_rng(1), 1, 6, 2, 16, 64)
    c = qlin.Kv8Cache(*t)
    before = [x.clone() for x in t]
    for count in (0, -1):
        qlin.qlin_kv8_copy_pages(c, c, up([[count, 0], [0, 1], [2, 3]]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(t, before))
    qlin.qlin_kv8_copy_pages(c, c, up([[1000, 0], [0, 1], [2, 3]]))
    torch.cuda.synchronize()
    for x, y in zip(t, before):
        assert torch.equal(x[1], y[0]) and torch.equal(x[3], y[2]) and torch.equal(x[[0, 2, 4, 5]], y[[0, 2, 4, 5]])


def test_a_captured_step_replays_on_the_book_as_it_stands():
    """Release, fork, grow, compact and copy in one graph, replayed as lengths change, against eager calls on a copy."""
    torch = torch_cuda()
    r = np.random.default_rng(6)
    b = Book(400, 9, 30)
    b.deal(r, [20, 11, 0, 0, 0, 0, 7, 0, 0])
    [t] = layers(r, 1, 400, 2, 16, 64)
    cache = qlin.Kv8Cache(*t)
    kids, parents, lens, grown = up([2, 3, 4, 5]), up([0, 0, 1, 6]), up([300, 17, 160, 112]), up([0] * 9)
    m_fork, m_grow, m_compact = b.moves(4), b.moves(0), b.moves(200)

    def step(book, cache):
        qlin.qlin_kv8_free(book, kids)
        qlin.qlin_kv8_fork(book, parents, kids, lens, m_fork)
        qlin.qlin_kv8_copy_pages(cache, cache, m_fork)
        qlin.qlin_kv8_grow(book, grown, m_grow)
        qlin.qlin_kv8_compact(book, m_compact)
        qlin.qlin_kv8_copy_pages(cache, cache, m_compact)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step(b.book, cache)
    for i in range(4):
        twin = [x.clone() for x in (b.d_refs, b.d_table, *t)]
        lens.copy_(up([300 - 30 * i, 17 + i, 160, 112 - 16 * i]))
        grown.copy_(up([0, 0, 0, 0, 0, 0, 112, 5 + 40 * i, 100 * i]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        moves = [x.clone() for x in (m_fork, m_grow, m_compact)]
        step(qlin.Kv8Book(twin[0], twin[1], 16), qlin.Kv8Cache(*twin[2:]))
        torch.cuda.synchronize()
        for x, y in zip((b.d_refs, b.d_table, *t, *moves), (*twin, m_fork, m_grow, m_compact)):
            assert torch.equal(x, y)
        assert int(moves[1][0, 1]) == 0 and int(moves[0][0, 1]) == 0


@pytest.mark.parametrize("rows,prefix", [(3, 700), (80, 40), (80, 700)])
def test_pages_that_a_fork_never_had_are_not_dealt_out(rows, prefix):
    """Prefixes that end in pages their parent gave back, grown by a token, by pages, and far; few rows and many, which are
    searched in different ways, and where the mark is among the entries that are looked at first."""
    b = Book(200 * rows, rows, 100)
    b.deal(np.random.default_rng(rows), [60] + [0] * (rows - 1))
    b.free([0], [0], [900])
    kids = np.arange(1, rows)
    lens = np.concatenate([[0], prefix + np.arange(rows - 1) % 33])
    assert b.fork([0] * len(kids), kids, lens[1:]) == (len(kids), 0)
    last = (lens[1:] - 1) // 16
    assert (b.table[kids, last] == pages.GONE).all()
    for more in (0, 1, 40, 700):
        assert b.grow(np.where(lens > 0, lens + more, 0))[1] == 0
        assert (b.table[kids, last] == pages.GONE).all() and all((b.table[k, :e] == -1).all() for k, e in zip(kids, last))
    b.compact(100)
    b.free([1])
    assert b.grow([0, 16 * 50] + [0] * (rows - 2)) == (50, 0)


def test_tokens_of_a_fork_whose_pages_are_gone_stay_hidden():
    """Book, append and attention together: a child whose prefix its parent had given back sees its own new tokens and
    nothing of what lies in the pool's pages."""
    torch = torch_cuda()
    P, D, H = 16, 64, 1
    b = Book(30, 2, 8, P)
    [t] = layers(np.random.default_rng(2), 1, 30, H, P, D)
    t[2].fill_(float("nan"))                                       # what others left: whoever sees it gets NaN
    cache = qlin.Kv8Cache(*t)
    b.grow([100, 0])
    b.free([0], [0], [48])
    b.fork([0], [1], [40])
    b.grow([0, 50])                                                # tokens 40 .. 47 have no page, 48 and 49 have
    x = torch.ones((10, 3 * H, D), dtype=torch.float16, device="cuda")
    y = torch.empty((10, H, D), dtype=torch.float16, device="cuda")
    batch = qlin.Kv8Batch(up([0, 0, 10]), up([100, 50]), b.d_table, 10, 10, 50)
    qlin.qlin_kv8_append(cache, batch, None, x[:, H:2 * H], x[:, 2 * H:], qlin.QLIN_F16, H, None, None, 0, qlin.QLIN_ROPE_HALF, None)
    need = qlin.qlin_kv8_attention_workspace_bytes(cache, batch, H)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    qlin.qlin_kv8_attention_scored(cache, batch, x[:, :H], qlin.QLIN_F16, H, 0.125, 0, 0, qlin.Kv8Scoring(20.0), y, ws)
    torch.cuda.synchronize()
    assert not y[:8].any()                                         # they see nothing, themselves among it
    assert torch.equal(y[8:], x[8:, :H])                           # ones, in codes of 127 and a scale of 1 / 127


def test_the_widest_table():
    """One row of as many entries as a table may have: ranges at its end, lists of padding, pages that move."""
    torch = torch_cuda()
    stride, n = (1 << 31) - 1, 64
    table = torch.full((1, stride), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(n, dtype=torch.int32, device="cuda")
    places = torch.tensor([0, 5, 1 << 27, stride - 20000, stride - 16384, stride - 300, stride - 1], device="cuda")
    pages_of = torch.tensor([50, 3, 60, 7, 20, 33, 63], dtype=torch.int32, device="cuda")
    table[0, places] = pages_of
    refs[pages_of.long()] = 1
    book = qlin.Kv8Book(refs, table, 16)
    say("kv8 pages: a row of 2^31 - 1 entries: fork of padding")
    m = up(np.full((2, 2), 77))
    qlin.qlin_kv8_fork(book, up([-1]), up([0]), up([5]), m)
    torch.cuda.synchronize()
    assert m.tolist() == [[1, 0], [-1, -1]] and int((refs == 1).sum()) == 7
    say("free of what lies behind 2^31 - 17 tokens")
    qlin.qlin_kv8_free(book, up([0]), up([(1 << 31) - 17]))
    torch.cuda.synchronize()
    assert table[0, places].tolist() == [50, 3] + [-1] * 5 and refs.nonzero().flatten().tolist() == [3, 50]
    table[0, places] = pages_of
    refs[pages_of.long()] = 1
    say("free up to 2^31 - 1 tokens, a range that ends before the row does")
    qlin.qlin_kv8_free(book, up([0]), None, up([(1 << 31) - 1]))
    torch.cuda.synchronize()
    assert table[0, places].tolist() == [-1, -1] + pages_of.tolist()[2:] and int((refs == 1).sum()) == 5
    say("compact and the rest")
    m = up(np.full((1 + 32, 2), 77))
    qlin.qlin_kv8_compact(book, m)
    torch.cuda.synchronize()
    assert table[0, places].tolist() == [-1, -1, 1, 4, 3, 2, 0] and m[0].tolist() == [5, 0]
    qlin.qlin_kv8_free(book, up([0]))
    torch.cuda.synchronize()
    assert not refs.any() and int(table.amax()) == -1


@pytest.mark.parametrize("num_pages,count", [(16380, 4095), (16384, 4096), (16388, 4097), (32772, 8193), (70000, 17500)])
def test_compactions_of_many_pages(num_pages, count):
    """Every other page in use: a quarter of the pool moves, more than LDS holds sources of at once.  The table looks its
    entries up in all of the moves or in some of them; also a small one, beside pages that are held outside of it."""
    r = np.random.default_rng(num_pages)
    used = np.arange(1, num_pages, 2)
    for rows, stride in ((5, 9000), (3, 300)):
        for most in (num_pages // 2, count, count - 1, 4100):
            b = Book(num_pages, rows, stride)
            flat = b.table.reshape(-1)
            n = min(len(flat), len(used))
            flat[r.permutation(len(flat))[:n]] = r.permutation(used)[:n]
            b.refs[used] = 1
            b.upload()
            assert b.compact(most) == (min(count, most), 0)
