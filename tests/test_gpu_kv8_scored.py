"""GPU parity of the 8-bit cache's attention with other scores and masks (capped scores, a bias by distance, prefixes,
documents) against the oracle, within bounds derived from its roundings; and of a serving history with forked sequences."""
import numpy as np
import pytest

from oracle import kv8 as okv
from oracle import kv8_pages as okp
from quantized_linear_layers_packed_amd import qlin
from tests.gpu_util import say, torch_cuda, workspace
from tests.test_gpu_kv8 import Setup, attention_bound, back, run_append, run_attention, to16
from tests.test_gpu_kv8_pages import Book, up

pytestmark = pytest.mark.gpu

F16, BF16 = qlin.QLIN_F16, qlin.QLIN_BF16
F = np.float32


def alibi(heads):
    return (2.0 ** (-8.0 * (np.arange(heads) + 1) / heads)).astype(F)


def scored_bound(A, Y, score, peak, far, D, L, dtype, cap):
    """attention_bound, and what capping and the bias add to a score's error, in the exponent's argument of numerator and
    denominator:

    cap:  tanh as 1 - 2 r with r = 1 / (E + 1), E = e^(2 x / cap): E, the sum and r are off by at most 2^-23, 2^-24 and
          2^-23 of themselves, so 2 cap r by 2 cap 2^-23 (E / (E + 1) + 1.5) r <= 3 cap 2^-23, and the last
          multiply-add by 2^-24 of a value below cap: under cap 2^-21 (x's own error counts as without a cap, tanh is flatter)
    sums: the capped score, the log2 of the value scale (below 8 here) and the bias added in fp32, 2^-24 of their
          magnitudes each, twice; the slope times log2(e) is off by 2^-23 of itself
    """
    extra = 2 * (cap * 2.0 ** -21 + 2.0 ** -22 * (far[..., None] + cap + 8))
    return attention_bound(A, Y, score, peak, D, L, dtype) + extra * A


def run_scored(s, G, dtype, Q=None, window=0, sinks=0, cap=0.0, slopes=None, prefix=None, starts=None, scale=None):
    torch = torch_cuda()
    Hq = s.Hk * G
    if Q is None:
        Q = (12.0 if cap else 3.0) * s.rng.standard_normal((s.T, Hq, s.D))
    d, Q = to16(Q, dtype)
    Y = torch.full((s.T, Hq, s.D), 7.0, dtype=d.dtype, device="cuda")
    scale = scale or 1.0 / np.sqrt(s.D)
    dev = [None if x is None else up(x, t) for x, t in ((slopes, F), (prefix, np.int32), (starts, np.int32))]
    need = qlin.qlin_kv8_attention_workspace_bytes(s.cache, s.batch, Hq, window, sinks)
    ws = workspace(need)
    qlin.qlin_kv8_attention_scored(s.cache, s.batch, d, dtype, Hq, scale, window, sinks, qlin.Kv8Scoring(cap, *dev), Y, ws)
    torch.cuda.synchronize()
    if need:
        assert not ws[:16384].any(), "arrival counters left behind"
    return Y, Q, scale


def check_scored(s, G, dtype, **kw):
    Y, Q, scale = run_scored(s, G, dtype, **kw)
    get = kw.get
    ref = okv.attention_scored(s.k, s.v, s.scales, s.offsets, s.kv_lens, s.table, Q, float(F(scale)), get("window", 0),
                               get("sinks", 0), float(F(get("cap", 0.0))), get("slopes"), get("prefix"), get("starts"))
    Yr, A, score, peak, far = ref
    tol = scored_bound(A, Yr, score, peak, far, s.D, max(s.kv + [1]), dtype, get("cap", 0.0))
    owned = slice(0, int(s.offsets[-1]))
    err = np.abs(back(Y).astype(np.float64)[owned] - Yr[owned])
    say(f"  worst error / bound: {float((err / np.maximum(tol[owned], 1e-30)).max()):.3f}")
    assert (err <= tol[owned]).all()
    return Y


def documents(s, every):
    """starts of the batch's tokens: a document of `every` tokens after another, in each sequence."""
    return np.array([p // every * every for n, m in zip(s.new, s.kv) for p in range(m - n, m)] + [0] * (s.T - sum(s.new)), np.int32)


SHAPES = [
    # dtype, D, P, Hk, G, new, kv
    (F16, 128, 64, 2, 4, [1, 1, 1], [1, 64, 300]),
    (BF16, 64, 16, 1, 7, [1, 2, 3], [40, 2, 515]),
    (F16, 256, 32, 1, 16, [1, 1], [31, 450]),
    (BF16, 256, 64, 2, 3, [1, 4], [260, 90]),
    (BF16, 128, 16, 1, 8, [5, 5], [5, 400]),                       # 40 rows
    (F16, 64, 128, 2, 4, [9, 1], [500, 129]),
    (F16, 128, 32, 1, 4, [200, 129, 1], [333, 129, 64]),           # prompts
    (BF16, 64, 16, 1, 8, [70, 90], [100, 300]),
    (F16, 256, 32, 1, 2, [130, 20], [190, 400]),
    (BF16, 128, 128, 2, 2, [257], [700]),
    (F16, 128, 64, 1, 8, [90, 1, 0, 9, 2, 40, 1, 5, 130], [300, 250, 9, 9, 2, 190, 63, 5, 200]),   # both kernels
]
FORMS = {
    "cap": dict(cap=20.0), "bias": dict(slopes=True), "cap bias": dict(cap=50.0, slopes=True),
    "prefix": dict(prefix=True), "documents": dict(starts=37), "documents prefix cap": dict(starts=150, prefix=True, cap=30.0),
    "window": dict(window=33, sinks=3, cap=30.0), "window prefix bias": dict(window=100, sinks=0, prefix=True, slopes=True),
    "window documents": dict(window=20, sinks=5, starts=90), "all": dict(window=50, sinks=70, starts=150, prefix=True, cap=10.0, slopes=True),
}


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dtype,D,P,Hk,G,new,kv", SHAPES)
def test_scored_attention_within_its_rounding_bounds(dtype, D, P, Hk, G, new, kv, form):
    say(f"kv8 scored attention {form}: D={D} P={P} Hk={Hk} G={G} new={new} kv={kv}")
    s = Setup(31, D, P, Hk, new, kv)
    kw = dict(FORMS[form])
    if "slopes" in kw:
        kw["slopes"] = alibi(Hk * G)
    if "prefix" in kw:                                               # inside the new tokens, all, none, past the end
        kw["prefix"] = [[m - n // 3, m, 0, m + 99][b % 4] for b, (n, m) in enumerate(zip(new, kv))]
    if "starts" in kw:
        kw["starts"] = documents(s, kw["starts"])
    check_scored(s, G, dtype, **kw)


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("cap", [0.0, 2.0 ** -10, 0.5, 1024.0])
def test_caps_at_their_limits(new, cap):
    s = Setup(32, 128, 32, 1, [new, new], [500, 77])
    check_scored(s, 4, F16, cap=cap)
    check_scored(s, 4, BF16, cap=cap, Q=300.0 * s.rng.standard_normal((s.T, 4, 128)))      # |x| far above small caps


@pytest.mark.parametrize("new", [1, 60])
def test_infinite_scores_are_capped(new):
    """Scores past fp32's range: cap or -cap by their sign, so a plain mean over the tokens of the higher one."""
    s = Setup(33, 64, 16, 1, [new], [300])
    s.scales[..., 0] = 2.0 ** 120
    s.upload()
    Q = np.zeros((s.T, 4, 64))
    Q[..., 0] = 2.0 ** 13
    Y = back(run_scored(s, 4, F16, Q=Q, cap=30.0, scale=1.0)[0])
    k, v, _ = okv.values(s.k, s.v, s.scales, s.table[0], 300, 0)
    for i in range(new):
        seen = k[:300 - new + i + 1, 0]
        top = np.sign(seen).max()
        ref = v[:len(seen)][np.sign(seen) == top].mean(axis=0)
        # -cap beside cap weighs e^-60; products of 0 with the infinite scale of a code of 0 do not occur: k is finite
        assert np.allclose(Y[i], ref, rtol=2.0 ** -9, atol=2.0 ** -9 * np.abs(v).max())


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("slopes", [[0.0, 0.0, 0.0, 0.0], [-0.05, 0.3, 8.0, 1e-3], [1e4, 0.0, -1e-9, 0.5]])
def test_slopes_of_either_sign_and_size(new, slopes):
    check_scored(Setup(34, 64, 16, 1, [new, 3], [300, 40]), 4, F16, slopes=np.array(slopes, F))


@pytest.mark.parametrize("new", [1, 60])
def test_sights_that_hold_nothing_give_zeros(new):
    """Starts behind the query, sequences longer in new tokens than in all, no pages; garbage in starts and prefixes."""
    torch_cuda()
    s = Setup(35, 64, 16, 2, [new, new + 3, 0, 2, new], [100, new, 30, 40, 100])
    s.table[3, :] = -1
    s.upload()
    starts = np.zeros(s.T, np.int32)
    o = s.offsets
    starts[o[0]:o[1]] = np.arange(100 - new, 100) + 1                       # each the position after it
    starts[o[4]:o[5]:2] = 1 << 30
    starts[o[4] + 1:o[5]:2] = -(1 << 30)
    for prefix in (None, [-5, -(1 << 31), 1 << 30, 3, 0]):
        Y = back(check_scored(s, 4, F16, starts=starts, prefix=prefix, slopes=alibi(8), cap=20.0))
        assert not Y[o[0]:o[1]].any() and not Y[o[1]:o[1] + 3].any() and not Y[o[3]:o[4]].any() and not Y[o[4]:o[5]:2].any()
        check_scored(s, 4, BF16, starts=starts, prefix=prefix, window=30, sinks=7)
    # a prefix makes what lies behind a query visible: rows whose sight begins there see it after all
    Y = back(check_scored(s, 4, F16, starts=starts, prefix=[100, 0, 0, 0, 0]))
    assert all(Y[i].any() for i in range(o[0], o[1] - 1)) and not Y[o[1] - 1].any()


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("garbage", [np.nan, np.inf, -np.inf, -1.0, 0.0])
def test_pages_out_of_sight_may_hold_anything(new, garbage):
    """Pages before the documents' first, given back or with garbage for scales, change nothing, bit for bit."""
    s = Setup(36, 64, 16, 1, [new], [400])
    starts = np.full(s.T, 400 - new - 70, np.int32)
    kw = dict(starts=starts, cap=30.0, slopes=alibi(4), Q=np.full((s.T, 4, 64), 0.5))
    clean = back(run_scored(s, 4, F16, **kw)[0])
    hidden = (400 - new - 70) // 16
    s.scales[s.table[0, :hidden // 2]] = garbage
    s.table[0, hidden // 2:hidden] = -1
    s.upload()
    assert np.array_equal(back(run_scored(s, 4, F16, **kw)[0]), clean)
    # garbage that only some rows see stays with them
    if new > 1 and garbage != garbage:
        s.scales[s.table[0, -1]] = garbage                                   # positions 384 .. 399
        s.upload()
        y = back(run_scored(s, 4, F16, **kw)[0])
        sees = np.arange(400 - new, 400) >= 384
        assert np.isnan(y[sees]).all() and np.array_equal(y[~sees], clean[~sees])


@pytest.mark.parametrize("dtype,D,P,G,new,kv", [(F16, 128, 64, 8, [1], [30000]), (BF16, 64, 16, 4, [5], [20000]),
                                                (F16, 256, 32, 8, [1, 1], [9000, 100]), (BF16, 128, 64, 8, [64], [9000])])
def test_long_sequences_in_many_splits(dtype, D, P, G, new, kv):
    """Far documents (few tiles of those planned), a window with first tokens of a document, a bias over the whole length;
    results do not depend on the order in which splits end."""
    s = Setup(37, D, P, 1, new, kv)
    T = s.T
    for kw in (dict(slopes=alibi(G)), dict(starts=documents(s, 7000), cap=30.0),
               dict(window=3000, sinks=300, starts=documents(s, 8500), slopes=alibi(G) / 64), dict(cap=50.0, prefix=kv)):
        kw["Q"] = 4.0 * np.random.default_rng(1).standard_normal((T, G, D))
        first = back(check_scored(s, G, dtype, **kw))
        for _ in range(3):
            assert np.array_equal(back(run_scored(s, G, dtype, **kw)[0]), first)


def test_packed_documents_equal_sequences_of_their_own():
    """Documents are computed as the sequences that they would be; each side is within its bound of the same values."""
    lens = [128, 64, 200, 56, 64]                                   # all of them begin where a page does
    s = Setup(38, 128, 64, 2, [sum(lens)], [sum(lens)])
    Q = s.rng.standard_normal((s.T, 8, 128))
    at = np.cumsum([0] + lens)
    packed = back(check_scored(s, 4, F16, Q=Q, starts=np.repeat(at[:-1], lens).astype(np.int32)))
    for a, n in zip(at[:-1], lens):
        if a % 64:
            continue
        t = Setup(38, 128, 64, 2, [sum(lens)], [sum(lens)])
        t.table = s.table[:, a // 64:].copy()
        t.new, t.kv = [n], [n]
        t.offsets, t.kv_lens, t.T = np.array([0, n], np.int32), np.array([n], np.int32), n
        t.counts = (n, n)
        t.upload()
        Y, Qr, scale = run_attention(t, 4, F16, Q=Q[a:a + n])
        ref, A, score, peak = okv.attention(t.k, t.v, t.scales, t.offsets, t.kv_lens, t.table, Qr, float(F(scale)), 0, 0)
        tol = attention_bound(A, ref, score, peak, 128, n, F16) + scored_bound(A, ref, score, peak, 0 * score, 128, sum(lens), F16, 0.0)
        assert (np.abs(back(Y).astype(np.float64) - packed[a:a + n]) <= tol).all()


def test_a_neutral_scoring_is_the_plain_attention():
    """No cap, no slopes (or slopes of 0), nothing before the prefix's or behind the document's end: the plain values."""
    for new, kv in (([1, 1], [300, 4000]), ([150, 3], [150, 700])):
        s = Setup(39, 128, 32, 2, new, kv)
        Q = 3.0 * s.rng.standard_normal((s.T, 8, 128))
        _, Qr, scale = run_attention(s, 4, F16, Q=Q)
        ref, A, score, peak = okv.attention(s.k, s.v, s.scales, s.offsets, s.kv_lens, s.table, Qr, float(F(scale)), 0, 0)
        tol = scored_bound(A, ref, score, peak, 0 * score, 128, max(kv), F16, 0.0)
        for kw in ({}, dict(slopes=np.zeros(8, F), prefix=[0, 0], starts=np.zeros(s.T, np.int32))):
            assert (np.abs(back(run_scored(s, 4, F16, Q=Q, **kw)[0]) - ref) <= tol).all()


@pytest.mark.parametrize("max_new,max_kv", [(1, 1), (3, 100), (20, 5000)])
def test_batches_beyond_or_below_the_plan(max_new, max_kv):
    s = Setup(40, 128, 32, 1, [70, 1, 9], [400, 600, 9], max_new=max_new, max_kv=max_kv)
    check_scored(s, 4, F16, cap=30.0, starts=documents(s, 99), prefix=[380, 0, 9], slopes=alibi(4))


def test_forked_sequences_go_on_by_themselves():
    """A serving history, book and cache together: prompts, forks of one of them at different lengths, tokens for all of
    them, a sequence that ends, compaction; append, attention and gather against host caches that know no sharing."""
    torch = torch_cuda()
    P, D, Hk, G, pages, rows, stride = 16, 64, 2, 4, 60, 6, 12
    r = np.random.default_rng(8)
    b = Book(pages, rows, stride, P)
    k, v, scales = (torch.zeros(x, dtype=t, device="cuda") for x, t in (((pages, Hk, P, D), torch.int8), ((pages, Hk, D, P), torch.int8),
                                                                        ((pages, Hk, 2), torch.float32)))
    cache = qlin.Kv8Cache(k, v, scales)
    # the host's sequences: a cache of its own for each row, entry e in page row * stride + e
    hk, hv, hs = np.zeros((rows * stride, Hk, P, D), np.int8), np.zeros((rows * stride, Hk, D, P), np.int8), np.zeros((rows * stride, Hk, 2), F)
    own = np.arange(rows * stride, dtype=np.int32).reshape(rows, stride)
    lens = np.zeros(rows, np.int64)
    slopes = alibi(Hk * G)
    cos, sin = okv.rope_tables(stride * P, D)
    dc, dn = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()

    def step(new):
        nonlocal lens
        lens = lens + new
        assert b.grow(lens)[1] == 0
        T, offsets = int(sum(new)), np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        x, xf = to16(r.standard_normal((T, Hk * (G + 2), D)), F16)
        batch = qlin.Kv8Batch(up(offsets), up(lens), b.d_table, T, int(max(new)), int(max(lens)))
        q, y = (torch.full((T, Hk * G, D), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
        qlin.qlin_kv8_append(cache, batch, x[:, :Hk * G], x[:, Hk * G:Hk * (G + 1)], x[:, Hk * (G + 1):], F16, Hk * G, dc, dn, D,
                             qlin.QLIN_ROPE_HALF, q)
        need = qlin.qlin_kv8_attention_workspace_bytes(cache, batch, Hk * G)
        scoring = qlin.Kv8Scoring(20.0, up(slopes, F), up(lens // 2))
        qlin.qlin_kv8_attention_scored(cache, batch, q, F16, Hk * G, 0.125, 0, 0, scoring, y, workspace(need))
        okv.append(hk, hv, hs, offsets, lens, own, xf[:, :Hk * G], xf[:, Hk * G:Hk * (G + 1)], xf[:, Hk * (G + 1):], cos, sin, D, False)
        ref = okv.attention_scored(hk, hv, hs, offsets, lens, own, back(q), 0.125, 0, 0, 20.0, slopes, lens // 2)
        assert (np.abs(back(y) - ref[0]) <= scored_bound(*(ref[i] for i in (1, 0, 2, 3, 4)), D, int(max(lens)), F16, 20.0)).all()
        check_all()

    def check_all():
        K, V = (torch.empty((int(lens.sum()), Hk, D), dtype=torch.float16, device="cuda") for _ in range(2))
        offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        qlin.qlin_kv8_gather(cache, qlin.Kv8Batch(up(offsets), up(lens), b.d_table, int(lens.sum()), int(max(lens)), int(max(lens))), K, V, F16)
        for i, got in enumerate((K, V)):
            want = [np.stack([okv.values(hk, hv, hs, own[row], int(m), h)[i] for h in range(Hk)], 1) for row, m in enumerate(lens)]
            assert np.array_equal(back(got), np.concatenate(want).astype(np.float16))

    def fork(parents, kids, part):
        m = b.moves(len(kids))
        qlin.qlin_kv8_fork(b.book, up(parents), up(kids), up(part), m)
        want = okp.fork(b.refs, b.table, P, parents, kids, part)
        b.check(want, m)
        qlin.qlin_kv8_copy_pages(cache, cache, m)
        for p, c, n in zip(parents, kids, part):
            lens[c] = n
            for x in (hk, hv, hs):
                x[own[c]] = x[own[p]]
        check_all()

    step([70, 33, 0, 0, 0, 0])
    fork([0, 0, 1], [2, 3, 4], [70, 41, 32])
    step([1, 1, 1, 1, 1, 0])
    step([5, 0, 20, 1, 17, 40])
    b.free([0, 1])
    lens[:2] = 0
    m = b.moves(pages // 2)
    qlin.qlin_kv8_compact(b.book, m)
    want = okp.compact(b.refs, b.table, pages // 2)
    b.check(want, m)
    assert want[0][0] > 0
    qlin.qlin_kv8_copy_pages(cache, cache, m)
    check_all()
    fork([2, 3], [0, 1], [60, 42])
    step([3, 1, 0, 9, 1, 1])


def test_graph_replays_with_other_lengths_documents_and_slopes():
    torch = torch_cuda()
    s = Setup(42, 64, 16, 2, [1, 1], [600, 300])
    G = 4
    q, _ = to16(3.0 * s.rng.standard_normal((2, 8, 64)), F16)
    y = torch.empty_like(q)
    slopes, prefix, starts = up(alibi(8), F), up([0, 0]), up([0, 0])
    scoring = qlin.Kv8Scoring(30.0, slopes, prefix, starts)
    need = qlin.qlin_kv8_attention_workspace_bytes(s.cache, s.batch, 8)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    call = lambda: qlin.qlin_kv8_attention_scored(s.cache, s.batch, q, F16, 8, 0.125, 0, 0, scoring, y, ws)   # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        s.kv = [600 - 50 * i, 300 - 90 * i]
        s.dev[1].copy_(up(s.kv))
        starts.copy_(up([100 * i, 7 * i]))
        slopes.mul_(0.5)
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = back(y)
        call()
        assert np.array_equal(back(y), got)
        s.kv_lens = np.array(s.kv, np.int32)
        ref = okv.attention_scored(s.k, s.v, s.scales, s.offsets, s.kv_lens, s.table, back(q), 0.125, 0, 0, 30.0,
                                   slopes.cpu().numpy(), [0, 0], starts.cpu().numpy())
        assert (np.abs(got - ref[0]) <= scored_bound(*(ref[k] for k in (1, 0, 2, 3, 4)), 64, 600, F16, 30.0)).all()


# Row tiles that are not split over the cache (planned for short sequences, so that small batches are not either): the
# kernels for whole prompts, of which heads of 256 and documents have their own.
WHOLE = [
    (F16, 256, 32, 1, 2, [130, 20], [190, 400]), (BF16, 256, 16, 2, 3, [90, 33, 1], [200, 33, 70]),
    (BF16, 256, 128, 1, 8, [65, 17], [300, 17]), (F16, 256, 64, 1, 1, [400], [650]),
    (F16, 128, 64, 1, 8, [90, 40], [300, 64]), (BF16, 128, 16, 2, 4, [129, 31], [129, 500]), (F16, 64, 32, 1, 4, [200, 70], [260, 70]),
]


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dtype,D,P,Hk,G,new,kv", WHOLE)
def test_whole_row_tiles_within_their_rounding_bounds(dtype, D, P, Hk, G, new, kv, form):
    say(f"kv8 scored attention, whole row tiles, {form}: D={D} P={P} Hk={Hk} G={G} new={new} kv={kv}")
    s = Setup(51, D, P, Hk, new, kv, max_kv=64)
    kw = dict(FORMS[form])
    if "slopes" in kw:
        kw["slopes"] = alibi(Hk * G)
    if "prefix" in kw:
        kw["prefix"] = [[m - n // 3, m, 0][b % 3] for b, (n, m) in enumerate(zip(new, kv))]
    if "starts" in kw:
        kw["starts"] = documents(s, kw["starts"])
    kw["Q"] = (12.0 if kw.get("cap") else 3.0) * s.rng.standard_normal((s.T, Hk * G, D))
    first = back(check_scored(s, G, dtype, **kw))
    assert np.array_equal(back(run_scored(s, G, dtype, **kw)[0]), first)


@pytest.mark.parametrize("D", [128, 256])
def test_whole_row_tiles_at_the_edges_of_sight(D):
    """Nothing in sight, tokens before the first position, a sequence without pages, garbage for starts and prefixes; pages
    out of sight that hold anything or nothing; queries that are not finite stay in their rows."""
    torch = torch_cuda()
    s = Setup(52, D, 16, 2, [60, 63, 0, 2, 60], [100, 60, 30, 40, 300], max_kv=64)
    s.table[3, :] = -1
    s.upload()
    o = s.offsets
    starts = np.zeros(s.T, np.int32)
    starts[o[0]:o[1]] = np.arange(40, 100) + 1
    starts[o[4]:o[5]:2] = 1 << 30
    starts[o[4] + 1:o[5]:2] = 130
    Q = 3.0 * s.rng.standard_normal((s.T, 8, D))
    for prefix in (None, [-5, -(1 << 31), 1 << 30, 3, 0]):
        Y = back(check_scored(s, 4, F16, Q=Q, starts=starts, prefix=prefix, slopes=alibi(8), cap=20.0))
        assert not Y[o[0]:o[1]].any() and not Y[o[1]:o[1] + 3].any() and not Y[o[3]:o[4]].any() and not Y[o[4]:o[5]:2].any()
        check_scored(s, 4, BF16, Q=Q, starts=starts, prefix=prefix, window=30, sinks=7)
    clean = back(run_scored(s, 4, F16, Q=Q, starts=starts, cap=20.0)[0])
    for i, garbage in enumerate((np.nan, np.inf, -np.inf, -1.0)):
        s.scales[s.table[4, i]] = garbage                                    # positions below 64, all before 130
    s.table[4, 4:8] = -1
    s.upload()
    assert np.array_equal(back(run_scored(s, 4, F16, Q=Q, starts=starts, cap=20.0)[0]), clean)
    Q[o[4] + 1, 3, 5], Q[o[4] + 3, 1, 0] = np.nan, np.inf
    Y = back(run_scored(s, 4, F16, Q=Q, starts=starts, slopes=alibi(8))[0])
    Z = back(run_scored(s, 4, F16, Q=np.nan_to_num(Q, nan=1.0, posinf=1.0), starts=starts, slopes=alibi(8))[0])
    bad = np.zeros(Y.shape[:2], bool)
    bad[o[4] + 1, 3] = bad[o[4] + 3, 1] = True
    assert np.isnan(Y[bad]).all() and np.array_equal(Y[~bad], Z[~bad])


@pytest.mark.parametrize("dtype,D,G,Hk,new,kv", [
    (F16, 128, 8, 4, [1070, 30], [1070, 90]),              # 67 row tiles: 33 pairs and one
    (BF16, 256, 8, 3, [1050, 0, 1], [1111, 5, 300]), (F16, 64, 4, 8, [600, 599, 1, 90], [600, 700, 40, 90]),
    (BF16, 128, 2, 30, [129, 700], [640, 700]),            # fewer than 64
])
def test_long_documents_first(dtype, D, G, Hk, new, kv):
    """Enough row tiles that those with the most tiles are begun with: each is computed once, whatever the starts say."""
    s = Setup(53, D, 16, Hk, new, kv, max_kv=64)
    r = np.random.default_rng(54)
    Q = 3.0 * r.standard_normal((s.T, Hk * G, D))
    wild = r.integers(-100, max(kv) + 100, s.T).astype(np.int32)           # rising and falling from token to token
    for kw in (dict(starts=documents(s, 333), slopes=alibi(Hk * G)), dict(starts=wild, prefix=[m // 2 for m in kv], window=200, sinks=9)):
        first = back(check_scored(s, G, dtype, Q=Q, **kw))
        assert np.array_equal(back(run_scored(s, G, dtype, Q=Q, **kw)[0]), first)


def test_two_streams_at_once():
    """Books, copies and attention of two serving programs side by side, each with its own buffers."""
    torch = torch_cuda()
    made = []
    for seed in (61, 62):
        r = np.random.default_rng(seed)
        s = Setup(seed, 128, 16, 2, [1, 40, 1], [900, 300, 77])
        b = Book(500, 8, 40)
        b.deal(r, [30, 17, 0, 0, 0, 0, 0, 0])
        q, _ = to16(3.0 * r.standard_normal((s.T, 8, 128)), F16)
        need = qlin.qlin_kv8_attention_workspace_bytes(s.cache, s.batch, 8)
        made.append(dict(s=s, b=b, q=q, y=torch.empty_like(q), ws=torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda"),
                         how=qlin.Kv8Scoring(25.0, up(alibi(8), F), up([0, 290, 0]), up(documents(s, 50))), moves=b.moves(3),
                         lists=[up([0, 1, 0]), up([2, 3, 4]), up([470, 100, 33])], lens=up([480, 300, 480, 0, 40, 0, 0, 5]), grown=b.moves(0),
                         stream=torch.cuda.Stream()))
    torch.cuda.synchronize()

    def step(m, stream):
        parents, kids, lens = m["lists"]
        for _ in range(3):
            qlin.qlin_kv8_free(m["b"].book, kids, stream=stream)
            qlin.qlin_kv8_fork(m["b"].book, parents, kids, lens, m["moves"], stream=stream)
            qlin.qlin_kv8_grow(m["b"].book, m["lens"], m["grown"], stream=stream)
            qlin.qlin_kv8_attention_scored(m["s"].cache, m["s"].batch, m["q"], F16, 8, 0.1, 0, 0, m["how"], m["y"], m["ws"], stream=stream)

    def result(m):
        return [x.clone() for x in (m["b"].d_table, m["b"].d_refs, m["moves"], m["grown"], m["y"])]

    for _ in range(4):
        for m in made:
            step(m, m["stream"])
    torch.cuda.synchronize()
    both = [result(m) for m in made]
    for m, got in zip(made, both):
        step(m, None)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(result(m)[2:3] + result(m)[4:], got[2:3] + got[4:]))
        table, refs = m["b"].d_table.cpu().numpy(), m["b"].d_refs.cpu().numpy()
        assert np.array_equal(np.bincount(table[table >= 0], minlength=500), refs) and int(m["grown"][0, 1]) == 0


@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 64, (1 << 31) - 400, 1 << 30])
@pytest.mark.parametrize("D,new,max_kv", [(64, 1, None), (128, 12, None), (128, 90, None), (128, 90, 64), (256, 90, 64)])
def test_windows_as_wide_as_int(D, new, max_kv, window):
    """A prefix behind the queries stays visible in them, in every kernel."""
    s = Setup(57, D, 16, 1, [new, new], [600, new], max_kv=max_kv)
    kw = dict(Q=3.0 * s.rng.standard_normal((s.T, 4, D)), prefix=[600, new], starts=documents(s, 300), cap=20.0)
    wide = back(check_scored(s, 4, F16, window=window, **kw))
    assert np.array_equal(back(run_scored(s, 4, F16, window=window, sinks=5, **kw)[0]), wide)
    check_scored(s, 4, F16, window=window, sinks=(1 << 31) - 1, **kw)


@pytest.mark.parametrize("slope", [2.3e38, 2.4e38, 3.4028234e38])
@pytest.mark.parametrize("D,new,max_kv", [(64, 1, None), (128, 90, None), (128, 90, 64), (256, 90, 64)])
def test_slopes_up_to_the_largest_float(D, new, max_kv, slope):
    """Beside such a slope a query sees its own position alone: its value, off by the roundings of the weight (2^-11) and of
    the output (2^-11) and a few of fp32."""
    s = Setup(58, D, 16, 1, [new, new], [600, new], max_kv=max_kv)
    Y = back(run_scored(s, 4, F16, slopes=np.full(4, slope, F))[0])
    for b, m in enumerate(s.kv):
        _, v, _ = okv.values(s.k, s.v, s.scales, s.table[b], m, 0)
        own = v[m - new:, None]
        assert (np.abs(Y[new * b:new * b + new] - own) <= (2.0 ** -10 + 2.0 ** -18) * np.abs(own)).all()


@pytest.mark.parametrize("dtype,D,G,Hk,new", [(F16, 128, 16, 2, 1100),       # 138 row tiles: 34 groups of four and two
                                              (BF16, 128, 16, 1, 2070),      # 259: 32 of eight and three
                                              (F16, 256, 16, 1, 2070), (F16, 64, 16, 2, 1040)])
def test_long_documents_first_of_many_row_tiles(dtype, D, G, Hk, new):
    s = Setup(59, D, 64, Hk, [new], [new], max_kv=64)
    r = np.random.default_rng(60)
    Q = 3.0 * r.standard_normal((s.T, Hk * G, D))
    wild = r.integers(-100, new + 100, s.T).astype(np.int32)
    for kw in (dict(starts=documents(s, 333), cap=20.0), dict(starts=wild, prefix=[new // 2], window=200, sinks=9)):
        first = back(check_scored(s, G, dtype, Q=Q, **kw))
        assert np.array_equal(back(run_scored(s, G, dtype, Q=Q, **kw)[0]), first)


def test_packed_documents_of_whole_pages_equal_sequences_of_their_own():
    lens = [128, 64, 192, 64, 256]
    s = Setup(38, 128, 64, 2, [sum(lens)], [sum(lens)])
    Q = s.rng.standard_normal((s.T, 8, 128))
    at = np.cumsum([0] + lens)
    packed = back(check_scored(s, 4, F16, Q=Q, starts=np.repeat(at[:-1], lens).astype(np.int32)))
    for a, n in zip(at[:-1], lens):
        t = Setup(38, 128, 64, 2, [sum(lens)], [sum(lens)])
        t.table = s.table[:, a // 64:].copy()
        t.new, t.kv = [n], [n]
        t.offsets, t.kv_lens, t.T = np.array([0, n], np.int32), np.array([n], np.int32), n
        t.counts = (n, n)
        t.upload()
        Y, Qr, scale = run_attention(t, 4, F16, Q=Q[a:a + n])
        ref, A, score, peak = okv.attention(t.k, t.v, t.scales, t.offsets, t.kv_lens, t.table, Qr, float(F(scale)), 0, 0)
        tol = attention_bound(A, ref, score, peak, 128, n, F16) + scored_bound(A, ref, score, peak, 0 * score, 128, sum(lens), F16, 0.0)
        assert (np.abs(back(Y).astype(np.float64) - packed[a:a + n]) <= tol).all()
