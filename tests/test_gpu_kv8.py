"""GPU parity of the 8-bit paged key/value cache against the oracle: scales, codes and read-back bit for bit, rotated
queries to their rounding, attention within bounds derived from its roundings."""
import numpy as np
import pytest

from oracle import kv8 as okv
from quantized_linear_layers_packed_amd import qlin
from tests.gpu_util import say, torch_cuda, workspace

pytestmark = pytest.mark.gpu

F16, BF16 = qlin.QLIN_F16, qlin.QLIN_BF16
F = np.float32


def to16(x, dtype):
    """fp32 array -> (device tensor of dtype, the same values as fp32)."""
    torch = torch_cuda()
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=F)).to(torch.float16 if dtype == F16 else torch.bfloat16)
    return t.cuda(), t.float().numpy()


def back(t):
    torch = torch_cuda()
    torch.cuda.synchronize()
    return t.float().cpu().numpy()


class Setup:
    """A pool of pages with earlier tokens, and a ragged batch on it, on host and device."""

    def __init__(self, seed, D, P, Hk, new, kv, max_new=None, max_kv=None, spare=3):
        r = self.rng = np.random.default_rng(seed)
        self.D, self.P, self.Hk = D, P, Hk
        self.new, self.kv = new, kv
        need = [-(-m // P) for m in kv]
        pages = sum(need) + spare
        order = r.permutation(pages)[:sum(need)].astype(np.int32)
        self.table = np.full((len(kv), max(max(need), 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.k = r.integers(-127, 128, (pages, Hk, P, D)).astype(np.int8)
        self.v = r.integers(-127, 128, (pages, Hk, D, P)).astype(np.int8)
        self.scales = r.uniform(0.005, 0.03, (pages, Hk, 2)).astype(F)
        self.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.kv_lens = np.array(kv, np.int32)
        self.T = max(int(self.offsets[-1]), 1)
        self.counts = (max_new or max(max(new), 1), max_kv or max(max(kv), 1))
        self.upload()

    def upload(self):
        torch = torch_cuda()
        self.dk, self.dv, self.ds = (torch.from_numpy(x.copy()).cuda() for x in (self.k, self.v, self.scales))
        self.dev = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (self.offsets, self.kv_lens, self.table)]
        self.cache = qlin.Kv8Cache(self.dk, self.dv, self.ds)
        self.batch = qlin.Kv8Batch(*self.dev, self.T, *self.counts)

    def check_cache(self):
        """Device cache against the host's: bit for bit where tokens live, and wherever no call may write."""
        torch = torch_cuda()
        torch.cuda.synchronize()
        k, v, s = self.dk.cpu().numpy(), self.dv.cpu().numpy(), self.ds.cpu().numpy()
        assert np.array_equal(s.view(np.uint32)[~np.isnan(s)], self.scales.view(np.uint32)[~np.isnan(self.scales)])
        assert np.array_equal(np.isnan(s), np.isnan(self.scales))
        live = np.ones(k.shape[:3], bool)                        # [page][head][slot]
        for b, m in enumerate(self.kv):
            if self.new[b] and m and m % self.P and 0 <= self.table[b, m // self.P] < len(k):
                live[self.table[b, m // self.P], :, m % self.P:] = False      # slots past the last token
        poisoned = np.isnan(self.scales)
        live_k, live_v = live & ~poisoned[..., :1], live & ~poisoned[..., 1:]
        assert np.array_equal(k[live_k], self.k[live_k])
        assert np.array_equal(v.transpose(0, 1, 3, 2)[live_v], self.v.transpose(0, 1, 3, 2)[live_v])


def run_append(s, Hq, dtype, rot, pairs, x=None, in_place=False, no_q=False):
    """Appends through the library and the oracle; returns the rotated queries of both."""
    torch = torch_cuda()
    if x is None:
        x = s.rng.standard_normal((s.T, Hq + 2 * s.Hk, s.D))
    d, x = to16(x, dtype)
    cos, sin = okv.rope_tables(max(s.kv + [1]), rot) if rot else (None, None)
    dc, dn = (torch.from_numpy(t).cuda() for t in (cos, sin)) if rot else (None, None)
    q = d[:, :Hq].contiguous() if in_place else d[:, :Hq]
    out = None if no_q else q if in_place else torch.full((s.T, Hq, s.D), 7.0, dtype=d.dtype, device="cuda")
    qlin.qlin_kv8_append(s.cache, s.batch, None if no_q else q, d[:, Hq:Hq + s.Hk], d[:, Hq + s.Hk:], dtype, Hq, dc, dn,
                         rot, qlin.QLIN_ROPE_PAIRS if pairs else qlin.QLIN_ROPE_HALF, out)
    ref = okv.append(s.k, s.v, s.scales, s.offsets, s.kv_lens, s.table, x[:, :Hq], x[:, Hq:Hq + s.Hk], x[:, Hq + s.Hk:],
                     cos, sin, rot, pairs)
    torch.cuda.synchronize()
    return out, ref


def check_round16(got, ref, dtype):
    """got is ref (fp32) rounded once to 16 bits."""
    torch = torch_cuda()
    want = torch.from_numpy(ref).to(torch.float16 if dtype == F16 else torch.bfloat16).float().numpy()
    assert np.array_equal(back(got), want, equal_nan=True)


@pytest.mark.parametrize("dtype,D,P,Hk,G,rot,pairs,new,kv", [
    (F16, 128, 64, 2, 4, 128, False, [1, 1, 1, 1], [1, 64, 65, 200]),              # single tokens: first, last, fresh, mid
    (BF16, 128, 64, 2, 1, 64, True, [1, 3, 64, 130], [128, 66, 64, 191]),
    (F16, 64, 16, 3, 3, 64, False, [37, 1, 15, 17], [37, 90, 31, 33]),
    (BF16, 64, 128, 1, 8, 16, True, [5, 300], [133, 300]),
    (F16, 256, 32, 2, 2, 256, True, [33, 1, 70], [40, 32, 101]),
    (BF16, 256, 128, 1, 2, 128, False, [129, 2, 250], [140, 129, 511]),
    (F16, 64, 32, 4, 1, 0, False, [7, 40], [9, 63]),
    (F16, 128, 16, 1, 7, 32, False, [1], [5]),
])
def test_append_matches_the_oracle_bit_for_bit(dtype, D, P, Hk, G, rot, pairs, new, kv):
    say(f"kv8 append D={D} P={P} Hk={Hk} G={G} rot={rot} new={new} kv={kv}")
    s = Setup(1, D, P, Hk, new, kv)
    q, q_ref = run_append(s, Hk * G, dtype, rot, pairs)
    s.check_cache()
    check_round16(q, q_ref, dtype)
    # the read-back of the same tokens
    torch = torch_cuda()
    K, V = (torch.full((s.T, Hk, D), 7.0, dtype=q.dtype, device="cuda") for _ in range(2))
    qlin.qlin_kv8_gather(s.cache, s.batch, K, V, dtype)
    k_ref, v_ref = np.zeros((s.T, Hk, D), F), np.zeros((s.T, Hk, D), F)
    for b, m in enumerate(kv):
        for h in range(Hk):
            k, v, _ = okv.values(s.k, s.v, s.scales, s.table[b], m, h)
            k_ref[s.offsets[b]:s.offsets[b + 1], h] = k[m - new[b]:]
            v_ref[s.offsets[b]:s.offsets[b + 1], h] = v[m - new[b]:]
    check_round16(K, k_ref, dtype)
    check_round16(V, v_ref, dtype)


def test_append_token_by_token_grows_the_scales_as_the_oracle_does():
    P, D, Hk = 32, 64, 2
    s = Setup(3, D, P, Hk, [1, 1], [1, 20])
    for step in range(40):
        s.kv = [1 + step, 20 + step]
        need = max(-(-m // P) for m in s.kv)
        free = [p for p in range(len(s.k)) if p not in s.table]
        if need > s.table.shape[1]:
            s.table = np.concatenate([s.table, np.full((2, 1), -1, np.int32)], axis=1)
        for b, m in enumerate(s.kv):
            if s.table[b, (m - 1) // P] < 0:
                s.table[b, (m - 1) // P] = free.pop()
        s.kv_lens = np.array(s.kv, np.int32)
        k, v, sc = s.dk, s.dv, s.ds
        s.upload()
        s.dk.copy_(k), s.dv.copy_(v), s.ds.copy_(sc)                # the device cache goes on from its own state
        gain = 1.0 + 0.2 * step                                    # most steps grow the scale
        run_append(s, Hk, BF16, 64, False, x=gain * s.rng.standard_normal((2, 3 * Hk, D)))
        s.check_cache()


def test_append_in_place_and_without_queries():
    for kw in ({"in_place": True}, {"no_q": True}):
        s = Setup(4, 128, 32, 2, [3, 40], [10, 50])
        q, q_ref = run_append(s, 6, F16, 128, False, **kw)
        s.check_cache()
        if q is not None:
            check_round16(q, q_ref, F16)


def test_append_zeros_tiny_and_non_finite_values():
    s = Setup(5, 64, 16, 2, [4, 4, 4, 4], [4, 20, 20, 7])
    x = s.rng.standard_normal((16, 6, 64)).astype(F)
    x[0:4] = 0.0                                         # an all-zero page: scale 0
    x[4:8] = 1e-39                                       # below the least scale: 0 (bf16 holds it as a subnormal)
    x[9, 2, 3] = np.inf                                  # keys of head 0, sequence 2
    x[13, 5, 60] = np.nan                                # values of head 1, sequence 3, whose page holds earlier tokens
    run_append(s, 2, BF16, 0, False, x=x)
    s.check_cache()
    assert np.isnan(s.scales).sum() == 2 and (s.scales == 0).sum() >= 8


def test_append_and_gather_keep_out_of_what_they_may_not_touch():
    """More new tokens than the sequence is long, no new tokens, pages that are not there, offsets out of range."""
    s = Setup(6, 64, 16, 2, [5, 0, 20, 6], [3, 12, 40, 6])
    s.table[2, 1] = -1                                   # positions 16 .. 31 of sequence 2 have no page
    s.table[3, 0] = len(s.k)                             # past the pool
    s.upload()
    q, q_ref = run_append(s, 4, F16, 64, False)
    s.check_cache()
    check_round16(q, q_ref, F16)
    torch = torch_cuda()
    K, V = (torch.full((s.T, 2, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    qlin.qlin_kv8_gather(s.cache, s.batch, K, V, F16)
    K, V = back(K), back(V)
    gone = list(range(0, 2)) + list(range(5, 5 + 12)) + list(range(25, 31))
    assert not K[gone].any() and not V[gone].any()
    assert (K[2:5] != 7).all() and K[17:25].any()
    # offsets past the tokens and out of order are clamped: the call stays inside its buffers
    s.offsets[:] = [-5, 1000, 3, 31, 2000000000]
    s.kv_lens[:] = [1 << 30, 50, -7, 6]
    s.upload()
    d, _ = to16(s.rng.standard_normal((s.T, 8, 64)), F16)
    out = torch.empty((s.T, 4, 64), dtype=torch.float16, device="cuda")
    qlin.qlin_kv8_append(s.cache, s.batch, d[:, :4], d[:, 4:6], d[:, 6:], F16, 4, None, None, 0, 0, out)
    Y = torch.empty_like(out)
    need = qlin.qlin_kv8_attention_workspace_bytes(s.cache, s.batch, 4)
    qlin.qlin_kv8_attention(s.cache, s.batch, out, F16, 4, 0.125, 0, 0, Y, workspace(need))
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# attention

def attention_bound(A, Y, score, peak, D, L, dtype):
    """Largest error of an output that the kernel's roundings allow.

    out:     half a unit of the output type
    weights: each rounded to fp16, 2^-11 of itself, or 2^-25 (subnormals) of the row's reference, times values of at
             most `peak` (that many times 2^8 / 2^8: the row's sum of weights is at least 1)
    scores:  D products summed in fp32 and a few fp32 operations after that, each within 2^-24 of sum |q k| scale, in
             the exponent's argument (so relative to the weight), in numerator and denominator
    sums:    fp32 accumulation over the tokens in tiles and the joins: 2^-24 each of at most L + 64 steps
    """
    u_out = 2.0 ** -11 if dtype == F16 else 2.0 ** -8
    rel = 2.0 ** -11 + 2 * (D + 16) * 2.0 ** -24 * (score[..., None] + 1) + 2 * (L + 64) * 2.0 ** -24
    return u_out * np.abs(Y) + rel * A + L * 2.0 ** -25 * peak[..., None] + (2.0 ** -25 if dtype == F16 else 0.0)


def run_attention(s, G, dtype, scale=None, window=0, sinks=0, Q=None, ws=None):
    torch = torch_cuda()
    Hq = s.Hk * G
    if Q is None:
        Q = 3.0 * s.rng.standard_normal((s.T, Hq, s.D))
    d, Q = to16(Q, dtype)
    Y = torch.full((s.T, Hq, s.D), 7.0, dtype=d.dtype, device="cuda")
    scale = scale or 1.0 / np.sqrt(s.D)
    need = qlin.qlin_kv8_attention_workspace_bytes(s.cache, s.batch, Hq, window, sinks)
    ws = workspace(need) if ws is None else ws
    qlin.qlin_kv8_attention(s.cache, s.batch, d, dtype, Hq, scale, window, sinks, Y, ws)
    torch.cuda.synchronize()
    if need:
        assert not ws[:16384].any(), "arrival counters left behind"
    return Y, Q, scale


def check_attention(s, G, dtype, **kw):
    Y, Q, scale = run_attention(s, G, dtype, **kw)
    args = (s.k, s.v, s.scales, s.offsets, s.kv_lens, s.table, Q, float(F(scale)), kw.get("window", 0), kw.get("sinks", 0))
    ref, A, score, peak = okv.attention(*args)
    tol = attention_bound(A, ref, score, peak, s.D, max(s.kv), dtype)
    owned = slice(0, int(s.offsets[-1]))
    err = np.abs(back(Y).astype(np.float64)[owned] - ref[owned])
    say(f"  worst error / bound: {float((err / np.maximum(tol[owned], 1e-30)).max()):.3f}")
    assert (err <= tol[owned]).all()
    return Y


CASES = [
    # dtype, D, P, Hk, G, new, kv, window, sinks
    (F16, 128, 64, 2, 4, [1, 1, 1], [1, 64, 300], 0, 0),
    (BF16, 128, 16, 1, 1, [1, 1, 1, 1], [5, 17, 333, 1000], 0, 0),
    (F16, 64, 128, 2, 8, [1, 1], [129, 700], 0, 0),
    (BF16, 64, 32, 3, 7, [1, 2, 3], [40, 2, 515], 0, 0),
    (F16, 256, 32, 1, 16, [1, 1], [31, 450], 0, 0),
    (BF16, 256, 64, 2, 3, [1, 4], [260, 90], 0, 0),
    (F16, 128, 64, 1, 8, [5, 5], [5, 400], 0, 0),                       # 40 rows
    (F16, 128, 16, 2, 4, [33, 7, 50], [33, 100, 177], 0, 0),
    (BF16, 64, 64, 1, 4, [100, 1], [100, 130], 0, 0),
    (F16, 128, 32, 1, 2, [1, 1, 1], [1000, 200, 70], 64, 4),            # window and first tokens
    (BF16, 128, 16, 1, 4, [1, 6, 20], [777, 300, 25], 100, 0),
    (F16, 64, 64, 2, 2, [40, 1], [500, 900], 33, 70),                   # more first tokens than a tile
    (F16, 64, 16, 1, 1, [3], [200], 1, 1),                              # a window of the token itself
    (BF16, 256, 128, 1, 2, [20, 1], [400, 600], 129, 3),
    (F16, 128, 64, 1, 1, [150], [150], 1 << 30, 5),                     # a window longer than anything
    (F16, 128, 32, 1, 4, [200, 129, 1], [333, 129, 64], 0, 0),          # prompts
    (BF16, 128, 64, 2, 2, [257], [700], 0, 0),
    (BF16, 64, 16, 1, 8, [70, 90], [100, 300], 40, 4),
    (F16, 256, 32, 1, 2, [130, 20], [190, 400], 0, 0),
    (BF16, 256, 16, 1, 3, [90], [200], 50, 20),
    (F16, 64, 128, 1, 3, [301], [640], 100, 130),
]


@pytest.mark.parametrize("dtype,D,P,Hk,G,new,kv,window,sinks", CASES)
def test_attention_within_its_rounding_bounds(dtype, D, P, Hk, G, new, kv, window, sinks):
    say(f"kv8 attention D={D} P={P} Hk={Hk} G={G} new={new} kv={kv} window={window} sinks={sinks}")
    check_attention(Setup(11, D, P, Hk, new, kv), G, dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_rows_that_see_nothing_give_zeros(new):
    torch = torch_cuda()
    s = Setup(12, 64, 16, 2, [new, new + 3, 0, 2], [0, new, 30, 40])
    s.table[3, :] = -1                                                  # a sequence without pages
    s.upload()
    Y = back(check_attention(s, 4, F16))
    o = s.offsets
    assert not Y[o[0]:o[1]].any() and not Y[o[1]:o[1] + 3].any() and not Y[o[3]:o[4]].any()


@pytest.mark.parametrize("new", [1, 60])
def test_attention_never_looks_at_what_the_mask_hides(new):
    """Pages outside the window given back (-1) or holding NaN scales, and stale codes past the last token, change
    nothing; a visible NaN page reaches exactly the rows that see it."""
    P, kv, window, sinks = 16, 400, 64, 4
    s = Setup(13, 64, P, 1, [new], [kv])
    clean = back(run_attention(s, 4, F16, window=window, sinks=sinks, Q=np.full((new, 4, 64), 0.5))[0])
    lo = (kv - new - window) // P                                       # pages 1 .. lo - 1 are hidden from every row
    s.scales[s.table[0, 1:lo // 2]] = np.nan
    s.table[0, lo // 2:lo] = -1
    s.k[:, :, :, :][[p for p in range(len(s.k)) if p not in s.table]] = 127
    s.upload()
    assert np.array_equal(back(run_attention(s, 4, F16, window=window, sinks=sinks, Q=np.full((new, 4, 64), 0.5))[0]), clean)
    if new > 1:
        for which in (0, 1):
            t = Setup(13, 64, P, 1, [new], [kv])
            t.scales[t.table[0, -1], :, which] = np.nan                 # the last page: positions 384 .. 399
            t.upload()
            y = back(run_attention(t, 4, F16, Q=np.full((new, 4, 64), 0.5))[0])
            sees = np.arange(kv - new, kv) >= kv - P
            assert np.isnan(y[sees]).all() and np.isfinite(y[~sees]).all()


def test_attention_non_finite_queries_stay_in_their_rows():
    for new in (1, 40):
        s = Setup(14, 128, 32, 1, [new, new], [100, 300])
        for dtype in (F16, BF16):
            Q = s.rng.standard_normal((2 * new, 4, 128))
            clean = back(run_attention(s, 4, dtype, Q=Q)[0])
            Q[0, 1, 7], Q[-1, 2, 0] = np.nan, np.inf
            y = back(run_attention(s, 4, dtype, Q=Q)[0])
            bad = np.zeros(y.shape, bool)
            bad[0, 1] = bad[-1, 2] = True
            assert np.isnan(y[bad]).all() and np.array_equal(y[~bad], clean[~bad])


def test_attention_large_and_small_scores_and_values():
    """Scores of +-thousands (all weight on few tokens), page scales over many orders, bf16 queries far outside fp16."""
    for new in (1, 30):
        s = Setup(15, 128, 16, 1, [new], [500])
        s.scales[..., 1] *= (10.0 ** s.rng.uniform(-3, 3, s.scales.shape[:2])).astype(F)
        s.scales[s.table[0, 3]] = 0.0
        s.upload()
        check_attention(s, 4, F16)
        check_attention(s, 4, F16, scale=20.0)
        s.scales[..., 0] *= F(1e-8)
        s.upload()
        check_attention(s, 4, BF16, Q=3e8 * s.rng.standard_normal((new, 4, 128)))
        s.scales[..., 0] *= F(1e16)
        s.upload()
        check_attention(s, 4, BF16, Q=3e-8 * s.rng.standard_normal((new, 4, 128)))


@pytest.mark.parametrize("max_new,max_kv", [(1, 1), (3, 100), (1, 5000)])
def test_plans_too_small_or_too_large_still_compute_everything(max_new, max_kv):
    s = Setup(16, 64, 16, 2, [40, 3, 1], [700, 90, 300], max_new=max_new, max_kv=max_kv)
    check_attention(s, 4, F16)
    q, q_ref = run_append(s, 4, F16, 64, False)
    s.check_cache()
    check_round16(q, q_ref, F16)


@pytest.mark.parametrize("dtype,D,P,G,window,sinks", [(F16, 64, 16, 4, 0, 0), (BF16, 128, 64, 8, 300, 4), (F16, 256, 32, 3, 0, 0)])
def test_prompts_among_single_tokens(dtype, D, P, G, window, sinks):
    """Eight and more sequences of very different lengths in one call: each kernel takes its own, long ones split."""
    new = [1, 90, 1, 0, 2, 40, 1, 5, 1, 300]
    kv = [2500, 300, 1, 50, 2, 1900, 63, 5, 700, 300]
    check_attention(Setup(21, D, P, 1, new, kv), G, dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("D,rows", [(128, 20), (128, 60), (128, 100), (64, 120), (256, 50), (128, 200)])
def test_every_kernel_choice_by_rows(D, rows):
    """Row counts around the limits between the kernels, few sequences and many."""
    for seqs, kv in ((1, 1500), (5, 400), (40, 130)):
        s = Setup(22, D, 32, 2 if seqs < 40 else 1, [rows // 4] * seqs, [kv + 7 * b for b in range(seqs)])
        check_attention(s, 4, F16)


@pytest.mark.parametrize("dtype,D,P,G,new,kv,window,sinks", [
    (F16, 128, 64, 8, [30], [33000], 0, 0),                             # a row tile split more than 64 times
    (BF16, 64, 16, 8, [13], [20011], 0, 0),
    (F16, 256, 32, 4, [25, 20], [20000, 70], 0, 0),                     # the second of one split
    (BF16, 256, 128, 8, [33, 5], [3000, 9000], 0, 0),
    (F16, 64, 64, 2, [200, 40, 1], [9000, 3000, 8000], 2000, 100),
    (BF16, 128, 32, 1, [70, 0, 3, 1, 200, 1, 1, 2], [12000, 9, 3, 5000, 200, 1, 77, 1600], 0, 0),
])
def test_few_rows_of_long_sequences_in_many_splits(dtype, D, P, G, new, kv, window, sinks):
    s = Setup(23, D, P, 1, new, kv)
    Q = s.rng.standard_normal((s.T, G, D))
    first = back(check_attention(s, G, dtype, Q=Q, window=window, sinks=sinks))
    for _ in range(3):
        assert np.array_equal(back(run_attention(s, G, dtype, Q=Q, window=window, sinks=sinks)[0]), first)


def test_attention_splits_are_deterministic_and_reuse_their_workspace():
    torch = torch_cuda()
    s = Setup(17, 128, 64, 2, [1, 1], [9000, 4100])
    need = qlin.qlin_kv8_attention_workspace_bytes(s.cache, s.batch, 8)
    assert need > 16384
    Q = s.rng.standard_normal((2, 8, 128))
    ys = [back(run_attention(s, 4, F16, Q=Q)[0]) for _ in range(5)]
    assert all(np.array_equal(y, ys[0]) for y in ys)
    check_attention(s, 4, F16, Q=Q)
    # two streams at once, a workspace each
    d, _ = to16(Q, F16)
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.zeros(need, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(4):
        for st, w in zip(streams, ws):
            y = torch.empty((2, 8, 128), dtype=torch.float16, device="cuda")
            y.record_stream(st)
            qlin.qlin_kv8_attention(s.cache, s.batch, d, F16, 8, 1.0 / np.sqrt(128), 0, 0, y, w, stream=st)
            outs.append(y)
    torch.cuda.synchronize()
    assert all(np.array_equal(back(y), ys[0]) for y in outs)


def test_offsets_past_32_bits():
    """Pages beyond 4 GiB of K codes: append, gather and attention there."""
    torch = torch_cuda()
    P, D, Hk, G = 128, 128, 4, 2
    pages = (1 << 32) // (Hk * P * D) + 40
    s = Setup(18, D, P, Hk, [1, 70], [300, 140])
    dk = torch.empty((pages, Hk, P, D), dtype=torch.int8, device="cuda")
    dv = torch.empty((pages, Hk, D, P), dtype=torch.int8, device="cuda")
    ds = torch.empty((pages, Hk, 2), dtype=torch.float32, device="cuda")
    n, shift = len(s.k), pages - len(s.k)
    dk[shift:], dv[shift:], ds[shift:] = s.dk, s.dv, s.ds
    s.dk, s.dv, s.ds = dk[shift:], dv[shift:], ds[shift:]
    s.cache = qlin.Kv8Cache(dk, dv, ds)
    table = torch.from_numpy(np.where(s.table >= 0, s.table + shift, -1).astype(np.int32)).cuda()
    s.batch = qlin.Kv8Batch(s.dev[0], s.dev[1], table, s.T, *s.counts)
    q, q_ref = run_append(s, Hk * G, F16, 128, False)
    s.check_cache()
    check_attention(s, G, F16)


def test_query_views_and_streams():
    """Queries as a slice of a fused projection, on a stream that is not the current one."""
    torch = torch_cuda()
    s = Setup(19, 64, 32, 2, [4, 1], [77, 130])
    x, xf = to16(s.rng.standard_normal((5, 12, 64)), F16)
    want = run_attention(s, 4, F16, Q=xf[:, :8])[0]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = torch.empty((5, 8, 64), dtype=torch.float16, device="cuda")
    need = qlin.qlin_kv8_attention_workspace_bytes(s.cache, s.batch, 8)
    qlin.qlin_kv8_attention(s.cache, s.batch, x[:, :8], F16, 8, 0.125, 0, 0, y, workspace(need), stream=st)
    torch.cuda.synchronize()
    assert np.array_equal(back(y), back(want))


def test_graph_replays_while_the_sequences_grow():
    """A captured append + attention step, replayed with device lengths that grow and work between the replays."""
    torch = torch_cuda()
    P, D, Hk, G, steps = 16, 64, 2, 4, 6
    s = Setup(20, D, P, Hk, [1, 1], [40 + steps, 9 + steps])
    s.kv = [40, 9]
    x = s.rng.standard_normal((steps, 2, Hk * (G + 2), D))
    xs = [to16(v, F16) for v in x]
    cos, sin = okv.rope_tables(64, D)
    dc, dn = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
    inp = torch.empty_like(xs[0][0])
    q = torch.empty((2, Hk * G, D), dtype=torch.float16, device="cuda")
    y = torch.empty_like(q)
    need = qlin.qlin_kv8_attention_workspace_bytes(s.cache, s.batch, Hk * G)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")

    def step():
        qlin.qlin_kv8_append(s.cache, s.batch, inp[:, :Hk * G], inp[:, Hk * G:Hk * (G + 1)], inp[:, Hk * (G + 1):], F16,
                             Hk * G, dc, dn, D, qlin.QLIN_ROPE_HALF, q)
        qlin.qlin_kv8_attention(s.cache, s.batch, q, F16, Hk * G, 0.125, 0, 0, y, ws)

    qlin.qlin_kv8_gather(s.cache, s.batch, *(torch.empty((2, Hk, D), dtype=torch.float16, device="cuda") for _ in range(2)), F16)
    qlin.qlin_kv8_attention(s.cache, s.batch, q.zero_(), F16, Hk * G, 0.125, 0, 0, y, ws)     # kernels are loaded
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        s.kv = [40 + i, 9 + i]
        s.kv_lens = np.array(s.kv, np.int32)
        s.dev[1].copy_(torch.from_numpy(s.kv_lens))
        inp.copy_(xs[i][0])
        graph.replay()
        torch.cuda.synchronize()
        xf = xs[i][1]
        q_ref = okv.append(s.k, s.v, s.scales, s.offsets, s.kv_lens, s.table, xf[:, :Hk * G], xf[:, Hk * G:Hk * (G + 1)],
                           xf[:, Hk * (G + 1):], cos, sin, D, False)
        s.check_cache()
        check_round16(q, q_ref, F16)
        ref, A, score, peak = okv.attention(s.k, s.v, s.scales, s.offsets, s.kv_lens, s.table, back(q), 0.125, 0, 0)
        assert (np.abs(back(y) - ref) <= attention_bound(A, ref, score, peak, D, max(s.kv), F16)).all()
