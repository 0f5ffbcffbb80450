"""The 8-bit cache's attention where its numbers are far apart: many small weights beside a large one, scores and value
scales near the ends of fp32's range.  Against fp64, within bounds derived from the kernels' roundings."""
import numpy as np
import pytest

from quantized_linear_layers_packed_amd import qlin
from tests.gpu_util import say, torch_cuda, workspace
from tests.test_gpu_kv8 import Setup, back, run_append, run_attention, to16

pytestmark = pytest.mark.gpu

F16, BF16 = qlin.QLIN_F16, qlin.QLIN_BF16
F = np.float32
LOG2E = np.log2(np.e)

# Calls by the kernel that serves them: head_dim, query heads of the one key/value head, sequences.  Up to 64 rows (heads
# of 256: 16) go to the kernel for few rows, more to the one for many; as many sequences as fit the device at once leave
# every sequence to one workgroup, a single one is split over the device; "two": 32 rows to a wave.
CALLS = {"few": (128, 4, 512), "few split": (128, 4, 1), "few two": (128, 32, 512), "few 64": (64, 16, 512), "few two 64": (64, 32, 512),
         "few 256": (256, 8, 300), "many": (128, 72, 256), "many split": (128, 72, 1),
         "many 64": (64, 72, 512), "many 256": (256, 40, 256)}


class Shared:
    """`seqs` single-token sequences that all read the same L cached tokens of one head (pages in a shuffled order)."""

    def __init__(self, D, P, L, seqs, k, v, key_scale, value_scales):
        """k, v: codes [L][D]; key_scale: one for all pages; value_scales: [pages]."""
        torch = torch_cuda()
        pages = -(-L // P)
        self.T, self.L, self.D = seqs, L, D
        order = np.random.default_rng(1).permutation(pages)
        pad = np.zeros((pages * P - L, D), np.int8)
        kc, vc = (np.concatenate([x, pad]).reshape(pages, P, D) for x in (k, v))
        K, V = np.empty((pages, 1, P, D), np.int8), np.empty((pages, 1, D, P), np.int8)
        S = np.empty((pages, 1, 2), F)
        K[order, 0], V[order, 0] = kc, vc.transpose(0, 2, 1)
        S[order, 0, 0], S[order, 0, 1] = key_scale, value_scales
        self.dev = [torch.from_numpy(x).cuda() for x in (K, V, S)]
        table = torch.from_numpy(np.broadcast_to(order.astype(np.int32), (seqs, pages)).copy()).cuda()
        lens = torch.full((seqs,), L, dtype=torch.int32, device="cuda")
        offsets = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
        self.cache, self.batch = qlin.Kv8Cache(*self.dev), qlin.Kv8Batch(offsets, lens, table, seqs, 1, L)
        self.k = k.astype(np.float64) * np.float64(F(key_scale))
        self.v = v.astype(np.float64) * np.repeat(np.asarray(value_scales, F).astype(np.float64), P)[:L, None]

    def run(self, q, G, dtype):
        """q [G][D], the same for every sequence -> outputs [seqs][G][D]; scale 1."""
        torch = torch_cuda()
        d, q = to16(np.broadcast_to(q, (self.T, G, self.D)), dtype)
        Y = torch.full((self.T, G, self.D), 7.0, dtype=d.dtype, device="cuda")
        need = qlin.qlin_kv8_attention_workspace_bytes(self.cache, self.batch, G)
        qlin.qlin_kv8_attention(self.cache, self.batch, d, dtype, G, 1.0, 0, 0, Y, workspace(need))
        return back(Y).astype(np.float64), q[0].astype(np.float64)

    def check(self, q, G, dtype):
        Y, q = self.run(q, G, dtype)
        ref, tol = self.reference(q, dtype)
        err = np.abs(Y - ref)
        say(f"  worst error / bound: {float((err / tol).max()):.3f}, relative error {float((err / np.abs(ref)).max()):.2e}")
        assert (err <= tol).all()

    def reference(self, q, dtype):
        """fp64 outputs [G][D] and the error that the kernels' roundings allow:

        out:     half a unit of the output type (the last term: its smallest subnormals)
        weights: rounded to fp16 where the row's largest is 2^7 at least, so each by 2^-11 of itself or, as a subnormal,
                 by 2^-25 / 2^7 of the largest (of a sum that is at least the largest), times values of at most `peak`
        scores:  D products summed in fp32 and a few fp32 operations after that, 2^-24 of sum |q k| each, in numerator
                 and denominator
        sums:    fp32, 16 tokens to a step, 2^-24 for each step and join, in numerator and denominator
        """
        x = q @ self.k.T
        w = np.exp(x - x.max(axis=1, keepdims=True))
        w /= w.sum(axis=1, keepdims=True)
        ref, A = w @ self.v, w @ np.abs(self.v)
        score = (np.abs(q) @ np.abs(self.k).T).max(axis=1)[:, None]
        u_out, least = (2.0 ** -11, 2.0 ** -25) if dtype == F16 else (2.0 ** -8, 2.0 ** -134)
        rel = 2.0 ** -11 + 2 * (self.D + 16) * 2.0 ** -24 * (score + 1) + 2 * (self.L / 16 + 64) * 2.0 ** -24
        return ref, u_out * np.abs(ref) + rel * A + self.L * 2.0 ** -32 * np.abs(self.v).max() + least


def by_first_dimension(D, codes):
    """Key codes [L][D] that are `codes` in dimension 0 and anything elsewhere, and a query that sees dimension 0 alone."""
    k = np.random.default_rng(2).integers(-127, 128, (len(codes), D)).astype(np.int8)
    k[:, 0] = codes
    return k, lambda x: np.concatenate([[x], np.zeros(D - 1)])[None]


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("below,dtype", [(20.6, F16), (25.1, F16), (20.6, BF16)])
def test_a_long_flat_tail_keeps_its_share(call, below, dtype):
    """A few tokens of large weight and 131 thousand of 2^-20.6 (or 2^-25.1) of it, each below an fp16 unit of the
    largest, together one to eight per cent of the output's weights."""
    D, G, seqs = CALLS[call]
    say(f"kv8 attention, flat tail: {call}, 2^-{below}")
    L = 131003
    codes = np.zeros(L, np.int64)
    codes[0 if call.startswith("many") else np.arange(0, 512, 64)] = 127    # one for every wave that walks by itself
    k, q = by_first_dimension(D, codes)
    v = np.where(codes[:, None] > 0, 10 + np.arange(D) % 3, 120 - np.arange(D) % 5).astype(np.int8)
    s = Shared(D, 64, L, seqs, k, v, 1.0 / 127, np.ones(-(-L // 64)))
    s.check(q(below / LOG2E), G, dtype)


@pytest.mark.parametrize("call", list(CALLS))
def test_many_tokens_without_values_do_not_overflow_the_sum_of_weights(call):
    """131 thousand tokens of all-zero values (scale 0), the first ones lower in score by almost the slack of the running
    reference, then a thousand tokens with values and a tenth of the weight."""
    D, G, seqs = CALLS[call]
    say(f"kv8 attention, values of zero: {call}")
    L, P = 132064, 32
    codes = np.full(L, 79, np.int64)
    codes[:512], codes[131072:] = 0, 119                                    # 0, 7.9 and 11.9 in log2
    k, q = by_first_dimension(D, codes)
    v = np.where(np.arange(L)[:, None] >= 131072, 100 - np.arange(D) % 7, 0).astype(np.int8)
    scales = np.where(np.arange(L // P) * P >= 131072, 1.0, 0.0)
    s = Shared(D, P, L, seqs, k, v, 0.1, scales)
    s.check(q(1.0 / LOG2E), G, F16)


def winner_takes_all(D, key_scale):
    """5003 cached tokens whose keys have codes -127 .. -64 in the one dimension that the query sees, but token 2400's -1."""
    L = 5003
    codes = -64 - np.arange(L) % 64
    codes[2400] = -1
    k, q = by_first_dimension(D, codes)
    v = (np.arange(L)[:, None] % 97 + np.arange(D) % 23).astype(np.int8)
    return L, k, v, key_scale, q


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("dtype,key_scale,x", [(BF16, 2.0 ** 60, 2.0 ** 50), (F16, 2.0 ** 100, 2.0 ** 15), (BF16, 2.0, 2.0 ** 118)])
def test_scores_far_below_zero_still_have_a_largest(call, dtype, key_scale, x):
    """Scores from -2^110 or -2^115 or -2^119 down: the row is its largest one's value, not zeros as if it saw nothing."""
    D, G, seqs = CALLS[call]
    say(f"kv8 attention, scores of -{key_scale * x:.1e}: {call}")
    L, k, v, key_scale, q = winner_takes_all(D, key_scale)
    Y, _ = Shared(D, 64, L, seqs, k, v, key_scale, np.ones(-(-L // 64))).run(q(x), G, dtype)
    assert np.array_equal(Y, np.broadcast_to(v[2400].astype(np.float64), Y.shape))


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("x", [2.0 ** 100, np.inf, -2.0 ** 100, -np.inf])
def test_scores_past_the_range_of_fp32_give_nan(call, x):
    """All scores -inf (or +inf) in fp32: no weights can be formed, and the row says so."""
    D, G, seqs = CALLS[call]
    say(f"kv8 attention, scores of -{x} 2^100: {call}")
    L, k, v, key_scale, q = winner_takes_all(D, 2.0 ** 100)
    Y, _ = Shared(D, 64, L, seqs, k, v, key_scale, np.ones(-(-L // 64))).run(q(x), G, BF16)
    assert np.isnan(Y).all()


@pytest.mark.parametrize("new,window", [(1, 64), (60, 64), (1, 0), (60, 0)])
@pytest.mark.parametrize("garbage", [np.nan, np.inf, -np.inf, -3e38, -1.0, 0.0, 1e-39, 1e-31])
def test_scales_of_hidden_pages_may_be_anything(new, window, garbage):
    """Pages outside the window, and those of the pool that table entries of -1 stand in for, do not reach a result."""
    say(f"kv8 attention, hidden scales of {garbage}: new={new} window={window}")
    P, kv = 16, 400
    s = Setup(31, 64, P, 1, [new], [kv])
    s.table[s.table == 0] = next(p for p in range(1, len(s.k)) if p not in s.table)   # page 0 stands in for -1
    s.table[0, 5:12] = -1
    s.upload()
    Q = np.full((new, 4, 64), 0.5)
    clean = back(run_attention(s, 4, F16, window=window, Q=Q)[0])
    s.scales[[p for p in range(len(s.k)) if p not in s.table]] = garbage
    if window:
        s.scales[s.table[0, 12:(kv - new - window) // P]] = garbage
    s.upload()
    assert np.isfinite(clean).all() and np.array_equal(back(run_attention(s, 4, F16, window=window, Q=Q)[0]), clean)


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("low,high", [(-80, -76), (-80, -60), (0, 20)])
def test_value_scales_down_to_the_least_that_append_keeps(call, low, high):
    D, G, seqs = CALLS[call]
    say(f"kv8 attention, value scales 2^{low} .. 2^{high}: {call}")
    L, P = 1801, 16
    r = np.random.default_rng(3)
    k, v = (r.integers(-127, 128, (L, D)).astype(np.int8) for _ in range(2))
    s = Shared(D, P, L, seqs, k, v, 0.02, 2.0 ** r.uniform(low, high, -(-L // P)))
    s.check(r.standard_normal((1, D)) / np.sqrt(D), G, BF16)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("exponent", [-133, -120, -110, -90, -81, -79, -70])
def test_attention_and_gather_agree_on_tiny_values(new, exponent):
    """bf16 values that need scales of 2^exponent: append keeps or drops them, and both readers say the same.  Every token
    has the same value, so any weights give it back; between the two lie the output's rounding and those of the sums."""
    torch = torch_cuda()
    say(f"kv8 append, gather, attention, value scales 2^{exponent}: new={new}")
    s = Setup(32, 64, 16, 1, [new, new], [new, new])
    x = s.rng.standard_normal((s.T, 6, 64))
    value = 2.0 ** exponent * 127 * (1 + np.arange(64) % 8) / 8
    x[:, 5] = value
    run_append(s, 4, BF16, 0, False, x=x)
    s.check_cache()
    K, V = (torch.empty((s.T, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qlin.qlin_kv8_gather(s.cache, s.batch, K, V, BF16)
    V = back(V).astype(np.float64)
    if exponent < -80:
        assert not V.any() and not s.scales[s.table[s.table >= 0], :, 1].any()
    else:
        assert (np.abs(V - value) <= 2.0 ** exponent / 2 * (1 + 2.0 ** -7) + 2.0 ** -8 * value).all()   # a code's, bf16's
    Y = back(run_attention(s, 4, BF16)[0])
    assert (np.abs(Y - V) <= (2 * 2.0 ** -8 + 2.0 ** -11 + 200 * 2.0 ** -24) * np.abs(V)).all()


@pytest.mark.parametrize("call", list(CALLS))
def test_tokens_without_values_keep_their_weight_beside_large_values(call):
    """131 thousand tokens of all-zero values (scale 0) and 2^-18.5 of the weight of a few whose page's scale is 2^15."""
    D, G, seqs = CALLS[call]
    say(f"kv8 attention, values of zero beside large ones: {call}")
    L, P = 131072, 64
    large = np.zeros(1) if call.startswith("many") else np.arange(0, 512, 64)
    codes = np.zeros(L, np.int64)
    codes[large.astype(int)] = 127
    k, q = by_first_dimension(D, codes)
    v = np.where(codes[:, None] > 0, np.ones(D, np.int64), 0).astype(np.int8)
    scales = np.where(v.reshape(-1, P * D).any(axis=1), 2.0 ** 15, 0.0)
    s = Shared(D, P, L, seqs, k, v, 1.0 / 127, scales)
    s.check(q(18.5 / LOG2E), G, F16)
