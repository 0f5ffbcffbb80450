"""Pins of the 8-bit cache oracle: hand-worked codes and scales, rotation against complex numbers, attention against a
direct sum."""
import numpy as np
import pytest

from oracle import kv8

F = np.float32


def cache(pages, H, P, D):
    return np.zeros((pages, H, P, D), np.int8), np.zeros((pages, H, D, P), np.int8), np.full((pages, H, 2), 9.0, F)


def test_append_by_hand():
    k, v, s = cache(2, 1, 16, 64)
    K = np.zeros((3, 1, 64), F)
    K[0, 0, :3] = [127.0, -63.5, 1.4]                 # scale 1: codes 127, -64 (half to even), 1
    K[1, 0, :2] = [1.0, -127.0]
    K[2, 0, :2] = [254.0, 5.0]                        # scale 2: its codes 127, 2 (2.5 to even)
    none = np.zeros((0, 0, 0), F)
    table = [[1]]
    kv8.append(k, v, s, [0, 2], [2], table, K[:2], K[:2], K[:2], None, None, 0, False)
    assert s[1, 0].tolist() == [1.0, 1.0] and s[0, 0].tolist() == [9.0, 9.0] and none.size == 0
    assert k[1, 0, 0, :4].tolist() == [127, -64, 1, 0] and k[1, 0, 1, :2].tolist() == [1, -127]
    assert v[1, 0, :3, 0].tolist() == [127, -64, 1] and v[1, 0, :2, 1].tolist() == [1, -127]
    kv8.append(k, v, s, [0, 1], [3], table, K[2:], K[2:], K[2:], None, None, 0, False)
    assert s[1, 0].tolist() == [2.0, 2.0]
    # earlier codes halved, halves to even: 127 -> 63.5 -> 64, -64 -> -32, 1 -> 0.5 -> 0
    assert k[1, 0, 0, :3].tolist() == [64, -32, 0] and k[1, 0, 1, :2].tolist() == [0, -64]
    assert k[1, 0, 2, :2].tolist() == [127, 2] and v[1, 0, :2, 2].tolist() == [127, 2]
    assert not k[0].any() and not v[0].any()


def test_append_starts_a_page_anew_and_poisons_it():
    k, v, s = cache(1, 1, 16, 64)
    s[:] = 50.0                                       # a scale of the page's earlier use does not count
    x = np.full((1, 1, 64), 127.0, F)
    kv8.append(k, v, s, [0, 1], [1], [[0]], x, x, x, None, None, 0, False)
    assert s[0, 0].tolist() == [1.0, 1.0]
    bad = x.copy()
    bad[0, 0, 5] = np.inf
    kv8.append(k, v, s, [0, 1], [2], [[0]], x, bad, x, None, None, 0, False)
    assert np.isnan(s[0, 0, 0]) and s[0, 0, 1] == 1.0
    kv8.append(k, v, s, [0, 1], [3], [[0]], x, x, x, None, None, 0, False)
    assert np.isnan(s[0, 0, 0])                       # until the page starts anew
    kv8.append(k, v, s, [0, 1], [1], [[0]], x, x, x, None, None, 0, False)
    assert s[0, 0, 0] == 1.0


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_is_a_complex_product(pairs):
    r = np.random.default_rng(1)
    x = r.standard_normal((3, 64)).astype(F)
    cos, sin = kv8.rope_tables(40, 32)
    y = kv8.rotate(x, cos[37], sin[37], 32, pairs)
    a, b = (x[:, 0:32:2], x[:, 1:32:2]) if pairs else (x[:, :16], x[:, 16:32])
    z = (a + 1j * b) * np.exp(1j * 37 * 10000.0 ** (-np.arange(16) / 16))
    ya, yb = (y[:, 0:32:2], y[:, 1:32:2]) if pairs else (y[:, :16], y[:, 16:32])
    # three fp32 roundings of products below 2^3
    assert np.abs(ya - z.real).max() < 2e-6 and np.abs(yb - z.imag).max() < 2e-6
    assert np.array_equal(y[:, 32:], x[:, 32:])


def test_attention_is_the_weighted_mean_of_visible_values():
    r = np.random.default_rng(2)
    k = r.integers(-127, 128, (4, 2, 16, 64)).astype(np.int8)
    v = r.integers(-127, 128, (4, 2, 64, 16)).astype(np.int8)
    s = r.uniform(0.01, 0.02, (4, 2, 2)).astype(F)
    Q = r.standard_normal((3, 4, 64)).astype(F)
    table = [[2, 0, 3]]
    Y, A, _, _ = kv8.attention(k, v, s, [0, 3], [41], table, Q, 0.125, 20, 2)
    h, i = 3, 1                                       # query 1 at position 39 sees 0, 1 and 20 .. 39
    js = [0, 1] + list(range(20, 40))
    num, den = np.zeros(64), 0.0
    for j in js:
        page = table[0][j // 16]
        w = np.exp(0.125 * float(Q[i, h].astype(float) @ (k[page, 1, j % 16] * float(s[page, 1, 0]))))
        num += w * v[page, 1, :, j % 16] * float(s[page, 1, 1])
        den += w
    assert np.allclose(Y[i, h], num / den, rtol=1e-12, atol=1e-12)
    assert (A >= np.abs(Y) - 1e-12).all()
    # a page given back and a query before the first position see nothing
    Y, _, _, _ = kv8.attention(k, v, s, [0, 3], [2], [[-1]], Q, 0.125, 0, 0)
    assert not Y.any()
