"""CPU-only checks of the 8-bit cache's entry points: sizes, workspaces and refusals, before anything is enqueued."""
import ctypes as C

import pytest
import torch

from quantized_linear_layers_packed_amd import qlin

EINVAL, EALIGN, EUNSUPPORTED = qlin.QLIN_EINVAL, qlin.QLIN_EALIGN, qlin.QLIN_EUNSUPPORTED
FAKE = 0x100000                   # aligned non-NULL addresses, never dereferenced by host-side validation
F16 = qlin.QLIN_F16


def cache(**kw):
    d = dict(k_codes=FAKE, v_codes=FAKE, scales=FAKE, num_pages=8, kv_heads=2, head_dim=128, page_size=64)
    d.update(kw)
    return qlin._KvCache(*(d[n] for n, _ in qlin._KvCache._fields_))


def batch(**kw):
    d = dict(offsets=FAKE, kv_lens=FAKE, block_table=FAKE, seqs=2, tokens=5, table_stride=4, max_new=3, max_kv=200)
    d.update(kw)
    return qlin._KvBatch(*(d[n] for n, _ in qlin._KvBatch._fields_))


def append(c=None, b=None, **kw):
    a = dict(Q=FAKE, K=FAKE, V=FAKE, dtype=F16, q_heads=4, q_stride=1024, k_stride=1024, v_stride=1024, cos=FAKE, sin=FAKE,
             max_pos=100, rot=128, style=0, out=FAKE << 4)
    a.update(kw)
    return qlin._lib.qlin_kv8_append(C.byref(c or cache()), C.byref(b or batch()), *a.values(), 0)


def attention(c=None, b=None, **kw):
    a = dict(Q=FAKE, dtype=F16, q_heads=4, q_stride=512, scale=0.1, window=0, sinks=0, Y=FAKE << 4, ws=None, ws_bytes=0)
    a.update(kw)
    return qlin._lib.qlin_kv8_attention(C.byref(c or cache()), C.byref(b or batch()), *a.values(), 0)


def gather(c=None, b=None, **kw):
    a = dict(K=FAKE, V=FAKE, dtype=F16)
    a.update(kw)
    return qlin._lib.qlin_kv8_gather(C.byref(c or cache()), C.byref(b or batch()), *a.values(), 0)


@pytest.mark.parametrize("call", [append, attention, gather])
def test_every_call_checks_cache_and_batch(call):
    for kw, want in (({"num_pages": 0}, EINVAL), ({"kv_heads": -1}, EINVAL), ({"head_dim": 96}, EUNSUPPORTED),
                     ({"page_size": 24}, EUNSUPPORTED), ({"page_size": 0}, EINVAL), ({"k_codes": 0}, EINVAL),
                     ({"v_codes": FAKE + 8}, EALIGN), ({"scales": 0}, EINVAL), ({"scales": FAKE + 4}, EALIGN),
                     ({"kv_heads": 40000}, EUNSUPPORTED), ({"num_pages": 1 << 30, "kv_heads": 4}, EUNSUPPORTED)):
        assert call(c=cache(**kw)) == want, kw
        assert next(iter(kw)) in qlin.last_error() or "cache" in qlin.last_error()
    for kw, want in (({"seqs": 0}, EINVAL), ({"tokens": 0}, EINVAL), ({"table_stride": 0}, EINVAL), ({"max_new": 0}, EINVAL),
                     ({"max_kv": -1}, EINVAL), ({"offsets": 0}, EINVAL), ({"kv_lens": FAKE + 4}, EALIGN),
                     ({"block_table": 0}, EINVAL), ({"seqs": 70000}, EUNSUPPORTED)):
        assert call(b=batch(**kw)) == want, kw
    assert call(dtype=qlin.QLIN_F32) == EINVAL


def test_append_refusals():
    for kw, want in (({"K": None}, EINVAL), ({"V": FAKE + 2}, EALIGN), ({"Q": None}, EINVAL), ({"out": None}, EINVAL),
                     ({"q_heads": 3}, EINVAL), ({"q_stride": 504}, EINVAL), ({"k_stride": 260}, EINVAL),
                     ({"v_stride": 128}, EINVAL), ({"rot": 24}, EINVAL), ({"rot": 144}, EINVAL), ({"rot": -16}, EINVAL),
                     ({"cos": None}, EINVAL), ({"sin": FAKE + 4}, EALIGN), ({"max_pos": 0}, EINVAL), ({"style": 2}, EINVAL),
                     ({"out": FAKE}, EINVAL),                        # in place needs contiguous queries
                     ({"out": FAKE + 1024}, EINVAL),
                     ({"K": FAKE << 4}, EINVAL),                     # keys under the rotated queries
                     ({"k_stride": 1 << 42}, EUNSUPPORTED)):
        assert append(**kw) == want, (kw, qlin.last_error())


def test_attention_refusals_and_workspace():
    for kw, want in (({"Q": None}, EINVAL), ({"Y": None}, EINVAL), ({"Y": FAKE + 2}, EALIGN), ({"Q": FAKE + 8}, EALIGN),
                     ({"q_heads": 0}, EINVAL), ({"q_heads": 5}, EINVAL), ({"q_stride": 508}, EINVAL),
                     ({"scale": 0.0}, EINVAL), ({"scale": float("nan")}, EINVAL), ({"scale": float("inf")}, EINVAL),
                     ({"q_heads": 1 << 29, "q_stride": 1 << 36}, EUNSUPPORTED), ({"window": -1}, EINVAL), ({"sinks": -1}, EINVAL), ({"sinks": 4}, EINVAL), ({"Y": FAKE + 512}, EINVAL)):
        assert attention(b=batch(max_kv=60), **kw) == want, (kw, qlin.last_error())
    need = C.c_size_t()
    long = batch(max_kv=100000, table_stride=2000, max_new=1)
    assert qlin._lib.qlin_kv8_attention_workspace_bytes(C.byref(cache(k_codes=0)), C.byref(long), 4, 0, 0, C.byref(need)) == 0
    assert need.value > 16384
    assert qlin._lib.qlin_kv8_attention_workspace_bytes(C.byref(cache()), C.byref(long), 4, 0, 0, None) == EINVAL
    assert attention(b=long) == EINVAL and str(need.value) in qlin.last_error()
    assert attention(b=long, ws=FAKE, ws_bytes=need.value - 1) == EINVAL
    assert attention(b=long, ws=FAKE + 8, ws_bytes=need.value) == EALIGN
    one = batch(max_kv=60, max_new=1)
    assert qlin._lib.qlin_kv8_attention_workspace_bytes(C.byref(cache()), C.byref(one), 4, 0, 0, C.byref(need)) == 0
    assert need.value == 0


def test_sizes():
    assert qlin.qlin_kv8_sizes(10, 8, 128, 64) == (10 * 8 * 128 * 64, 10 * 8 * 128 * 64, 10 * 8 * 8)
    assert qlin.qlin_kv8_sizes(1 << 20, 8, 128, 64)[0] == 1 << 36
    with pytest.raises(qlin.QlinError):
        qlin.qlin_kv8_sizes(10, 8, 80, 64)


def test_binding_checks_shapes():
    k, v, s = (torch.zeros(shape, dtype=t) for shape, t in (((4, 2, 16, 64), torch.int8), ((4, 2, 64, 16), torch.int8),
                                                           ((4, 2, 2), torch.float32)))
    i = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    c = qlin.Kv8Cache(k, v, s)
    b = qlin.Kv8Batch(i(3), i(2), i(2, 4), 5, 3, 60)
    with pytest.raises(ValueError):
        qlin.Kv8Cache(k, k, s)
    with pytest.raises(ValueError):
        qlin.Kv8Cache(k, v, s.double())
    with pytest.raises(ValueError):
        qlin.Kv8Batch(i(2), i(2), i(2, 4), 5, 3, 60)
    with pytest.raises(ValueError):
        qlin.Kv8Batch(i(3).long(), i(2), i(2, 4), 5, 3, 60)
    x = torch.zeros((5, 4, 64), dtype=torch.float16)
    for bad in (x[:4], x.float(), x.transpose(1, 2), torch.zeros((5, 4, 128), dtype=torch.float16)[..., ::2]):
        with pytest.raises(ValueError):
            qlin.qlin_kv8_attention(c, b, bad, F16, 4, 0.1, 0, 0, x, stream=0)
    with pytest.raises(ValueError):
        qlin.qlin_kv8_attention(c, b, x, F16, 4, 0.1, 0, 0, x[:4].contiguous(), stream=0)
    with pytest.raises(ValueError):
        qlin.qlin_kv8_append(c, b, x, x[:, :2], x[:, 2:], F16, 4, torch.zeros(9, 16), torch.zeros(9, 16), 64, 0, x, stream=0)
    with pytest.raises(qlin.QlinError):                                # a slice of Q is K: fine for reading, not as Q_out
        qlin.qlin_kv8_append(c, b, x, x[:, :2], x[:, 2:], F16, 4, None, None, 0, 0, x, stream=0)
