"""CPU-only checks of the attention with other scores and masks: refusals before anything is enqueued."""
import ctypes as C

import pytest
import torch

from quantized_linear_layers_packed_amd import qlin
from tests.test_abi_kv8 import EALIGN, EINVAL, EUNSUPPORTED, F16, FAKE, batch, cache


def scored(c=None, b=None, how=None, **kw):
    a = dict(Q=FAKE, dtype=F16, q_heads=4, q_stride=512, scale=0.1, window=0, sinks=0, scoring=None, Y=FAKE << 4, ws=None, ws_bytes=0)
    a.update(kw)
    s = dict(cap=0.0, slopes=None, prefix_lens=None, starts=None)
    s.update(how or {})
    if a["scoring"] is None:
        a["scoring"] = C.byref(qlin._KvScoring(*s.values()))
    return qlin._lib.qlin_kv8_attention_scored(C.byref(c or cache()), C.byref(b or batch(max_kv=60)), *a.values(), 0)


def test_scoring_is_checked():
    nan, inf = float("nan"), float("inf")
    for how, want in (({"cap": -1.0}, EINVAL), ({"cap": nan}, EINVAL), ({"cap": inf}, EINVAL), ({"cap": 2.0 ** -11}, EINVAL),
                      ({"cap": 1025.0}, EINVAL), ({"slopes": FAKE + 4}, EALIGN), ({"prefix_lens": FAKE + 8}, EALIGN),
                      ({"starts": FAKE + 4}, EALIGN)):
        assert scored(how=how) == want, how
        assert next(iter(how)) in qlin.last_error()
    assert scored(scoring=C.c_void_p(None)) == EINVAL and "scoring" in qlin.last_error()


def test_what_the_plain_attention_refuses_is_refused_here_too():
    for kw, want in (({"Q": None}, EINVAL), ({"Y": None}, EINVAL), ({"Y": FAKE + 2}, EALIGN), ({"q_heads": 5}, EINVAL),
                     ({"q_stride": 508}, EINVAL), ({"scale": 0.0}, EINVAL), ({"scale": float("nan")}, EINVAL),
                     ({"window": -1}, EINVAL), ({"sinks": 4}, EINVAL), ({"Y": FAKE + 512}, EINVAL), ({"dtype": qlin.QLIN_F32}, EINVAL),
                     ({"q_heads": 1 << 29, "q_stride": 1 << 36}, EUNSUPPORTED)):
        assert scored(**kw) == want, (kw, qlin.last_error())
    assert scored(c=cache(head_dim=96)) == EUNSUPPORTED
    long = batch(max_kv=100000, table_stride=2000, max_new=1)
    assert scored(b=long) == EINVAL and "workspace" in qlin.last_error()
    # what the kernels hold has to be finite: 2 log2(e) scale / cap
    assert scored(b=long, scale=1.2e35, how={"cap": 2.0 ** -10}) == EINVAL and "cap" in qlin.last_error()
    assert scored(b=long, scale=1.2e35, how={"cap": 50.0}) == EINVAL and "workspace" in qlin.last_error()


def test_binding_checks_the_tensors():
    i = lambda *n: torch.zeros(n, dtype=torch.int32)                                              # noqa: E731
    for bad in (dict(slopes=i(4)), dict(prefix_lens=torch.zeros(2)), dict(starts=i(5).long()), dict(slopes=torch.zeros(4, 1)),
                dict(starts=i(10)[::2])):
        with pytest.raises(ValueError):
            qlin.Kv8Scoring(0.0, **bad)
    c = qlin.Kv8Cache(torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2, 64, 16, dtype=torch.int8), torch.zeros(4, 2, 2))
    b = qlin.Kv8Batch(i(3), i(2), i(2, 4), 5, 3, 60)
    x = torch.zeros((5, 4, 64), dtype=torch.float16)
    call = lambda s, q=x, y=x: qlin.qlin_kv8_attention_scored(c, b, q, F16, 4, 0.1, 0, 0, s, y, stream=0)   # noqa: E731
    for bad in (dict(slopes=torch.zeros(3)), dict(prefix_lens=i(3)), dict(starts=i(4))):
        with pytest.raises(ValueError, match=next(iter(bad))):
            call(qlin.Kv8Scoring(1.0, **bad))
    for kw in (dict(q=x.bfloat16()), dict(y=x[:4].contiguous()), dict(q=x[:4])):
        with pytest.raises(ValueError):
            call(qlin.Kv8Scoring(1.0), **kw)
    with pytest.raises(qlin.QlinError):                                # Y is Q
        call(qlin.Kv8Scoring(1.0, torch.zeros(4), i(2), i(5)))
