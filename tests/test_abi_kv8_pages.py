"""CPU-only checks of the page book's entry points: refusals before anything is enqueued, and what the binding takes."""
import ctypes as C

import pytest
import torch

from quantized_linear_layers_packed_amd import qlin
from tests.test_abi_kv8 import EALIGN, EINVAL, EUNSUPPORTED, FAKE, cache

lib = qlin._lib


def book(**kw):
    d = dict(refs=FAKE, block_table=FAKE, num_pages=8, page_size=16, rows=3, table_stride=4)
    d.update(kw)
    return C.byref(qlin._KvBook(*(d[n] for n, _ in qlin._KvBook._fields_)))


def grow(b=None, lens=FAKE, moves=FAKE):
    return lib.qlin_kv8_grow(b or book(), lens, moves, 0)


def fork(b=None, parents=FAKE, children=FAKE, lens=FAKE, count=2, moves=FAKE):
    return lib.qlin_kv8_fork(b or book(), parents, children, lens, count, moves, 0)


def free(b=None, rows=FAKE, begin=None, end=None, count=2):
    return lib.qlin_kv8_free(b or book(), rows, begin, end, count, 0)


def compact(b=None, most=4, moves=FAKE):
    return lib.qlin_kv8_compact(b or book(), most, moves, 0)


@pytest.mark.parametrize("call", [grow, fork, free, compact])
def test_every_call_checks_the_book(call):
    for kw, want in (({"refs": 0}, EINVAL), ({"refs": FAKE + 4}, EALIGN), ({"block_table": 0}, EINVAL),
                     ({"block_table": FAKE + 8}, EALIGN), ({"num_pages": 0}, EINVAL), ({"num_pages": (1 << 30) + 1}, EUNSUPPORTED),
                     ({"page_size": 24}, EUNSUPPORTED), ({"page_size": -16}, EINVAL), ({"rows": 0}, EINVAL),
                     ({"rows": 32768}, EUNSUPPORTED), ({"table_stride": 0}, EINVAL),
                     ({"rows": 32767, "table_stride": 65540}, EUNSUPPORTED)):
        assert call(book(**kw)) == want, kw
        assert next(iter(kw)) in qlin.last_error()


def test_lists():
    for call, kw, want in ((grow, {"lens": None}, EINVAL), (grow, {"moves": None}, EINVAL), (grow, {"moves": FAKE + 8}, EALIGN),
                           (fork, {"parents": None}, EINVAL), (fork, {"children": FAKE + 4}, EALIGN), (fork, {"lens": None}, EINVAL),
                           (fork, {"count": 0}, EINVAL), (fork, {"count": 16385}, EUNSUPPORTED), (fork, {"moves": None}, EINVAL),
                           (free, {"rows": None}, EINVAL), (free, {"begin": FAKE + 4}, EALIGN), (free, {"end": FAKE + 4}, EALIGN),
                           (free, {"count": -1}, EINVAL), (free, {"count": 65536}, EUNSUPPORTED),
                           (compact, {"most": 0}, EINVAL), (compact, {"moves": None}, EINVAL)):
        assert call(**kw) == want, (call, kw)


def test_copy_pages_refusals():
    two = lambda a, b=None: (qlin._KvCache * 2)(a, b or cache())                                   # noqa: E731

    def copy(to=None, source=None, layers=2, moves=FAKE, most=4):
        return lib.qlin_kv8_copy_pages(to or two(cache()), source or two(cache()), layers, moves, most, 0)

    for kw, want in (({"layers": 0}, EINVAL), ({"most": 0}, EINVAL), ({"moves": None}, EINVAL), ({"moves": FAKE + 4}, EALIGN),
                     ({"to": two(cache(kv_heads=4))}, EINVAL), ({"source": two(cache(page_size=32))}, EINVAL),
                     ({"source": two(cache(), cache(head_dim=64))}, EINVAL), ({"source": two(cache(), cache(num_pages=9))}, EINVAL),
                     ({"to": two(cache(), cache(k_codes=0))}, EINVAL), ({"to": two(cache(scales=FAKE + 8))}, EALIGN),
                     ({"source": two(cache(head_dim=80))}, EUNSUPPORTED)):
        assert copy(**kw) == want, (kw, qlin.last_error())
    big = cache(kv_heads=32767, num_pages=2, head_dim=256, page_size=128)
    assert lib.qlin_kv8_copy_pages(C.byref(big), C.byref(big), 1, None, 1, 0) == EINVAL      # (chunks fit: the list is at fault)
    assert lib.qlin_kv8_copy_pages(None, C.byref(big), 1, FAKE, 1, 0) == EINVAL


def test_binding_checks_shapes_and_types():
    i = lambda *n: torch.zeros(n, dtype=torch.int32)                                              # noqa: E731
    b = qlin.Kv8Book(i(8), i(3, 4), 16)
    for bad in ((i(8, 1), i(3, 4)), (i(8), i(12)), (i(8).float(), i(3, 4)), (i(8), i(3, 4).long()), (i(8), i(4, 3).T)):
        with pytest.raises(ValueError):
            qlin.Kv8Book(*bad, 16)
    k, v, s = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2, 64, 16, dtype=torch.int8), torch.zeros(4, 2, 2)
    c = qlin.Kv8Cache(k, v, s)
    for call in (lambda: qlin.qlin_kv8_grow(b, i(4), i(1, 2), stream=0), lambda: qlin.qlin_kv8_grow(b, i(3), i(2), stream=0),
                 lambda: qlin.qlin_kv8_grow(b, i(3).long(), i(1, 2), stream=0), lambda: qlin.qlin_kv8_grow(b, i(3), i(0, 2), stream=0), lambda: qlin.qlin_kv8_grow(b, i(3), i(5, 2), stream=0),
                 lambda: qlin.qlin_kv8_fork(b, i(2), i(3), i(2), i(3, 2), stream=0),
                 lambda: qlin.qlin_kv8_fork(b, i(2), i(2), i(2), i(2, 2), stream=0),
                 lambda: qlin.qlin_kv8_free(b, i(2), i(1), stream=0), lambda: qlin.qlin_kv8_free(b, i(2), None, i(2).float(), stream=0),
                 lambda: qlin.qlin_kv8_compact(b, i(1, 2), stream=0), lambda: qlin.qlin_kv8_compact(b, i(3, 3), stream=0),
                 lambda: qlin.qlin_kv8_copy_pages(c, qlin.Kv8Caches([c, c]), i(3, 2), stream=0),
                 lambda: qlin.qlin_kv8_copy_pages(c, c, i(1, 2), stream=0)):
        with pytest.raises(ValueError):
            call()
