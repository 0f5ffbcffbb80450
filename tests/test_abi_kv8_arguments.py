"""CPU-only checks of the 8-bit cache's arguments: limits of numbers, and the types that the binding takes."""
import pytest
import torch

from quantized_linear_layers_packed_amd import qlin
from tests.test_abi_kv8 import EINVAL, attention, batch


@pytest.mark.parametrize("scale,fits", [(2.3e38, True), (2.4e38, False), (3.4e38, False)])
def test_a_scale_is_finite_in_the_exponent_of_two_as_well(scale, fits):
    """scale * log2(e) is what the kernels hold; one that fits gets as far as the missing workspace."""
    long = batch(max_kv=100000, table_stride=2000, max_new=1)
    assert attention(b=long, scale=scale) == EINVAL
    assert ("workspace" if fits else "scale") in qlin.last_error()


def tensors(**types):
    """A small cache, batch and projection on the host, of the types that the calls take but for those given."""
    t = dict(k=torch.int8, v=torch.int8, scales=torch.float32, offsets=torch.int32, kv_lens=torch.int32, table=torch.int32)
    t.update(types)
    shapes = dict(k=(4, 2, 16, 64), v=(4, 2, 64, 16), scales=(4, 2, 2), offsets=(3,), kv_lens=(2,), table=(2, 4))
    x = {n: torch.zeros(s, dtype=t[n]) for n, s in shapes.items()}
    cache = lambda: qlin.Kv8Cache(x["k"], x["v"], x["scales"])                                    # noqa: E731
    batch = lambda: qlin.Kv8Batch(x["offsets"], x["kv_lens"], x["table"], 5, 3, 60)               # noqa: E731
    return cache, batch


@pytest.mark.parametrize("name,bad", [("k", torch.bool), ("v", torch.float8_e4m3fn), ("scales", torch.int32)])
def test_cache_tensors_of_another_type_are_refused(name, bad):
    cache, _ = tensors()
    cache()
    cache, _ = tensors(**{name: bad})
    with pytest.raises(ValueError, match=str(bad)):
        cache()


@pytest.mark.parametrize("name", ["offsets", "kv_lens", "table"])
def test_batch_tensors_of_another_type_are_refused(name):
    _, batch = tensors()
    batch()
    _, batch = tensors(**{name: torch.float32})
    with pytest.raises(ValueError, match="torch.float32"):
        batch()


@pytest.mark.parametrize("dtype,right,wrong", [(qlin.QLIN_F16, torch.float16, torch.bfloat16),
                                               (qlin.QLIN_BF16, torch.bfloat16, torch.float16)])
def test_rows_of_the_other_16_bit_type_are_refused(dtype, right, wrong):
    """Each of the calls' tensors in turn; 16-bit integers pass as bits, as everywhere in the binding.  Calls of the right
    types get as far as the library's own refusals (a scale of 0, a rotation of 8 dimensions, head sizes that differ)."""
    cache, batch = tensors()
    c, b = cache(), batch()
    rows = lambda heads, t: torch.zeros((5, heads, 64), dtype=t)                                  # noqa: E731
    table = torch.zeros(9, 4)
    refused = 96
    wide = qlin.Kv8Cache(torch.zeros((4, 2, 16, refused), dtype=torch.int8), torch.zeros((4, 2, refused, 16), dtype=torch.int8),
                         torch.zeros((4, 2, 2)))

    def attention(q=right, y=right):
        qlin.qlin_kv8_attention(c, b, rows(4, q), dtype, 4, 0.0, 0, 0, rows(4, y), stream=0)

    def append(q=right, k=right, v=right, out=right, cos=torch.float32, sin=torch.float32):
        qlin.qlin_kv8_append(c, b, rows(4, q), rows(2, k), rows(2, v), dtype, 4, table.to(cos), table.to(sin), 8, 0,
                             rows(4, out), stream=0)

    def gather(k=right, v=right):
        qlin.qlin_kv8_gather(wide, b, *(torch.zeros((5, 2, refused), dtype=t) for t in (k, v)), dtype, stream=0)

    for call, names in ((attention, "q y"), (append, "q k v out"), (gather, "k v")):
        with pytest.raises(qlin.QlinError):
            call()
        for name in names.split():
            with pytest.raises(qlin.QlinError):
                call(**{name: torch.int16})
            with pytest.raises(ValueError, match=str(wrong)):
                call(**{name: wrong})
    for name in ("cos", "sin"):
        with pytest.raises(ValueError, match="torch.int32"):
            append(**{name: torch.int32})
