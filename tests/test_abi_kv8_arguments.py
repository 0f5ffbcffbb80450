"""CPU-only checks of the 8-bit cache's arguments: limits of numbers, and the types that the binding takes."""
import pytest

from quantized_linear_layers_packed_amd import qlin
from tests.test_abi_kv8 import EINVAL, attention, batch


@pytest.mark.parametrize("scale,fits", [(2.3e38, True), (2.4e38, False), (3.4e38, False)])
def test_a_scale_is_finite_in_the_exponent_of_two_as_well(scale, fits):
    """scale * log2(e) is what the kernels hold; one that fits gets as far as the missing workspace."""
    long = batch(max_kv=100000, table_stride=2000, max_new=1)
    assert attention(b=long, scale=scale) == EINVAL
    assert ("workspace" if fits else "scale") in qlin.last_error()
