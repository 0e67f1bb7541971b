"""Host-side tests of strides that no memory has (no GPU needed)."""
import pytest

from routed_moe_decode_router_gb300 import build as B
from routed_moe_decode_router_gb300 import native as N

P = 1 << 28      # a well-aligned address that no refused call may touch


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return N.lib()


@pytest.mark.parametrize("stride", [1 << 39, 1 << 62, (1 << 62) + 4096, (1 << 63) - 16])
@pytest.mark.parametrize("name", ["k_stride", "v_stride"])
def test_strides_of_a_cache_whose_bytes_pass_64_bits(stride, name):
    """A stride times the elements' size is not what is checked if it wraps around."""
    d = dict(k=P, v=2 * P, k_scales=0, v_scales=0, k_stride=4096, v_stride=4096, k_scales_stride=0,
             v_scales_stride=0, pages=8, heads=2, page=32, dim=64, type=N.MOEOP_BF16)
    d[name] = stride
    with pytest.raises(N.MoeError, match="strides"):
        N.moeop_kv_write(N.KvCache(**d), 0, 128, 6 * P, 128, 0, 7 * P, 4)
