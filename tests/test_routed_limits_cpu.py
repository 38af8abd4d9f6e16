"""Sizes that the routed operators' 32-bit indices cannot hold are refused on the host (placeholder addresses,
nothing is launched or read)."""
import pytest

UNSUPPORTED = 2
P = 1 << 20  # aligned placeholder addresses
Q = P + 4096
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    from weight_only_int4_w4a16_amd import binding
    assert binding.ERR_UNSUPPORTED == UNSUPPORTED
    return binding.lib()


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("width", [INT_MAX, INT_MAX - 200, INT_MAX - 600, INT_MAX - 1022])
def test_rows_too_wide_to_index(L, width, dtype):
    """The last items' lanes index up to 1023 elements past the row before they are held back to it."""
    head = (Q, 1, 1, 8)
    assert L.w4a16_dispatch(P, *head, width, dtype, 2 * P, None) == UNSUPPORTED
    assert L.w4a16_dispatch_backward(P, *head, width, dtype, 2 * P, None) == UNSUPPORTED
    assert L.w4a16_combine(P, *head, P, width, dtype, 2 * P, dtype, None) == UNSUPPORTED
    assert L.w4a16_combine_backward(P, 3 * P, *head, P, width, dtype, 2 * P, P, None) == UNSUPPORTED


@pytest.mark.parametrize("K,N", [(32, 2 ** 31 - 16), (32, 2 ** 31 - 2032), (2 ** 31 - 32, 16), (2 ** 31 - 96, 16)])
@pytest.mark.parametrize("M", [1, 300])
def test_adapters_too_wide_to_index(L, M, K, N):
    assert L.w4a16_lora_add(P, P, M, K, N, 0, 0, P, P, 1, 8, P, P, None, P, Q, 2 ** 62, None) == UNSUPPORTED
    assert L.w4a16_lora_workspace_bytes(M, K, N, 1, 8, 0) == 0
