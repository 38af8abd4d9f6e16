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


# The library takes C ints, and ctypes drops what is above 32 bits: a size of 2^32 + 8 would run as one of 8 and leave
# the rest of the output as it was. (Meta tensors: sizes without memory.)
BIG = 2 ** 32


def _meta_routing(tokens, topk, groups):
    import torch
    import weight_only_int4_w4a16_amd as w4
    n = w4.lib().w4a16_route_bytes(tokens, topk, groups) // 4
    return w4.Routing(torch.empty(n, dtype=torch.int32, device="meta"), tokens, topk, groups)


def _too_large(fn):
    from weight_only_int4_w4a16_amd import W4A16Error
    with pytest.raises(W4A16Error, match="2\\^31") as e:
        fn()
    assert e.value.status == UNSUPPORTED


def test_binding_refuses_rows_past_a_c_int():
    import torch
    import weight_only_int4_w4a16_amd as w4
    r = _meta_routing(1, 2, 3)
    x = torch.empty(1, BIG + 8, dtype=torch.bfloat16, device="meta")
    ys = torch.empty(2, BIG + 8, dtype=torch.bfloat16, device="meta")
    w = torch.empty(1, 2, device="meta")
    _too_large(lambda: w4.dispatch(x, r))
    _too_large(lambda: w4.dispatch_backward(ys, r))
    _too_large(lambda: w4.combine(ys, r, w))
    _too_large(lambda: w4.combine_backward(x, ys, r, w))


def test_binding_refuses_ids_past_a_c_int():
    import torch
    import weight_only_int4_w4a16_amd as w4
    ids = torch.empty(BIG + 4, 2, dtype=torch.int32, device="meta")
    for i, groups in ((ids, 8), (ids.t().contiguous(), 8), (ids[:4], BIG + 8)):
        _too_large(lambda: w4.route(i, groups))


def test_binding_refuses_weights_past_a_c_int():
    import torch
    import weight_only_int4_w4a16_amd as w4
    r = _meta_routing(4, 1, 2)
    m = lambda *s, d=torch.float16: torch.empty(s, dtype=d, device="meta")  # noqa: E731
    _too_large(lambda: w4.pack_grouped(m(2, 4, BIG + 16, d=torch.int32)))
    _too_large(lambda: w4.pack_grouped(m(2, BIG // 8 + 4, 16, d=torch.int32)))
    _too_large(lambda: w4.gemm_grouped(m(4, 32), r, m(2, 64, d=torch.int32), m(2, 1, BIG + 16), None, 32))
    _too_large(lambda: w4.gemm_grouped(m(4, BIG + 32), r, m(2, 64, d=torch.int32), m(2, BIG // 32 + 1, 16), None, 32))


def test_binding_refuses_adapters_past_a_c_int(monkeypatch):
    import torch
    import weight_only_int4_w4a16_amd as w4
    from weight_only_int4_w4a16_amd import binding
    monkeypatch.setattr(binding, "_need_device", lambda *a: None)  # meta tensors stand for device tensors
    m = lambda *s, d=torch.float16: torch.empty(s, dtype=d, device="meta")  # noqa: E731
    ids = lambda n: m(n, d=torch.int32)  # noqa: E731
    s = lambda n: m(n, d=torch.float32)  # noqa: E731
    _too_large(lambda: w4.lora_add(m(4, BIG + 16), m(4, 32), m(2, 8, 32), m(2, BIG + 16, 8), ids(4), s(2)))
    _too_large(lambda: w4.lora_add(m(4, 16), m(4, BIG + 32), m(2, 8, BIG + 32), m(2, 16, 8), ids(4), s(2)))
    _too_large(lambda: w4.lora_add(m(BIG + 4, 16), m(BIG + 4, 32), m(2, 8, 32), m(2, 16, 8), ids(BIG + 4), s(2)))
    _too_large(lambda: w4.lora_add(m(4, 16), m(4, 32), m(BIG + 2, 8, 32), m(BIG + 2, 16, 8), ids(4), s(BIG + 2)))
    _too_large(lambda: w4.lora_add(m(4, 16), m(4, 32), m(2, BIG + 8, 32), m(2, 16, BIG + 8), ids(4), s(2)))
    assert w4.lora_workspace_bytes(BIG + 300, 4096, 4096, 8, 16) == 0
    assert w4.grouped_kernel_name(BIG + 16, 4096, 4096, 8, 128) == "none"
