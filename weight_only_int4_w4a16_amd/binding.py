"""ctypes binding over ``libw4a16.so`` (the C ABI in ``include/w4a16.h``).

Argument marshalling only: tensors are passed as device pointers with the caller's
current HIP stream; every step of the computation runs in the library's HIP kernels.
The library is loaded on first use and a missing or unloadable library raises
:class:`W4A16Error`; there is no other code path.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libw4a16.so")

F16, BF16, F32 = 0, 1, 2
OK, ERR_ARG, ERR_UNSUPPORTED, ERR_HIP, ERR_WORKSPACE = 0, 1, 2, 3, 4

_lib = None
_workspaces = {}   # device index -> uint8 scratch tensor


class W4A16Error(RuntimeError):
    def __init__(self, msg, status=None):
        super().__init__(msg)
        self.status = status


def lib() -> ctypes.CDLL:
    """Load ``libw4a16.so`` once; raise if it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise W4A16Error(f"{LIB_PATH} is missing: build it with "
                         "`python -m weight_only_int4_w4a16_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.w4a16_packed_bytes.argtypes = [i32, i32]
    L.w4a16_packed_bytes.restype = sz
    L.w4a16_pack.argtypes = [vp, i32, i32, vp, vp]
    L.w4a16_pack.restype = i32
    L.w4a16_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.w4a16_workspace_bytes.restype = sz
    L.w4a16_gemm.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, i32, vp, sz, vp]
    L.w4a16_gemm.restype = i32
    L.w4a16_gemm_static.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, i32, vp]
    L.w4a16_gemm_static.restype = i32
    L.w4a16_gemm_nf4.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, i32, vp, sz, vp]
    L.w4a16_gemm_nf4.restype = i32
    L.w4a16_awq_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.w4a16_awq_workspace_bytes.restype = sz
    L.w4a16_gemm_awq.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, i32, vp, sz, vp]
    L.w4a16_gemm_awq.restype = i32
    L.w4a16_w4a8_workspace_bytes.argtypes = [i32, i32, i32]
    L.w4a16_w4a8_workspace_bytes.restype = sz
    L.w4a16_gemm_w4a8.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, sz, vp]
    L.w4a16_gemm_w4a8.restype = i32
    L.w4a16_w4a8_kernel_name.argtypes = [i32, i32, i32]
    L.w4a16_w4a8_kernel_name.restype = ctypes.c_char_p
    L.w4a16_quantize_act_int8.argtypes = [vp, i32, i32, i32, vp, vp, vp]
    L.w4a16_quantize_act_int8.restype = i32
    L.w4a16_gemm_swiglu.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, i32, vp, sz, vp]
    L.w4a16_gemm_swiglu.restype = i32
    L.w4a16_gemm_nf4_swiglu.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, i32, vp, sz, vp]
    L.w4a16_gemm_nf4_swiglu.restype = i32
    L.w4a16_dequant.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp]
    L.w4a16_dequant.restype = i32
    L.w4a16_dequant_nf4.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp]
    L.w4a16_dequant_nf4.restype = i32
    L.w4a16_kernel_name.argtypes = [i32, i32, i32, i32]
    L.w4a16_kernel_name.restype = ctypes.c_char_p
    L.w4a16_status_string.argtypes = [i32]
    L.w4a16_status_string.restype = ctypes.c_char_p
    L.w4a16_route_bytes.argtypes = [i32, i32, i32]
    L.w4a16_route_bytes.restype = sz
    L.w4a16_route.argtypes = [vp, i32, i32, i32, vp, sz, vp]
    L.w4a16_route.restype = i32
    L.w4a16_dispatch.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp]
    L.w4a16_dispatch.restype = i32
    L.w4a16_dispatch_backward.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp]
    L.w4a16_dispatch_backward.restype = i32
    L.w4a16_combine.argtypes = [vp, vp, i32, i32, i32, vp, i32, i32, vp, i32, vp]
    L.w4a16_combine.restype = i32
    L.w4a16_combine_backward.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, i32, vp, vp, vp]
    L.w4a16_combine_backward.restype = i32
    L.w4a16_gemm_grouped.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp, vp, i32, i32, vp, i32, vp]
    L.w4a16_gemm_grouped.restype = i32
    L.w4a16_gemm_grouped_nf4.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp, vp, i32, i32, vp, i32, vp]
    L.w4a16_gemm_grouped_nf4.restype = i32
    L.w4a16_grouped_kernel_name.argtypes = [i32, i32, i32, i32, i32]
    L.w4a16_grouped_kernel_name.restype = ctypes.c_char_p
    L.w4a16_lora_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    L.w4a16_lora_workspace_bytes.restype = sz
    L.w4a16_lora_add.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.w4a16_lora_add.restype = i32
    L.w4a16_read_probe.argtypes = [vp, sz, vp, vp]
    L.w4a16_read_probe.restype = i32
    L.w4a16_version.argtypes = []
    L.w4a16_version.restype = ctypes.c_char_p
    _lib = L
    return L


def _check(status: int, what: str) -> None:
    if status != OK:
        msg = lib().w4a16_status_string(status).decode()
        raise W4A16Error(f"{what}: {msg} (status {status})", status)


def _torch():
    import torch
    return torch


def _dt(t) -> int:
    torch = _torch()
    m = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
    if t not in m:
        raise W4A16Error(f"unsupported dtype {t}", ERR_ARG)
    return m[t]


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise W4A16Error("tensors must be contiguous device tensors", ERR_ARG)
    return ctypes.c_void_p(t.data_ptr())


def _fail(msg):
    raise W4A16Error(msg, ERR_ARG)


def _expect(t, name, shape, dtypes, device=None):
    """Check one tensor argument on the host, before any pointer reaches the library: the
    C ABI receives no buffer sizes, so a tensor of the wrong shape would make a kernel read
    or write past its end."""
    if t is None:
        _fail(f"{name} is required")
    if t.dtype not in dtypes:
        _fail(f"{name}: dtype {t.dtype}, expected one of {[str(d) for d in dtypes]}")
    if tuple(t.shape) != tuple(shape):
        _fail(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        _fail(f"{name} must be contiguous")
    if device is not None and t.device != device:
        _fail(f"{name} is on {t.device}, expected {device}")


def _expect_packed(packed, K, N, device):
    """The device-layout weight: int32, at least ``packed_bytes(K, N)`` bytes."""
    torch = _torch()
    if packed is None or packed.dtype != torch.int32 or not packed.is_contiguous():
        _fail("packed must be a contiguous int32 tensor (the output of pack)")
    need = packed_bytes(K, N)
    if need == 0:
        raise W4A16Error(f"unsupported shape K={K} N={N}", ERR_UNSUPPORTED)
    if packed.numel() * 4 < need:
        _fail(f"packed holds {packed.numel() * 4} bytes, K={K} N={N} needs {need}")
    if packed.device != device:
        _fail(f"packed is on {packed.device}, expected {device}")


def _expect_x(x, name="x"):
    torch = _torch()
    if x is None or x.dim() != 2:
        _fail(f"{name} must be a 2-D [M, K] tensor")
    if x.dtype not in (torch.float16, torch.bfloat16):
        _fail(f"{name}: dtype {x.dtype}, expected float16 or bfloat16")
    if not x.is_contiguous():
        _fail(f"{name} must be contiguous")
    return x.shape[0], x.shape[1]


def _groups(K, g, what="group_size"):
    if g <= 0 or K % g:
        _fail(f"K={K} is not a multiple of {what}={g}")
    return K // g


def _out(out, M, N, out_dtype, x):
    """The caller's ``out`` checked against (M, N) and the requested dtype, or a new one."""
    torch = _torch()
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    if out_dtype not in (x.dtype, torch.float32):
        _fail(f"out dtype {out_dtype}: must be the activation dtype or float32")
    if out is None:
        return torch.empty((M, N), dtype=out_dtype, device=x.device)
    _expect(out, "out", (M, N), (out_dtype,), x.device)
    return out


def _expect_workspace(ws, need, device):
    if ws is None:
        return
    torch = _torch()
    if ws.device != device or not ws.is_contiguous():
        _fail("workspace must be a contiguous tensor on the activations' device")
    if ws.numel() * ws.element_size() < need:
        _fail(f"workspace holds {ws.numel() * ws.element_size()} bytes, {need} needed")


def _stream(t):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _raw_stream(device):
    """The current stream's handle on ``device``, without the 2 us a stream object takes to make
    (a small routed call takes 4 us in all)."""
    torch = _torch()
    try:
        return torch._C._cuda_getCurrentRawStream(device.index)
    except AttributeError:
        return torch.cuda.current_stream(device).cuda_stream


def packed_bytes(K: int, N: int) -> int:
    return int(lib().w4a16_packed_bytes(K, N))


def workspace_bytes(M: int, K: int, N: int, group_size: int) -> int:
    return int(lib().w4a16_workspace_bytes(M, K, N, group_size))


def awq_workspace_bytes(M: int, K: int, N: int, group_size: int) -> int:
    return int(lib().w4a16_awq_workspace_bytes(M, K, N, group_size))


def _workspace(device, nbytes: int, workspace=None):
    """The caller's workspace, or a cached scratch buffer for the device.

    The library keeps nothing in a workspace between calls, so one buffer serves all calls
    that do not run concurrently; callers that launch GEMMs on several streams at
    once pass their own ``workspace`` per stream. It is never allocated while a HIP graph
    is being captured (warm up eagerly first).
    """
    torch = _torch()
    if workspace is not None:
        return workspace
    if nbytes == 0:
        return None
    key = device.index if device.index is not None else torch.cuda.current_device()
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        if torch.cuda.is_current_stream_capturing():
            raise W4A16Error("workspace must be allocated before graph capture: run the same "
                             "calls once eagerly on this stream first", ERR_WORKSPACE)
        ws = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def pack(qweight):
    """Canonical ``qweight[K/8, N]`` int32 -> the library's device layout (int32 tensor)."""
    torch = _torch()
    if qweight.dtype != torch.int32 or qweight.dim() != 2:
        raise W4A16Error("qweight must be a 2-D int32 tensor [K/8, N]", ERR_ARG)
    if not qweight.is_contiguous():
        _fail("qweight must be contiguous")
    K, N = qweight.shape[0] * 8, qweight.shape[1]
    nb = packed_bytes(K, N)
    if nb == 0:
        raise W4A16Error(f"unsupported shape K={K} N={N}", ERR_UNSUPPORTED)
    out = torch.empty(nb // 4, dtype=torch.int32, device=qweight.device)
    _check(lib().w4a16_pack(_ptr(qweight), K, N, _ptr(out), _stream(qweight)), "w4a16_pack")
    return out


def _affine_operands(x, packed, scales, qzeros, group_size, n_cols):
    """Shapes of an affine/symmetric GEMM's operands: x [M, K], scales [K/g, N] in x's
    dtype, qzeros [K/g, N/8] int32 or None, packed for (K, N). Returns (M, K, N)."""
    torch = _torch()
    M, K = _expect_x(x)
    if scales is None or scales.dim() != 2:
        _fail("scales must be a 2-D [K/g, N] tensor")
    N = scales.shape[1] if n_cols is None else n_cols
    G = _groups(K, group_size)
    _expect(scales, "scales", (G, N), (x.dtype,), x.device)
    if N % 8:
        _fail(f"N={N} is not a multiple of 8")
    if qzeros is not None:
        _expect(qzeros, "qzeros", (G, N // 8), (torch.int32,), x.device)
    _expect_packed(packed, K, N, x.device)
    return M, K, N


def _nf4_operands(x, packed, absmax, codebook, block_size):
    """NF4 operands: absmax [K/b, N] fp16, codebook (16,) fp16, packed for (K, N)."""
    torch = _torch()
    M, K = _expect_x(x)
    if absmax is None or absmax.dim() != 2:
        _fail("absmax must be a 2-D [K/block_size, N] tensor")
    N = absmax.shape[1]
    _expect(absmax, "absmax", (_groups(K, block_size, "block_size"), N), (torch.float16,), x.device)
    _expect(codebook, "codebook", (16,), (torch.float16,), x.device)
    _expect_packed(packed, K, N, x.device)
    return M, K, N


def _ws_args(ws):
    return _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size()


def gemm(x, packed, scales, qzeros, group_size: int, out_dtype=None, out=None, workspace=None):
    """``y = x @ W_hat`` with affine (``qzeros`` given) or symmetric (``qzeros=None``) INT4.

    ``x[M, K]`` fp16/bf16, ``scales[K/g, N]`` in x's dtype, ``qzeros[K/g, N/8]`` int32.
    ``workspace``: optional uint8 device tensor of ``workspace_bytes(M, K, N, group_size)``.
    Every tensor's shape, dtype and device is checked before anything is launched.
    """
    M, K, N = _affine_operands(x, packed, scales, qzeros, group_size, None)
    out = _out(out, M, N, out_dtype, x)
    need = workspace_bytes(M, K, N, group_size) if M else 0
    _expect_workspace(workspace, need, x.device)
    ws = _workspace(x.device, need, workspace)
    st = lib().w4a16_gemm(_ptr(x), M, K, N, _dt(x.dtype), _ptr(packed), _ptr(scales),
                          _ptr(qzeros), group_size, _ptr(out), _dt(out.dtype), *_ws_args(ws),
                          _stream(x))
    _check(st, "w4a16_gemm")
    return out


def gemm_static(x, packed, scales, qzeros, group_size: int, out_dtype=None, out=None):
    """:func:`gemm` through ``w4a16_gemm_static``: the library's split-K scratch comes from its
    own static device array, so the call allocates nothing (``out`` is allocated here only
    when not given). Calls that overlap on one GPU race on that array."""
    M, K, N = _affine_operands(x, packed, scales, qzeros, group_size, None)
    out = _out(out, M, N, out_dtype, x)
    st = lib().w4a16_gemm_static(_ptr(x), M, K, N, _dt(x.dtype), _ptr(packed), _ptr(scales),
                                 _ptr(qzeros), group_size, _ptr(out), _dt(out.dtype), _stream(x))
    _check(st, "w4a16_gemm_static")
    return out


def gemm_nf4(x, packed, absmax, codebook, block_size: int = 64, out_dtype=None, out=None,
             workspace=None):
    """``y = x @ W_hat`` with NF4 weights: fp16 ``absmax[K/b, N]``, fp16 ``codebook[16]``."""
    M, K, N = _nf4_operands(x, packed, absmax, codebook, block_size)
    out = _out(out, M, N, out_dtype, x)
    need = workspace_bytes(M, K, N, block_size) if M else 0
    _expect_workspace(workspace, need, x.device)
    ws = _workspace(x.device, need, workspace)
    st = lib().w4a16_gemm_nf4(_ptr(x), M, K, N, _dt(x.dtype), _ptr(packed), _ptr(absmax),
                              _ptr(codebook), block_size, _ptr(out), _dt(out.dtype),
                              *_ws_args(ws), _stream(x))
    _check(st, "w4a16_gemm_nf4")
    return out


def gemm_awq(x, s_inv, packed, scales, qzeros, group_size: int, out_dtype=None, out=None,
             workspace=None):
    """``y = RN(x * s_inv) @ W_hat``: the GEMM of AWQ-scaled activations, ``s_inv[K]`` the
    per-input-channel S^-1 in x's dtype, the weight the INT4 format of S W (as for
    :func:`gemm`). ``workspace``: optional, ``awq_workspace_bytes(M, K, N, group_size)``."""
    M, K, N = _affine_operands(x, packed, scales, qzeros, group_size, None)
    _expect(s_inv, "s_inv", (K,), (x.dtype,), x.device)
    out = _out(out, M, N, out_dtype, x)
    need = awq_workspace_bytes(M, K, N, group_size) if M else 0
    _expect_workspace(workspace, need, x.device)
    ws = _workspace(x.device, need, workspace)
    st = lib().w4a16_gemm_awq(_ptr(x), _ptr(s_inv), M, K, N, _dt(x.dtype), _ptr(packed),
                              _ptr(scales), _ptr(qzeros), group_size, _ptr(out), _dt(out.dtype),
                              *_ws_args(ws), _stream(x))
    _check(st, "w4a16_gemm_awq")
    return out


def w4a8_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().w4a16_w4a8_workspace_bytes(M, K, N))


def gemm_w4a8(x, packed, wscale, out_dtype=None, out=None, workspace=None):
    """W4A8: ``y = sx * sw * (xq @ q)`` with x quantized per token to INT8 inside the call,
    symmetric INT4 codes (packed as for :func:`gemm` with ``qzeros=None``) and one scale per
    output channel ``wscale[N]`` in x's dtype."""
    M, K = _expect_x(x)
    if wscale is None or wscale.dim() != 1:
        _fail("wscale must be a 1-D (N,) tensor")
    N = wscale.shape[0]
    _expect(wscale, "wscale", (N,), (x.dtype,), x.device)
    _expect_packed(packed, K, N, x.device)
    out = _out(out, M, N, out_dtype, x)
    need = w4a8_workspace_bytes(M, K, N) if M else 0
    _expect_workspace(workspace, need, x.device)
    ws = _workspace(x.device, need, workspace)
    st = lib().w4a16_gemm_w4a8(_ptr(x), M, K, N, _dt(x.dtype), _ptr(packed), _ptr(wscale),
                               _ptr(out), _dt(out.dtype), *_ws_args(ws), _stream(x))
    _check(st, "w4a16_gemm_w4a8")
    return out


def w4a8_kernel_name(M: int, K: int, N: int) -> str:
    return lib().w4a16_w4a8_kernel_name(M, K, N).decode()


def quantize_act_int8(x):
    """The per-token INT8 quantization of the W4A8 path: ``(xq[M, K] int8, sx[M] float32)``."""
    torch = _torch()
    M, K = _expect_x(x)
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    sx = torch.empty((M,), dtype=torch.float32, device=x.device)
    st = lib().w4a16_quantize_act_int8(_ptr(x), M, K, _dt(x.dtype), _ptr(xq), _ptr(sx), _stream(x))
    _check(st, "w4a16_quantize_act_int8")
    return xq, sx


def _glu_out(out, M, N2, out_dtype, x):
    if N2 % 2:
        _fail(f"N2={N2} must be even (gate and up halves)")
    return _out(out, M, N2 // 2, out_dtype, x)


def gemm_swiglu(x, packed, scales, qzeros, group_size: int, out_dtype=None, out=None,
                workspace=None):
    """``h = SiLU(x @ W_gate) * (x @ W_up)`` for a fused gate+up weight ``[K, N2]`` (gate
    columns first; ``scales[K/g, N2]``, ``qzeros[K/g, N2/8]`` or None); ``h[M, N2/2]``."""
    M, K, N2 = _affine_operands(x, packed, scales, qzeros, group_size, None)
    out = _glu_out(out, M, N2, out_dtype, x)
    need = workspace_bytes(M, K, N2, group_size) if M else 0
    _expect_workspace(workspace, need, x.device)
    ws = _workspace(x.device, need, workspace)
    st = lib().w4a16_gemm_swiglu(_ptr(x), M, K, N2, _dt(x.dtype), _ptr(packed), _ptr(scales),
                                 _ptr(qzeros), group_size, _ptr(out), _dt(out.dtype),
                                 *_ws_args(ws), _stream(x))
    _check(st, "w4a16_gemm_swiglu")
    return out


def gemm_nf4_swiglu(x, packed, absmax, codebook, block_size: int = 64, out_dtype=None, out=None,
                    workspace=None):
    """NF4 counterpart of :func:`gemm_swiglu`."""
    M, K, N2 = _nf4_operands(x, packed, absmax, codebook, block_size)
    out = _glu_out(out, M, N2, out_dtype, x)
    need = workspace_bytes(M, K, N2, block_size) if M else 0
    _expect_workspace(workspace, need, x.device)
    ws = _workspace(x.device, need, workspace)
    st = lib().w4a16_gemm_nf4_swiglu(_ptr(x), M, K, N2, _dt(x.dtype), _ptr(packed), _ptr(absmax),
                                     _ptr(codebook), block_size, _ptr(out), _dt(out.dtype),
                                     *_ws_args(ws), _stream(x))
    _check(st, "w4a16_gemm_nf4_swiglu")
    return out


def dequant(packed, scales, qzeros, K: int, group_size: int):
    """Test hook: W_hat[K, N] in the scales' dtype, from the GEMM's own dequant routine."""
    torch = _torch()
    if scales is None or scales.dim() != 2:
        _fail("scales must be a 2-D [K/g, N] tensor")
    N = scales.shape[1]
    G = _groups(K, group_size)
    _expect(scales, "scales", (G, N), (torch.float16, torch.bfloat16))
    if qzeros is not None:
        _expect(qzeros, "qzeros", (G, N // 8), (torch.int32,), scales.device)
    _expect_packed(packed, K, N, scales.device)
    w = torch.empty((K, N), dtype=scales.dtype, device=scales.device)
    st = lib().w4a16_dequant(_ptr(packed), _ptr(scales), _ptr(qzeros), K, N, group_size,
                             _dt(scales.dtype), _ptr(w), _stream(scales))
    _check(st, "w4a16_dequant")
    return w


def dequant_nf4(packed, absmax, codebook, K: int, block_size: int = 64, wdtype=None):
    """Test hook: NF4 W_hat[K, N] (fp16 by default, or bf16)."""
    torch = _torch()
    if absmax is None or absmax.dim() != 2:
        _fail("absmax must be a 2-D [K/block_size, N] tensor")
    N = absmax.shape[1]
    _expect(absmax, "absmax", (_groups(K, block_size, "block_size"), N), (torch.float16,))
    _expect(codebook, "codebook", (16,), (torch.float16,), absmax.device)
    _expect_packed(packed, K, N, absmax.device)
    wdtype = torch.float16 if wdtype is None else wdtype
    if wdtype not in (torch.float16, torch.bfloat16):
        _fail(f"wdtype {wdtype}: float16 or bfloat16")
    w = torch.empty((K, N), dtype=wdtype, device=absmax.device)
    st = lib().w4a16_dequant_nf4(_ptr(packed), _ptr(absmax), _ptr(codebook), K, N, block_size,
                                 _dt(wdtype), _ptr(w), _stream(absmax))
    _check(st, "w4a16_dequant_nf4")
    return w


# ---- routed operators: rows of one batch that go to different weights ----
#
# Decode calls of these take a few microseconds on the GPU, as long as a launch takes on the
# host, so their checks compare what is expected first and look for what is wrong only after that fails.
#
# As everywhere in this binding, autograd is not told of a call: a result never requires a gradient, whatever its inputs do.
# dispatch_backward and combine_backward are calls for a training loop to make (or to put into a
# torch.autograd.Function); there is none that takes a gradient through 4-bit weights or through an adapter.

_dtypes = {}      # torch dtype -> w4a16_dtype
_act_dtypes = ()  # what activations may be


def _load_dtypes():
    global _act_dtypes
    torch = _torch()
    _act_dtypes = (torch.float16, torch.bfloat16)
    _dtypes.update({torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32})


def _need(t, name, shape, dtype, device):
    """A contiguous ``t`` of this shape and dtype on ``device``; returns its address."""
    if t is None or t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _expect(t, name, shape, (dtype,), device)
    return t.data_ptr()


_INT_MAX = 2 ** 31 - 1


def _need_ints(*sizes):
    """Sizes that the library's C ints hold: ctypes drops the bits above them without a word. (The calls of a decode
    step make this one only where the sizes' sum is past it: 0.4 us each.)"""
    if max(sizes) > _INT_MAX:
        raise W4A16Error(f"unsupported size {max(sizes)}: sizes must be below 2^31", ERR_UNSUPPORTED)


def _need_rows(t, name, rows):
    """A contiguous 2-D tensor of ``rows`` rows of fp16, bf16 or fp32; returns its width and w4a16 dtype."""
    if not _dtypes:
        _load_dtypes()
    if t is None or t.dim() != 2:
        _fail(f"{name} must be a 2-D tensor")
    n, width = t.shape
    dt = _dtypes.get(t.dtype)
    if dt is None or n != rows or not t.is_contiguous():
        _expect(t, name, (rows, width), tuple(_dtypes))
    if width < 1:
        _fail(f"{name} has rows of no elements")
    if width > _INT_MAX:
        _need_ints(width)
    return width, dt


def _need_device(device, what="tensors"):
    if device.type != "cuda":
        _fail(f"{what} must be contiguous device tensors")


def _apart(out, name, others):
    """``out`` shares no memory with the tensors a call reads."""
    lo, hi = out.data_ptr(), out.data_ptr() + out.numel() * out.element_size()
    for t in others:
        if t.data_ptr() < hi and lo < t.data_ptr() + t.numel() * t.element_size():
            _fail(f"{name} overlaps an input")


class Routing:
    """A batch's plan (:func:`route`): which sorted row each slot (token, choice) has.

    ``offsets`` int32 ``[groups + 1]``: group ``e``'s sorted rows are ``offsets[e]`` to ``offsets[e + 1]``;
    ``order`` int32 ``[rows]``: the slot of each sorted row, the slots of no group last; ``slot`` int32 ``[tokens,
    topk]``: the sorted row of each slot, -1 for a slot of no group (``rows = tokens * topk``). They
    are views of ``plan``, the buffer the kernels read, and are not to be written."""

    __slots__ = ("plan", "tokens", "topk", "groups", "rows", "device", "_views")

    def __init__(self, plan, tokens: int, topk: int, groups: int):
        self.plan, self.tokens, self.topk, self.groups = plan, tokens, topk, groups
        self.rows, self.device, self._views = tokens * topk, plan.device, None

    def _split(self):
        if self._views is None:
            e, n = self.groups + 1, self.rows
            e64, n64 = -e % 64, -n % 64
            at = e + e64 + n + n64 + n
            parts = self.plan.split_with_sizes((e, e64, n, n64, n, self.plan.numel() - at))
            self._views = parts[0], parts[2], parts[4].view(self.tokens, self.topk)
        return self._views

    @property
    def offsets(self):
        return self._split()[0]

    @property
    def order(self):
        return self._split()[1]

    @property
    def slot(self):
        return self._split()[2]


def _need_routing(routing):
    if not isinstance(routing, Routing):
        _fail("routing must be the result of route()")


def route(ids, groups: int) -> Routing:
    """Sort a batch's slots by group: ``ids`` int32 ``[tokens, topk]`` (or ``[tokens]``, one choice
    each), a value outside ``[0, groups)`` being no group. The plan serves any number of the calls
    below."""
    torch = _torch()
    if ids is None or ids.dtype is not torch.int32 or ids.dim() not in (1, 2):
        _fail("ids must be an int32 tensor [tokens, topk] or [tokens]")
    if not ids.is_contiguous():
        _fail("ids must be contiguous")
    tokens, topk = ids.shape if ids.dim() == 2 else (ids.shape[0], 1)
    if tokens + topk + groups > _INT_MAX:
        _need_ints(tokens, topk, groups)
    device = ids.device
    _need_device(device, "ids")
    if topk < 1 or groups < 1:
        _fail(f"topk={topk}, groups={groups}: both must be at least 1")
    L = lib()
    need = L.w4a16_route_bytes(tokens, topk, groups)
    if need == 0:
        raise W4A16Error(f"unsupported routing: {tokens} x {topk} slots, {groups} groups", ERR_UNSUPPORTED)
    plan = ids.new_empty(need // 4)
    st = L.w4a16_route(ids.data_ptr(), tokens, topk, groups, plan.data_ptr(), need, _raw_stream(device))
    if st:
        _check(st, "w4a16_route")
    return Routing(plan, tokens, topk, groups)


def dispatch(x, routing: Routing, out=None):
    """Tokens' rows into sorted order: ``xs[rows, width]``, ``xs[p] = x[order[p] // topk]``, zeros in the
    rows of no group. ``x[tokens, width]`` fp16, bf16 or fp32, any width. The result has no autograd history."""
    _need_routing(routing)
    r = routing
    width, dt = _need_rows(x, "x", r.tokens)
    if x.device != r.device:
        _fail(f"x is on {x.device}, expected {r.device}")
    if out is None:
        out = x.new_empty((r.rows, width))
    else:
        _need(out, "out", (r.rows, width), x.dtype, r.device)
        _apart(out, "out", (x,))
    st = lib().w4a16_dispatch(x.data_ptr(), r.plan.data_ptr(), r.tokens, r.topk, r.groups, width, dt, out.data_ptr(),
                              _raw_stream(r.device))
    if st:
        _check(st, "w4a16_dispatch")
    return out


def dispatch_backward(dxs, routing: Routing, out=None):
    """Gradient of :func:`dispatch`: ``dx[t] = sum_j dxs[slot[t, j]]``, summed in fp32. ``dxs`` comes from the
    experts' own backward pass, which for 4-bit weights is not in this library."""
    _need_routing(routing)
    r = routing
    width, dt = _need_rows(dxs, "dxs", r.rows)
    if dxs.device != r.device:
        _fail(f"dxs is on {dxs.device}, expected {r.device}")
    if out is None:
        out = dxs.new_empty((r.tokens, width))
    else:
        _need(out, "out", (r.tokens, width), dxs.dtype, r.device)
        _apart(out, "out", (dxs,))
    st = lib().w4a16_dispatch_backward(dxs.data_ptr(), r.plan.data_ptr(), r.tokens, r.topk, r.groups, width, dt,
                                       out.data_ptr(), _raw_stream(r.device))
    if st:
        _check(st, "w4a16_dispatch_backward")
    return out


def combine(ys, routing: Routing, weights, out_dtype=None, out=None):
    """Sorted rows back to their tokens: ``y[t] = sum_j weights[t, j] * ys[slot[t, j]]`` in fp32,
    rounded once to ``ys``'s dtype (fp32 ``ys``: to any ``out_dtype``). ``weights`` fp32
    ``[tokens, topk]``; the weight of a slot of no group is not used. The result has no autograd history."""
    _need_routing(routing)
    torch, r = _torch(), routing
    width, dt = _need_rows(ys, "ys", r.rows)
    if ys.device != r.device:
        _fail(f"ys is on {ys.device}, expected {r.device}")
    w = _need(weights, "weights", (r.tokens, r.topk), torch.float32, r.device)
    if out_dtype is None:
        out_dtype = ys.dtype if out is None else out.dtype
    if out_dtype is not ys.dtype and (dt != F32 or out_dtype not in _act_dtypes):
        _fail(f"out dtype {out_dtype} for {ys.dtype} rows")
    if out is None:
        out = ys.new_empty((r.tokens, width), dtype=out_dtype)
    else:
        _need(out, "out", (r.tokens, width), out_dtype, r.device)
        _apart(out, "out", (ys, weights))
    st = lib().w4a16_combine(ys.data_ptr(), r.plan.data_ptr(), r.tokens, r.topk, r.groups, w, width, dt,
                             out.data_ptr(), _dtypes[out_dtype], _raw_stream(r.device))
    if st:
        _check(st, "w4a16_combine")
    return out


def combine_backward(dy, ys, routing: Routing, weights):
    """Gradients of :func:`combine` for ``dy[tokens, width]`` in ``ys``'s dtype: ``(dys, dweights)``,
    ``dys[slot[t, j]] = weights[t, j] * dy[t]`` and the fp32 ``dweights[t, j] = <dy[t], ys[slot[t, j]]>``.
    ``dweights`` trains a gate over frozen 4-bit experts; ``dys`` is for experts whose backward pass the caller has."""
    _need_routing(routing)
    torch, r = _torch(), routing
    width, dt = _need_rows(ys, "ys", r.rows)
    if ys.device != r.device:
        _fail(f"ys is on {ys.device}, expected {r.device}")
    g = _need(dy, "dy", (r.tokens, width), ys.dtype, r.device)
    w = _need(weights, "weights", (r.tokens, r.topk), torch.float32, r.device)
    dys = torch.empty_like(ys)
    dweights = torch.empty_like(weights)
    st = lib().w4a16_combine_backward(g, ys.data_ptr(), r.plan.data_ptr(), r.tokens, r.topk, r.groups, w, width, dt,
                                      dys.data_ptr(), dweights.data_ptr(), _raw_stream(r.device))
    if st:
        _check(st, "w4a16_combine_backward")
    return dys, dweights


def pack_grouped(qweight):
    """Canonical ``qweight[groups, K/8, N]`` int32 -> the groups' device layouts, one after another."""
    torch = _torch()
    if qweight is None or qweight.dtype != torch.int32 or qweight.dim() != 3 or not qweight.is_contiguous():
        _fail("qweight must be a contiguous int32 tensor [groups, K/8, N]")
    K, N = qweight.shape[1] * 8, qweight.shape[2]
    _need_ints(K, N)
    nb = packed_bytes(K, N)
    if nb == 0:
        raise W4A16Error(f"unsupported shape K={K} N={N}", ERR_UNSUPPORTED)
    out = torch.empty((qweight.shape[0], nb // 4), dtype=torch.int32, device=qweight.device)
    for e in range(qweight.shape[0]):
        _check(lib().w4a16_pack(_ptr(qweight[e]), K, N, _ptr(out[e]), _stream(qweight)), "w4a16_pack")
    return out


def _grouped(x, routing, packed, scales, tail, group_size, glu, gather, out_dtype, out, nf4):
    _need_routing(routing)
    torch, r = _torch(), routing
    if not _dtypes:
        _load_dtypes()
    device = r.device
    rows, K = _expect_x(x)
    want = r.tokens if gather else r.rows
    if rows != want:
        _fail(f"x has {rows} rows, expected {want} ({'tokens' if gather else 'sorted rows'})")
    if x.device != device:
        _fail(f"x is on {x.device}, expected {device}")
    if scales is None or scales.dim() != 3:
        _fail("scales must be a 3-D [groups, K/g, N] tensor")
    E, N, G = r.groups, scales.shape[2], _groups(K, group_size)
    if K + N > _INT_MAX:
        _need_ints(K, N)
    sp = _need(scales, "scales", (E, G, N), torch.float16 if nf4 else x.dtype, device)
    if N % 8:
        _fail(f"N={N} is not a multiple of 8")
    if nf4:
        tp = _need(tail, "codebook", (16,), torch.float16, device)
    else:
        tp = None if tail is None else _need(tail, "qzeros", (E, G, N // 8), torch.int32, device)
    L = lib()
    need = L.w4a16_packed_bytes(K, N)
    if need == 0:
        raise W4A16Error(f"unsupported shape K={K} N={N}", ERR_UNSUPPORTED)
    pp = _need(packed, "packed", (E, need // 4), torch.int32, device)
    if glu and N % 2:
        _fail(f"N={N} must be even (gate and up halves)")
    width = N // 2 if glu else N
    if out is None and out_dtype is None:
        out = x.new_empty((r.rows, width))
    else:
        out = _out(out, r.rows, width, out_dtype, x)
        _apart(out, "out", (x,))
    f = L.w4a16_gemm_grouped_nf4 if nf4 else L.w4a16_gemm_grouped
    st = f(x.data_ptr(), r.plan.data_ptr(), r.tokens, r.topk, E, int(gather), K, N, _dtypes[x.dtype], pp, sp, tp,
           group_size, int(glu), out.data_ptr(), _dtypes[out.dtype], _raw_stream(device))
    if st:
        _check(st, "w4a16_gemm_grouped_nf4" if nf4 else "w4a16_gemm_grouped")
    return out


def gemm_grouped(x, routing: Routing, packed, scales, qzeros, group_size: int, gather: bool = False,
                 out_dtype=None, out=None):
    """The experts' products: ``out[rows, N]``, ``out[p] = row(p) @ W_hat[e]`` for group ``e``'s sorted rows,
    zeros in the rows of no group. ``x[rows, K]`` holds the sorted rows, or with ``gather`` the tokens'
    ``[tokens, K]``, read through the plan. ``packed`` from :func:`pack_grouped`, ``scales[groups, K/g, N]`` in
    x's dtype, ``qzeros[groups, K/g, N/8]`` int32 or None (symmetric)."""
    return _grouped(x, routing, packed, scales, qzeros, group_size, False, gather, out_dtype, out, False)


def gemm_grouped_swiglu(x, routing: Routing, packed, scales, qzeros, group_size: int, gather: bool = False,
                        out_dtype=None, out=None):
    """:func:`gemm_grouped` of fused gate+up weights (gate columns first) with the SwiGLU epilogue:
    ``h[rows, N/2]``."""
    return _grouped(x, routing, packed, scales, qzeros, group_size, True, gather, out_dtype, out, False)


def gemm_grouped_nf4(x, routing: Routing, packed, absmax, codebook, block_size: int = 64, gather: bool = False,
                     out_dtype=None, out=None):
    """NF4 counterpart of :func:`gemm_grouped`: fp16 ``absmax[groups, K/b, N]``, one fp16 ``codebook[16]``."""
    return _grouped(x, routing, packed, absmax, codebook, block_size, False, gather, out_dtype, out, True)


def gemm_grouped_nf4_swiglu(x, routing: Routing, packed, absmax, codebook, block_size: int = 64,
                            gather: bool = False, out_dtype=None, out=None):
    """NF4 counterpart of :func:`gemm_grouped_swiglu`."""
    return _grouped(x, routing, packed, absmax, codebook, block_size, True, gather, out_dtype, out, True)


def grouped_kernel_name(rows: int, K: int, N: int, groups: int, group_size: int) -> str:
    if max(rows, K, N, groups, group_size) > _INT_MAX:
        return "none"
    return lib().w4a16_grouped_kernel_name(rows, K, N, groups, group_size).decode()


def lora_workspace_bytes(M: int, K: int, N: int, adapters: int, rank: int, planned: bool = False) -> int:
    if max(M, K, N, adapters, rank) > _INT_MAX:
        return 0
    return int(lib().w4a16_lora_workspace_bytes(M, K, N, adapters, rank, int(planned)))


def lora_add(y, x, lora_a, lora_b, ids, scaling, routing: Routing | None = None, out=None, workspace=None):
    """Low-rank adapters of many requests beside a shared projection: ``out[m] = y[m] + scaling[a] *
    (x[m] @ lora_a[a].T) @ lora_b[a].T`` with ``a = ids[m]``, ``out[m] = y[m]`` where ``a`` is outside
    ``[0, adapters)``.

    ``y[M, N]`` the projection's output (x's dtype or fp32), ``x[M, K]`` fp16/bf16,
    ``lora_a[adapters, rank, K]``, ``lora_b[adapters, N, rank]`` in x's dtype, ``ids`` int32 ``[M]``,
    ``scaling`` fp32 ``[adapters]``. ``routing``: ``route(ids, adapters)``, made once for the projections of a step
    that share the ids. ``out`` may be ``y``. ``workspace``: optional, ``lora_workspace_bytes(...)``. The
    result has no autograd history."""
    torch = _torch()
    if not _dtypes:
        _load_dtypes()
    M, K = _expect_x(x)
    device, dtype = x.device, x.dtype
    _need_device(device)
    if lora_a is None or lora_a.dim() != 3:
        _fail("lora_a must be a 3-D [adapters, rank, K] tensor")
    adapters, rank, _ = lora_a.shape
    ap = _need(lora_a, "lora_a", (adapters, rank, K), dtype, device)
    if y is None or y.dim() != 2:
        _fail("y must be a 2-D [M, N] tensor")
    N = y.shape[1]
    if M + K + N + adapters + rank > _INT_MAX:
        _need_ints(M, K, N, adapters, rank)
    if y.dtype is not dtype:
        _expect(y, "y", (M, N), (dtype, torch.float32), device)
    yp = _need(y, "y", (M, N), y.dtype, device)
    bp = _need(lora_b, "lora_b", (adapters, N, rank), dtype, device)
    sp = _need(scaling, "scaling", (adapters,), torch.float32, device)
    if routing is None:
        ip, plan = _need(ids, "ids", (M,), torch.int32, device), None
    else:
        _need_routing(routing)
        if (routing.tokens, routing.topk, routing.groups) != (M, 1, adapters):
            _fail("routing must be route(ids, adapters) of these rows")
        if routing.device != device:
            _fail(f"the routing is on {routing.device}, expected {device}")
        ip, plan = None, routing.plan.data_ptr()
    if out is None:
        out = torch.empty_like(y)
    else:
        _need(out, "out", (M, N), y.dtype, device)
        _apart(out, "out", (x,) if out.data_ptr() == yp else (x, y))
    L = lib()
    need = L.w4a16_lora_workspace_bytes(M, K, N, adapters, rank, plan is not None)
    if workspace is None:
        wp = None
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
            wp = workspace.data_ptr()
    else:
        _expect_workspace(workspace, need, device)
        wp, need = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = L.w4a16_lora_add(x.data_ptr(), yp, M, K, N, _dtypes[dtype], _dtypes[y.dtype], ap, bp, adapters, rank, ip, sp,
                          plan, out.data_ptr(), wp, need, _raw_stream(device))
    if st:
        _check(st, "w4a16_lora_add")
    return out


def read_probe(buf, sink):
    """Measurement hook: stream every byte of the contiguous device tensor ``buf`` once (its
    size a multiple of 16 bytes), XOR-folding the words into ``sink`` (a contiguous 256-element
    int32/uint32 device tensor); for timing the device's practical HBM read rate."""
    if not buf.is_contiguous() or not sink.is_contiguous() or sink.numel() != 256 \
            or sink.element_size() != 4:
        _fail("buf must be contiguous and sink 256 contiguous 32-bit elements")
    nbytes = buf.numel() * buf.element_size()
    st = lib().w4a16_read_probe(_ptr(buf), nbytes, _ptr(sink), _stream(buf))
    _check(st, "w4a16_read_probe")


def kernel_name(M: int, K: int, N: int, group_size: int) -> str:
    return lib().w4a16_kernel_name(M, K, N, group_size).decode()


def version() -> str:
    return lib().w4a16_version().decode()
