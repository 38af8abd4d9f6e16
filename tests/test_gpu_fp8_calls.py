"""GPU checks of the 8-bit floating point calls at their rarer plans, values and arguments, against the fp64 oracle and with the
bounds of test_gpu_fp8.py (derived there)."""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import fp8 as F

from gpu_common import require_gpu, torch_mod
import test_gpu_fp8 as T

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# ------------------------------------------------------------------ pinned tiles

def check_pinned():
    """Products of few rows, where the kernel that quantizes x by itself ends, on whatever tile is pinned."""
    import weight_only_int4_w4a16_amd as w4
    for M, K, N in [(1, 272, 260), (2, 1040, 100), (3, 400, 64), (40, 272, 260)]:
        for halves in (1, 2):
            T._announce(f"pinned {os.environ.get('W4A16_FP8_ROWS')} {M}x{K}x{N} {halves}")
            x, xv = T._rows((M, K), "bf16", M + K)
            xv = F.rows_value(*F.quantize_rows(xv))
            codes, scales, wv = T._weight((), N, K, N, halves=halves)
            f = w4.gemm_fp8 if halves == 1 else w4.gemm_fp8_swiglu
            for kind in ("bf16", "f32"):
                if halves == 1:
                    ref, bound = F.gemm_fp8_ref(xv, wv), T._sum_bound(xv, wv, kind)
                else:
                    ref, bound = T._glu_bound(xv, wv, kind)
                y = f(x, codes, scales, out_dtype=T._dtype(kind))
                T._within(y.cpu().double().numpy(), ref, T._stored(ref, bound, kind), kind)


def _pinned(rows, check):
    """The pin is read once a process: a child runs its products."""
    here = os.path.dirname(os.path.abspath(__file__))
    env = {**os.environ, "W4A16_FP8_ROWS": str(rows), "PYTHONPATH": os.pathsep.join([ROOT, here])}
    run = subprocess.run([sys.executable, "-u", "-c", f"import test_gpu_fp8_calls as t; t.{check}()"], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=100)
    print(run.stdout, flush=True)
    assert run.returncode == 0, run.stderr[-3000:]


@pytest.mark.parametrize("rows", [16, 32, 64, 128, 256])
def test_pinned_tiles(rows):
    _pinned(rows, "check_pinned")


def _check_gradients(M, K, N, kind, n_some=None, k_some=None):
    """Both gradients, dw in some of its rows and columns."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    x, xv = T._rows((M, K), kind, M + K)
    dy, dyv = T._rows((M, N), kind, M + N)
    codes_t, scales_t, wt = T._weight((), K, N, K + N)
    dx, dw = w4.gemm_fp8_backward(dy, x, codes_t, scales_t)
    m = np.unique(np.concatenate([np.arange(0, M, 17), [M - 1]]))
    v = F.rows_value(*F.quantize_rows(dyv[m]))
    ref = F.gemm_fp8_ref(v, wt)
    T._within(dx[torch.from_numpy(m).cuda()].cpu().double().numpy(), ref, T._stored(ref, T._sum_bound(v, wt, kind), kind), "dx")
    n = np.arange(N) if n_some is None else n_some
    k = np.arange(K) if k_some is None else k_some
    ref, bound = T._dw_bound(dyv[:, n], xv[:, k])
    T._within(dw.cpu().double().numpy()[np.ix_(n, k)], ref, bound, "dw")


def _edges(size, step, tile):
    """Indices all over 0 .. size - 1, both sides of the tiles' edges among them."""
    at = np.arange(tile, size, tile)
    return np.unique(np.concatenate([np.arange(0, size, step), at - 1, at, [size - 1]]))


def check_pinned_families():
    """Each kind of product on one tile: plain in 16 and 32 bits, SwiGLU and its codes, routed, and the gradients; a weight's
    gradient on more tiles than the chip has compute units where the pinned tile loops."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    rows = int(os.environ["W4A16_FP8_ROWS"])
    M, K, N = 300, 400, 1000
    x, xv = T._rows((M, K), "f16", 1)
    xv = F.rows_value(*F.quantize_rows(xv))
    for halves, width in ((1, N), (2, 640)):
        T._announce(f"pinned {rows}: {M}x{K}x{width}")
        codes, scales, wv = T._weight((), width, K, 2, halves=halves)
        f = w4.gemm_fp8 if halves == 1 else w4.gemm_fp8_swiglu
        for kind in ("f16", "f32"):
            ref, bound = (F.gemm_fp8_ref(xv, wv), T._sum_bound(xv, wv, kind)) if halves == 1 else T._glu_bound(xv, wv, kind)
            y = f(x, codes, scales, out_dtype=T._dtype(kind))
            T._within(y.cpu().double().numpy(), ref, T._stored(ref, bound, kind), kind)
    q, s = w4.gemm_fp8_swiglu(x, codes, scales, quantized=True)
    T._check_quantized(q, s, ref, bound, "quantized h")

    tokens, topk, E, N2 = 300, 2, 5, 640
    T._announce(f"pinned {rows}: routed {tokens}x{topk} groups={E} {K}x{N2}")
    r, (offsets, order, _) = T._routed(T._ids(tokens, topk, E, 4), E)
    n = int(offsets[-1])
    sorted_rows = xv[order // topk]
    codes, scales, wv = T._weight((E,), N2, K, 3, halves=2)
    h, dh = T._each(lambda v, w: T._glu_bound(v, w, "f32"), offsets, sorted_rows, wv)
    q, s = w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True, quantized=True)
    T._check_quantized(q, s, h, dh, "quantized h of routed rows")
    assert not T._bits(q)[n:].any()
    codes, scales, wv = T._weight((E,), N2, K, 5)
    for kind in ("f16", "f32"):
        ref, bound = T._each(lambda v, w: (F.gemm_fp8_ref(v, w), T._sum_bound(v, w, kind)), offsets, sorted_rows, wv)
        y = w4.gemm_fp8_grouped(x, r, codes, scales, gather=True, out_dtype=T._dtype(kind))
        T._within(y.cpu().double().numpy(), ref, T._stored(ref, bound, kind), f"routed {kind}")

    if rows < 128:
        T._announce(f"pinned {rows}: gradients of 300x272x400")
        _check_gradients(300, 272, 400, "bf16")
    elif rows == 128:
        M, K, N = 700, 2064, 4112
        cus = torch.cuda.get_device_properties(0).multi_processor_count
        assert -(-N // 128) * -(-K // 256) > cus
        T._announce(f"pinned {rows}: gradients of {M}x{K}x{N}")
        _check_gradients(M, K, N, "bf16", _edges(N, 97, 128), _edges(K, 61, 256))


@pytest.mark.parametrize("rows", [32, 64, 128, 256])
def test_every_family_on_each_tile(rows):
    _pinned(rows, "check_pinned_families")


@pytest.mark.parametrize("M,K,N", [(700, 2064, 4112), (1030, 4112, 4208)])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_gradients_of_many_tiles(M, K, N, kind):
    """Weights' gradients of several times as many tiles of any height as the chip has compute units, whose sizes no tile divides."""
    T._announce(f"gemm_fp8_backward {M}x{K}x{N} {kind}")
    _check_gradients(M, K, N, kind, _edges(N, 97, 128), _edges(K, 61, 256))


@pytest.mark.parametrize("tokens,groups,K,N,how", [(1500, 12, 528, 1040, "skewed"), (2600, 40, 272, 1168, "mixed"), (3000, 40, 528, 1040, "skewed"), (900, 300, 16, 16, "mixed")])
def test_grouped_gradients_of_many_tiles(tokens, groups, K, N, how):
    """Weights' gradients by group on tiles of 128 x 256 that workgroups take in turn: more of them than compute units, of groups of
    no row, of a few and of several blocks of 128."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert -(-N // 128) * -(-K // 256) * groups > cus
    T._announce(f"grouped backward {tokens} groups={groups} {K}x{N} {how}")
    ids = T._ids(tokens, 1, groups, tokens, how)
    ids[ids == 1] = 0  # a group of no rows among the first
    ids[:300] = 2      # and one of more than two blocks
    ids[300:310] = -1
    ids[-50:] = groups - 1
    r, (offsets, _, _) = T._routed(ids, groups)
    n = int(offsets[-1])
    sizes = np.diff(offsets)
    assert n < tokens and sizes.min() == 0 and sizes.max() > 256 and np.any((0 < sizes) & (sizes < 128))
    x, xv = T._rows((tokens, K), "bf16", tokens + K)
    dy, dyv = T._rows((tokens, N), "bf16", tokens + N)
    x[n:], dy[n:] = float("nan"), float("inf")  # rows of no group reach nothing
    codes_t, scales_t, _ = T._weight((groups,), K, N, K + N)
    _, dw = w4.gemm_fp8_grouped_backward(dy, x, r, codes_t, scales_t)
    rows, cols = _edges(N, 97, 128), _edges(K, 61, 256)
    got = dw[:, torch.from_numpy(rows).cuda()][:, :, torch.from_numpy(cols).cuda()].cpu().double().numpy()
    for e in range(groups):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            assert not bool(dw[e].any()), f"group {e}"
        else:
            ref, bound = T._dw_bound(dyv[a:b][:, rows], xv[a:b][:, cols])
            T._within(got[e], ref, bound, f"dw of group {e}")


# ------------------------------------------------------------------ SwiGLU far below zero

@pytest.mark.parametrize("M,K,N2", [(2, 128, 256), (20, 128, 256), (64, 128, 256), (300, 256, 512), (2100, 256, 4096)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_swiglu_of_large_negative_gates(M, K, N2, kind):
    """Gates down to -88.6, where SiLU(g) is 1e-36 and less and exp(-g) nears fp32's largest, under up values of 2^100: h is an
    ordinary number and has to be right to the bounds of every other h. One code a row is not zero, so g and u are exact."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    T._announce(f"gemm_fp8_swiglu {M}x{K}x{N2} {kind}, gates from -88.6 to 8")
    N = N2 // 2
    x = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    x[:, 0] = 0x38  # 1
    size = torch.linspace(-8, 88.6, M, device="cuda")
    xs = torch.ones(K // 128, M, device="cuda")
    xs[0] = size.abs()
    x[size < 0, 0] = 0xB8  # -1
    codes = torch.zeros(N2, K, dtype=torch.uint8, device="cuda")
    codes[:N, 0], codes[N:, 0] = 0xB8, 0x38
    scales = torch.ones(2 * -(-N // 128), K // 128, device="cuda")
    scales[len(scales) // 2:] = 2.0 ** 100
    h = w4.gemm_fp8_swiglu(x.view(torch.float8_e4m3fn), codes.view(torch.float8_e4m3fn), scales, x_scales=xs, out_dtype=T._dtype(kind))
    v = size.cpu().double().numpy()
    g, u = -v, v * 2.0 ** 100
    want = g / (1 + np.exp(-g)) * u
    bound = (np.abs(g) + 8) * 2.0 ** -22 * np.abs(want)
    T._within(h.cpu().double().numpy(), want[:, None] + np.zeros(N), T._stored(want, bound, kind)[:, None], "h")


@pytest.mark.parametrize("tokens", [40, 600])
def test_grouped_swiglu_of_large_negative_gates(tokens):
    """The same of routed rows."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    K, N2, E = 128, 256, 2
    T._announce(f"gemm_fp8_grouped_swiglu {tokens} rows, gates from -88.6 to -1")
    r = w4.route(torch.zeros(tokens, 1, dtype=torch.int32, device="cuda"), E)
    x = torch.zeros(tokens, K, dtype=torch.uint8, device="cuda")
    x[:, 0] = 0x38
    size = torch.linspace(1, 88.6, tokens, device="cuda")
    codes = torch.zeros(E, N2, K, dtype=torch.uint8, device="cuda")
    codes[:, :N2 // 2, 0], codes[:, N2 // 2:, 0] = 0xB8, 0x38
    scales = torch.ones(E, 2, 1, device="cuda")
    scales[:, 1] = 2.0 ** 100
    h = w4.gemm_fp8_grouped_swiglu(x.view(torch.float8_e4m3fn), r, codes.view(torch.float8_e4m3fn), scales, x_scales=size[None],
                                   gather=True, out_dtype=torch.float32)
    v = size.cpu().double().numpy()
    want = -v / (1 + np.exp(v)) * v * 2.0 ** 100
    bound = (v + 8) * 2.0 ** -22 * np.abs(want)
    T._within(h.cpu().double().numpy(), want[:, None] + np.zeros(N2 // 2), T._stored(want, bound, "f32")[:, None], "h")


# ------------------------------------------------------------------ columns past the last row

@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 5), (130, 40), (249, 300)])
def test_codes_past_the_last_row_are_zeros(M, K, kind):
    """Also of a column that holds an infinity or a NaN, whose own codes are NaN."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    T._announce(f"columns {M}x{K} {kind}")
    x, _ = T._rows((M, K), kind, M)
    x[-1, 0], x[-1, 2], x[-1, 4] = float("inf"), float("nan"), float("-inf")
    codes, scales = w4.quantize_fp8_columns(x)
    want, wants = F.quantize_columns(x.cpu().float().numpy())
    T._same_codes(T._bits(codes), want, "codes")
    assert np.array_equal(scales.cpu().numpy(), wants, equal_nan=True)
    assert not T._bits(codes)[:, M:].any()


# ------------------------------------------------------------------ sizes next to the limits

def test_a_square_of_2_to_the_34_results():
    """131072 rows and columns: one kernel, whose grid is far from its limit."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    M = N = 1 << 17
    K = 16
    T._announce(f"gemm_fp8 {M}x{K}x{N}")
    big = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x, xv = T._rows((70, K), "bf16", 1)
    at = torch.cat([torch.arange(3), torch.arange(M - 67, M)]).cuda()
    big[at] = x
    codes, scales, wv = T._weight((), N, K, 2)
    y = w4.gemm_fp8(big, codes, scales)
    v = F.rows_value(*F.quantize_rows(xv))
    some = np.concatenate([np.arange(300), np.arange(N - 300, N)])
    ref = F.gemm_fp8_ref(v, wv[some])
    got = y[at][:, torch.from_numpy(some).cuda()].cpu().double().numpy()
    T._within(got, ref, T._stored(ref, T._sum_bound(v, wv[some], "bf16"), "bf16"), "corners")
    assert not bool(y[3:1000].any()) and not bool(y[M - 1000:M - 67].any())


def test_rows_next_to_their_limit():
    """2^27 - 8 rows, the most that one launch takes."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    M, K = (1 << 27) - 8, 16
    T._announce(f"rows {M}x{K}")
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    last, lv = T._rows((9, K), "bf16", 3)
    x[-9:] = last
    codes, scales = w4.quantize_fp8(x)
    want, wants = F.quantize_rows(lv)
    T._same_codes(T._bits(codes[-9:]), want, "codes")
    assert np.array_equal(scales[:, -9:].cpu().numpy(), wants)
    assert not bool(codes[:1000].view(torch.uint8).any()) and bool((scales[0, :1000] == 2.0 ** -126).all())
    with pytest.raises(w4.W4A16Error, match="unsupported"):
        w4.quantize_fp8(torch.empty(M + 1, K, dtype=torch.bfloat16, device="cuda"))


# ------------------------------------------------------------------ memory that a call reads and writes

def _refused(fn, match):
    import weight_only_int4_w4a16_amd as w4
    with pytest.raises(w4.W4A16Error, match=match) as e:
        fn()
    assert e.value.status == 1


def _inside(t, shape, dtype):
    """A tensor over t's first bytes."""
    torch = torch_mod()
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    return t.view(-1).view(torch.uint8)[:n].view(dtype).view(shape)


def test_out_and_workspace_overlap_nothing_that_is_read():
    """Results are stored while other workgroups still read: sharing memory with any input is refused, and so is a
    workspace that shares it with an input or the output."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    M, K, N = 24, 512, 256
    bf16, u8 = torch.bfloat16, torch.uint8
    x, _ = T._rows((M, K), "bf16", 1)
    q, s = w4.quantize_fp8(x)
    codes, scales, _ = T._weight((), N, K, 2)
    # scales next to a buffer of its own, so that an output can lie over them
    room = torch.zeros(M * N + 4096, device="cuda")
    own = room[:scales.numel()].view(scales.shape).copy_(scales)
    own_s = room[64:64 + s.numel()].view(s.shape).copy_(s)
    for out in (_inside(codes, (M, N), bf16), _inside(room, (M, N), bf16), _inside(x, (M, N), bf16)):
        _refused(lambda: w4.gemm_fp8(x, codes, own, out=out), "out overlaps an input")
    _refused(lambda: w4.gemm_fp8(q, codes, scales, x_scales=own_s, out=_inside(room, (M, N), bf16)), "out overlaps an input")
    _refused(lambda: w4.gemm_fp8(q, codes, scales, x_scales=s, out=_inside(q, (M, N), bf16)), "out overlaps an input")
    need = w4.fp8_workspace_bytes(M, K, N, bf16)
    out = torch.empty(M, N, dtype=bf16, device="cuda")
    big = torch.zeros(need + M * K * 2, dtype=u8, device="cuda")
    inside = big[:M * K * 2].view(bf16).view(M, K).copy_(x)
    over = big[:M * N * 2].view(bf16).view(M, N)
    _refused(lambda: w4.gemm_fp8(inside, codes, scales, workspace=big), "workspace overlaps")
    _refused(lambda: w4.gemm_fp8(x, codes, scales, out=over, workspace=big), "workspace overlaps")
    _refused(lambda: w4.gemm_fp8(x, codes, room[:scales.numel()].view(scales.shape), workspace=room.view(u8)), "workspace overlaps")
    assert torch.equal(w4.gemm_fp8(x, codes, scales, out=out, workspace=big), w4.gemm_fp8(x, codes, scales))

    E = 2
    r = w4.route(torch.arange(M, device="cuda", dtype=torch.int32).reshape(-1, 1) % E, E)
    ecodes, escales, _ = T._weight((E,), N, K, 3)
    eown = room[:escales.numel()].view(escales.shape).copy_(escales)
    for out in (_inside(ecodes, (M, N), bf16), _inside(room, (M, N), bf16)):
        _refused(lambda: w4.gemm_fp8_grouped(x, r, ecodes, eown, out=out), "out overlaps an input")
    _refused(lambda: w4.gemm_fp8_grouped(inside, r, ecodes, escales, workspace=big), "workspace overlaps")
    deep, _ = T._rows((4, 16), "bf16", 1)  # an output no larger than the plan
    small = w4.route(torch.zeros(4, 1, dtype=torch.int32, device="cuda"), 1)
    c1, s1, _ = T._weight((1,), 16, 16, 4)
    _refused(lambda: w4.gemm_fp8_grouped(deep, small, c1, s1, out=_inside(small.plan, (4, 16), bf16)), "out overlaps an input")

    codes_t, scales_t, _ = T._weight((), K, N, 5)
    dy, _ = T._rows((M, N), "bf16", 6)
    from weight_only_int4_w4a16_amd import binding
    need = binding.lib().w4a16_fp8_backward_workspace_bytes(M, K, N)
    big = torch.zeros(need + M * K * 2, dtype=u8, device="cuda")
    inside = big[:M * K * 2].view(bf16).view(M, K).copy_(x)
    _refused(lambda: w4.gemm_fp8_backward(dy, inside, codes_t, scales_t, workspace=big), "workspace overlaps")
    a, b = w4.gemm_fp8_backward(dy, inside, codes_t, scales_t, workspace=big[(M * K * 2 + 255) // 256 * 256:])
    c, d = w4.gemm_fp8_backward(dy, x, codes_t, scales_t)
    assert torch.equal(a, c) and torch.equal(b, d)


def test_workspaces_of_the_public_sizes():
    """Each call with a workspace of the bytes that its size function names, for every result type."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    tokens, topk, E, K, N = 40, 2, 3, 256, 192

    def space(n):
        ws, ends = T._guarded((max(n, 1),), torch.uint8)
        return ws, ends

    r = w4.route(torch.from_numpy(T._ids(tokens, topk, E, 1)).cuda(), E)
    x, _ = T._rows((tokens, K), "f16", 1)
    codes, scales, _ = T._weight((E,), N, K, 2, halves=2)
    ws, ends = space(w4.fp8_grouped_workspace_bytes(tokens, topk, E, K, N, x.dtype, swiglu=True, gather=True))
    for dtype in (torch.float16, torch.float32):
        got = w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True, out_dtype=dtype, workspace=ws)
        assert torch.equal(got, w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True, out_dtype=dtype))
    ends("SwiGLU")
    ws, ends = space(w4.fp8_grouped_workspace_bytes(tokens, topk, E, K, N, x.dtype, swiglu=True, quantized=True, gather=True))
    q, s = w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True, quantized=True, workspace=ws)
    q2, s2 = w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True, quantized=True)
    ends("quantized")
    assert np.array_equal(T._bits(q), T._bits(q2)) and torch.equal(s, s2)
    S = tokens * topk
    dy, _ = T._rows((S, N), "f16", 3)
    xs, _ = T._rows((S, K), "f16", 4)
    codes_t, scales_t, _ = T._weight((E,), K, N, 5)
    ws, ends = space(w4.fp8_grouped_backward_workspace_bytes(tokens, topk, E, K, N))
    got = w4.gemm_fp8_grouped_backward(dy, xs, r, codes_t, scales_t, workspace=ws)
    ends("routed gradients")
    assert all(map(torch.equal, got, w4.gemm_fp8_grouped_backward(dy, xs, r, codes_t, scales_t)))
    ws, ends = space(w4.fp8_backward_workspace_bytes(S, K, N))
    got = w4.gemm_fp8_backward(dy, xs, codes_t[0], scales_t[0], workspace=ws)
    ends("gradients")
    assert all(map(torch.equal, got, w4.gemm_fp8_backward(dy, xs, codes_t[0], scales_t[0])))
