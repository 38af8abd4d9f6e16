"""CPU checks of the 8-bit floating point operators: the oracle against the format's definition, torch's own cast,
brute force and differences, and the refusals of the C ABI and of the binding (nothing is launched)."""
import numpy as np
import pytest

from oracle import fp8 as F

OK, ARG, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
F16, BF16, F32, E4M3 = 0, 1, 2, 3
P = 1 << 20  # aligned placeholder addresses, never dereferenced
Q = P + 4096


# ------------------------------------------------------------------ oracle

def test_codes_are_torchs():
    import torch
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(F.e4m3_values(), want, equal_nan=True)
    assert np.nanmax(F.e4m3_values()) == F.LARGEST
    # every value, the middle between neighbours (to the even code) and both sides of it
    v = F.e4m3_values()[:127].astype(np.float32)
    mid = ((v[:-1] + v[1:]) / 2).astype(np.float32)  # exact: four bits and one more
    tests = np.concatenate([v, mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9))])
    tests = np.concatenate([tests, -tests])
    want = torch.from_numpy(tests).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(F.to_e4m3(tests), want)
    assert np.array_equal(F.to_e4m3(v), codes[:127])


def test_groups_are_scaled_and_rounded_once():
    g = np.random.default_rng(0)
    x = (g.standard_normal((5, 300)) * 10.0 ** g.integers(-6, 6, size=(5, 1))).astype(np.float32)
    x[3, 128:256] = 0
    codes, scales = F.quantize_rows(x)
    assert scales.shape == (3, 5) and scales[1, 3] == F.LEAST and not codes[3, 128:256].any()
    for m in range(5):
        for b in range(3):
            k = slice(128 * b, 128 * b + 128)
            if not x[m, k].any():
                continue
            assert scales[b, m] == np.float32(np.abs(x[m, k]).max() / np.float32(448))
            assert np.abs(F.from_e4m3(codes[m, k])).max() == 448  # the largest takes the largest code
            # half a step: 2^-4 of the value, or of the least normal number 2^-6
            bound = np.maximum(np.abs(x[m, k]) * 2.0 ** -4, scales[b, m] * 2.0 ** -10) * (1 + 2.0 ** -22)
            assert np.all(np.abs(F.from_e4m3(codes[m, k]) * scales[b, m] - x[m, k]) <= bound)


def test_columns_and_blocks():
    g = np.random.default_rng(1)
    x = g.standard_normal((150, 9)).astype(np.float32)
    codes, scales = F.quantize_columns(x)
    assert codes.shape == (9, 160) and scales.shape == (2, 9) and not codes[:, 150:].any()
    for k in range(9):
        for b in range(2):
            part = x[128 * b: 128 * b + 128, k]
            assert scales[b, k] == F.scale_of(part)
            assert np.array_equal(codes[k, 128 * b: 128 * b + 128][: len(part)], F.to_e4m3((part / scales[b, k]).astype(np.float32)))
    w = g.standard_normal((130, 140)).astype(np.float32)
    codes, scales = F.quantize_weight(w)
    assert scales.shape == (2, 2) and scales[1, 0] == F.scale_of(w[128:, :128])
    # a weight and its transpose have the same codes
    ct, st = F.quantize_weight(w.T)
    assert np.array_equal(ct, codes.T) and np.array_equal(st, scales.T)


def test_groups_that_are_not_finite():
    x = np.zeros((3, 256), dtype=np.float32)
    x[0, 5], x[1, 200], x[2, 0] = np.inf, np.nan, -np.inf
    codes, scales = F.quantize_rows(x)
    for m, b in [(0, 0), (1, 1), (2, 0)]:
        assert np.isnan(scales[b, m]) and np.isnan(F.from_e4m3(codes[m, 128 * b: 128 * b + 128])).all()
        assert scales[1 - b, m] == F.LEAST and not codes[m, 128 * (1 - b): 128 * (1 - b) + 128].any()
    assert np.isnan(F.gemm_fp8_ref(F.rows_value(codes, scales), np.ones((2, 256)))).all()


def test_products_by_loops():
    g = np.random.default_rng(2)
    x, w = g.standard_normal((3, 144)).astype(np.float32), g.standard_normal((5, 144)).astype(np.float32)
    xc, xs = F.quantize_rows(x)
    wc, ws = F.quantize_weight(w)
    y = F.gemm_fp8_ref(F.rows_value(xc, xs), F.weight_value(wc, ws))
    for m in range(3):
        for n in range(5):
            want = sum(float(xs[k // 128, m]) * float(ws[0, k // 128]) * F.from_e4m3(xc[m, k]) * F.from_e4m3(wc[n, k])
                       for k in range(144))
            assert abs(y[m, n] - want) < 1e-12 * 144
    # near the product of the values themselves: each factor off by 2^-4 at most, its group's least by 2^-10 of the scale
    assert np.abs(y - x.astype(float) @ w.T.astype(float)).max() < (2 * 2.0 ** -4 + 2.0 ** -8) * (np.abs(x) @ np.abs(w).T).max()
    # halves with blocks of their own
    a, b = g.standard_normal((6, 32)).astype(np.float32), g.standard_normal((6, 32)).astype(np.float32)
    (ac, as_), (bc, bs) = F.quantize_weight(a), F.quantize_weight(b)
    both = F.weight_value(np.concatenate([ac, bc]), np.concatenate([as_, bs]), 2)
    assert np.array_equal(both, np.concatenate([F.weight_value(ac, as_), F.weight_value(bc, bs)]))
    v = g.standard_normal((2, 32))
    gate, up = v @ both[:6].T, v @ both[6:].T
    assert np.allclose(F.swiglu_fp8_ref(v, both), gate / (1 + np.exp(-gate)) * up, rtol=1e-13, atol=0)


def test_gradients_against_differences():
    """y = x W^T is linear in each, so central differences of <dy, y> are exact up to rounding; the quantized gradients
    are those of the values that the codes stand for."""
    g = np.random.default_rng(3)
    dy, x = g.standard_normal((40, 32)).astype(np.float32), g.standard_normal((40, 48)).astype(np.float32)
    wt = F.weight_value(*F.quantize_weight(g.standard_normal((48, 32)).astype(np.float32)))
    dx, dw = F.backward_fp8_ref(dy, x, wt)
    dyv = F.rows_value(*F.quantize_rows(dy))
    dyc, xc = (F.rows_value(*F.quantize_columns(v))[:, :40].T for v in (dy, x))

    def slope(f, a, at, h=0.5):
        up, down = a.copy(), a.copy()
        up[at] += h
        down[at] -= h
        return (f(up) - f(down)) / (2 * h)

    xd = x.astype(np.float64)
    for at in [(0, 0), (39, 47), (7, 20)]:
        assert abs(slope(lambda v: np.sum(dyv * (v @ wt)), xd, at) - dx[at]) < 1e-9
    w0 = np.zeros((32, 48))
    for at in [(0, 0), (31, 47), (5, 9)]:
        assert abs(slope(lambda v: np.sum(dyc * (xc @ v.T)), w0, at) - dw[at]) < 1e-9


# ------------------------------------------------------------------ refusals of the C ABI

@pytest.fixture(scope="module")
def L():
    from weight_only_int4_w4a16_amd import binding
    return binding.lib()


QUANT = dict(x=P, M=4, K=64, dtype=BF16, codes=2 * P, scales=Q)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), ARG), (dict(K=0), ARG), (dict(dtype=3), ARG), (dict(dtype=-1), ARG), (dict(x=0), ARG),
    (dict(codes=0), ARG), (dict(scales=0), ARG), (dict(codes=2 * P + 8), ARG), (dict(scales=Q + 2), ARG),
    (dict(M=0, x=0, codes=0, scales=0), OK), (dict(M=2 ** 31 - 1, K=1 << 20), UNSUPPORTED),
])
def test_quantizers_refuse(L, kw, status):
    a = {**QUANT, **kw}
    args = (a["x"] or None, a["M"], a["K"], a["dtype"], a["codes"] or None, a["scales"] or None)
    assert L.w4a16_quantize_fp8(*args, None) == status
    assert L.w4a16_quantize_fp8_columns(*args, None) == status
    assert L.w4a16_quantize_fp8_weight(*args, None, None, None) == status


def test_quantizers_of_special_forms(L):
    # rows: vectors of eight values; the others take any width and any address of an element
    assert L.w4a16_quantize_fp8(P, 4, 72, BF16, 2 * P, Q, None) == UNSUPPORTED
    assert L.w4a16_quantize_fp8(P + 8, 4, 64, BF16, 2 * P, Q, None) == ARG
    assert L.w4a16_quantize_fp8_columns(P + 1, 4, 7, BF16, 2 * P, Q, None) == ARG
    assert L.w4a16_quantize_fp8_weight(P + 2, 4, 7, F32, 2 * P, Q, None, None, None) == ARG
    # transposed codes and scales come together
    assert L.w4a16_quantize_fp8_weight(P, 4, 64, F32, 2 * P, Q, 3 * P, None, None) == ARG
    assert L.w4a16_quantize_fp8_weight(P, 4, 64, F32, 2 * P, Q, None, 3 * P, None) == ARG
    assert L.w4a16_quantize_fp8_weight(P, 4, 64, F32, 2 * P, Q, 3 * P + 4, Q, None) == ARG


GEMM = dict(x=P, xdt=BF16, xs=0, M=4, K=256, N=64, codes=2 * P, scales=Q, glu=0, out=3 * P, odt=BF16, os=0, ws=4 * P, nb=1 << 20)

GEMM_CASES = [
    (dict(M=-1), ARG), (dict(K=0), ARG), (dict(N=0), ARG), (dict(xdt=F32), ARG), (dict(xdt=4), ARG), (dict(odt=7), ARG),
    (dict(odt=F16), ARG), (dict(odt=E4M3), ARG), (dict(glu=1, N=63), ARG), (dict(K=264), UNSUPPORTED),
    (dict(x=0), ARG), (dict(x=P + 8), ARG), (dict(codes=0), ARG), (dict(codes=2 * P + 4), ARG), (dict(scales=0), ARG),
    (dict(scales=Q + 2), ARG), (dict(out=0), ARG), (dict(out=3 * P + 8), ARG), (dict(out=P), ARG),
    (dict(xdt=E4M3, xs=0), ARG), (dict(xdt=E4M3, xs=Q + 1), ARG), (dict(glu=1, odt=E4M3, os=0), ARG),
    (dict(glu=1, odt=E4M3, os=Q, N=48), UNSUPPORTED), (dict(ws=0), WORKSPACE), (dict(ws=4 * P + 64), WORKSPACE),
    (dict(nb=1023), WORKSPACE), (dict(glu=1, odt=E4M3, os=Q, nb=1791), WORKSPACE), (dict(K=1 << 23), UNSUPPORTED),
    (dict(M=1 << 27, K=1 << 16), UNSUPPORTED), (dict(K=16, N=(1 << 30) + 16), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", GEMM_CASES)
def test_products_refuse(L, kw, status):
    a = {**GEMM, **kw}
    assert L.w4a16_gemm_fp8(a["x"] or None, a["xdt"], a["xs"] or None, a["M"], a["K"], a["N"], a["codes"] or None,
                            a["scales"] or None, a["glu"], a["out"] or None, a["odt"], a["os"] or None, a["ws"] or None,
                            a["nb"], None) == status


@pytest.mark.parametrize("kw,status", GEMM_CASES + [
    (dict(tokens=-1), ARG), (dict(topk=0), ARG), (dict(groups=0), ARG), (dict(groups=1025), UNSUPPORTED),
    (dict(plan=0), ARG), (dict(plan=Q + 64), ARG), (dict(tokens=1 << 23, K=256, gather=1), UNSUPPORTED),
    (dict(tokens=1 << 26), UNSUPPORTED),
])
def test_grouped_products_refuse(L, kw, status):
    a = {**GEMM, "plan": Q, "tokens": 2, "topk": 2, "groups": 3, "gather": 0, **kw}
    if "M" in kw:
        a["tokens"] = kw["M"] if kw["M"] < 0 else 1 << 26
    assert L.w4a16_gemm_fp8_grouped(a["x"] or None, a["xdt"], a["xs"] or None, a["plan"] or None, a["tokens"], a["topk"],
                                    a["groups"], a["gather"], a["K"], a["N"], a["codes"] or None, a["scales"] or None, a["glu"],
                                    a["out"] or None, a["odt"], a["os"] or None, a["ws"] or None, a["nb"], None) == status


def test_products_of_no_rows(L):
    assert L.w4a16_gemm_fp8(None, BF16, None, 0, 64, 32, None, None, 0, None, BF16, None, None, 0, None) == OK
    assert L.w4a16_gemm_fp8_grouped(None, BF16, None, None, 0, 2, 3, 0, 64, 32, None, None, 0, None, BF16, None, None, 0, None) == OK
    assert L.w4a16_gemm_fp8_backward(None, None, 0, 64, 32, BF16, None, None, None, None, None, 0, None) == OK


BACK = dict(dy=P, x=2 * P, M=4, K=64, N=32, act=BF16, codes=3 * P, scales=Q, dx=4 * P, dw=5 * P, ws=6 * P, nb=1 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), ARG), (dict(K=0), ARG), (dict(N=0), ARG), (dict(act=F32), ARG), (dict(act=E4M3), ARG), (dict(K=72), UNSUPPORTED),
    (dict(N=40), UNSUPPORTED), (dict(dy=0), ARG), (dict(dy=P + 8), ARG), (dict(x=0), ARG), (dict(x=2 * P + 2), ARG),
    (dict(codes=0), ARG), (dict(scales=0), ARG), (dict(dx=P), ARG), (dict(dx=4 * P + 4), ARG), (dict(dw=5 * P + 8), ARG),
    (dict(ws=0), WORKSPACE), (dict(nb=255), WORKSPACE), (dict(M=2 ** 31 - 1), UNSUPPORTED),
    (dict(K=(1 << 30) + 16, N=16), UNSUPPORTED), (dict(M=1 << 22, K=1 << 17, N=16), UNSUPPORTED),
])
def test_gradients_refuse(L, kw, status):
    a = {**BACK, **kw}
    rest = (a["K"], a["N"], a["act"], a["codes"] or None, a["scales"] or None, a["dx"] or None, a["dw"] or None, a["ws"] or None, a["nb"], None)
    assert L.w4a16_gemm_fp8_backward(a["dy"] or None, a["x"] or None, a["M"], *rest) == status
    tokens = a["M"] if a["M"] < 1 << 20 else 1 << 26
    assert L.w4a16_gemm_fp8_grouped_backward(a["dy"] or None, a["x"] or None, Q, tokens, 1, 3, *rest) == status


def test_sizes_and_names(L):
    assert L.w4a16_fp8_workspace_bytes(0, 64, 32, BF16, 0, BF16) == 0
    assert L.w4a16_fp8_workspace_bytes(4, 72, 32, BF16, 0, BF16) == 0
    assert L.w4a16_fp8_workspace_bytes(4, 64, 32, E4M3, 0, BF16) == 0
    assert L.w4a16_fp8_workspace_bytes(4, 256, 32, BF16, 0, BF16) >= 4 * 256 + 2 * 4 * 4
    assert L.w4a16_fp8_backward_workspace_bytes(4, 64, 40) == 0
    assert L.w4a16_fp8_kernel_name(0, 64, 32, 0) == b"none" and L.w4a16_fp8_kernel_name(1, 64, 32, 0) != b"none"
    assert L.w4a16_fp8_kernel_name(1, 60, 32, 0) == b"none"


def test_gradients_have_room_for_partial_sums(L):
    """Products whose depth is cut keep fp32 sums of every slice beside the codes that all of them read."""
    most = 0
    for M, K, N in [(2085, 256, 128), (1500, 128, 160), (40, 256, 8192), (2048, 128, 128), (8192, 256, 256), (64, 512, 16384)]:
        depth = (M + 15) // 16 * 16
        sums = max(L.w4a16_fp8_workspace_bytes(N, depth, K, E4M3, 0, F32) if N > 16 else 0,
                   L.w4a16_fp8_workspace_bytes(M, N, K, E4M3, 0, BF16))
        assert L.w4a16_fp8_backward_workspace_bytes(M, K, N) >= sums + M * N + depth * (K + N)
        most = max(most, sums)
    assert most > 0


def test_workspace_covers_every_out_dtype(L):
    import torch
    import weight_only_int4_w4a16_amd as w4
    for M, K, N in [(1, 256, 64), (20, 8192, 1024), (40, 2048, 4096), (64, 14336, 4096), (333, 2896, 5001)]:
        for x, dt in ((torch.bfloat16, BF16), (torch.float8_e4m3fn, E4M3)):
            have = w4.fp8_workspace_bytes(M, K, N, x)
            assert have == max(L.w4a16_fp8_workspace_bytes(M, K, N, dt, 0, o) for o in (BF16, F32))


# ------------------------------------------------------------------ refusals of the binding (meta and host tensors)

def _refused(fn, match, status=ARG):
    from weight_only_int4_w4a16_amd import W4A16Error
    with pytest.raises(W4A16Error, match=match) as e:
        fn()
    assert e.value.status == status


def test_binding_refuses():
    import torch
    import weight_only_int4_w4a16_amd as w4
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for f in (w4.quantize_fp8, w4.quantize_fp8_columns, w4.quantize_fp8_weight):
        _refused(lambda: f(x), "device")
        _refused(lambda: f(None), "2-D")
        _refused(lambda: f(x[0]), "2-D")
        _refused(lambda: f(x.t()), "contiguous")
        _refused(lambda: f(x.to(torch.float64)), "dtype")
        _refused(lambda: f(x[:, :0]), "no elements")
        _refused(lambda: f(torch.empty(2 ** 31, 16, dtype=torch.bfloat16, device="meta")), "2\\^31", UNSUPPORTED)
    codes, scales = torch.zeros(32, 64, dtype=torch.float8_e4m3fn), torch.zeros(1, 1)
    _refused(lambda: w4.gemm_fp8(x, codes, scales), "device")
    _refused(lambda: w4.gemm_fp8(x.t(), codes, scales), "contiguous")
    _refused(lambda: w4.gemm_fp8(x[0], codes, scales), "2-D")
    _refused(lambda: w4.gemm_fp8_grouped(x, None, codes, scales), "route")
    _refused(lambda: w4.gemm_fp8_grouped_backward(x, x, None, codes, scales), "route")
    _refused(lambda: w4.gemm_fp8_backward(x, x.float(), codes, scales), "dtype")
    _refused(lambda: w4.gemm_fp8_backward(None, x, codes, scales), "2-D")
