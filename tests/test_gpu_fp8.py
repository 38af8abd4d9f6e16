"""GPU checks of the 8-bit floating point operators against the fp64 oracle (oracle/fp8.py).

Codes and scales of quantizers are equal to the oracle's, bit for bit. Bounds of products, elementwise, on the values that
the codes stand for (eps the fp32 unit roundoff 2^-24, u the output type's, 2^-11 fp16 and 2^-8 bf16, d half the type's
least subnormal):

* a sum of n fp32 terms is off by at most 2 n eps times the sum of the terms' magnitudes, whatever its order; a block's two
  scales add two roundings: 2 (K + 2) eps in all;
* results of 16 bits: the 8-bit matrix instructions keep 17 bits below the leading one of a block's largest product
  (measured in every lane and position, on codes of all sizes), so each of 128 products loses less than 2^-17 of it and the
  block 2^-10 of its largest product, times its scales;
* storing in a 16-bit type adds u |value| + d;
* SwiGLU of sums off by dg, du: |dh| <= 1.1 dg |u| + (|SiLU(g)| + 1.1 dg) du, and the fp32 exponential, division and
  products add (|g| + 8) 2^-22 |h|;
* h quantized from fp32: its scale is off by what the largest |h| of the group is, and a code by half a step, 2^-4 of the
  value or 2^-10 of the scale.
"""
import numpy as np
import pytest

from oracle import fp8 as F
from oracle import routed as R
from weight_only_int4_w4a16_amd import synth

from gpu_common import assert_graph_replays_match_eager, require_gpu, torch_mod

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": EPS}
D = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _announce(msg):
    print(f"[case] {msg}", flush=True)


def _dtype(kind):
    torch = torch_mod()
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[kind]


def _rows(shape, kind, seed, spread=True):
    """(device tensor, its fp32 values): normal values, some columns ten times as large."""
    torch = torch_mod()
    g = synth.generator(seed)
    a = g.standard_normal(shape)
    if spread:
        a = a * np.where(g.random(shape[-1]) < 0.05, 10.0, 1.0)
    t = torch.from_numpy(a.astype(np.float32)).cuda().to(_dtype(kind))
    return t, t.cpu().float().numpy()


def _bits(codes):
    torch = torch_mod()
    return codes.cpu().view(torch.uint8).numpy()


def _same_codes(got, want, what):
    """Equal codes; a NaN may have either sign."""
    got, want = got.copy(), want.copy()
    got[got == 255] = 127
    want[want == 255] = 127
    assert np.array_equal(got, want), f"{what}: {np.mean(got != want):.2e} of the codes differ"


def _weight(lead, N, K, seed, halves=1):
    """(codes, scales) on the device and the fp64 values [*lead, N, K]."""
    torch = torch_mod()
    g = synth.generator(seed)
    table = np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)
    codes = F.to_e4m3(np.clip(112 * g.standard_normal((*lead, N, K)), -448, 448))
    some = g.random(codes.shape) < 0.05
    codes[some] = g.choice(table, size=int(some.sum()))  # of all sizes
    blocks = halves * -(-(N // halves) // 128)
    scales = ((0.5 + g.random((*lead, blocks, -(-K // 128)))) / (112 * K ** 0.5)).astype(np.float32)
    if lead:
        value = np.stack([F.weight_value(c, s, halves) for c, s in zip(codes, scales)])
    else:
        value = F.weight_value(codes, scales, halves)
    return torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scales).cuda(), value


def _sum_bound(xv, wv, kind):
    """What the sums of a product may be off by (before rounding to the output type)."""
    K = xv.shape[1]
    bound = 2 * (K + 2) * EPS * (np.abs(xv) @ np.abs(wv).T)
    if kind != "f32":
        for b in range(0, K, 128):
            k = slice(b, b + 128)
            bound += 2.0 ** -10 * (np.abs(xv[:, k]).max(1)[:, None] * np.abs(wv[:, k]).max(1)[None, :])
    return bound


def _stored(ref, bound, kind):
    return bound + U[kind] * (np.abs(ref) + bound) + D[kind]


def _glu_bound(xv, wv, kind):
    y, dy = F.gemm_fp8_ref(xv, wv), _sum_bound(xv, wv, kind)
    (g, u), (dg, du) = np.split(y, 2, 1), np.split(dy, 2, 1)
    h = F.silu(g) * u
    return h, 1.1 * dg * np.abs(u) + (np.abs(F.silu(g)) + 1.1 * dg) * du + (np.abs(g) + 8) * 2.0 ** -22 * (np.abs(h) + 1.1 * dg * np.abs(u))


def _within(got, ref, bound, what):
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    over = np.abs(got - ref) - bound
    assert np.all(over <= 0), f"{what}: off by {np.abs(got - ref).max():.3e}, {over.max():.3e} past the bound"


def _check_quantized(codes, scales, h, dh, what):
    """Codes and scales of an fp32 h that is within dh of the reference."""
    codes, scales = _bits(codes), scales.cpu().double().numpy()
    M, N = h.shape
    for b in range(-(-N // 128)):
        n = slice(128 * b, 128 * b + 128)
        most, off = np.abs(h[:, n]).max(1), dh[:, n].max(1)
        least = float(F.LEAST)
        assert np.all(scales[b] <= np.maximum((most + off) / 448 * (1 + 2 * EPS), least)), what
        assert np.all(scales[b] >= np.maximum((most - off) / 448 * (1 - 2 * EPS), least)), what
        v = F.from_e4m3(codes[:, n]) * scales[b][:, None]
        size = np.abs(h[:, n]) + dh[:, n]
        bound = dh[:, n] + np.maximum(2.0 ** -4 * size, 2.0 ** -10 * scales[b][:, None]) * (1 + 2.0 ** -20)
        _within(v, h[:, n], bound, what)


# ------------------------------------------------------------------ quantizers

@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (3, 128), (5, 144), (33, 1040), (17, 656), (1100, 4112)])
def test_rows(M, K, kind):
    import weight_only_int4_w4a16_amd as w4
    _announce(f"rows {M}x{K} {kind}")
    x, xv = _rows((M, K), kind, M + K)
    codes, scales = w4.quantize_fp8(x)
    some = np.unique(np.concatenate([np.arange(min(M, 40)), [M - 1]]))  # the oracle's loops are slow
    want, wants = F.quantize_rows(xv[some])
    _same_codes(_bits(codes)[some], want, "codes")
    assert np.array_equal(scales.cpu().numpy()[:, some], wants)


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 9), (16, 128), (127, 7), (128, 136), (129, 130), (300, 33), (500, 260)])
def test_columns_and_blocks(M, K, kind):
    import weight_only_int4_w4a16_amd as w4
    _announce(f"columns {M}x{K} {kind}")
    x, xv = _rows((M, K), kind, M * 3 + K)
    codes, scales = w4.quantize_fp8_columns(x)
    want, wants = F.quantize_columns(xv)
    _same_codes(_bits(codes), want, "columns")
    assert np.array_equal(scales.cpu().numpy(), wants)
    want, wants = F.quantize_weight(xv)
    codes, scales = w4.quantize_fp8_weight(x)
    _same_codes(_bits(codes), want, "blocks")
    assert np.array_equal(scales.cpu().numpy(), wants)
    codes, scales, codes_t, scales_t = w4.quantize_fp8_weight(x, transposed=True)
    _same_codes(_bits(codes), want, "blocks")
    _same_codes(_bits(codes_t), want.T, "transposed blocks")
    assert np.array_equal(scales.cpu().numpy(), wants) and np.array_equal(scales_t.cpu().numpy(), wants.T)


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
def test_values_of_all_sizes(kind):
    """Each group at its own power of two, from the least numbers of the type to its largest, and groups that are not
    finite: quotients next to and at the middle between codes are rounded as the definition says."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    g = synth.generator(77)
    lo, hi = {"f16": (-30, 15), "bf16": (-139, 126), "f32": (-155, 126)}[kind]
    rows = []
    for e in range(lo, hi, 3):
        rows.append(np.ldexp(g.standard_normal(128), e))
        # fractions of eight bits: the quotients of bf16 values lie at and around the middles
        rows.append(np.ldexp(1.0 + g.integers(0, 128, 128) / 128, e) * g.choice([1.0, 0.5, 0.25, 0.125, 2.0 ** -7, 2.0 ** -13], 128))
    x = np.array(rows, dtype=np.float64)
    x = np.where(np.abs(x) > 2.0 ** 15 * 1.9 if kind == "f16" else np.abs(x) > 1.6e38, 1.0, x)
    with np.errstate(over="ignore"):
        t = torch.from_numpy(x.astype(np.float32)).to(_dtype(kind))
    t[-1, 3], t[-2, 5], t[-3, 127] = float("inf"), float("nan"), float("-inf")
    xv = t.float().numpy()
    codes, scales = w4.quantize_fp8(t.cuda())
    want, wants = F.quantize_rows(xv)
    _same_codes(_bits(codes), want, "codes")
    assert np.array_equal(scales.cpu().numpy(), wants, equal_nan=True)
    codes, scales = w4.quantize_fp8_columns(t.t().contiguous().cuda())
    _same_codes(_bits(codes), want, "columns")
    assert np.array_equal(scales.cpu().numpy(), wants, equal_nan=True)
    for i in range(0, len(rows) - 4, 7):  # one block each
        codes, scales = w4.quantize_fp8_weight(t[i:i + 1].cuda())
        _same_codes(_bits(codes), want[i:i + 1], "block")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_every_quotient_of_16_bits(kind):
    """Every significand under every largest value of a group, at every exponent that has a code: the codes of 16-bit values
    (one step of the division) are those of the same values in 32 bits (two), and some rows' the oracle's."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    n = 1024 if kind == "f16" else 128
    m = (1 + torch.arange(n, dtype=torch.float64, device="cuda") / n)
    values = torch.cat([m * 2.0 ** (10 - e) for e in range(21)])
    values = torch.cat([values, torch.zeros(-len(values) % 127, dtype=torch.float64, device="cuda")]).reshape(-1, 127)
    values[:, 1::2] *= -1
    for top in range(0, n, 128):
        largest = (m[top:top + 128] * 2.0 ** 10).reshape(-1, 1, 1).expand(-1, len(values), 1)
        v = values.expand(len(largest), -1, -1)
        v = torch.where(v.abs() > largest, 0.0, v)
        x = torch.cat([largest, v], dim=2).reshape(len(largest), -1).to(_dtype(kind))
        codes, scales = w4.quantize_fp8(x)
        codes32, scales32 = w4.quantize_fp8(x.float())
        assert torch.equal(scales, scales32)
        assert torch.equal(codes.view(torch.uint8), codes32.view(torch.uint8)), f"largest from {top}"
        codes, _ = w4.quantize_fp8_columns(x.t().contiguous())
        assert torch.equal(codes.view(torch.uint8), codes32.view(torch.uint8)), f"columns, largest from {top}"
        some = [0, 5, 77]
        want, wants = F.quantize_rows(x[some].float().cpu().numpy())
        assert np.array_equal(_bits(codes[some]), want) and np.array_equal(scales[:, some].cpu().numpy(), wants)


def test_quantizers_at_odd_addresses():
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    buf = torch.randn(40 * 72 + 1, device="cuda")
    for kind in ("f32", "bf16"):
        x = buf.to(_dtype(kind))[1:].view(40, 72)
        want, wants = F.quantize_columns(x.cpu().float().numpy())
        codes, scales = w4.quantize_fp8_columns(x)
        _same_codes(_bits(codes), want, "columns")
        want, wants = F.quantize_weight(x.cpu().float().numpy())
        codes, scales = w4.quantize_fp8_weight(x)
        _same_codes(_bits(codes), want, "blocks")


# ------------------------------------------------------------------ products

PRODUCTS = [
    # M, K, N: one token to many, depths and widths that divide nothing
    (1, 16, 1), (1, 4096, 512), (1, 14352, 96), (1, 33024, 48), (2, 144, 33), (2, 4112, 300), (2, 16400, 40), (3, 1040, 100), (5, 144, 28800), (16, 256, 32768), (7, 2048, 640), (15, 528, 1000), (16, 256, 256), (17, 4112, 130),
    (18, 1040, 4608), (20, 144, 100), (32, 8208, 48), (31, 128, 2048), (33, 384, 129), (48, 640, 777), (63, 896, 128), (64, 1024, 384), (65, 512, 257), (100, 272, 1024),
    (127, 1152, 255), (128, 2176, 512), (129, 160, 640), (200, 1280, 1001), (48, 1680, 300), (64, 8208, 200), (90, 3600, 400), (333, 2896, 700), (256, 640, 2048), (257, 400, 512), (333, 656, 501),
]


@pytest.mark.parametrize("M,K,N", PRODUCTS)
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_products(M, K, N, kind):
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    _announce(f"gemm_fp8 {M}x{K}x{N} {kind} {w4.fp8_kernel_name(M, K, N)}")
    x, xv = _rows((M, K), kind, M + 3 * K + N)
    xq, xs = F.quantize_rows(xv)
    xv = F.rows_value(xq, xs)
    codes, scales, wv = _weight((), N, K, M * 5 + K + N)
    ref = F.gemm_fp8_ref(xv, wv)
    y = w4.gemm_fp8(x, codes, scales)
    assert y.dtype == x.dtype
    _within(y.cpu().double().numpy(), ref, _stored(ref, _sum_bound(xv, wv, kind), kind), "16-bit out")
    y32 = w4.gemm_fp8(x, codes, scales, out_dtype=torch.float32)
    _within(y32.cpu().double().numpy(), ref, _stored(ref, _sum_bound(xv, wv, "f32"), "f32"), "fp32 out")
    # from codes, the same bits
    q, s = w4.quantize_fp8(x)
    assert torch.equal(w4.gemm_fp8(q, codes, scales, x_scales=s, out_dtype=torch.float32), y32)
    assert torch.equal(w4.gemm_fp8(q, codes, scales, x_scales=s, out_dtype=x.dtype), y)
    out = torch.full((M + 2, N), 7.0, dtype=x.dtype, device="cuda")
    if N % 8 == 0:  # rows around the output stay
        w4.gemm_fp8(x, codes, scales, out=out[1:-1])
        assert torch.equal(out[1:-1], y) and bool((out[0] == 7).all()) and bool((out[-1] == 7).all())


@pytest.mark.parametrize("M,K,N2", [(1, 256, 2), (1, 2048, 512), (2, 4112, 160), (5, 144, 100), (9, 272, 28672), (16, 640, 704), (17, 528, 98), (32, 4112, 288), (33, 1040, 258), (48, 1680, 1056), (64, 8208, 512), (100, 4112, 1024), (64, 512, 96),
                                    (70, 272, 640), (130, 384, 1000), (257, 256, 1024), (300, 528, 288)])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_swiglu(M, K, N2, kind):
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    _announce(f"gemm_fp8_swiglu {M}x{K}x{N2} {kind}")
    x, xv = _rows((M, K), kind, M + K + N2)
    xv = F.rows_value(*F.quantize_rows(xv))
    codes, scales, wv = _weight((), N2, K, M + 7 * K + N2, halves=2)
    h, dh = _glu_bound(xv, wv, kind)
    _within(w4.gemm_fp8_swiglu(x, codes, scales).cpu().double().numpy(), h, _stored(h, dh, kind), "h")
    h, dh = _glu_bound(xv, wv, "f32")
    _within(w4.gemm_fp8_swiglu(x, codes, scales, out_dtype=torch.float32).cpu().double().numpy(), h, _stored(h, dh, "f32"), "fp32 h")
    if N2 % 32 == 0:
        q, s = w4.gemm_fp8_swiglu(x, codes, scales, quantized=True)
        assert q.shape == h.shape and s.shape == (-(-h.shape[1] // 128), M)
        _check_quantized(q, s, h, dh, "quantized h")


@pytest.mark.parametrize("M,K,N2", [(2100, 256, 4096), (2049, 144, 3904), (4096, 384, 2560)])
def test_swiglu_on_large_tiles(M, K, N2):
    """Enough tiles of 256 x 256 to fill the chip: h is quantized where it is made."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    _announce(f"gemm_fp8_swiglu {M}x{K}x{N2}, large tiles")
    x, xv = _rows((M, K), "bf16", M)
    codes, scales, wv = _weight((), N2, K, K, halves=2)
    q, s = w4.gemm_fp8_swiglu(x, codes, scales, quantized=True)
    h16 = w4.gemm_fp8_swiglu(x, codes, scales)
    some = np.unique(np.concatenate([np.arange(0, M, 37), [255, 256, M - 1]]))
    xv = F.rows_value(*F.quantize_rows(xv[some]))
    at = torch.from_numpy(some).cuda()
    h, dh = _glu_bound(xv, wv, "f32")
    _check_quantized(q.view(torch.uint8)[at].view(torch.float8_e4m3fn), s[:, at], h, dh, "quantized h")
    h, dh = _glu_bound(xv, wv, "bf16")
    _within(h16[at].cpu().double().numpy(), h, _stored(h, dh, "bf16"), "h")


LARGE = [(2048, 256, 4100), (4000, 400, 2056), (1000, 640, 1300), (3000, 144, 3000), (4096, 512, 9000), (4100, 256, 5000), (530, 4096, 520), (500, 512, 9000), (250, 4096, 9000)]


@pytest.mark.parametrize("M,K,N", LARGE)
def test_products_on_large_tiles(M, K, N):
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    _announce(f"gemm_fp8 {M}x{K}x{N}, {w4.fp8_kernel_name(M, K, N)}")
    x, xv = _rows((M, K), "f16", M)
    codes, scales, wv = _weight((), N, K, K)
    some = np.unique(np.concatenate([np.arange(0, M, 31), [127, 128, M - 1]]))
    xv = F.rows_value(*F.quantize_rows(xv[some]))
    ref = F.gemm_fp8_ref(xv, wv)
    at = torch.from_numpy(some).cuda()
    y = w4.gemm_fp8(x, codes, scales)
    _within(y[at].cpu().double().numpy(), ref, _stored(ref, _sum_bound(xv, wv, "f16"), "f16"), "16-bit out")
    y = w4.gemm_fp8(x, codes, scales, out_dtype=torch.float32)
    _within(y[at].cpu().double().numpy(), ref, _stored(ref, _sum_bound(xv, wv, "f32"), "f32"), "fp32 out")


def test_every_kernel_is_reached():
    """The shapes of these tests run on tiles of each height, with k whole and in slices."""
    import weight_only_int4_w4a16_amd as w4
    names = {w4.fp8_kernel_name(M, K, N) for M, K, N in PRODUCTS + LARGE}
    assert names >= {"w4a16_fp8_16", "w4a16_fp8_32x128", "w4a16_fp8_64x128", "w4a16_fp8_128x256", "w4a16_fp8_256x256"}, names
    assert {n.split("_")[2] for n in names if n.endswith("splitk")} >= {"32x128", "64x128"}, names


def test_not_finite_rows():
    """An infinity or NaN in a row of x makes that row NaN and no other."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    for M, K, N in [(4, 256, 64), (200, 384, 300)]:
        x, xv = _rows((M, K), "bf16", 5)
        codes, scales, _ = _weight((), N, K, 6)
        y = w4.gemm_fp8(x, codes, scales)
        x[1, 7], x[3, 200] = float("inf"), float("nan")
        z = w4.gemm_fp8(x, codes, scales)
        assert bool(z[[1, 3]].isnan().all())
        keep = [m for m in range(M) if m not in (1, 3)]
        assert torch.equal(z[keep], y[keep])


# ------------------------------------------------------------------ grouped products

def _ids(tokens, topk, groups, seed, how="mixed"):
    g = synth.generator(seed)
    ids = g.integers(0, groups, size=(tokens, topk))
    if how == "mixed":
        ids = np.where(g.random((tokens, topk)) < 0.2, g.choice([-1, -7, groups, 2 ** 31 - 1], size=(tokens, topk)), ids)
    elif how == "one":
        ids[:] = groups - 1
    elif how == "none":
        ids[:] = -1
    elif how == "skewed":
        ids = np.minimum(ids, g.integers(0, groups, size=(tokens, topk)) // 3)
    return ids.astype(np.int32)


def _routed(ids, groups):
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    return w4.route(torch.from_numpy(ids).cuda(), groups), R.route_ref(ids, groups)


GROUPED = [
    # tokens, topk, groups, K, N2, how
    (1, 1, 1, 256, 64, "all"), (1, 2, 8, 512, 256, "all"), (5, 2, 3, 144, 96, "mixed"), (16, 4, 8, 640, 512, "mixed"),
    (33, 2, 7, 272, 160, "one"), (40, 1, 5, 256, 128, "none"), (64, 8, 64, 256, 96, "all"), (200, 3, 9, 528, 704, "mixed"),
    (300, 2, 4, 384, 288, "skewed"), (700, 2, 3, 256, 320, "mixed"),
]


def _each(ref, offsets, rows, values):
    """A per-group reference for the sorted rows, zeros past the last group; ``ref(rows, w)`` gives arrays."""
    n = int(offsets[-1])
    parts = [ref(rows[offsets[e]:offsets[e + 1]], w) for e, w in enumerate(values)]
    out = []
    for arrays in zip(*parts):
        a = np.concatenate(arrays)
        out.append(np.concatenate([a, np.zeros((len(rows) - n, a.shape[1]))]))
    return out


@pytest.mark.parametrize("tokens,topk,groups,K,N2,how", GROUPED)
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_grouped(tokens, topk, groups, K, N2, how, kind):
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    _announce(f"grouped {tokens}x{topk} groups={groups} K={K} N2={N2} {how} {kind}")
    r, (offsets, order, _) = _routed(_ids(tokens, topk, groups, tokens + K, how), groups)
    n = int(offsets[-1])
    x, xv = _rows((tokens, K), kind, tokens + N2)
    q, s = F.quantize_rows(xv)
    rows = F.rows_value(q, s)[order // topk]
    codes, scales, wv = _weight((groups,), N2, K, groups + N2, halves=1)

    ref, bound = _each(lambda v, w: (F.gemm_fp8_ref(v, w), _sum_bound(v, w, kind)), offsets, rows, wv)
    y = w4.gemm_fp8_grouped(x, r, codes, scales, gather=True)
    got = y.cpu().double().numpy()
    _within(got, ref, _stored(ref, bound, kind), "gathered")
    assert np.all(got[n:] == 0)
    # sorted rows and codes give the same bits
    xs = w4.dispatch(x, r)
    assert torch.equal(w4.gemm_fp8_grouped(xs, r, codes, scales), y)
    xq, xsc = w4.quantize_fp8(x)
    assert torch.equal(w4.gemm_fp8_grouped(xq, r, codes, scales, x_scales=xsc, gather=True, out_dtype=x.dtype), y)
    ref, bound = _each(lambda v, w: (F.gemm_fp8_ref(v, w), _sum_bound(v, w, "f32")), offsets, rows, wv)
    y = w4.gemm_fp8_grouped(x, r, codes, scales, gather=True, out_dtype=torch.float32)
    _within(y.cpu().double().numpy(), ref, _stored(ref, bound, "f32"), "fp32")

    codes, scales, wv = _weight((groups,), N2, K, groups + N2 + 1, halves=2)
    h, dh = _each(lambda v, w: _glu_bound(v, w, kind), offsets, rows, wv)
    _within(w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True).cpu().double().numpy(), h, _stored(h, dh, kind), "h")
    if N2 % 32 == 0:
        h, dh = _each(lambda v, w: _glu_bound(v, w, "f32"), offsets, rows, wv)
        hq, hs = w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True, quantized=True)
        _check_quantized(hq, hs, h, dh, "quantized h")
        assert not _bits(hq)[n:].any() and np.all(hs.cpu().numpy()[:, n:] == F.LEAST)


@pytest.mark.parametrize("tokens,topk,groups,K,N2", [(3000, 2, 5, 256, 2560), (4096, 1, 9, 144, 4096), (2500, 4, 20, 256, 1408)])
def test_grouped_on_large_tiles(tokens, topk, groups, K, N2):
    """Hundreds of rows a group: tiles of 256 rows that start at any multiple of 128 of the list."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    _announce(f"grouped {tokens}x{topk} groups={groups} K={K} N2={N2}, large tiles")
    r, (offsets, order, _) = _routed(_ids(tokens, topk, groups, tokens + K), groups)
    n, S = int(offsets[-1]), tokens * topk
    x, xv = _rows((tokens, K), "bf16", tokens)
    some = np.unique(np.concatenate([np.arange(0, S, 29), offsets[:-1], offsets[1:] - 1, [n, S - 1]]))
    some = some[some < S]
    rows = F.rows_value(*F.quantize_rows(xv[order[some] // topk]))
    at = np.searchsorted(some, offsets)  # the sampled rows' groups
    pick = torch.from_numpy(some).cuda()
    codes, scales, wv = _weight((groups,), N2, K, groups, halves=2)
    h, dh = _each(lambda v, w: _glu_bound(v, w, "bf16"), at, rows, wv)
    got = w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True)
    _within(got[pick].cpu().double().numpy(), h, _stored(h, dh, "bf16"), "h")
    assert bool((got[n:] == 0).all())
    h, dh = _each(lambda v, w: _glu_bound(v, w, "f32"), at, rows, wv)
    hq, hs = w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True, quantized=True)
    _check_quantized(hq.view(torch.uint8)[pick].view(torch.float8_e4m3fn), hs[:, pick], h, dh, "quantized h")
    assert not _bits(hq)[n:].any() and np.all(hs.cpu().numpy()[:, n:] == F.LEAST)
    codes, scales, wv = _weight((groups,), N2 + 8, K, groups + 1)
    ref, bound = _each(lambda v, w: (F.gemm_fp8_ref(v, w), _sum_bound(v, w, "bf16")), at, rows, wv)
    got = w4.gemm_fp8_grouped(x, r, codes, scales, gather=True)
    _within(got[pick].cpu().double().numpy(), ref, _stored(ref, bound, "bf16"), "product")


# ------------------------------------------------------------------ gradients

def _dw_bound(dy, x):
    """(dw, its bound) of dy[M, N] and x[M, K]: fp32 sums over M."""
    M = len(x)
    a, b = (F.rows_value(*F.quantize_columns(v)) for v in (dy, x))
    return a @ b.T, 2 * (M + 2) * EPS * (np.abs(a) @ np.abs(b).T) + 2 * EPS * np.abs(a @ b.T) + D["f32"]


@pytest.mark.parametrize("M,K,N", [(1, 16, 16), (7, 128, 144), (128, 256, 128), (129, 144, 272), (300, 400, 160), (515, 512, 640)])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_gradients(M, K, N, kind):
    import weight_only_int4_w4a16_amd as w4
    _announce(f"gemm_fp8_backward {M}x{K}x{N} {kind}")
    x, xv = _rows((M, K), kind, M + K)
    dy, dyv = _rows((M, N), kind, M + N)
    codes_t, scales_t, wt = _weight((), K, N, K + N)
    dx, dw = w4.gemm_fp8_backward(dy, x, codes_t, scales_t)
    v = F.rows_value(*F.quantize_rows(dyv))
    ref = F.gemm_fp8_ref(v, wt)
    _within(dx.cpu().double().numpy(), ref, _stored(ref, _sum_bound(v, wt, kind), kind), "dx")
    ref, bound = _dw_bound(dyv, xv)
    _within(dw.cpu().double().numpy(), ref, bound, "dw")


@pytest.mark.parametrize("M,K,N", [(1100, 144, 160), (2085, 256, 128), (5000, 272, 16), (9000, 272, 160), (4100, 48, 16), (40, 256, 8192), (3, 64, 16384)])
def test_gradients_with_few_tiles(M, K, N):
    """Deep products of few tiles, whose depth is cut: their partial sums have room of their own."""
    import weight_only_int4_w4a16_amd as w4
    _announce(f"gemm_fp8_backward {M}x{K}x{N}")
    x, xv = _rows((M, K), "bf16", M + K)
    dy, dyv = _rows((M, N), "bf16", M + N)
    codes_t, scales_t, wt = _weight((), K, N, K + N)
    dx, dw = w4.gemm_fp8_backward(dy, x, codes_t, scales_t)
    v = F.rows_value(*F.quantize_rows(dyv))
    ref = F.gemm_fp8_ref(v, wt)
    _within(dx.cpu().double().numpy(), ref, _stored(ref, _sum_bound(v, wt, "bf16"), "bf16"), "dx")
    ref, bound = _dw_bound(dyv, xv)
    _within(dw.cpu().double().numpy(), ref, bound, "dw")


@pytest.mark.parametrize("M,K,N", [(130, 144, 272), (1500, 128, 160)])
def test_one_gradient_alone(M, K, N):
    """A call for dx or dw alone (NULL for the other, and for what only that one reads) gives the bits of the call for both."""
    import weight_only_int4_w4a16_amd as w4
    from weight_only_int4_w4a16_amd import binding
    torch = torch_mod()
    L = binding.lib()
    x, _ = _rows((M, K), "bf16", M + K)
    dy, _ = _rows((M, N), "bf16", M + N)
    codes_t, scales_t, _ = _weight((), K, N, K + N)
    dx, dw = w4.gemm_fp8_backward(dy, x, codes_t, scales_t)
    s = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(L.w4a16_fp8_backward_workspace_bytes(M, K, N), dtype=torch.uint8, device="cuda")
    at = (ws.data_ptr(), ws.numel(), s)
    one, other = torch.full_like(dx, 7), torch.full_like(dw, 7)
    assert L.w4a16_gemm_fp8_backward(dy.data_ptr(), None, M, K, N, 1, codes_t.data_ptr(), scales_t.data_ptr(), one.data_ptr(), None, *at) == 0
    assert L.w4a16_gemm_fp8_backward(dy.data_ptr(), x.data_ptr(), M, K, N, 1, None, None, None, other.data_ptr(), *at) == 0
    assert np.array_equal(_bits(one), _bits(dx)) and np.array_equal(_bits(other), _bits(dw))
    r = w4.route(torch.arange(M, device="cuda", dtype=torch.int32).reshape(-1, 1) % 4, 3)
    codes_t, scales_t, _ = _weight((3,), K, N, K)
    dx, dw = w4.gemm_fp8_grouped_backward(dy, x, r, codes_t, scales_t)
    ws = torch.empty(L.w4a16_fp8_grouped_backward_workspace_bytes(M, 1, 3, K, N), dtype=torch.uint8, device="cuda")
    at = (ws.data_ptr(), ws.numel(), s)
    one, other = torch.full_like(dx, 7), torch.full_like(dw, 7)
    plan = (r.plan.data_ptr(), M, 1, 3, K, N, 1)
    assert L.w4a16_gemm_fp8_grouped_backward(dy.data_ptr(), None, *plan, codes_t.data_ptr(), scales_t.data_ptr(), one.data_ptr(), None, *at) == 0
    assert L.w4a16_gemm_fp8_grouped_backward(dy.data_ptr(), x.data_ptr(), *plan, None, None, None, other.data_ptr(), *at) == 0
    assert np.array_equal(_bits(one), _bits(dx)) and np.array_equal(_bits(other), _bits(dw))


def test_gradients_against_differences():
    """Operands that their codes hold exactly (small whole numbers, each group's largest 448 / 64): then the calls are
    the gradients of <dy, x W^T> and central differences of the product itself give them."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    g = synth.generator(11)
    M, K, N = 128, 128, 128

    def whole(shape):
        a = g.integers(-3, 4, size=shape).astype(np.float32)
        np.fill_diagonal(a, 7.0)  # every row and column of 128 has the largest: all scales are 1/64
        return a

    x, dy, w = whole((M, K)), whole((M, N)), whole((N, K))
    xt, dyt = (torch.from_numpy(a).cuda().bfloat16() for a in (x, dy))
    codes, scales, codes_t, scales_t = w4.quantize_fp8_weight(torch.from_numpy(w).cuda(), transposed=True)
    dx, dw = w4.gemm_fp8_backward(dyt, xt, codes_t, scales_t)

    def loss(a, c, s):
        return float((dyt.double() * w4.gemm_fp8(a, c, s, out_dtype=torch.float32).double()).sum())

    for at in [(0, 1), (100, 3), (127, 126)]:
        up, down = x.copy(), x.copy()
        up[at] += 2
        down[at] -= 2
        got = (loss(torch.from_numpy(up).cuda().bfloat16(), codes, scales) - loss(torch.from_numpy(down).cuda().bfloat16(), codes, scales)) / 4
        assert abs(got - float(dx[at])) <= 2.0 ** -8 * abs(got) + 1e-3  # dx is rounded to bf16
        up, down = w.copy(), w.copy()
        up[at] += 2
        down[at] -= 2
        got = (loss(xt, *w4.quantize_fp8_weight(torch.from_numpy(up).cuda())) - loss(xt, *w4.quantize_fp8_weight(torch.from_numpy(down).cuda()))) / 4
        assert abs(got - float(dw[at])) <= 1e-3


@pytest.mark.parametrize("tokens,topk,groups,K,N,how", [
    (1, 1, 1, 16, 16, "all"), (9, 2, 4, 144, 128, "mixed"), (100, 2, 3, 256, 272, "mixed"), (200, 1, 5, 128, 160, "none"),
    (260, 1, 3, 272, 128, "one"), (300, 4, 9, 256, 144, "skewed"), (600, 2, 2, 512, 256, "all"),
])
def test_grouped_gradients(tokens, topk, groups, K, N, how):
    import weight_only_int4_w4a16_amd as w4
    _announce(f"grouped backward {tokens}x{topk} groups={groups} {K}x{N} {how}")
    r, (offsets, _, _) = _routed(_ids(tokens, topk, groups, tokens, how), groups)
    n, S = int(offsets[-1]), tokens * topk
    x, xv = _rows((S, K), "bf16", tokens + K)
    dy, dyv = _rows((S, N), "bf16", tokens + N)
    x[n:], dy[n:] = float("nan"), float("inf")  # rows of no group reach nothing
    codes_t, scales_t, wt = _weight((groups,), K, N, K + N)
    dx, dw = w4.gemm_fp8_grouped_backward(dy, x, r, codes_t, scales_t)
    v = F.rows_value(*F.quantize_rows(np.where(np.arange(S)[:, None] < n, dyv, 0)))
    ref, bound = _each(lambda a, w: (F.gemm_fp8_ref(a, w), _sum_bound(a, w, "bf16")), offsets, v, wt)
    got = dx.cpu().double().numpy()
    _within(got, ref, _stored(ref, bound, "bf16"), "dx")
    assert np.all(got[n:] == 0)
    dw = dw.cpu().double().numpy()
    for e in range(groups):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            assert np.all(dw[e] == 0)
        else:
            ref, bound = _dw_bound(dyv[a:b], xv[a:b])
            _within(dw[e], ref, bound, f"dw of group {e}")


def test_no_rows():
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    codes, scales, _ = _weight((), 64, 128, 1)
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    assert w4.gemm_fp8(x, codes, scales).shape == (0, 64)
    assert w4.quantize_fp8(x)[0].shape == (0, 128) and w4.quantize_fp8_columns(x)[0].shape == (128, 0)
    dx, dw = w4.gemm_fp8_backward(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), x, *_weight((), 128, 64, 2)[:2])
    assert dx.shape == (0, 128) and dw.shape == (64, 128) and bool((dw == 0).all())
    r = w4.route(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 3)
    codes, scales, _ = _weight((3,), 64, 128, 3)
    assert w4.gemm_fp8_grouped(x, r, codes, scales, gather=True).shape == (0, 64)
    dx, dw = w4.gemm_fp8_grouped_backward(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), x, r, *_weight((3,), 128, 64, 4)[:2])
    assert dw.shape == (3, 64, 128) and bool((dw == 0).all())


# ------------------------------------------------------------------ offsets past 32 bits

def test_rows_of_more_than_2_to_the_32_values():
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    M, K = 262500, 16384
    assert M * K > 2 ** 32
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    last, lv = _rows((5, K), "bf16", 1)
    x[-5:] = last
    codes, scales = w4.quantize_fp8(x)
    q, s = F.quantize_rows(lv)
    assert np.array_equal(_bits(codes[-5:]), q) and np.array_equal(scales[:, -5:].cpu().numpy(), s)
    assert not bool(codes[:16].view(torch.uint8).any())
    del codes, scales
    codes, scales = w4.quantize_fp8_columns(x)
    q, s = F.quantize_columns(np.concatenate([np.zeros((M % 128 - 5, 64), np.float32), lv[:, :64]]))
    assert np.array_equal(_bits(codes[:64, M // 128 * 128:M]), q[:, :M % 128])
    assert np.array_equal(scales[-1, :64].cpu().numpy(), s[0])


def test_a_product_of_more_than_2_to_the_32_results():
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    M, K, N = 134300, 128, 32008
    assert M * N > 2 ** 32
    x, xv = _rows((300, K), "bf16", 1)
    codes, scales, wv = _weight((), N, K, 2)
    big = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    big[-300:] = x
    y = w4.gemm_fp8(big, codes, scales)
    v = F.rows_value(*F.quantize_rows(xv))
    ref = F.gemm_fp8_ref(v, wv)
    _within(y[-300:].cpu().double().numpy(), ref, _stored(ref, _sum_bound(v, wv, "bf16"), "bf16"), "last rows")
    assert not bool(y[:1000].any())


@pytest.mark.parametrize("M", [1, 9, 16, 25, 40, 64])
def test_weights_read_past_the_caches(M):
    """Weights of 128 MiB and more, plain, SwiGLU and routed: some columns of each."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    K, N = 4096, 33000
    g = torch.Generator(device="cuda").manual_seed(M)
    codes = torch.randint(0, 0x48, (N, K), dtype=torch.uint8, device="cuda", generator=g)
    codes[::3] += 128  # and negative ones
    scales = torch.rand(-(-N // 128), K // 128, device="cuda", generator=g) / 64 + 2.0 ** -7
    x, xv = _rows((M, K), "bf16", M)
    v = F.rows_value(*F.quantize_rows(xv))
    w8 = codes.view(torch.float8_e4m3fn)

    def rows_of(s, half, n):  # values of n rows of the weight from row 128 b of a half on
        at, b = half * (N // 2) if half is not None else 0, n[0] // 128
        c = codes[at + 128 * b:at + 128 * b + len(n)].cpu().numpy()
        return F.weight_value(c, s[b:b + 1].cpu().numpy())

    for dtype in ("bf16", "f32"):
        y = w4.gemm_fp8(x, w8, scales, out_dtype=_dtype(dtype))
        for b in (0, 100, N // 128):
            n = np.arange(128 * b, min(128 * b + 128, N))
            wv = rows_of(scales, None, n)
            ref = F.gemm_fp8_ref(v, wv)
            _within(y[:, n[0]:n[-1] + 1].cpu().double().numpy(), ref, _stored(ref, _sum_bound(v, wv, dtype), dtype), f"{dtype}, block {b}")
    half = -(-N // 256)
    gs, us = (torch.rand(half, K // 128, device="cuda", generator=g) / 4096 + 2.0 ** -13 for _ in range(2))
    h = w4.gemm_fp8_swiglu(x, w8, torch.cat([gs, us]))
    for b in (0, 60, half - 1):
        n = np.arange(128 * b, min(128 * b + 128, N // 2))
        wv = np.concatenate([rows_of(gs, 0, n), rows_of(us, 1, n)])
        ref, bound = _glu_bound(v, wv, "bf16")
        _within(h[:, n[0]:n[-1] + 1].cpu().double().numpy(), ref, _stored(ref, bound, "bf16"), f"h, block {b}")
    if M < 16:
        return
    E = 3  # 11000 rows each
    r = w4.route(torch.arange(M, device="cuda", dtype=torch.int32).reshape(-1, 1) % E, E)
    es = torch.rand(E, -(-11000 // 128), K // 128, device="cuda", generator=g) / 64 + 2.0 ** -7
    y = w4.gemm_fp8_grouped(x, r, w8.view(E, 11000, K), es, gather=True)
    first = 0
    for e in range(E):
        mine = v[e::E]
        wv = F.weight_value(codes[11000 * e + 128:11000 * e + 256].cpu().numpy(), es[e, 1:2].cpu().numpy())
        ref = F.gemm_fp8_ref(mine, wv)
        _within(y[first:first + len(mine), 128:256].cpu().double().numpy(), ref, _stored(ref, _sum_bound(mine, wv, "bf16"), "bf16"), f"group {e}")
        first += len(mine)


def test_experts_of_more_than_2_to_the_32_codes():
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    E, N, K = 33, 8192, 16384
    assert E * N * K > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    for e in range(E):  # magnitudes up to 4: no NaN among them
        codes[e] = torch.randint(0, 0x48, (N, K), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.rand(E, N // 128, K // 128, device="cuda", generator=g) + 0.5
    x, xv = _rows((60, K), "bf16", 4)
    ids = torch.tensor([0, 16, 32] * 20, dtype=torch.int32, device="cuda").reshape(-1, 1)
    r = w4.route(ids, E)
    y = w4.gemm_fp8_grouped(x, r, codes.view(torch.float8_e4m3fn), scales, gather=True)
    v = F.rows_value(*F.quantize_rows(xv))
    for i, e in enumerate([0, 16, 32]):
        wv = F.weight_value(codes[e, -128:].cpu().numpy(), scales[e, -1:].cpu().numpy())[28:]
        ref = F.gemm_fp8_ref(v[i::3], wv)
        got = y[20 * i:20 * i + 20, -100:].cpu().double().numpy()
        _within(got, ref, _stored(ref, _sum_bound(v[i::3], wv, "bf16"), "bf16"), f"group {e}")


# ------------------------------------------------------------------ as they are used

def test_expert_layer_and_its_replays():
    """Routed rows through their experts' projections and back to their tokens, on a stream of its own and from a graph."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    tokens, topk, E, K, inner = 50, 2, 6, 256, 192
    ids = torch.from_numpy(_ids(tokens, topk, E, 3)).cuda()
    x, xv = _rows((tokens, K), "bf16", 4)
    gate = torch.rand(tokens, topk, device="cuda")
    up, ups, upv = _weight((E,), 2 * inner, K, 5, halves=2)
    down, downs, downv = _weight((E,), K, inner, 6)
    y = torch.empty(tokens, K, dtype=torch.bfloat16, device="cuda")

    def layer():
        r = w4.route(ids, E)
        h, hs = w4.gemm_fp8_grouped_swiglu(x, r, up, ups, gather=True, quantized=True)
        w4.combine(w4.gemm_fp8_grouped(h, r, down, downs, x_scales=hs, out_dtype=torch.float32), r, gate, out_dtype=torch.bfloat16, out=y)

    layer()
    offsets, order, slot = R.route_ref(ids.cpu().numpy(), E)
    rows = F.rows_value(*F.quantize_rows(xv))[order // topk]
    h, = _each(lambda v, w: (F.swiglu_fp8_ref(v, w),), offsets, rows, upv)
    ys, = _each(lambda v, w: (F.gemm_fp8_ref(v, w),), offsets, F.rows_value(*F.quantize_rows(h.astype(np.float32))), downv)
    ref = R.combine_ref(ys, slot, gate.cpu().numpy())
    got = y.cpu().double().numpy()
    # a value of h near the middle between two codes may fall either way: a step of 2^-3 in one of 192 terms
    assert np.linalg.norm(got - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    assert_graph_replays_match_eager(layer, [y])
    first = y.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y.zero_()
        layer()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, first)


def test_training_step_replays():
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    M, K, N = 140, 256, 272
    w = torch.randn(N, K, device="cuda")
    x, _ = _rows((M, K), "bf16", 1)
    dy, _ = _rows((M, N), "bf16", 2)
    out = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, K, dtype=torch.bfloat16, device="cuda"),
           torch.empty(N, K, device="cuda")]

    def step():
        c, s, ct, st = w4.quantize_fp8_weight(w, transposed=True)
        w4.gemm_fp8(x, c, s, out=out[0])
        dx, dw = w4.gemm_fp8_backward(dy, x, ct, st)
        out[1].copy_(dx)
        out[2].copy_(dw)

    assert_graph_replays_match_eager(step, out)


def test_two_streams_at_once():
    """Calls on two streams, each with torch's own scratch, give what they give alone."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    sets = []
    for i, (M, K, N) in enumerate([(40, 512, 640), (300, 256, 512)]):
        x, _ = _rows((M, K), "bf16", i)
        codes, scales, _ = _weight((), N, K, i + 5)
        sets.append((x, codes, scales, w4.gemm_fp8(x, codes, scales)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(20):
        for i, (x, codes, scales, _) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(w4.gemm_fp8(x, codes, scales))
    torch.cuda.synchronize()
    for i, s in enumerate(sets):
        assert all(torch.equal(y, s[3]) for y in got[i])


GUARD = 4096


def _guarded(shape, dtype):
    """An uninitialised tensor with bytes behind it that a call must leave alone, and a check of them."""
    torch = torch_mod()
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf[:n].view(dtype).view(shape), lambda what: bool((buf[n:] == 0xA5).all()) or pytest.fail(f"{what}: written past the end")


@pytest.mark.parametrize("M,K,N", [(1, 4096, 300), (2, 512, 4), (5, 1040, 36), (16, 512, 1000), (20, 8192, 1020), (20, 512, 100), (40, 4096, 300), (64, 8208, 404),
                                   (100, 2048, 132), (333, 2896, 700), (300, 256, 1001), (257, 4096, 516), (2049, 256, 1300)])
def test_nothing_past_the_ends(M, K, N):
    """Outputs and workspaces of exactly the bytes they need, with bytes behind them that stay."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    x, _ = _rows((M, K), "bf16", M + N)
    codes, scales, _ = _weight((), N, K, N)
    q, s = w4.quantize_fp8(x)
    for a, xs in ((x, None), (q, s)):
        for dtype in (torch.bfloat16, torch.float32):
            want = w4.gemm_fp8(a, codes, scales, x_scales=xs, out_dtype=dtype)
            out, out_ends = _guarded((M, N), dtype)
            ws, ws_ends = _guarded((max(1, w4.fp8_workspace_bytes(M, K, N, a.dtype)),), torch.uint8)
            w4.gemm_fp8(a, codes, scales, x_scales=xs, out=out, workspace=ws)
            out_ends(f"out {dtype}"), ws_ends(f"workspace {dtype}")
            assert torch.equal(out, want)


@pytest.mark.parametrize("M,K,N", [(3, 64, 16384), (40, 256, 8192), (333, 272, 144), (9000, 272, 160)])
def test_gradients_stay_in_their_workspace(M, K, N):
    import weight_only_int4_w4a16_amd as w4
    from weight_only_int4_w4a16_amd import binding
    torch = torch_mod()
    L = binding.lib()
    x, _ = _rows((M, K), "bf16", 1)
    dy, _ = _rows((M, N), "bf16", 2)
    codes_t, scales_t, _ = _weight((), K, N, 3)
    dx, dw = w4.gemm_fp8_backward(dy, x, codes_t, scales_t)
    ws, ends = _guarded((L.w4a16_fp8_backward_workspace_bytes(M, K, N),), torch.uint8)
    a, b = w4.gemm_fp8_backward(dy, x, codes_t, scales_t, workspace=ws)
    ends("workspace")
    assert torch.equal(a, dx) and torch.equal(b, dw)
    if M > 1000:
        return
    r = w4.route(torch.arange(M, device="cuda", dtype=torch.int32).reshape(-1, 1) % 4, 3)
    codes_t, scales_t, _ = _weight((3,), K, N, 4)
    dx, dw = w4.gemm_fp8_grouped_backward(dy, x, r, codes_t, scales_t)
    ws, ends = _guarded((L.w4a16_fp8_grouped_backward_workspace_bytes(M, 1, 3, K, N),), torch.uint8)
    a, b = w4.gemm_fp8_grouped_backward(dy, x, r, codes_t, scales_t, workspace=ws)
    ends("workspace of routed rows")
    assert torch.equal(a, dx) and torch.equal(b, dw)


def test_routed_products_stay_in_their_ends():
    import weight_only_int4_w4a16_amd as w4
    from weight_only_int4_w4a16_amd import binding
    torch = torch_mod()
    L = binding.lib()
    for tokens, topk, E, K, N2 in [(7, 2, 3, 144, 96), (100, 2, 4, 256, 288), (600, 1, 2, 128, 416)]:
        r = w4.route(torch.from_numpy(_ids(tokens, topk, E, tokens)).cuda(), E)
        x, _ = _rows((tokens, K), "bf16", 1)
        codes, scales, _ = _weight((E,), N2, K, 2, halves=2)
        S = tokens * topk
        for dtype, n in ((torch.bfloat16, 1), (torch.float32, 2)):
            want = w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True, out_dtype=dtype)
            out, ends = _guarded((S, N2 // 2), dtype)
            ws, ws_ends = _guarded((L.w4a16_fp8_grouped_workspace_bytes(tokens, topk, E, 1, K, N2, 1, 1, n),), torch.uint8)
            w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True, out=out, workspace=ws)
            ends("out"), ws_ends("workspace")
            assert torch.equal(out, want)
        want = w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True, quantized=True)
        ws, ws_ends = _guarded((L.w4a16_fp8_grouped_workspace_bytes(tokens, topk, E, 1, K, N2, 1, 1, 3),), torch.uint8)
        got = w4.gemm_fp8_grouped_swiglu(x, r, codes, scales, gather=True, quantized=True, workspace=ws)
        ws_ends("workspace")
        assert np.array_equal(_bits(got[0]), _bits(want[0])) and torch.equal(got[1], want[1])


def test_caller_workspace_and_refusals_on_the_device():
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    x, _ = _rows((9, 256), "f16", 1)
    codes, scales, _ = _weight((), 96, 256, 2)
    y = w4.gemm_fp8(x, codes, scales)
    need = w4.fp8_workspace_bytes(9, 256, 96, x.dtype)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(w4.gemm_fp8(x, codes, scales, workspace=ws), y)

    def refused(fn, match):
        with pytest.raises(w4.W4A16Error, match=match):
            fn()

    refused(lambda: w4.gemm_fp8(x, codes, scales, workspace=ws[:-1]), "workspace")
    refused(lambda: w4.gemm_fp8(x, codes.view(torch.uint8), scales), "dtype")
    refused(lambda: w4.gemm_fp8(x, codes[:, :128], scales), "shape")
    refused(lambda: w4.gemm_fp8(x, codes, scales.double()), "dtype")
    refused(lambda: w4.gemm_fp8(x, codes, scales[:, :1]), "shape")
    refused(lambda: w4.gemm_fp8(x, codes, scales, x_scales=scales), "x_scales")
    refused(lambda: w4.gemm_fp8(x, codes, scales, out_dtype=torch.bfloat16), "out dtype")
    refused(lambda: w4.gemm_fp8(x, codes, scales, out=y[:, :8]), "shape")
    refused(lambda: w4.gemm_fp8(x[:, :200].contiguous(), codes[:, :200].contiguous(), scales), "unsupported")
    refused(lambda: w4.gemm_fp8_swiglu(x, codes, scales), "shape")  # the halves' blocks are their own
    refused(lambda: w4.gemm_fp8_swiglu(x, codes[:95], scales), "even")
    q, s = w4.quantize_fp8(x)
    refused(lambda: w4.gemm_fp8(q, codes, scales), "x_scales")
    refused(lambda: w4.gemm_fp8(q, codes, scales, x_scales=s[:1]), "shape")
    refused(lambda: w4.gemm_fp8_backward(x, x, codes, scales), "shape|codes_t")
    r = w4.route(torch.zeros(9, 1, dtype=torch.int32, device="cuda"), 2)
    refused(lambda: w4.gemm_fp8_grouped(x, r, codes, scales), "3-D")
    refused(lambda: w4.gemm_fp8_grouped(x[:8], r, codes[None], scales[None]), "rows")
    refused(lambda: w4.gemm_fp8_grouped(x, r, codes[None], scales[None]), "shape")
