"""GPU checks of the routed kernels' forms that few shapes reach, against the fp64 oracle with the bounds of
test_gpu_routed.py: the 128 x 512 tile of the grouped products, the eight waves that share a deep K, fp32 rows
combined to 16 bits past the caches."""
import numpy as np
import pytest

from weight_only_int4_w4a16_amd import synth

from gpu_common import require_gpu, torch_mod
from test_gpu_routed import D, EPS, U, _announce, _check_grouped, _dtype, _experts, _ids, _routed, _rows, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _kernel(rows, K, N, groups, g):
    import weight_only_int4_w4a16_amd as w4
    name = w4.grouped_kernel_name(rows, K, N, groups, g)
    _announce(f"grouped rows={rows} K={K} N={N} groups={groups} g={g} {name}")
    return name


@pytest.mark.parametrize("act,fmt,g,K,glu", [
    ("f16", "asym", 32, 1440, False), ("bf16", "asym", 64, 1472, False), ("bf16", "sym", 32, 1440, True),
    ("f16", "nf4", 64, 1472, True), ("bf16", "nf4", 32, 1440, True), ("f16", "sym", 128, 1536, False),
])
def test_grouped_on_the_128_row_tile(act, fmt, g, K, glu):
    """Part-filled tiles, a ragged last block of K and column tile, rows of no group; both ways to read x."""
    assert _kernel(2100, K, 7584, 2, g) == "w4a16_grouped_128x512"
    _check_grouped(2100, 1, 2, K, 7584, g, act, fmt, glu, gather=fmt != "asym")


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("fmt,g,K", [("asym", 32, 8224), ("asym", 64, 8256), ("sym", 128, 8320), ("sym", 32, 8224),
                                     ("nf4", 64, 8256), ("nf4", 32, 8224)])
@pytest.mark.parametrize("glu", [False, True])
def test_grouped_deep_k_over_eight_waves(act, fmt, g, K, glu):
    """65 blocks of K, the last ragged, in eight shares that are not all as long."""
    assert _kernel(9, K, 96, 3, g) == "w4a16_grouped_16x64"
    _check_grouped(9, 1, 3, K, 96, g, act, fmt, glu, gather=not glu)


@pytest.mark.parametrize("width", [4096, 4001])  # whole cache lines and not
@pytest.mark.parametrize("to", ["f16", "bf16"])
def test_combine_of_fp32_rows_past_the_caches_to_16_bits(to, width):
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    _announce(f"combine 2100x2 width={width} f32 -> {to}")
    ids = _ids(2100, 2, 5, 3)
    r, (offsets, _, _) = _routed(ids, 5)
    ys, _ = _rows((4200, width), "f32", 4)
    ys[int(offsets[-1]):] = float("nan")
    w = torch.rand(2100, 2, device="cuda")
    y32 = w4.combine(ys, r, w)
    assert np.isfinite(y32.cpu().numpy()).all()
    assert torch.equal(w4.combine(ys, r, w, out_dtype=_dtype(to)), y32.to(_dtype(to)))


# Outputs of more than 2^32 elements: every offset from a row number has to be a 64-bit one. Rows near the ends and the
# places where 31 and 32 bits of elements or bytes end are checked.

def _samples(rows, width, seed):
    g = synth.generator(seed)
    at = [0, 1, rows - 1, rows - 2] + [v // width + d for v in (2 ** 30, 2 ** 31, 2 ** 32) for d in (-1, 0, 1)]
    return np.unique([p for p in at + g.integers(0, rows, size=40).tolist() if 0 <= p < rows])


def test_rows_of_more_than_32_bits_of_elements():
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    tokens, topk, groups, width = 66000, 8, 7, 8200
    _announce(f"rows {tokens}x{topk} width={width}")
    ids = _ids(tokens, topk, groups, 91)
    r, (offsets, order, slot) = _routed(ids, groups)
    n = int(offsets[-1])
    x = torch.randn(tokens, width, device="cuda", dtype=torch.bfloat16)
    xs = w4.dispatch(x, r)
    assert xs.numel() > 2 ** 32
    for a in range(0, tokens * topk, 1 << 16):
        b = min(a + (1 << 16), tokens * topk)
        want = x[torch.from_numpy(order[a:b] // topk).cuda().long()]
        want[max(n - a, 0):] = 0
        assert torch.equal(xs[a:b], want), f"rows {a} to {b}"
    # x itself times the sum of its live weights, powers of two whose sums of eight are exact
    w = torch.from_numpy(2.0 ** synth.generator(92).integers(-3, 3, size=(tokens, topk))).float().cuda()
    total = torch.where(torch.from_numpy(slot >= 0).cuda(), w, 0).sum(1, keepdim=True)
    assert torch.equal(w4.combine(xs, r, w), (x.float() * total).bfloat16())
    dys, dw = w4.combine_backward(x, xs, r, w)
    for t in _samples(tokens, width, 93):
        for j in range(topk):
            p = int(slot[t, j])
            if p < 0:
                assert float(dw[t, j]) == 0
                continue
            assert torch.equal(dys[p], (x[t].float() * w[t, j]).bfloat16())
            square = float((x[t].double() ** 2).sum())
            assert abs(float(dw[t, j]) - square) <= 2 * width * 2.0 ** -24 * square
    assert not dys[n:].any()


@pytest.mark.parametrize("K,kernel", [(32, "w4a16_grouped_64x64"), (2048, "w4a16_grouped_128x512")])
def test_grouped_of_more_than_32_bits_of_elements(K, kernel):
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    rows, groups, N, g = 2 ** 19 + 21, 3, 8208, 32
    if K > 32:
        g = 128
    assert _kernel(rows, K, N, groups, g) == kernel
    d, w = _experts(K, N, g, "f16", "asym", groups, 95)
    ids = _ids(rows, 1, groups, 96)
    r, (offsets, order, _) = _routed(ids, groups)
    n = int(offsets[-1])
    x = torch.randn(rows, K, device="cuda", dtype=torch.float16)
    y = w4.gemm_grouped(x, r, d["packed"], d["scales"], d["tail"], g)
    assert y.numel() > 2 ** 32 and not y[n:].any()
    for p in _samples(rows, N, 97):
        if p >= n:
            continue
        e = int(ids[order[p], 0])
        xv = x[p].cpu().double().numpy()
        ref, mag = xv @ w[e], np.abs(xv) @ np.abs(w[e])
        dsum = 2 * K * EPS * mag
        _within(y[p].cpu().double().numpy(), ref, dsum + U["f16"] * (np.abs(ref) + dsum) + D["f16"], f"row {p}")


def test_adapters_of_more_than_32_bits_of_elements():
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    M, K, N, L, rank = 2 ** 18 + 37, 64, 16400, 3, 8
    _announce(f"lora M={M} K={K} N={N}")
    ids = np.repeat(np.array([1, -1, 0, 2], dtype=np.int32), [100001, 777, 120005, M - 100001 - 777 - 120005])
    x = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    y = torch.randn(M, N, device="cuda", dtype=torch.bfloat16)
    a = torch.randn(L, rank, K, device="cuda").mul_(K ** -0.5).bfloat16()
    b = torch.randn(L, N, rank, device="cuda").mul_(rank ** -0.5).bfloat16()
    s = torch.tensor([0.5, 1.25, 2.0], device="cuda")
    out = w4.lora_add(y, x, a, b, torch.from_numpy(ids).cuda(), s)
    assert out.numel() > 2 ** 32
    av, bv = a.cpu().double().numpy(), b.cpu().double().numpy()
    for m in np.append(_samples(M, N, 98), [100000, 100001, 100777, 100778]):
        e, yv = int(ids[m]), y[m].cpu().double().numpy()
        got = out[m].cpu().double().numpy()
        if e < 0:
            assert np.array_equal(got, yv)
            continue
        xv, sv = x[m].cpu().double().numpy(), float(s[e])
        t = av[e] @ xv
        ref = yv + sv * (bv[e] @ t)
        dt = 2 * K * EPS * (np.abs(av[e]) @ np.abs(xv))
        dt = dt + 2.0 ** -16 * (np.abs(t) + dt).max()
        mag = np.abs(bv[e]) @ (np.abs(t) + dt)
        bound = sv * (np.abs(bv[e]) @ dt + 2 * 3 * (rank + 2) * EPS * mag) + 4 * EPS * (np.abs(yv) + sv * mag)
        _within(got, ref, bound + U["bf16"] * (np.abs(ref) + bound) + D["bf16"], f"row {m}")
