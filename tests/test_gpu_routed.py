"""GPU checks of the routed operators against the fp64 oracle (oracle/routed.py).

Bounds, elementwise, from the arithmetic the kernels document (eps the fp32 unit roundoff 2^-24,
u the output type's, 2^-11 fp16 and 2^-8 bf16, d half the type's least subnormal):

* a sum of n fp32 terms is off by at most 2 n eps times the sum of the terms' magnitudes (one
  rounding for each product and one for each addition), whatever its order;
* storing in a 16-bit type adds u |value| + d;
* SwiGLU of sums off by dg, du: |dh| <= 1.1 dg |u| + (|SiLU(g)| + 1.1 dg) du, and the fp32
  exponential, division and products add (|g| + 8) 2^-22 |h|;
* an adapter's t, split into 16-bit parts, is off by 2^-21 max|t| (fp16, two parts), 2^-16 |t|
  (bf16, two) or 2^-23 |t| (bf16, three), whichever the largest |t| of the row bounds.
"""
import numpy as np
import pytest

import oracle
from oracle import routed as R
from weight_only_int4_w4a16_amd import synth

from gpu_common import assert_graph_replays_match_eager, from_dev, out_values, require_gpu, rtn_case, to_dev, torch_mod

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


def _rows(shape, kind, seed, scale=1.0):
    """(device tensor, its fp64 values) of normal rows."""
    torch = torch_mod()
    a = (synth.generator(seed).standard_normal(shape) * scale).astype(np.float32)
    t = torch.from_numpy(a).cuda().to(_dtype(kind))
    return t, t.cpu().double().numpy()


def _ids(tokens, topk, groups, seed, how="mixed"):
    g = synth.generator(seed)
    ids = g.integers(0, groups, size=(tokens, topk))
    if how == "mixed":  # some of no group, on both sides of the range
        ids = np.where(g.random((tokens, topk)) < 0.2, g.choice([-1, -7, groups, 2 ** 31 - 1], size=(tokens, topk)), ids)
    elif how == "one":
        ids[:] = groups - 1
    elif how == "none":
        ids[:] = -1
    elif how == "skewed":
        ids = np.minimum(ids, g.integers(0, groups, size=(tokens, topk)) // 3)
    elif how == "steps":  # 1, 16, 17, 32, 33 .. rows, the rest in the last group: every share of a tile
        ids = np.repeat(np.arange(groups), [16 * (e // 2) + (1 if e % 2 == 0 else 16) for e in range(groups)])[:tokens * topk]
        ids = np.concatenate([ids, np.full(tokens * topk - len(ids), groups - 1)])
        ids = ids[g.permutation(len(ids))].reshape(tokens, topk)
    return ids.astype(np.int32)


def _within(got, ref, bound, what):
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    over = np.abs(got - ref) - bound
    assert np.all(over <= 0), f"{what}: off by {np.abs(got - ref).max():.3e}, {over.max():.3e} past the bound"


def _routed(ids, groups):
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    r = w4.route(torch.from_numpy(ids).cuda(), groups)
    torch.cuda.synchronize()
    return r, R.route_ref(ids, groups)


# ------------------------------------------------------------------ the plan

@pytest.mark.parametrize("tokens,topk,groups,how", [
    (0, 2, 4, "all"), (1, 1, 1, "all"), (1, 2, 8, "all"), (1, 1, 1024, "mixed"), (7, 3, 5, "mixed"),
    (16, 4, 8, "none"), (33, 2, 7, "one"), (64, 8, 64, "all"), (100, 1, 63, "skewed"),
    (1000, 3, 64, "mixed"), (4095, 2, 1024, "mixed"), (8192, 1, 3, "mixed"),   # one workgroup
    (8193, 1, 3, "mixed"), (20011, 4, 130, "skewed"), (40000, 1, 1024, "mixed"), (9000, 2, 5, "none"),
    (256, 2, 9, "mixed"), (257, 2, 9, "mixed"), (4096, 1, 70, "mixed"), (4097, 1, 70, "mixed"),
    (200000, 1, 1024, "mixed"),                                                # counts scanned by a kernel
])
def test_route_is_the_stable_sort(tokens, topk, groups, how):
    _announce(f"route {tokens}x{topk} groups={groups} {how}")
    ids = _ids(tokens, topk, groups, tokens + groups, how)
    r, (offsets, order, slot) = _routed(ids, groups)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.order.cpu().numpy(), order)
    assert np.array_equal(r.slot.cpu().numpy(), slot)
    # behind them the sorted rows' tokens (the order itself for topk 1), then the lists of row tiles
    plan, S = r.plan.cpu().numpy(), tokens * topk
    up = lambda n: (n + 63) // 64 * 64
    at = up(groups + 1) + 2 * up(S)
    if topk > 1:
        assert np.array_equal(plan[at:at + S], order // topk)
        at += up(S)
    bounds = np.append(offsets, S)  # the slots of no group are the last
    for rows in (16, 32, 64, 128):
        want = [(e, p, min(p + rows, bounds[e + 1]), 0) for e in range(groups + 1)
                for p in range(bounds[e], bounds[e + 1], rows)]
        assert plan[at] == len(want)
        assert np.array_equal(plan[at + 4:at + 4 + 4 * len(want)].reshape(-1, 4), np.array(want, np.int32).reshape(-1, 4))
        at += up(4 + 4 * (S // rows + min(groups + 1, S)))


# ------------------------------------------------------------------ rows into order and back

ROW_CASES = [
    (1, 1, 1, 8, "f16"), (1, 2, 8, 4096, "bf16"), (5, 2, 3, 1, "f16"), (9, 3, 4, 7, "bf16"), (40, 2, 6, 2885, "bf16"),
    (17, 8, 64, 1030, "f16"), (70, 4, 16, 512, "f32"), (33, 5, 9, 1027, "f32"), (12, 9, 11, 264, "f16"),
    (300, 1, 40, 2048, "bf16"),
    # narrower than a vector, just wider, and one wave's share and one element
    (7, 3, 4, 3, "f32"), (6, 6, 5, 2, "bf16"), (8, 8, 3, 5, "f32"), (10, 4, 5, 9, "f16"), (21, 6, 4, 1025, "f16"),
    # sorted rows past the size where they are streamed, in whole cache lines and not
    (8256, 2, 5, 2048, "bf16"), (4200, 2, 9, 4001, "f16"), (4200, 1, 3, 4096, "f32"),
]


@pytest.mark.parametrize("tokens,topk,groups,width,kind", ROW_CASES)
def test_rows_into_order_and_back(tokens, topk, groups, width, kind):
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    _announce(f"rows {tokens}x{topk} groups={groups} width={width} {kind}")
    seed = tokens * 7 + width
    ids = _ids(tokens, topk, groups, seed)
    r, (offsets, order, slot) = _routed(ids, groups)
    n = int(offsets[-1])
    x, xv = _rows((tokens, width), kind, seed + 1)
    ys, ysv = _rows((tokens * topk, width), kind, seed + 2)
    dy, dyv = _rows((tokens, width), kind, seed + 3)
    # what belongs to no group must not reach any result
    ys[n:] = float("nan")
    w = synth.generator(seed + 4).random((tokens, topk)).astype(np.float32) - 0.3
    w[slot < 0] = np.nan
    wt = torch.from_numpy(w).cuda()

    xs = w4.dispatch(x, r)
    assert np.array_equal(xs.cpu().double().numpy(), R.dispatch_ref(xv, offsets, order, topk))

    y = w4.combine(ys, r, wt).cpu().double().numpy()
    live = slot >= 0
    mag = R.combine_ref(np.abs(ysv), slot, np.abs(w))
    ref = R.combine_ref(ysv, slot, w)
    _within(y, ref, 2 * topk * EPS * mag + U[kind] * np.abs(ref) * (1 + 2 * topk * EPS) + D[kind] + U[kind] * 2 * topk * EPS * mag, "y")

    dys, dw = w4.combine_backward(dy, ys, r, wt)
    rdys, rdw = R.combine_backward_ref(dyv, ysv, slot, w)
    _within(dys.cpu().double().numpy(), rdys, (U[kind] + 2 * EPS) * np.abs(rdys) + D[kind], "dys")
    _, mdw = R.combine_backward_ref(np.abs(dyv), np.abs(ysv), slot, np.abs(w))
    _within(dw.cpu().double().numpy(), rdw, 2 * width * EPS * mdw, "dweights")
    assert np.all(dw.cpu().numpy()[~live] == 0)

    dxs, dxsv = _rows((tokens * topk, width), kind, seed + 5)
    dxs[n:] = float("inf")
    dx = w4.dispatch_backward(dxs, r).cpu().double().numpy()
    ref = R.dispatch_backward_ref(dxsv, slot)
    mag = R.dispatch_backward_ref(np.abs(dxsv), slot)
    _within(dx, ref, 2 * topk * EPS * mag * (1 + U[kind]) + U[kind] * np.abs(ref) + D[kind], "dx")


@pytest.mark.parametrize("width", [333, 3, 6])
@pytest.mark.parametrize("to", ["f16", "bf16"])
def test_combine_of_fp32_rows_to_16_bits(to, width):
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    ids = _ids(30, 2, 5, 3)
    r, (_, _, slot) = _routed(ids, 5)
    ys, _ = _rows((60, width), "f32", 4)
    w = torch.rand(30, 2, device="cuda")
    y32 = w4.combine(ys, r, w)
    y16 = w4.combine(ys, r, w, out_dtype=_dtype(to))
    assert torch.equal(y16, y32.to(_dtype(to)))  # the same sums, rounded once


def test_rows_at_odd_addresses():
    """Rows that start two bytes after a 16-byte boundary."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    ids = _ids(20, 2, 5, 9)
    r, (offsets, order, slot) = _routed(ids, 5)
    buf = torch.randn(20 * 72 + 1, device="cuda").to(torch.bfloat16)
    x = buf[1:].view(20, 72)
    out = torch.empty(40 * 72 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(40, 72)
    w4.dispatch(x, r, out=out)
    assert np.array_equal(out.cpu().double().numpy(), R.dispatch_ref(x.cpu().double().numpy(), offsets, order, 2))
    w = torch.ones(20, 2, device="cuda")
    assert torch.equal(w4.combine(out, r, w), w4.dispatch_backward(out, r))


def test_gradients_against_differences():
    """combine is linear in ys and in weights, dispatch in x: a difference quotient of fp32 rows is the
    derivative up to the rounding of the sums (2 n eps of their magnitudes, divided by the step)."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    tokens, topk, groups, width, h = 11, 3, 4, 37, 0.5
    ids = _ids(tokens, topk, groups, 21)
    r, (offsets, _, slot) = _routed(ids, groups)
    n = int(offsets[-1])
    ys, _ = _rows((tokens * topk, width), "f32", 22)
    dy, dyv = _rows((tokens, width), "f32", 23)
    step, _ = _rows((tokens * topk, width), "f32", 24)
    w = torch.rand(tokens, topk, device="cuda")
    dys, dw = w4.combine_backward(dy, ys, r, w)

    def loss(ys, w):
        return float((w4.combine(ys, r, w).double() * dy.double()).sum())

    terms = float((w4.combine(ys.abs() + h * step.abs(), r, w).double() * dy.abs().double()).sum())
    tol = 4 * (2 * topk + 2) * EPS * terms / h
    got = (loss(ys + h * step, w) - loss(ys - h * step, w)) / (2 * h)
    assert abs(got - float((dys[:n].double() * step[:n].double()).sum())) <= tol + 4 * EPS * terms / h
    for t, j in [(0, 0), (5, 1), (10, 2)]:
        e = torch.zeros_like(w)
        e[t, j] = h
        got = (loss(ys, w + e) - loss(ys, w - e)) / (2 * h)
        assert abs(got - float(dw[t, j])) <= 4 * (2 * topk + 2 + width) * EPS * (terms + float(dy.abs().sum())) / h
    # dispatch: <dxs, dispatch(x)> has the gradient dispatch_backward(dxs)
    x, _ = _rows((tokens, width), "f32", 25)
    dxs, _ = _rows((tokens * topk, width), "f32", 26)
    dxs[n:] = 0
    left = float((w4.dispatch(x, r).double() * dxs.double()).sum())
    right = float((w4.dispatch_backward(dxs, r).double() * x.double()).sum())
    assert abs(left - right) <= 2 * topk * EPS * float((w4.dispatch(x.abs(), r).double() * dxs.abs().double()).sum())


# ------------------------------------------------------------------ the groups' products

def _experts(K, N, g, act, fmt, groups, seed):
    """Device operands of `groups` quantized weights and their W_hat as fp64."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    cases = [rtn_case(1, K, N, g, act, sym=fmt == "sym", seed=seed + 10 * e, nf4=fmt == "nf4") for e in range(groups)]
    kind = "f16" if fmt == "nf4" else act
    qw = torch.stack([to_dev(c["qweight"], "i32") for c in cases])
    d = {"packed": w4.pack_grouped(qw), "scales": torch.stack([to_dev(c["scales"], kind) for c in cases])}
    d["tail"] = to_dev(cases[0]["codebook"], "f16") if fmt == "nf4" else (
        torch.stack([to_dev(c["qzeros"], "i32") for c in cases]) if fmt == "asym" else None)
    w = [oracle.bf16_bits_to_f64(c["w_hat"]) if act == "bf16" else c["w_hat"].astype(np.float64) for c in cases]
    return d, w


def _grouped_call(fmt, glu):
    import weight_only_int4_w4a16_amd as w4
    return {(False, False): w4.gemm_grouped, (False, True): w4.gemm_grouped_swiglu,
            (True, False): w4.gemm_grouped_nf4, (True, True): w4.gemm_grouped_nf4_swiglu}[(fmt == "nf4", glu)]


def _check_grouped(tokens, topk, groups, K, N, g, act, fmt, glu, gather, how="mixed"):
    torch = torch_mod()
    import weight_only_int4_w4a16_amd as w4
    name = w4.grouped_kernel_name(tokens * topk, K, N, groups, g)
    _announce(f"grouped {tokens}x{topk} E={groups} K={K} N={N} g={g} {act} {fmt} glu={glu} gather={gather} {how} {name}")
    seed = tokens + K + N
    d, w = _experts(K, N, g, act, fmt, groups, seed)
    ids = _ids(tokens, topk, groups, seed + 5, how)
    r, (offsets, order, _) = _routed(ids, groups)
    n = int(offsets[-1])
    x, xv = _rows((tokens if gather else tokens * topk, K), act, seed + 6)
    rows = xv[order // topk] if gather else xv
    call = _grouped_call(fmt, glu)
    y = call(x, r, d["packed"], d["scales"], d["tail"], g, gather=gather, out_dtype=torch.float32)
    got = y.cpu().double().numpy()
    ref = R.grouped_ref(rows, offsets, w, glu)
    mag = R.grouped_ref(np.abs(rows), offsets, [np.abs(v) for v in w])
    dsum = 2 * K * EPS * mag
    if glu:
        plain = R.grouped_ref(rows, offsets, w)
        gate, up = oracle.swiglu_split(plain)
        dg, du = oracle.swiglu_split(dsum)
        bound = 1.1 * dg * np.abs(up) + (np.abs(oracle.silu(gate)) + 1.1 * dg) * du + (np.abs(gate) + 8) * 2.0 ** -22 * np.abs(ref)
    else:
        bound = dsum
    _within(got, ref, bound + 1e-30, "fp32 output")
    assert np.all(got[n:] == 0)
    # the 16-bit output is the fp32 one rounded once, and runs repeat bit for bit
    z = call(x, r, d["packed"], d["scales"], d["tail"], g, gather=gather)
    assert torch.equal(z, y.to(_dtype(act)))
    assert torch.equal(y, call(x, r, d["packed"], d["scales"], d["tail"], g, gather=gather, out_dtype=torch.float32))


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("fmt,g", [("asym", 32), ("asym", 64), ("asym", 128), ("sym", 32), ("sym", 64), ("sym", 128),
                                   ("nf4", 32), ("nf4", 64), ("nf4", 128)])
@pytest.mark.parametrize("glu", [False, True])
def test_grouped_every_format(act, fmt, g, glu):
    _check_grouped(20, 2, 5, 384, 96, g, act, fmt, glu, gather=True)


@pytest.mark.parametrize("tokens,topk,groups,K,N,g,how", [
    (1, 1, 1, 32, 16, 32, "all"),        # the least of everything
    (1, 2, 8, 1024, 512, 128, "all"),    # one token
    (3, 1, 4, 352, 48, 32, "mixed"),     # K not a multiple of 128, N not of a tile
    (16, 1, 1, 256, 80, 64, "one"), (17, 1, 1, 256, 80, 64, "one"), (33, 1, 2, 416, 144, 32, "one"),
    (9, 3, 200, 256, 64, 128, "all"),    # most groups empty
    (24, 2, 3, 2048, 272, 128, "none"),  # no row at all has a group
    (150, 2, 4, 512, 320, 128, "skewed"), (400, 2, 3, 1184, 560, 32, "mixed"), (700, 1, 2, 640, 1040, 64, "skewed"),
    (64, 2, 2, 4224, 64, 128, "mixed"),
    (5, 1, 2, 8320, 96, 128, "all"),                                              # a deep K over eight waves
    (500, 1, 8, 160, 12560, 32, "mixed"),                                         # 64-row tiles, waves side by side
    (2100, 1, 2, 160, 4112, 32, "mixed"),                                         # 128-row tiles
])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_sizes(tokens, topk, groups, K, N, g, how, gather):
    _check_grouped(tokens, topk, groups, K, N, g, "f16", "asym", False, gather, how)


@pytest.mark.parametrize("tokens,groups,K,N", [(40, 1, 512, 96), (200, 2, 352, 608), (600, 3, 640, 1056)])
@pytest.mark.parametrize("act,fmt,g", [("bf16", "asym", 32), ("f16", "sym", 32), ("bf16", "nf4", 64 // 2)])
def test_grouped_more_rows(tokens, groups, K, N, act, fmt, g):
    _check_grouped(tokens, 1, groups, K, N, g, act, fmt, True, gather=False)


@pytest.mark.parametrize("act,fmt,g", [("bf16", "asym", 64), ("bf16", "sym", 32), ("f16", "nf4", 64), ("bf16", "nf4", 32)])
@pytest.mark.parametrize("tokens,groups,K,N", [(500, 8, 192, 12576), (2100, 2, 192, 4128)])
def test_grouped_many_rows_in_every_format(tokens, groups, K, N, act, fmt, g):
    _check_grouped(tokens, 1, groups, K, N, g, act, fmt, fmt != "asym", gather=True)


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("fmt,g", [("asym", 32), ("asym", 64), ("sym", 32), ("sym", 128), ("nf4", 32), ("nf4", 64)])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("tokens,groups", [(70, 4), (330, 8)])  # tiles of 32 and of 64 rows
def test_grouped_every_share_of_a_tile(tokens, groups, act, fmt, g, glu):
    _check_grouped(tokens, 1, groups, 384, 96, g, act, fmt, glu, False, "steps")


@pytest.mark.parametrize("act,fmt,g,glu", [("f16", "asym", 64, False), ("f16", "nf4", 64, True), ("bf16", "sym", 128, True),
                                           ("bf16", "nf4", 32, False)])
def test_grouped_every_share_of_a_tile_side_by_side(act, fmt, g, glu):
    _check_grouped(500, 1, 8, 256, 12576, g, act, fmt, glu, True, "steps")


def test_no_tokens():
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    d, _ = _experts(256, 64, 128, "f16", "asym", 3, 7)
    r = w4.route(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 3)
    assert r.offsets.tolist() == [0, 0, 0, 0] and r.order.numel() == 0 and r.slot.shape == (0, 2)
    x, w = torch.zeros(0, 256, device="cuda").half(), torch.zeros(0, 2, device="cuda")
    assert w4.dispatch(x, r).shape == (0, 256) and w4.dispatch_backward(x, r).shape == (0, 256)
    assert w4.combine(x, r, w).shape == (0, 256) and w4.combine_backward(x, x, r, w)[1].shape == (0, 2)
    assert w4.gemm_grouped(x, r, d["packed"], d["scales"], d["tail"], 128, gather=True).shape == (0, 64)
    a, b = torch.zeros(2, 8, 256, device="cuda").half(), torch.zeros(2, 64, 8, device="cuda").half()
    y = w4.lora_add(x[:, :64].contiguous(), x, a, b, torch.zeros(0, dtype=torch.int32, device="cuda"), torch.ones(2, device="cuda"))
    assert y.shape == (0, 64)


def test_grouped_rows_do_not_mix():
    """A NaN or an infinity in a token stays in that token's rows."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    for tokens in (5, 60, 300):
        d, _ = _experts(256, 64, 128, "f16", "asym", 3, 7)
        ids = _ids(tokens, 2, 3, 8)
        r, (offsets, order, _) = _routed(ids, 3)
        x, _ = _rows((tokens, 256), "f16", 9)
        clean = w4.gemm_grouped(x, r, d["packed"], d["scales"], d["tail"], 128, gather=True)
        bad = x.clone()
        bad[2] = float("nan")
        bad[4] = float("inf")
        y = w4.gemm_grouped(bad, r, d["packed"], d["scales"], d["tail"], 128, gather=True)
        keep = torch.from_numpy(~np.isin(order // 2, [2, 4])).cuda()
        assert torch.equal(y[keep], clean[keep])


# ------------------------------------------------------------------ adapters

def _check_lora(M, K, N, L, rank, act, ykind, ids, seed, scale=1.0, planned=False, alias=False):
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    _announce(f"lora M={M} K={K} N={N} L={L} R={rank} {act}->{ykind} planned={planned} alias={alias}")
    x, xv = _rows((M, K), act, seed, scale)
    y, yv = _rows((M, N), ykind, seed + 1, scale)
    a, av = _rows((L, rank, K), act, seed + 2, K ** -0.5)
    b, bv = _rows((L, N, rank), act, seed + 3, rank ** -0.5)
    s = (synth.generator(seed + 4).random(L) + 0.25).astype(np.float32)
    idt, st = torch.from_numpy(ids).cuda(), torch.from_numpy(s).cuda()
    out = y.clone() if alias else None
    got = w4.lora_add(out if alias else y, x, a, b, idt, st, routing=w4.route(idt, L) if planned else None, out=out)
    got = got.cpu().double().numpy()
    ref = R.lora_ref(yv, xv, av, bv, ids, s)
    bound = np.zeros((M, N))
    for m, e in enumerate(ids.tolist()):
        if 0 <= e < L:
            t = np.abs(av[e] @ xv[m])
            dt = 2 * K * EPS * (np.abs(av[e]) @ np.abs(xv[m]))
            split = 2.0 ** -21 if act == "f16" else 2.0 ** -16 if ykind == "bf16" else 2.0 ** -23
            dt = dt + split * (t + dt).max()
            mag = np.abs(bv[e]) @ (t + dt)
            bound[m] = s[e] * (np.abs(bv[e]) @ dt + 2 * 3 * (rank + 2) * EPS * mag) + 4 * EPS * (np.abs(yv[m]) + s[e] * mag)
    bound += U[ykind] * (np.abs(ref) + bound) + D[ykind]
    bound[[not 0 <= e < L for e in ids.tolist()]] = 0  # rows of no adapter are y itself
    _within(got, ref, bound, "out")


@pytest.mark.parametrize("act,ykind", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("M,K,N,L,rank", [
    (1, 32, 16, 1, 8), (1, 1024, 512, 8, 16), (5, 352, 80, 3, 24), (130, 256, 272, 64, 32), (100, 4096, 144, 2, 40),
    (300, 512, 336, 4, 64), (77, 288, 112, 5, 72), (50, 256, 64, 3, 256), (700, 192, 528, 2, 136),
])
def test_lora_every_size(M, K, N, L, rank, act, ykind):
    ids = _ids(M, 1, L, M + rank)[:, 0].copy()
    _check_lora(M, K, N, L, rank, act, ykind, ids, M + N, planned=M % 2 == 0)


@pytest.mark.parametrize("how", ["none", "one", "skewed", "all"])
def test_lora_ids(how):
    ids = _ids(90, 1, 6, 5, how)[:, 0].copy()
    _check_lora(90, 256, 208, 6, 16, "bf16", "bf16", ids, 31)
    _check_lora(90, 256, 208, 6, 16, "f16", "f16", ids, 32, alias=True)


def test_lora_runs_of_rows():
    """Prefill: long runs of one request's rows."""
    ids = np.repeat(np.array([2, -1, 0, 2, 1], dtype=np.int32), [333, 40, 7, 290, 130])
    _check_lora(800, 1024, 400, 3, 64, "bf16", "bf16", ids, 41)
    _check_lora(800, 1024, 400, 3, 32, "f16", "f16", ids, 42, planned=True)


@pytest.mark.parametrize("act,ykind,N,rank", [("bf16", "bf16", 16288, 16), ("f16", "f32", 8208, 40), ("f16", "f16", 16288, 8)])
def test_lora_of_rows_past_the_caches(act, ykind, N, rank):
    """So many rows that y and out are streamed, in place as well."""
    ids = np.repeat(np.array([1, -1, 0, 2], dtype=np.int32), [1001, 30, 333, 700])
    _check_lora(2064, 128, N, 3, rank, act, ykind, ids, 43, alias=ykind == "f16")


@pytest.mark.parametrize("scale", [2.0 ** -12, 2.0 ** 9])
def test_lora_scales_of_t(scale):
    """t far from 1: its fp16 parts are taken on a power-of-two scale."""
    ids = _ids(20, 1, 3, 6, "all")[:, 0].copy()
    _check_lora(20, 512, 96, 3, 16, "f16", "f32", ids, 51, scale=scale)


def test_lora_rows_do_not_mix():
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    for M in (6, 200):
        x, _ = _rows((M, 256), "f16", 61)
        y, _ = _rows((M, 64), "f16", 62)
        a, _ = _rows((2, 16, 256), "f16", 63, 0.06)
        b, _ = _rows((2, 64, 16), "f16", 64, 0.25)
        ids = torch.from_numpy(_ids(M, 1, 2, 65, "all")[:, 0].copy()).cuda()
        s = torch.ones(2, device="cuda")
        clean = w4.lora_add(y, x, a, b, ids, s)
        x[1] = float("nan")
        x[3] = float("inf")
        got = w4.lora_add(y, x, a, b, ids, s)
        keep = [m for m in range(M) if m not in (1, 3)]
        assert torch.equal(got[keep], clean[keep])
        assert not torch.isfinite(got[1].float()).any()


# ------------------------------------------------------------------ streams and graphs

def test_one_layer_in_a_graph_and_on_a_side_stream():
    """A layer of routed experts with adapters on the shared projection, captured and replayed."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    tokens, topk, groups, K, I = 24, 2, 4, 256, 192
    up, _ = _experts(K, 2 * I, 64, "bf16", "sym", groups, 71)
    down, _ = _experts(I, K, 64, "bf16", "sym", groups, 72)
    ids = torch.from_numpy(_ids(tokens, topk, groups, 73)).cuda()
    x, _ = _rows((tokens, K), "bf16", 74)
    w = torch.rand(tokens, topk, device="cuda")
    a, _ = _rows((3, 8, K), "bf16", 75, 0.06)
    b, _ = _rows((3, K, 8), "bf16", 76, 0.3)
    aid = torch.from_numpy(_ids(tokens, 1, 3, 77)[:, 0].copy()).cuda()
    s = torch.ones(3, device="cuda")
    y = torch.empty(tokens, K, device="cuda", dtype=torch.bfloat16)
    z = torch.empty_like(y)
    dys, dw = torch.empty(tokens * topk, K, device="cuda", dtype=torch.bfloat16), torch.empty_like(w)

    def step():
        r = w4.route(ids, groups)
        h = w4.gemm_grouped_swiglu(x, r, up["packed"], up["scales"], None, 64, gather=True)
        e = w4.gemm_grouped(h, r, down["packed"], down["scales"], None, 64)
        w4.combine(e, r, w, out=y)
        w4.lora_add(y, x, a, b, aid, s, out=z)
        g = w4.combine_backward(x, e, r, w)
        dys.copy_(g[0])
        dw.copy_(g[1])

    assert_graph_replays_match_eager(step, [y, z, dys, dw])
    step()
    torch.cuda.synchronize()
    eager = [t.clone() for t in (y, z, dys, dw)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    for t, e in zip((y, z, dys, dw), eager):
        assert torch.equal(t, e)


def test_the_example_layer():
    """The example runs the operators together; five roundings to bf16 (y, its adapter's sum, h, e and z; 2^-9 each in
    the mean square, and h's and e's gains near one) keep the whole within 5 * 2^-9 of fp64."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import routed_layer
    assert routed_layer.main(rows=40, width=512, inner=256, experts=5, adapters=3, rank=8) < 5 * 2.0 ** -9


# ------------------------------------------------------------------ refusals that need device tensors

def test_refusals_on_the_device():
    """Checked on the host before anything is launched."""
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    M, K, N, L, rank = 4, 64, 48, 3, 8
    x, y = torch.zeros(M, K, device="cuda").half(), torch.zeros(M, N, device="cuda").half()
    a, b = torch.zeros(L, rank, K, device="cuda").half(), torch.zeros(L, N, rank, device="cuda").half()
    ids, s = torch.zeros(M, device="cuda", dtype=torch.int32), torch.ones(L, device="cuda")

    def refused(match, fn):
        with pytest.raises(w4.W4A16Error, match=match):
            fn()

    refused("lora_b", lambda: w4.lora_add(y, x, a, b[:, :, :4].contiguous(), ids, s))
    refused("lora_a", lambda: w4.lora_add(y, x, a.float(), b, ids, s))
    refused("ids", lambda: w4.lora_add(y, x, a, b, ids.long(), s))
    refused("ids", lambda: w4.lora_add(y, x, a, b, None, s))
    refused("scaling", lambda: w4.lora_add(y, x, a, b, ids, s[:2]))
    refused("out", lambda: w4.lora_add(y, x, a, b, ids, s, out=y.float()))
    refused("routing", lambda: w4.lora_add(y, x, a, b, ids, s, routing=w4.route(ids, L + 1)))
    refused("unsupported", lambda: w4.lora_add(y[:, :24].contiguous(), x, a, b[:, :24].contiguous(), ids, s))
    r = w4.route(ids, L)
    refused("expected", lambda: w4.dispatch(x.cpu(), r))
    refused("expected", lambda: w4.combine(y, r, torch.ones(M, 1)))
    refused("overlaps", lambda: w4.dispatch_backward(x, r, out=x))
    big = torch.zeros(3 * M, N, device="cuda").half()
    refused("overlaps", lambda: w4.lora_add(big[:M], x, a, b, ids, s, out=big[1:M + 1]))
    refused("unsupported", lambda: w4.route(ids, 1025))
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    refused("bytes", lambda: w4.lora_add(y, x, a, b, None, s, routing=r, workspace=ws))
