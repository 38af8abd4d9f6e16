"""CPU checks of the routed operators: the oracle against brute force and differences, and the refusals of the
C ABI and of the binding (nothing is launched)."""
import ctypes

import numpy as np
import pytest

from oracle import routed as R

ids_cases = [np.array([[2, 0], [1, 2], [-1, 5], [0, 0]]), np.zeros((0, 3), dtype=int), np.full((3, 2), 9)]


# ------------------------------------------------------------------ oracle

@pytest.mark.parametrize("ids", ids_cases)
def test_route_ref_is_numpys_stable_sort(ids):
    offsets, order, slot = R.route_ref(ids, 3)
    key = np.where((ids >= 0) & (ids < 3), ids, 3).reshape(-1)
    assert np.array_equal(order, np.argsort(key, kind="stable"))
    assert np.array_equal(offsets, np.searchsorted(np.sort(key), np.arange(4)))
    flat = slot.reshape(-1)
    assert np.array_equal(flat < 0, key == 3)
    assert all(order[p] == i for i, p in enumerate(flat) if p >= 0)


def test_rows_go_there_and_back():
    g = np.random.default_rng(0)
    ids = ids_cases[0]
    offsets, order, slot = R.route_ref(ids, 3)
    x = g.standard_normal((4, 5))
    xs = R.dispatch_ref(x, offsets, order, 2)
    # weights that sum to one over a token's live slots give the token back
    live = slot >= 0
    w = live / np.maximum(live.sum(1, keepdims=True), 1)
    assert np.allclose(R.combine_ref(xs, slot, w)[live.any(1)], x[live.any(1)], rtol=0, atol=1e-15)


def test_gradients_against_differences():
    """Both moves are linear, so central differences are exact up to fp64 rounding."""
    g = np.random.default_rng(1)
    ids = g.integers(-1, 4, size=(6, 3))
    offsets, order, slot = R.route_ref(ids, 4)
    x, dxs = g.standard_normal((6, 4)), g.standard_normal((18, 4))
    ys, dy, w = g.standard_normal((18, 4)), g.standard_normal((6, 4)), g.standard_normal((6, 3))
    n = int(offsets[-1])
    dys, dw = R.combine_backward_ref(dy, ys, slot, w)
    dx = R.dispatch_backward_ref(dxs, slot)

    def diff(f, a, at, h=0.25):
        up, down = a.copy(), a.copy()
        up[at] += h
        down[at] -= h
        return (f(up) - f(down)) / (2 * h)

    for at in [(0, 0), (n - 1, 3), (17, 1)]:
        assert abs(diff(lambda v: np.sum(dy * R.combine_ref(v, slot, w)), ys, at) - dys[at]) < 1e-12
    for at in [(0, 0), (3, 2), (5, 1)]:
        assert abs(diff(lambda v: np.sum(dy * R.combine_ref(ys, slot, v)), w, at) - dw[at]) < 1e-12
        assert abs(diff(lambda v: np.sum(dxs[:n] * R.dispatch_ref(v, offsets, order, 3)[:n]), x, at) - dx[at]) < 1e-12


def test_grouped_and_adapters_by_loops():
    g = np.random.default_rng(2)
    ids = np.array([[1], [0], [-1], [1]])
    offsets, order, _ = R.route_ref(ids, 2)
    x = g.standard_normal((4, 6))
    w = [g.standard_normal((6, 4)) for _ in range(2)]
    out = R.grouped_ref(x[order], offsets, w)
    for p, i in enumerate(order):
        want = np.zeros(4) if ids[i, 0] < 0 else np.array([sum(x[i, k] * w[ids[i, 0]][k, n] for k in range(6)) for n in range(4)])
        assert np.allclose(out[p], want, rtol=0, atol=1e-13)
    h = R.grouped_ref(x[order], offsets, w, glu=True)
    gate, up = out[:, :2], out[:, 2:]
    assert np.allclose(h, gate / (1 + np.exp(-gate)) * up, rtol=1e-14, atol=0)
    a, b, s = g.standard_normal((2, 3, 6)), g.standard_normal((2, 4, 3)), [2.0, 0.5]
    y = g.standard_normal((4, 4))
    got = R.lora_ref(y, x, a, b, ids[:, 0], s)
    for m, e in enumerate(ids[:, 0]):
        want = y[m] if e < 0 else y[m] + s[e] * (b[e] @ (a[e] @ x[m]))
        assert np.allclose(got[m], want, rtol=0, atol=1e-13)


# ------------------------------------------------------------------ refusals of the C ABI

@pytest.fixture(scope="module")
def L():
    from weight_only_int4_w4a16_amd import binding
    return binding.lib()


OK, ARG, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
P = 1 << 20  # aligned placeholder addresses, never dereferenced
Q = P + 4096


def test_plan_sizes(L):
    assert L.w4a16_route_bytes(-1, 2, 8) == 0 and L.w4a16_route_bytes(4, 0, 8) == 0
    assert L.w4a16_route_bytes(4, 2, 0) == 0 and L.w4a16_route_bytes(4, 2, 1025) == 0
    assert L.w4a16_route_bytes(1 << 26, 2, 8) == 0
    # offsets, order and slot at their documented places, within the plan
    for tokens, topk, groups in [(0, 1, 1), (1, 2, 8), (5000, 3, 1024)]:
        r = lambda n: -(-n // 64) * 64  # noqa: E731
        assert L.w4a16_route_bytes(tokens, topk, groups) >= 4 * (r(groups + 1) + 2 * r(tokens * topk))


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), ARG), (dict(topk=0), ARG), (dict(groups=0), ARG), (dict(groups=1025), UNSUPPORTED),
    (dict(tokens=1 << 26), UNSUPPORTED), (dict(ids=0), ARG), (dict(ids=P + 2), ARG),
    (dict(plan=0), WORKSPACE), (dict(plan=P + 64), WORKSPACE), (dict(nbytes=255), WORKSPACE),
])
def test_route_refuses(L, kw, status):
    a = dict(ids=P, tokens=4, topk=2, groups=8, plan=Q, nbytes=1 << 20)
    a.update(kw)
    assert L.w4a16_route(a["ids"] or None, a["tokens"], a["topk"], a["groups"], a["plan"] or None, a["nbytes"], None) == status


ROWS = dict(src=P, plan=Q, tokens=4, topk=2, groups=8, width=64, dtype=1, dst=P + (1 << 16), w=P + (1 << 18), out_dtype=1,
            dw=P + (1 << 19), dy=P + (1 << 17))


def _rows_call(L, name, a):
    head = (a["plan"] or None, a["tokens"], a["topk"], a["groups"])
    if name in ("dispatch", "dispatch_backward"):
        return getattr(L, "w4a16_" + name)(a["src"] or None, *head, a["width"], a["dtype"], a["dst"] or None, None)
    if name == "combine":
        return L.w4a16_combine(a["src"] or None, *head, a["w"] or None, a["width"], a["dtype"], a["dst"] or None, a["out_dtype"], None)
    return L.w4a16_combine_backward(a["dy"] or None, a["src"] or None, *head, a["w"] or None, a["width"], a["dtype"],
                                    a["dst"] or None, a["dw"] or None, None)


@pytest.mark.parametrize("name", ["dispatch", "dispatch_backward", "combine", "combine_backward"])
@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), ARG), (dict(topk=0), ARG), (dict(groups=1025), UNSUPPORTED), (dict(width=0), ARG),
    (dict(dtype=3), ARG), (dict(src=0), ARG), (dict(dst=0), ARG), (dict(plan=0), ARG), (dict(plan=Q + 4), ARG),
    (dict(src=P + 1), ARG), (dict(dst=P), ARG), (dict(tokens=1 << 25, width=1 << 20), UNSUPPORTED),
    (dict(tokens=1 << 24, topk=1, width=8), UNSUPPORTED),
])
def test_rows_refuse(L, name, kw, status):
    assert _rows_call(L, name, {**ROWS, **kw}) == status


@pytest.mark.parametrize("name,kw", [
    ("combine", dict(w=0)), ("combine", dict(w=P + 2)), ("combine", dict(out_dtype=2)), ("combine", dict(dtype=0, out_dtype=1)),
    ("combine_backward", dict(w=0)), ("combine_backward", dict(dy=0)), ("combine_backward", dict(dw=0)),
    ("combine_backward", dict(dst=P + (1 << 17))),
])
def test_weighted_rows_refuse(L, name, kw):
    assert _rows_call(L, name, {**ROWS, **kw}) == ARG


@pytest.mark.parametrize("name", ["dispatch", "dispatch_backward", "combine", "combine_backward"])
def test_rows_of_no_tokens_are_a_noop(L, name):
    assert _rows_call(L, name, {**ROWS, "tokens": 0, "src": 0, "dst": 0, "plan": 0, "dy": 0, "dw": 0}) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(K=100), ARG), (dict(K=96, g=128), ARG), (dict(g=48), ARG), (dict(N=4100), ARG), (dict(N=4104), UNSUPPORTED),
    (dict(act=2), ARG), (dict(act=0, odt=1), ARG), (dict(glu=1, N=4112), UNSUPPORTED), (dict(tokens=-1), ARG),
    (dict(groups=0), ARG), (dict(topk=0), ARG), (dict(x=0), ARG), (dict(x=P + 8), ARG), (dict(plan=0), ARG),
    (dict(packed=0), ARG), (dict(scales=0), ARG), (dict(out=0), ARG), (dict(qzeros=P + 2), ARG),
    (dict(tokens=1 << 18, gather=1), UNSUPPORTED),  # 2 GiB of rows read in place
])
def test_grouped_refuses(L, kw, status):
    a = dict(x=P, plan=Q, tokens=4, topk=2, groups=8, gather=0, K=4096, N=4096, act=0, packed=P, scales=P, qzeros=P, g=128,
             glu=0, out=P, odt=0)
    a.update(kw)
    got = L.w4a16_gemm_grouped(a["x"] or None, a["plan"] or None, a["tokens"], a["topk"], a["groups"], a["gather"], a["K"],
                               a["N"], a["act"], a["packed"] or None, a["scales"] or None, a["qzeros"], a["g"], a["glu"],
                               a["out"] or None, a["odt"], None)
    assert got == status


def test_grouped_nf4_needs_a_codebook(L):
    assert L.w4a16_gemm_grouped_nf4(P, Q, 4, 2, 8, 0, 4096, 4096, 0, P, P, None, 64, 0, P, 0, None) == ARG
    assert L.w4a16_gemm_grouped_nf4(P, Q, 0, 2, 8, 0, 4096, 4096, 0, None, None, None, 64, 0, None, 0, None) == OK


def test_grouped_kernel_names(L):
    import weight_only_int4_w4a16_amd as w4
    assert w4.grouped_kernel_name(0, 4096, 4096, 8, 128) == "none"
    assert w4.grouped_kernel_name(16, 100, 4096, 8, 128) == "none"
    # the tile grows with the rows a group can expect
    names = [w4.grouped_kernel_name(8 * m, 4096, 14336, 8, 128) for m in (1, 20, 100, 1000)]
    assert names == ["w4a16_grouped_16x64", "w4a16_grouped_32x64", "w4a16_grouped_64x64", "w4a16_grouped_128x512"]


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), ARG), (dict(K=100), ARG), (dict(K=4104), UNSUPPORTED), (dict(N=4100), ARG), (dict(N=4104), UNSUPPORTED),
    (dict(rank=0), ARG), (dict(rank=12), UNSUPPORTED), (dict(rank=264), UNSUPPORTED), (dict(adapters=0), ARG),
    (dict(adapters=1025), UNSUPPORTED), (dict(M=1 << 26, N=1 << 20), UNSUPPORTED), (dict(act=2), ARG), (dict(act=0, ydt=1), ARG), (dict(x=0), ARG), (dict(y=0), ARG),
    (dict(a=0), ARG), (dict(b=0), ARG), (dict(ids=0), ARG), (dict(scaling=0), ARG), (dict(out=0), ARG),
    (dict(x=P + 8), ARG), (dict(out=P + 8), ARG), (dict(ids=P + 2), ARG), (dict(plan=Q + 4), ARG),
    (dict(ws=0), WORKSPACE), (dict(ws=Q + 64), WORKSPACE), (dict(wsb=64), WORKSPACE),
])
def test_lora_refuses(L, kw, status):
    v = dict(x=P, y=P, M=300, K=4096, N=4096, act=0, ydt=0, a=P, b=P, adapters=8, rank=16, ids=P, scaling=P, plan=0, out=P,
             ws=Q, wsb=1 << 30)
    v.update(kw)
    n = lambda k: v[k] or None  # noqa: E731
    got = L.w4a16_lora_add(n("x"), n("y"), v["M"], v["K"], v["N"], v["act"], v["ydt"], n("a"), n("b"), v["adapters"], v["rank"],
                           n("ids"), n("scaling"), n("plan"), n("out"), n("ws"), v["wsb"], None)
    assert got == status


def test_lora_of_no_rows_is_a_noop(L):
    assert L.w4a16_lora_add(None, None, 0, 4096, 4096, 0, 0, None, None, 8, 16, None, None, None, None, None, 0, None) == OK


# ------------------------------------------------------------------ refusals of the binding

def _raises(fn, match):
    from weight_only_int4_w4a16_amd import W4A16Error
    with pytest.raises(W4A16Error, match=match) as e:
        fn()
    assert e.value.status in (ARG, UNSUPPORTED)


def _routing(tokens, topk, groups):
    """A plan's object on the CPU: enough for the checks, which come before any launch."""
    import torch
    import weight_only_int4_w4a16_amd as w4
    n = w4.lib().w4a16_route_bytes(tokens, topk, groups) // 4
    return w4.Routing(torch.zeros(n, dtype=torch.int32), tokens, topk, groups)


def test_route_binding_refuses():
    import torch
    import weight_only_int4_w4a16_amd as w4
    ids = torch.zeros(4, 2, dtype=torch.int32)
    _raises(lambda: w4.route(ids, 8), "device")                       # a CPU tensor
    _raises(lambda: w4.route(ids.long(), 8), "int32")
    _raises(lambda: w4.route(ids[None], 8), "int32")
    _raises(lambda: w4.route(ids.t(), 8), "contiguous")
    _raises(lambda: w4.route(None, 8), "int32")


def test_rows_binding_refuses():
    import torch
    import weight_only_int4_w4a16_amd as w4
    r = _routing(4, 2, 8)
    assert r.offsets.shape == (9,) and r.order.shape == (8,) and r.slot.shape == (4, 2)
    x, ys, w = torch.zeros(4, 16), torch.zeros(8, 16), torch.zeros(4, 2)
    _raises(lambda: w4.dispatch(x, None), "route")
    _raises(lambda: w4.dispatch(ys, r), "shape")
    _raises(lambda: w4.dispatch(x[:, :0], r), "no elements")
    _raises(lambda: w4.dispatch(x[0], r), "2-D")
    _raises(lambda: w4.dispatch(x.double(), r), "dtype")
    _raises(lambda: w4.dispatch(torch.zeros(16, 4).t(), r), "contiguous")
    _raises(lambda: w4.dispatch(x, r, out=torch.zeros(8, 15)), "shape")
    big = torch.zeros(12, 16)
    _raises(lambda: w4.dispatch(big[:4], r, out=big[2:10]), "overlaps")
    _raises(lambda: w4.dispatch_backward(x, r), "shape")
    _raises(lambda: w4.combine(ys, r, w[:, :1]), "shape")
    _raises(lambda: w4.combine(ys, r, w.half()), "dtype")
    _raises(lambda: w4.combine(ys.half(), r, w, out_dtype=torch.float32), "dtype")
    _raises(lambda: w4.combine(ys, r, w, out=big[:4], out_dtype=torch.float16), "dtype")
    _raises(lambda: w4.combine_backward(x[:3], ys, r, w), "shape")
    _raises(lambda: w4.combine_backward(x.half(), ys, r, w), "dtype")


def test_grouped_binding_refuses():
    import torch
    import weight_only_int4_w4a16_amd as w4
    r = _routing(4, 2, 3)
    K, N, g = 256, 64, 128
    x = torch.zeros(8, K, dtype=torch.float16)
    pk = torch.zeros(3, w4.packed_bytes(K, N) // 4, dtype=torch.int32)
    sc = torch.zeros(3, 2, N, dtype=torch.float16)
    qz = torch.zeros(3, 2, N // 8, dtype=torch.int32)
    cb = torch.zeros(16, dtype=torch.float16)
    _raises(lambda: w4.gemm_grouped(x[:4], r, pk, sc, qz, g), "rows")
    _raises(lambda: w4.gemm_grouped(x, r, pk, sc, qz, g, gather=True), "rows")
    _raises(lambda: w4.gemm_grouped(x, r, pk[:2], sc, qz, g), "shape")
    _raises(lambda: w4.gemm_grouped(x, r, pk, sc[:2], qz, g), "shape")
    _raises(lambda: w4.gemm_grouped(x, r, pk, sc.bfloat16(), qz, g), "dtype")
    _raises(lambda: w4.gemm_grouped(x, r, pk, sc, qz[:, :1], g), "shape")
    _raises(lambda: w4.gemm_grouped(x, r, pk, sc, qz, 64), "shape")
    _raises(lambda: w4.gemm_grouped(x.float(), r, pk, sc, qz, g), "dtype")
    _raises(lambda: w4.gemm_grouped(x, r, pk, sc, qz, g, out=torch.zeros(7, N, dtype=torch.float16)), "shape")
    _raises(lambda: w4.gemm_grouped_swiglu(x, r, pk, sc, qz, g, out=torch.zeros(8, N, dtype=torch.float16)), "shape")
    _raises(lambda: w4.gemm_grouped_nf4(x, r, pk, sc, cb[:8], g), "shape")
    _raises(lambda: w4.gemm_grouped_nf4(x, r, pk, sc, None, g), "required")
    _raises(lambda: w4.pack_grouped(torch.zeros(3, 8, 24, dtype=torch.int32)), "unsupported")
    _raises(lambda: w4.pack_grouped(torch.zeros(8, 16, dtype=torch.int32)), "int32")


def test_lora_binding_refuses():
    """The shape checks need a device; what is refused before that is checked here."""
    import torch
    import weight_only_int4_w4a16_amd as w4
    x = torch.zeros(4, 64, dtype=torch.float16)
    _raises(lambda: w4.lora_add(x, x, None, None, None, None), "device")
    _raises(lambda: w4.lora_add(x, x.float(), None, None, None, None), "dtype")
    _raises(lambda: w4.lora_add(x, x[0], None, None, None, None), "2-D")
    assert w4.lora_workspace_bytes(4, 64, 64, 8, 12) == 0
    assert w4.lora_workspace_bytes(300, 4096, 4096, 8, 16) > w4.lora_workspace_bytes(300, 4096, 4096, 8, 16, planned=True) > 0
