"""One decoder layer's projections on 4-bit weights, with what differs between the rows of a batch:
a shared projection with each request's low-rank adapter beside it, and an MLP of routed experts.

    y = x W + s[a] (x A[a]^T) B[a]^T                     (a = the row's adapter, or none)
    p = softmax of the topk gate scores of y
    z = y + sum_j p[t, j] E[ids[t, j]](y[t]),  E(v) = (SiLU(v G) * (v U)) D

``python examples/routed_layer.py`` runs it on random weights, checks it against fp64 and times it;
:func:`layer` is what a server would capture in a graph.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import weight_only_int4_w4a16_amd as w4


def random_weight(K, N, group, dtype, gen, groups=None):
    """Symmetric 4-bit codes and scales of one weight, or of ``groups`` of them."""
    lead = () if groups is None else (groups,)
    codes = torch.randint(-2 ** 31, 2 ** 31, (*lead, K // 8, N), generator=gen, device="cuda", dtype=torch.int32)
    # scales that keep a product's size near its input's: codes - 8 have a spread of about 4.6
    scales = (0.5 + torch.rand(*lead, K // group, N, generator=gen, device="cuda")) / (4.6 * K ** 0.5)
    return codes, scales.to(dtype)


def make_layer(width, inner, experts, adapters, rank, group=128, dtype=torch.bfloat16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    m = {"group": group, "experts": experts}
    for name, K, N, n in (("proj", width, width, None), ("up", width, 2 * inner, experts), ("down", inner, width, experts)):
        codes, m[name + "_scales"] = random_weight(K, N, group, dtype, gen, n)
        m[name + "_codes"] = codes
        m[name] = w4.pack(codes) if n is None else w4.pack_grouped(codes)
    m["gate"] = torch.randn(width, experts, generator=gen, device="cuda") / width ** 0.5
    m["lora_a"] = (torch.randn(adapters, rank, width, generator=gen, device="cuda") / width ** 0.5).to(dtype)
    m["lora_b"] = (torch.randn(adapters, width, rank, generator=gen, device="cuda") / rank ** 0.5).to(dtype)
    m["scaling"] = torch.full((adapters,), 0.5, device="cuda")
    return m


def layer(m, x, adapter_ids, topk=2):
    """``(z, ids)`` for ``x[rows, width]`` and each row's adapter (int32, -1: none)."""
    y = w4.gemm(x, m["proj"], m["proj_scales"], None, m["group"])
    w4.lora_add(y, x, m["lora_a"], m["lora_b"], adapter_ids, m["scaling"], out=y)
    scores, ids = torch.topk(y.float() @ m["gate"], topk, dim=1)
    ids = ids.to(torch.int32)
    routing = w4.route(ids, m["experts"])
    h = w4.gemm_grouped_swiglu(y, routing, m["up"], m["up_scales"], None, m["group"], gather=True)
    e = w4.gemm_grouped(h, routing, m["down"], m["down_scales"], None, m["group"])
    return y + w4.combine(e, routing, torch.softmax(scores, dim=1)), ids


def layer_fp64(m, x, adapter_ids, ids, topk=2):
    """The same in fp64 from the codes, for given choices of experts (a near tie of two scores may fall
    either way)."""
    def weight(name, e=None):
        codes, scales = m[name + "_codes"], m[name + "_scales"]
        if e is not None:
            codes, scales = codes[e], scales[e]
        q = torch.stack([(codes >> (4 * i)) & 15 for i in range(8)], 1).flatten(0, 1).double() - 8
        return (q * scales.double().repeat_interleave(m["group"], 0)).to(scales.dtype).double()

    x = x.double()
    y = x @ weight("proj")
    for a in range(len(m["scaling"])):
        rows = adapter_ids == a
        y[rows] += m["scaling"][a].double() * (x[rows] @ m["lora_a"][a].double().t()) @ m["lora_b"][a].double().t()
    p = torch.softmax((y @ m["gate"].double()).gather(1, ids.long()), dim=1)
    z = y.clone()
    for e in range(m["experts"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            g, u = (y[t] @ weight("up", e)).chunk(2, dim=1)
            z.index_add_(0, t, p[t, j][:, None] * ((g * torch.sigmoid(g) * u) @ weight("down", e)))
    return z


def main(rows=64, width=4096, inner=2048, experts=8, adapters=16, rank=16):
    m = make_layer(width, inner, experts, adapters, rank)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, width, generator=gen, device="cuda").to(torch.bfloat16)
    adapter_ids = torch.randint(-1, adapters, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    z, ids = layer(m, x, adapter_ids)
    ref = layer_fp64(m, x, adapter_ids, ids)
    error = float((z.double() - ref).norm() / ref.norm())
    for _ in range(5):
        layer(m, x, adapter_ids)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(20):
        layer(m, x, adapter_ids)
    end.record()
    torch.cuda.synchronize()
    print(f"{rows} rows, {experts} experts of {width}x{2 * inner} and {inner}x{width}, {adapters} adapters of rank {rank}: "
          f"error {error:.2e} of fp64, {start.elapsed_time(end) / 20 * 1e3:.1f} us a layer")
    return error


if __name__ == "__main__":
    main()
