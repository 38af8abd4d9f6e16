"""Cases that time the routed operators: tokens sorted by expert and back with its gradient, the
experts' 4-bit products, and the low-rank adapters of many requests.

A case is a plain dict; ``op`` names the operator:

* ``route``: the tokens' rows go into expert order and the experts' rows come back weighted
  (``train``: with the gradients of both moves);
* ``experts``: routed rows times each expert's packed 4-bit weight (``glu``: the fused gate+up
  projection with its SwiGLU);
* ``lora``: every row's own low-rank adapter beside a projection the rows share.

``run`` computes the plain form with elementary torch operations in 32 bits, or, where ``own`` is
set, calls the framework. ``exact`` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # a decode step of 16 sequences over a few large experts: launch latency counts
        dict(name="route-decode", op="route", tokens=16, topk=2, experts=8, width=4096, dtype="bf16",
             drop=0.0, train=False),
        # the same with many small experts and eight choices each
        dict(name="route-decode-wide", op="route", tokens=64, topk=8, experts=64, width=2048,
             dtype="fp16", drop=0.0, train=False),
        # a prefill batch with padding tokens that belong to no expert
        dict(name="route-prefill", op="route", tokens=8192, topk=2, experts=8, width=4096,
             dtype="fp16", drop=0.1, train=False),
        # training with sizes that divide nothing, some choices dropped by a capacity limit
        dict(name="route-train-ragged", op="route", tokens=4099, topk=3, experts=60, width=2885,
             dtype="bf16", drop=0.2, train=True),
        # a large training batch over many experts
        dict(name="route-train", op="route", tokens=16384, topk=8, experts=128, width=2048,
             dtype="bf16", drop=0.0, train=True),
        # one token through the two experts it chose
        dict(name="experts-token", op="experts", tokens=1, topk=2, experts=8, k=4096, n=14336,
             format="asym", group=128, dtype="fp16", glu=False),
        # a decode batch through the fused gate+up projection: every expert's weight is read
        dict(name="experts-decode", op="experts", tokens=32, topk=2, experts=8, k=4096, n=28672,
             format="sym", group=128, dtype="bf16", glu=True),
        # many small NF4 experts with a few dozen rows each
        dict(name="experts-wide-nf4", op="experts", tokens=200, topk=8, experts=64, k=2048, n=2816,
             format="nf4", group=64, dtype="bf16", glu=False),
        # prefill: each expert's product is bound by arithmetic
        dict(name="experts-prefill", op="experts", tokens=4096, topk=2, experts=8, k=4096, n=14336,
             format="asym", group=128, dtype="fp16", glu=False),
        # one request's adapter at decode
        dict(name="lora-token", op="lora", rows=1, requests=1, adapters=8, rank=16, k=4096, n=4096,
             dtype="fp16", out="fp16", none=0.0),
        # a decode batch, nearly every request with an adapter of its own
        dict(name="lora-decode", op="lora", rows=96, requests=96, adapters=64, rank=32, k=4096,
             n=14336, dtype="bf16", out="bf16", none=0.1),
        # prefill of several prompts, each with its adapter
        dict(name="lora-prefill", op="lora", rows=4096, requests=9, adapters=16, rank=64, k=8192,
             n=8192, dtype="bf16", out="bf16", none=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "experts", "lora"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "route":
        experts = _log_int(rng, 2, 256)
        topk = min(experts, rng.choice([1, 2, 3, 4, 6, 8]))
        width = _log_int(rng, 256, 8192)
        if rng.random() < 0.7:  # most models' widths divide by 64; the others are any size
            width = max(64, width // 64 * 64)
        tokens = min(_log_int(rng, 1, 16384), max(1, (1 << 28) // (topk * width)))
        return dict(op=op, tokens=tokens, topk=topk, experts=experts, width=width, dtype=dtype,
                    drop=rng.choice([0.0, 0.0, 0.1, 0.3]), train=rng.random() < 0.5)
    if op == "experts":
        fmt = rng.choice(["asym", "sym", "nf4"])
        group = 64 if fmt == "nf4" else rng.choice([32, 64, 128])
        glu = rng.random() < 0.5
        k = max(group, _log_int(rng, 512, 8192) // group * group)
        n = max(32, _log_int(rng, 512, 28672) // 32 * 32)
        experts = max(2, min(_log_int(rng, 2, 64), (1 << 30) // (k * n)))
        topk = min(experts, rng.choice([1, 2, 4, 8]))
        tokens = min(_log_int(rng, 1, 4096), max(1, 400 * 10 ** 9 // (2 * k * n * topk)))
        return dict(op=op, tokens=tokens, topk=topk, experts=experts, k=k, n=n, format=fmt,
                    group=group, dtype=dtype, glu=glu)
    rows = _log_int(rng, 1, 4096)
    adapters = _log_int(rng, 1, 64)
    rank = rng.choice([8, 16, 16, 24, 32, 64, 128])
    k = max(32, _log_int(rng, 512, 8192) // 32 * 32)
    n = max(16, _log_int(rng, 512, 14336) // 16 * 16)
    # decode batches have one row a request, prefill batches a run of rows each
    requests = rows if rows <= 256 and rng.random() < 0.7 else max(1, min(rows, _log_int(rng, 1, 32)))
    return dict(op=op, rows=rows, requests=requests, adapters=adapters, rank=rank, k=k, n=n,
                dtype=dtype, out=rng.choice([dtype, dtype, "fp32"]), none=rng.choice([0.0, 0.1, 0.5]))


def work(case):
    if case["op"] == "route":
        slots = case["tokens"] * case["topk"]
        row = case["width"] * 2
        live = slots * (1.0 - case["drop"])
        moved = case["tokens"] * row + slots * row + live * row + case["tokens"] * row
        flops = 2.0 * live * case["width"]
        if case["train"]:
            moved += case["tokens"] * row + live * row + slots * row  # dy, ys, dys
            moved += live * row + case["tokens"] * row                # dxs, dx
            flops += 4.0 * live * case["width"]
        return {"bytes": moved + slots * 16.0, "flops": flops}
    if case["op"] == "experts":
        slots = case["tokens"] * case["topk"]
        hit = case["experts"] * (1.0 - (1.0 - case["topk"] / case["experts"]) ** case["tokens"])
        k, n, groups = case["k"], case["n"], case["k"] // case["group"]
        weight = k * n / 2 + groups * n * 2 + (groups * n / 2 if case["format"] == "asym" else 0)
        n_out = n // 2 if case["glu"] else n
        return {"bytes": hit * weight + 2.0 * case["tokens"] * k + 2.0 * slots * n_out,
                "flops": 2.0 * slots * k * n}
    live = case["rows"] * (1.0 - case["none"])
    # runs of one request share an adapter; requests draw theirs at random
    used = case["adapters"] * (1.0 - (1.0 - 1.0 / case["adapters"]) ** (case["requests"] * (1.0 - case["none"])))
    wide = 4 if case["out"] == "fp32" else 2
    moved = used * case["rank"] * (case["k"] + case["n"]) * 2 + live * case["k"] * 2
    return {"bytes": moved + 2.0 * case["rows"] * case["n"] * wide,
            "flops": 2.0 * live * case["rank"] * (case["k"] + case["n"])}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _choices(gen, tokens, topk, experts):
    """The experts of each token: the largest of noisy scores, some experts liked more."""
    liked = 0.7 * torch.randn(experts, generator=gen, device="cuda")
    scores = torch.randn(tokens, experts, generator=gen, device="cuda") + liked
    top, ids = torch.topk(scores, topk, dim=1)
    return ids.to(torch.int32), torch.softmax(top, dim=1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    s = dict(case)
    if case["op"] == "route":
        tokens, topk, width = case["tokens"], case["topk"], case["width"]
        s["ids"], s["weights"] = _choices(gen, tokens, topk, case["experts"])
        if case["drop"]:
            lost = torch.rand(tokens, topk, generator=gen, device="cuda") < case["drop"]
            s["ids"] = torch.where(lost, -1, s["ids"])
        s["x"] = normal(tokens, width)
        s["ys"] = normal(tokens * topk, width)
        if case["train"]:
            s["dy"] = normal(tokens, width)
            s["dxs"] = normal(tokens * topk, width)
    elif case["op"] == "experts":
        experts, k, n = case["experts"], case["k"], case["n"]
        groups = k // case["group"]
        s["ids"], _ = _choices(gen, case["tokens"], case["topk"], experts)
        s["x"] = normal(case["tokens"], k)
        s["qweight"] = torch.randint(-2 ** 31, 2 ** 31, (experts, k // 8, n), generator=gen,
                                     device="cuda", dtype=torch.int32)
        u = torch.rand(experts, groups, n, generator=gen, device="cuda")
        s["qzeros"] = s["codebook"] = None
        if case["format"] == "nf4":
            s["scales"] = (0.02 + 0.07 * u).to(torch.float16)
            q = torch.linspace(0.03, 0.97, 16, device="cuda")
            level = torch.erfinv(2 * q - 1)
            s["codebook"] = (level / level.max()).to(torch.float16)
        else:
            s["scales"] = (0.004 + 0.005 * u).to(dt)
            if case["format"] == "asym":
                s["qzeros"] = torch.randint(-2 ** 31, 2 ** 31, (experts, groups, n // 8),
                                            generator=gen, device="cuda", dtype=torch.int32)
        # the largest number of rows one expert gets: the plain form's padded batch
        s["rows"] = int(torch.bincount(s["ids"].flatten().long(), minlength=experts).max())
        if own:  # the load-time layout of the weights, kept by a program that serves them
            import weight_only_int4_w4a16_amd as w4
            s["packed"] = w4.pack_grouped(s["qweight"])
    else:
        rows, requests, adapters = case["rows"], case["requests"], case["adapters"]
        chosen = torch.randint(0, adapters, (requests,), generator=gen, device="cuda", dtype=torch.int32)
        chosen = torch.where(torch.rand(requests, generator=gen, device="cuda") < case["none"], -1, chosen)
        if requests == rows:
            s["ids"] = chosen
        else:  # requests' rows lie one after another, at random lengths
            ends = torch.sort(torch.randint(0, rows, (requests - 1,), generator=gen, device="cuda"))[0]
            s["ids"] = chosen[torch.searchsorted(ends, torch.arange(rows, device="cuda"), right=True)]
        s["x"] = normal(rows, case["k"])
        s["y"] = torch.randn(rows, case["n"], generator=gen, device="cuda").to(TYPES[case["out"]])
        s["lora_a"] = (torch.randn(adapters, case["rank"], case["k"], generator=gen, device="cuda")
                       / math.sqrt(case["k"])).to(dt)
        s["lora_b"] = (torch.randn(adapters, case["n"], case["rank"], generator=gen, device="cuda")
                       / math.sqrt(case["rank"])).to(dt)
        s["scaling"] = 0.25 + torch.rand(adapters, generator=gen, device="cuda")
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(state):
    if own:
        return _OWN[state["op"]](state)
    return _PLAIN[state["op"]](state)


def _own_route(s):
    import weight_only_int4_w4a16_amd as w4
    r = w4.route(s["ids"], s["experts"])
    out = {"offsets": r.offsets, "order": r.order, "slot": r.slot, "xs": w4.dispatch(s["x"], r),
           "y": w4.combine(s["ys"], r, s["weights"])}
    if s["train"]:
        out["dys"], out["dweights"] = w4.combine_backward(s["dy"], s["ys"], r, s["weights"])
        out["dx"] = w4.dispatch_backward(s["dxs"], r)
    return out


def _own_experts(s):
    import weight_only_int4_w4a16_amd as w4
    r = w4.route(s["ids"], s["experts"])
    if s["format"] == "nf4":
        f = w4.gemm_grouped_nf4_swiglu if s["glu"] else w4.gemm_grouped_nf4
        return f(s["x"], r, s["packed"], s["scales"], s["codebook"], s["group"], gather=True)
    f = w4.gemm_grouped_swiglu if s["glu"] else w4.gemm_grouped
    return f(s["x"], r, s["packed"], s["scales"], s["qzeros"], s["group"], gather=True)


def _own_lora(s):
    import weight_only_int4_w4a16_amd as w4
    return w4.lora_add(s["y"], s["x"], s["lora_a"], s["lora_b"], s["ids"], s["scaling"])


_OWN = {"route": _own_route, "experts": _own_experts, "lora": _own_lora}


def _sort_plain(ids, experts):
    """Slots in expert order (ties by slot, those of no expert last): offsets, the slot of each row, the
    row of each slot and whether it has one."""
    flat = ids.flatten().long()
    live = (flat >= 0) & (flat < experts)
    expert, order = torch.sort(torch.where(live, flat, experts), stable=True)
    offsets = (expert[:, None] < torch.arange(experts + 1, device=flat.device)).sum(0)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=flat.device)
    return offsets, order, row, live


def _route_plain(s):
    dt, topk = s["x"].dtype, s["topk"]
    offsets, order, row, live = _sort_plain(s["ids"], s["experts"])
    token, filled = order // topk, live[order][:, None]
    shape = (s["tokens"], topk, s["width"])
    weights = s["weights"].flatten()
    back = torch.where(live[:, None], s["ys"].float()[row], 0.0)
    out = {"offsets": offsets.to(torch.int32), "order": order.to(torch.int32),
           "slot": torch.where(live, row, -1).to(torch.int32).view(s["tokens"], topk),
           "xs": torch.where(filled, s["x"][token], 0),
           "y": (torch.where(live, weights, 0.0)[:, None] * back).view(shape).sum(1).to(dt)}
    if s["train"]:
        dy = s["dy"].float()
        out["dys"] = torch.where(filled, weights[order][:, None] * dy[token], 0.0).to(dt)
        out["dweights"] = (back.view(shape) * dy[:, None, :]).sum(2)
        dxs = torch.where(live[:, None], s["dxs"].float()[row], 0.0)
        out["dx"] = dxs.view(shape).sum(1).to(dt)
    return out


def _weights_plain(s):
    """The experts' weights as the values their codes stand for, rounded once to the activations' type."""
    e, kw, n = s["qweight"].shape
    bits = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    codes = ((s["qweight"][:, :, None, :] >> bits[:, None]) & 15).view(e, kw * 8, n)
    groups = s["scales"].shape[1]
    scales = s["scales"].float()[:, :, None, :]
    if s["codebook"] is not None:
        w = s["codebook"].float()[codes].view(e, groups, -1, n) * scales
    else:
        zeros = 8
        if s["qzeros"] is not None:
            zeros = ((s["qzeros"][..., None] >> bits) & 15).view(e, groups, 1, n)
        w = (codes.view(e, groups, -1, n) - zeros).float() * scales
    return w.to(s["x"].dtype).view(e, kw * 8, n).float()


def _experts_plain(s):
    dt = s["x"].dtype
    offsets, order, _, _ = _sort_plain(s["ids"], s["experts"])
    expert = s["ids"].flatten().long()[order]
    place = torch.arange(order.numel(), device="cuda") - offsets[expert]
    padded = torch.zeros(s["experts"], s["rows"], s["k"], device="cuda")
    padded[expert, place] = s["x"].float()[order // s["topk"]]
    y = torch.bmm(padded, _weights_plain(s))[expert, place]
    if s["glu"]:
        gate, up = y[:, : s["n"] // 2], y[:, s["n"] // 2:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y.to(dt)


def _lora_plain(s):
    adapters, rank, k = s["lora_a"].shape
    ids = s["ids"].long()
    live = (ids >= 0) & (ids < adapters)
    mine = (ids[:, None] == torch.arange(adapters, device="cuda")) & live[:, None]
    # every adapter's product, of which each row keeps its own
    t = s["x"].float() @ s["lora_a"].float().view(adapters * rank, k).t()
    t = (t.view(-1, adapters, rank) * (mine * s["scaling"])[:, :, None]).view(-1, adapters * rank)
    b = s["lora_b"].float().transpose(0, 1).reshape(s["n"], adapters * rank)
    return (s["y"].float() + t @ b.t()).to(s["y"].dtype)


_PLAIN = {"route": _route_plain, "experts": _experts_plain, "lora": _lora_plain}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _route_exact, "experts": _experts_exact, "lora": _lora_exact}[case["op"]](s)


def _sorted_slots(s):
    """For each expert in turn, its slots in rising order (a list of index tensors)."""
    flat = s["ids"].flatten()
    return [torch.nonzero(flat == e)[:, 0] for e in range(s["experts"])]


def _route_exact(s):
    slots = torch.cat(_sorted_slots(s))
    token = slots // s["topk"]
    count, tokens, width = s["ids"].numel(), s["tokens"], s["width"]
    w = s["weights"].double().flatten()[slots][:, None]

    def total(rows):
        """The rows of a token added up, over its slots."""
        acc = torch.zeros(tokens, width, dtype=torch.float64, device="cuda")
        return acc.index_add_(0, token, rows)

    xs = torch.zeros(count, width, dtype=torch.float64, device="cuda")
    xs[: len(slots)] = s["x"].double()[token]
    ys = s["ys"][: len(slots)].double()
    out = {"offsets": None, "order": None, "slot": None, "xs": xs, "y": total(w * ys)}
    if s["train"]:
        dy = s["dy"].double()[token]
        dys = torch.zeros(count, width, dtype=torch.float64, device="cuda")
        dys[: len(slots)] = w * dy
        dw = torch.zeros(count, dtype=torch.float64, device="cuda")
        dw[slots] = torch.linalg.vecdot(dy, ys)
        out.update(dys=dys, dweights=dw.view(tokens, s["topk"]), dx=total(s["dxs"][: len(slots)].double()))
    return out


def _experts_exact(s):
    dt, parts = s["x"].dtype, []
    for e, slots in enumerate(_sorted_slots(s)):
        if not len(slots):
            continue
        codes = torch.stack([(s["qweight"][e] >> (4 * i)) & 15 for i in range(8)], 1).flatten(0, 1)
        scale = s["scales"][e].repeat_interleave(s["group"], 0).double()
        if s["codebook"] is not None:
            level = s["codebook"].double()[codes.long()]
        elif s["qzeros"] is None:
            level = codes.double() - 8
        else:
            zero = torch.stack([(s["qzeros"][e] >> (4 * i)) & 15 for i in range(8)], 2).flatten(1, 2)
            level = codes.double() - zero.repeat_interleave(s["group"], 0).double()
        # level * scale has at most 22 significant bits, so 32 bits hold it exactly and the
        # rounding to the activations' type is the definition's only one
        w = (level * scale).float().to(dt).double()
        y = s["x"][slots // s["topk"]].double() @ w
        if s["glu"]:
            gate, up = y.chunk(2, dim=1)
            y = gate * torch.sigmoid(gate) * up
        parts.append(y)
    return torch.cat(parts)


def _lora_exact(s):
    y = s["y"].double()
    for a in range(s["adapters"]):
        rows = torch.nonzero(s["ids"] == a)[:, 0]
        if len(rows):
            low = s["x"][rows].double() @ s["lora_a"][a].double().t()
            y[rows] += s["scaling"][a].double() * (low @ s["lora_b"][a].double().t())
    return y
