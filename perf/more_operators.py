"""Cases that time the 8-bit floating point operators: the quantizers that give every 128 values (or block
of 128 x 128) a scale, products of what they make, the same product for routed rows, and its gradients.

A case is a plain dict; ``op`` names the operator:

* ``quantize``: 16- or 32-bit values to e4m3 codes and their scales (``form``: ``rows``, one scale for 128
  values of a row, as activations go into a product; ``columns``, one for 128 values of a column, the codes
  transposed, as both sides go into the weight's gradient; ``weight``, one for a block of 128 x 128, with the
  transposed codes that the activations' gradient multiplies with);
* ``linear``: a 16-bit activation quantized and multiplied with an 8-bit weight (``glu``: the fused gate+up
  projection with its SwiGLU);
* ``experts``: routed rows through their experts' SwiGLU projection, quantized, and through the second one;
* ``train``: the gradients of the product for its activation and its weight (``experts`` over 0: of the routed
  product, whose rows are in expert order).

A scale is s = max|v| / 448 in 32 bits, at least 2^-126, and a code is v / s rounded to 32 bits and then to
the nearest e4m3 (ties to even). ``run`` computes the plain form with elementary torch operations in 32
bits, or, where ``own`` is set, calls the framework. ``exact`` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
LEAST = 2.0 ** -126


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # a decode batch's activations: launch latency counts
        dict(name="quantize-decode", op="quantize", form="rows", m=16, k=8192, dtype="bf16"),
        # a training batch of a size that divides nothing, on its way into a weight's gradient
        dict(name="quantize-columns", op="quantize", form="columns", m=4099, k=2885, dtype="bf16"),
        # a master weight, quantized after each optimizer step for both directions
        dict(name="quantize-weight", op="quantize", form="weight", m=14336, k=4096, dtype="fp32"),
        # one token through a small projection
        dict(name="linear-token", op="linear", m=1, k=4096, n=4096, dtype="bf16", out="bf16", glu=False),
        # a decode batch of 16 sequences
        dict(name="linear-decode", op="linear", m=16, k=8192, n=10240, dtype="fp16", out="fp16", glu=False),
        # a larger decode batch through a fused gate+up projection
        dict(name="linear-swiglu", op="linear", m=64, k=8192, n=57344, dtype="bf16", out="bf16", glu=True),
        # sizes that divide nothing, in 32 bits for a loss
        dict(name="linear-ragged", op="linear", m=333, k=2896, n=5001, dtype="bf16", out="fp32", glu=False),
        # prefill: bound by arithmetic
        dict(name="linear-prefill", op="linear", m=2048, k=8192, n=28672, dtype="bf16", out="bf16", glu=False),
        # a decode batch over a few large experts: every expert's weights are read
        dict(name="experts-decode", op="experts", tokens=32, topk=2, experts=8, k=4096, inner=14336,
             dtype="bf16", drop=0.0),
        # a prefill batch over many small experts, with padding tokens that belong to none
        dict(name="experts-prefill", op="experts", tokens=4096, topk=8, experts=64, k=2048, inner=1408,
             dtype="fp16", drop=0.05),
        # a training step's gradients of a projection
        dict(name="train-linear", op="train", m=4096, topk=1, experts=0, k=4096, n=14336, dtype="bf16", drop=0.0),
        # and of routed experts
        dict(name="train-experts", op="train", m=4096, topk=2, experts=16, k=2048, n=2816, dtype="bf16", drop=0.05),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _depth(rng, lo, hi):
    """A product's depth: any multiple of 16, most often of 128 as models' widths are."""
    k = _log_int(rng, lo, hi)
    return max(128, k // 128 * 128) if rng.random() < 0.7 else max(16, k // 16 * 16)


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "experts", "train"])
    dtype = rng.choice(["fp16", "bf16"])
    most = 450 * 10 ** 9  # multiplications of a drawn case
    if op == "quantize":
        form = rng.choice(["rows", "columns", "weight"])
        k = _log_int(rng, 128, 16384)
        if form == "rows" or rng.random() < 0.7:
            k = k // 16 * 16
        m = min(_log_int(rng, 1, 16384), max(1, (1 << 25) // k))
        return dict(op=op, form=form, m=m, k=k, dtype=rng.choice([dtype, dtype, "fp32"]))
    if op == "linear":
        k, n = _depth(rng, 256, 16384), _log_int(rng, 128, 32768)
        glu = rng.random() < 0.4
        if glu or rng.random() < 0.7:
            n = max(32, n // 32 * 32)
        m = min(_log_int(rng, 1, 8192), max(1, most // (k * n)))
        return dict(op=op, m=m, k=k, n=n, dtype=dtype, out=rng.choice([dtype, dtype, "fp32"]), glu=glu)
    if op == "experts":
        k, inner = _depth(rng, 256, 4096), _depth(rng, 256, 14336)
        experts = max(2, min(_log_int(rng, 2, 64), (1 << 29) // (k * inner)))
        topk = min(experts, rng.choice([1, 2, 4, 8]))
        tokens = min(_log_int(rng, 1, 4096), max(1, most // (3 * k * inner * topk)))
        return dict(op=op, tokens=tokens, topk=topk, experts=experts, k=k, inner=inner, dtype=dtype,
                    drop=rng.choice([0.0, 0.0, 0.1]))
    k, n = _depth(rng, 256, 8192), _depth(rng, 256, 14336)
    experts = 0 if rng.random() < 0.5 else max(2, min(_log_int(rng, 2, 64), (1 << 27) // (k * n)))
    topk = min(experts, rng.choice([1, 2, 4])) if experts else 1
    m = min(_log_int(rng, 1, 8192), max(1, most // (2 * k * n * topk)))
    return dict(op=op, m=m, topk=topk, experts=experts, k=k, n=n, dtype=dtype,
                drop=rng.choice([0.0, 0.1]) if experts else 0.0)


def _hit(case, tokens):
    return case["experts"] * (1.0 - (1.0 - case["topk"] * (1.0 - case["drop"]) / case["experts"]) ** tokens)


def work(case):
    k = case["k"]
    if case["op"] == "quantize":
        m, values = case["m"], case["m"] * k
        wide = 4 if case["dtype"] == "fp32" else 2
        out = {"rows": values + 4 * m * -(-k // 128), "columns": (m + -m % 16) * k + 4 * k * -(-m // 128),
               "weight": 2 * values + 8 * -(-m // 128) * -(-k // 128)}[case["form"]]
        return {"bytes": float(wide * values + out), "flops": 2.0 * values}
    if case["op"] == "linear":
        m, n = case["m"], case["n"]
        wide = 4 if case["out"] == "fp32" else 2
        moved = 2 * m * k + n * k + 4 * (n // 128 + 1) * (k // 128 + 1) + wide * m * (n // 2 if case["glu"] else n)
        return {"bytes": float(moved), "flops": 2.0 * m * n * k}
    if case["op"] == "experts":
        slots, inner = case["tokens"] * case["topk"], case["inner"]
        live = slots * (1.0 - case["drop"])
        moved = _hit(case, case["tokens"]) * 3 * k * inner + 2 * case["tokens"] * k + slots * (inner + 2 * k)
        return {"bytes": float(moved), "flops": 6.0 * live * k * inner}
    n, rows = case["n"], case["m"] * case["topk"]
    live = rows * (1.0 - case["drop"])
    weights = _hit(case, case["m"]) if case["experts"] else 1
    moved = live * (2 * n + 2 * k) + 2 * rows * k + weights * n * k + 4 * max(1, case["experts"]) * n * k
    return {"bytes": float(moved), "flops": 4.0 * live * n * k}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _choices(gen, tokens, topk, experts, drop):
    """The experts of each token: the largest of noisy scores, some experts liked more; -1: no expert."""
    liked = 0.7 * torch.randn(experts, generator=gen, device="cuda")
    scores = torch.randn(tokens, experts, generator=gen, device="cuda") + liked
    ids = torch.topk(scores, topk, dim=1)[1].to(torch.int32)
    lost = torch.rand(tokens, topk, generator=gen, device="cuda") < drop
    return torch.where(lost, -1, ids)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def rows(m, width):
        """Normal values; one channel in 64 is ten times as large, as in models' activations."""
        size = torch.where(torch.rand(width, generator=gen, device="cuda") < 1 / 64, 10.0, 1.0)
        return (torch.randn(m, width, generator=gen, device="cuda") * size).to(dt)

    def weight(*shape, blocks):
        """Codes of an 8-bit weight and one scale for each block of 128 x 128."""
        codes = (112 * torch.randn(*shape, generator=gen, device="cuda")).clamp_(-448, 448).to(E4M3)
        kb = -(-shape[-1] // 128)
        scales = 0.5 + torch.rand(*shape[:-2], blocks, kb, generator=gen, device="cuda")
        return codes, scales / (112 * math.sqrt(shape[-1]))

    s = dict(case)
    k = case["k"]
    if case["op"] == "quantize":
        s["x"] = rows(case["m"], k)
    elif case["op"] == "linear":
        n = case["n"]
        s["x"] = rows(case["m"], k)
        s["codes"], s["scales"] = weight(n, k, blocks=2 * -(-n // 256) if case["glu"] else -(-n // 128))
    elif case["op"] == "experts":
        experts, inner = case["experts"], case["inner"]
        s["ids"] = _choices(gen, case["tokens"], case["topk"], experts, case["drop"])
        s["x"] = rows(case["tokens"], k)
        s["up"], s["up_scales"] = weight(experts, 2 * inner, k, blocks=2 * -(-inner // 128))
        s["down"], s["down_scales"] = weight(experts, k, inner, blocks=-(-k // 128))
    else:
        experts, n = case["experts"], case["n"]
        lead = (experts,) if experts else ()
        s["x"], s["dy"] = rows(case["m"] * case["topk"], k), rows(case["m"] * case["topk"], n)
        # the transposed weight, as the quantizer leaves it for this direction
        s["codes"], s["scales"] = weight(*lead, k, n, blocks=-(-k // 128))
        if experts:
            s["ids"] = _choices(gen, case["m"], case["topk"], experts, case["drop"])
    if "ids" in s:
        # the largest number of rows one expert gets: the plain form's padded batch
        flat = s["ids"].flatten().long()
        s["rows"] = max(1, int(torch.bincount(flat[flat >= 0], minlength=case["experts"]).max()))
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(state):
    if own:
        return _OWN[state["op"]](state)
    return _PLAIN[state["op"]](state)


def _own_quantize(s):
    import weight_only_int4_w4a16_amd as w4
    if s["form"] == "rows":
        return w4.quantize_fp8(s["x"])
    if s["form"] == "columns":
        return w4.quantize_fp8_columns(s["x"])
    return w4.quantize_fp8_weight(s["x"], transposed=True)


def _own_linear(s):
    import weight_only_int4_w4a16_amd as w4
    f = w4.gemm_fp8_swiglu if s["glu"] else w4.gemm_fp8
    return f(s["x"], s["codes"], s["scales"], out_dtype=TYPES[s["out"]])


def _own_experts(s):
    import weight_only_int4_w4a16_amd as w4
    r = w4.route(s["ids"], s["experts"])
    h, h_scales = w4.gemm_fp8_grouped_swiglu(s["x"], r, s["up"], s["up_scales"], gather=True, quantized=True)
    y = w4.gemm_fp8_grouped(h, r, s["down"], s["down_scales"], x_scales=h_scales, out_dtype=s["x"].dtype)
    return {"h": h, "h_scales": h_scales, "y": y}


def _own_train(s):
    import weight_only_int4_w4a16_amd as w4
    if s["experts"]:
        r = w4.route(s["ids"], s["experts"])
        return w4.gemm_fp8_grouped_backward(s["dy"], s["x"], r, s["codes"], s["scales"])
    return w4.gemm_fp8_backward(s["dy"], s["x"], s["codes"], s["scales"])


_OWN = {"quantize": _own_quantize, "linear": _own_linear, "experts": _own_experts, "train": _own_train}


def _padded(x, dim):
    """``x`` in 32 bits with zeros behind it up to a multiple of 128 along ``dim``."""
    lack = -x.shape[dim] % 128
    x = x.float()
    if not lack:
        return x
    shape = list(x.shape)
    shape[dim] = lack
    return torch.cat([x, x.new_zeros(shape)], dim)


def _scale_plain(most):
    # a tensor of 448s: by a number, torch multiplies with the rounded reciprocal
    return (most / torch.full_like(most, 448.0)).clamp(min=LEAST)


def _rows_plain(x):
    """Codes ``[..., m, k]`` (the values they are, in 32 bits) and scales ``[..., k / 128, m]`` of 128 values of a row."""
    v = _padded(x, -1).unflatten(-1, (-1, 128))
    s = _scale_plain(v.abs().amax(-1))
    q = (v / s[..., None]).to(E4M3).float().flatten(-2)
    return q[..., : x.shape[-1]], s.transpose(-1, -2)


def _times_rows(q, s):
    return q * s.transpose(-1, -2).repeat_interleave(128, -1)[..., : q.shape[-1]]


def _columns_plain(x):
    """The same along columns ``[..., m, k]``, in place: codes ``[..., m, k]``, scales ``[..., m / 128, k]``."""
    q, s = _rows_plain(x.transpose(-1, -2))
    return q.transpose(-1, -2), s


def _quantize_plain(s):
    x = s["x"]
    if s["form"] == "rows":
        q, scales = _rows_plain(x)
        return q.to(E4M3), scales.contiguous()
    if s["form"] == "columns":
        q, scales = _columns_plain(x)
        codes = torch.zeros(s["k"], s["m"] + -s["m"] % 16, dtype=E4M3, device="cuda")
        codes[:, : s["m"]] = q.t().to(E4M3)
        return codes, scales.contiguous()
    v = _padded(_padded(x, 0), 1).unflatten(1, (-1, 128)).unflatten(0, (-1, 128))
    scales = _scale_plain(v.abs().amax((1, 3)))
    q = (v / scales[:, None, :, None]).flatten(2).flatten(0, 1)[: s["m"], : s["k"]].to(E4M3)
    return q, scales, q.t().contiguous(), scales.t().contiguous()


def _weight_plain(codes, scales, halves=1):
    """The weight its codes and blocks' scales stand for; each half has blocks of its own."""
    w = codes.float().unflatten(-2, (halves, -1))
    up = scales.unflatten(-2, (halves, -1)).repeat_interleave(128, -2)[..., : w.shape[-2], :]
    return (w * up.repeat_interleave(128, -1)[..., : w.shape[-1]]).flatten(-3, -2)


def _swiglu_plain(y):
    gate, up = y.chunk(2, dim=-1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _linear_plain(s):
    x = _times_rows(*_rows_plain(s["x"]))
    y = x @ _weight_plain(s["codes"], s["scales"], 2 if s["glu"] else 1).t()
    return (_swiglu_plain(y) if s["glu"] else y).to(TYPES[s["out"]])


def _sorted_plain(s):
    """Each sorted row's slot and expert (those of no expert last), and its place among its expert's rows."""
    flat = s["ids"].flatten().long()
    expert, order = torch.sort(torch.where(flat >= 0, flat, s["experts"]), stable=True)
    first = (expert[:, None] < torch.arange(s["experts"] + 1, device="cuda")).sum(0)
    return order, expert, torch.arange(order.numel(), device="cuda") - first[expert]


def _batched(rows, expert, place, experts, most):
    """The experts' rows as a batch ``[experts, most, width]``, zeros where there are none."""
    out = torch.zeros(experts + 1, most, rows.shape[1], device="cuda")
    live = expert < experts
    out[torch.where(live, expert, experts), torch.where(live, place, 0)] = torch.where(live[:, None], rows, 0.0)
    return out[:experts]


def _unbatched(batch, expert, place):
    live = expert < batch.shape[0]
    got = batch[torch.where(live, expert, 0), torch.where(live, place, 0)]
    return torch.where(live[:, None], got, 0.0)


def _experts_plain(s):
    dt, experts = s["x"].dtype, s["experts"]
    order, expert, place = _sorted_plain(s)
    x = _times_rows(*_rows_plain(s["x"]))[order // s["topk"]]
    up = _weight_plain(s["up"], s["up_scales"], 2).transpose(1, 2)
    h = _swiglu_plain(torch.bmm(_batched(x, expert, place, experts, s["rows"]), up))
    q, scales = _rows_plain(_unbatched(h, expert, place))
    down = _weight_plain(s["down"], s["down_scales"]).transpose(1, 2)
    y = torch.bmm(_batched(_times_rows(q, scales), expert, place, experts, s["rows"]), down)
    return {"h": q.to(E4M3), "h_scales": scales.contiguous(), "y": _unbatched(y, expert, place).to(dt)}


def _train_plain(s):
    dt = s["x"].dtype
    dy = _times_rows(*_rows_plain(s["dy"]))
    back = _weight_plain(s["codes"], s["scales"])
    if not s["experts"]:
        dyc, xc = (_both_columns(s[name]) for name in ("dy", "x"))
        return (dy @ back.t()).to(dt), dyc.t() @ xc
    order, expert, place = _sorted_plain(s)
    most = s["rows"] + -s["rows"] % 128

    def batch(rows):
        return _batched(rows, expert, place, s["experts"], most)

    dx = _unbatched(torch.bmm(batch(dy), back.transpose(1, 2)), expert, place)
    dyc, xc = (_both_columns(batch(s[name].float())) for name in ("dy", "x"))
    return dx.to(dt), torch.bmm(dyc.transpose(1, 2), xc)


def _both_columns(v):
    """The values that the codes of 128 rows a scale stand for."""
    q, s = _columns_plain(v)
    return q * s.repeat_interleave(128, -2)[..., : q.shape[-2], :]


_PLAIN = {"quantize": _quantize_plain, "linear": _linear_plain, "experts": _experts_plain, "train": _train_plain}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"quantize": _quantize_exact, "linear": _linear_exact, "experts": _experts_exact,
            "train": _train_exact}[case["op"]](s)


def _e4m3_exact(v):
    """The nearest e4m3 of values up to 448 and a little more: three fraction bits from 2^-6 on, steps of 2^-9 below."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _scale_exact(most):
    # 64 bits hold twice 32 bits' digits and more, so rounding their quotient again gives the 32-bit one
    return (most / 448.0).float().double().clamp(min=LEAST)


def _along(v, dim):
    """Codes and scales along the last or first dimension of a matrix, 128 values at a time."""
    codes, scales = [], []
    for part in v.double().split(128, dim):
        s = _scale_exact(part.abs().amax(dim, keepdim=True))
        codes.append(_e4m3_exact((part / s).float().double()))
        scales.append(s)
    return codes, scales


def _values(v, dim):
    codes, scales = _along(v, dim)
    return torch.cat([q * s for q, s in zip(codes, scales)], dim)


def _quantize_exact(s):
    x, m, k = s["x"], s["m"], s["k"]
    if s["form"] == "rows":
        codes, scales = _along(x, 1)
        return torch.cat(codes, 1), torch.cat(scales, 1).t().contiguous()
    if s["form"] == "columns":
        codes, scales = _along(x, 0)
        out = torch.zeros(k, m + -m % 16, dtype=torch.float64, device="cuda")
        out[:, :m] = torch.cat(codes, 0).t()
        return out, torch.cat(scales, 0)
    q = torch.empty(m, k, dtype=torch.float64, device="cuda")
    scales = torch.empty(-(-m // 128), -(-k // 128), dtype=torch.float64, device="cuda")
    for j, part in enumerate(x.split(128, 1)):
        most = part.double().abs().amax(1)
        most = torch.stack([p.amax() for p in most.split(128)])
        scales[:, j] = _scale_exact(most)
        per_row = scales[:, j].repeat_interleave(128)[:m, None]
        q[:, 128 * j: 128 * j + 128] = _e4m3_exact((part.double() / per_row).float().double())
    return q, scales, q.t().contiguous(), scales.t().contiguous()


def _half_exact(codes, scales):
    """One matrix of codes times its blocks' scales."""
    wide = scales.double().repeat_interleave(128, 0)[: codes.shape[0]]
    return codes.double() * wide.repeat_interleave(128, 1)[:, : codes.shape[1]]


def _glu_exact(x, codes, scales):
    half, blocks = codes.shape[0] // 2, scales.shape[0] // 2
    gate = x @ _half_exact(codes[:half], scales[:blocks]).t()
    return gate * torch.sigmoid(gate) * (x @ _half_exact(codes[half:], scales[blocks:]).t())


def _linear_exact(s):
    x = _values(s["x"], 1)
    if s["glu"]:
        return _glu_exact(x, s["codes"], s["scales"])
    return x @ _half_exact(s["codes"], s["scales"]).t()


def _expert_slots(s):
    """For each expert in turn, its slots in rising order."""
    flat = s["ids"].flatten()
    return [torch.nonzero(flat == e)[:, 0] for e in range(s["experts"])]


def _experts_exact(s):
    slots_of = _expert_slots(s)
    x, k = _values(s["x"], 1), s["k"]
    h = torch.zeros(s["ids"].numel(), s["inner"], dtype=torch.float64, device="cuda")
    y = torch.zeros(s["ids"].numel(), k, dtype=torch.float64, device="cuda")
    at = 0
    for e, slots in enumerate(slots_of):
        if len(slots):
            h[at: at + len(slots)] = _glu_exact(x[slots // s["topk"]], s["up"][e], s["up_scales"][e])
        at += len(slots)
    codes, scales = _along(h, 1)
    hv = torch.cat([q * c for q, c in zip(codes, scales)], 1)
    at = 0
    for e, slots in enumerate(slots_of):
        rows = slice(at, at + len(slots))
        y[rows] = hv[rows] @ _half_exact(s["down"][e], s["down_scales"][e]).t()
        at += len(slots)
    return {"h": torch.cat(codes, 1), "h_scales": torch.cat(scales, 1).t().contiguous(), "y": y}


def _train_exact(s):
    if not s["experts"]:
        dx = _values(s["dy"], 1) @ _half_exact(s["codes"], s["scales"]).t()
        return dx, _values(s["dy"], 0).t() @ _values(s["x"], 0)
    k, n, at = s["k"], s["n"], 0
    dx = torch.zeros(s["dy"].shape[0], k, dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["experts"], n, k, dtype=torch.float64, device="cuda")
    for e, slots in enumerate(_expert_slots(s)):
        if len(slots):
            rows = slice(at, at + len(slots))
            dx[rows] = _values(s["dy"][rows], 1) @ _half_exact(s["codes"][e], s["scales"][e]).t()
            dw[e] = _values(s["dy"][rows], 0).t() @ _values(s["x"][rows], 0)
            at += len(slots)
    return dx, dw
