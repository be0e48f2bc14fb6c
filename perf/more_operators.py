"""Cases and plain forms of the operators around the expert products.

The operators: the root-mean-square norm ahead of the layer with the residual's addition
(``norm``), its rows in the input type or in 8 bits with a scale per 128, and its gradients; rows
in 8 bits times 8-bit weights with a scale per 128 x 128, dense or per expert (``linear``), and
the gradient to the rows (``linear_grad``); the experts' activation (``swiglu``), in the input
type or in 8 bits, and its gradient; the router's balance loss with the experts' counts
(``balance``) and its gradient.

``run`` computes a case in plain 32-bit torch operations, or, with ``own`` set, through the
library's entry points.  ``exact`` computes it in 64 bits.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_E4M3 = torch.float8_e4m3fn
_BLOCK = 128  # elements of a row, and rows of a weight, that share a scale
_LARGEST = 448.0  # of E4M3
_LEAST = 2.0 ** -100  # a block's largest magnitude counts as this at least
_EPS = 1e-5
_ALPHA, _LIMIT = 1.702, 7.0


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the norm ahead of a decode step's experts: four tokens, latency alone counts
        {"name": "norm_decode_fp8", "op": "norm", "tokens": 4, "hidden": 2880, "dtype": "bf16", "fp8": True,
         "train": False},
        # a training step's norm of float32 rows of an odd width, with its gradients
        {"name": "norm_train_ragged", "op": "norm", "tokens": 777, "hidden": 1001, "dtype": "f32", "fp8": False,
         "train": True},
        # the 120b long prefill in a training step: rows out in 8 bits, then the gradients
        {"name": "norm_train_prefill", "op": "norm", "tokens": 4096, "hidden": 2880, "dtype": "bf16", "fp8": True,
         "train": True},
        # the activation between the products of a 20b decode step, out in 8 bits
        {"name": "swiglu_decode_fp8", "op": "swiglu", "rows": 16, "inner": 2880, "dtype": "bf16", "split": False,
         "fp8": True, "train": False},
        # the activation of the 120b long prefill's pairs in a training step, with its gradient
        {"name": "swiglu_train_prefill", "op": "swiglu", "rows": 16384, "inner": 2880, "dtype": "bf16",
         "split": False, "fp8": False, "train": True},
        # one token of bf16 through a dense 8-bit projection
        {"name": "linear_one_token", "op": "linear", "tokens": 1, "top_k": 1, "experts": 0, "n": 2880, "k": 4096,
         "bias": True, "quantize": True, "skew": 0.0},
        # a decode batch of 20b through its experts' gate and up rows
        {"name": "linear_decode_experts", "op": "linear", "tokens": 4, "top_k": 4, "experts": 32, "n": 5760,
         "k": 2880, "bias": True, "quantize": False, "skew": 0.0},
        # the 120b long prefill through its experts' gate and up rows
        {"name": "linear_prefill_experts", "op": "linear", "tokens": 4096, "top_k": 4, "experts": 128, "n": 5760,
         "k": 2880, "bias": True, "quantize": False, "skew": 0.2},
        # a small fine-tuning batch over few experts with ragged sizes
        {"name": "linear_grad_ragged", "op": "linear_grad", "tokens": 150, "top_k": 2, "experts": 8, "n": 1000,
         "k": 736, "bias": False, "quantize": False, "skew": 0.0},
        # fine-tuning through the frozen down projections of the 120b long prefill
        {"name": "linear_grad_prefill_experts", "op": "linear_grad", "tokens": 4096, "top_k": 4, "experts": 128,
         "n": 2880, "k": 2880, "bias": False, "quantize": False, "skew": 0.2},
        # the balance loss and its gradient: a 20b prefill batch, and a long padded one over 120b's experts
        {"name": "balance_256", "op": "balance", "tokens": 256, "experts": 32, "top_k": 4, "masked": False},
        {"name": "balance_long", "op": "balance", "tokens": 32768, "experts": 128, "top_k": 4, "masked": True},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "swiglu", "linear", "linear", "linear_grad", "balance"])
    if op == "norm":
        return {"op": op, "tokens": _spread(rng, 1, 4096), "hidden": _spread(rng, 64, 2880),
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "fp8": rng.random() < 0.5,
                "train": rng.random() < 0.6}
    if op == "swiglu":
        return {"op": op, "rows": _spread(rng, 1, 16384), "inner": _spread(rng, 64, 2880),
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "split": rng.random() < 0.3,
                "fp8": rng.random() < 0.5, "train": rng.random() < 0.5}
    if op == "balance":
        experts = _spread(rng, 8, 128)
        return {"op": op, "tokens": _spread(rng, 1, 32768), "experts": experts, "top_k": rng.randint(1, 8),
                "masked": rng.random() < 0.5}
    dense = rng.random() < 0.4
    experts = 0 if dense else _spread(rng, 2, 128)
    return {"op": op, "tokens": _spread(rng, 1, 4096), "top_k": 1 if dense else rng.randint(1, min(4, experts)),
            "experts": experts, "n": _spread(rng, 64, 2880), "k": 16 * _spread(rng, 4, 180),
            "bias": op == "linear" and rng.random() < 0.5, "quantize": op == "linear" and rng.random() < 0.5,
            "skew": 0.0 if dense else 0.1 * rng.randint(0, 2)}


# ----------------------------------------------------------------- the inputs

def _logits(gen, tokens, experts, skew):
    rank = torch.arange(1, experts + 1, device="cuda", dtype=torch.float32)
    return torch.randn((tokens, experts), generator=gen, device="cuda") - skew * rank.log()


def _blocks(size):
    return (size + _BLOCK - 1) // _BLOCK


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    op, s = case["op"], {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def activations(rows, width):
        # channels of unequal size, as a residual stream has them
        return normal(rows, width) * torch.exp(0.5 * normal(width))

    if op in ("linear", "linear_grad"):
        tokens, top_k, experts, n, k = (case[q] for q in ("tokens", "top_k", "experts", "n", "k"))
        rows, lead = tokens * top_k, (experts,) if experts else ()
        # a block's largest weight lies at the largest code, four deviations out
        s["weight"] = (normal(*lead, n, k) * (_LARGEST / 4)).clamp_(-_LARGEST, _LARGEST).to(_E4M3)
        s["weight_scales"] = (torch.rand((*lead, _blocks(n), _blocks(k)), generator=gen, device="cuda") + 0.5) * 2e-4
        s["bias"] = (normal(*lead, n) * 0.02).bfloat16() if case["bias"] else None
        if op == "linear_grad":
            s["rows"] = normal(rows, n).bfloat16()
        else:
            s["rows"] = activations(rows, k).bfloat16()
            if not case["quantize"]:  # rows that arrive in 8 bits
                s["rows"], s["row_scales"] = _quantize(s["rows"].float())
        s["offsets"] = None
        if experts:
            ids = _logits(gen, tokens, experts, case["skew"]).topk(top_k, dim=1).indices
            counts = torch.bincount(ids.reshape(-1), minlength=experts)
            offsets = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
            offsets[1:] = counts.cumsum(0)
            s["offsets"] = offsets.to(torch.int32)
            # the plan of a padded batched product over the experts that hold rows: every row's expert
            # among those, and its place there
            s["capacity"], s["used"] = int(counts.max()), torch.nonzero(counts).reshape(-1)
            s["expert"] = torch.repeat_interleave(torch.arange(len(s["used"]), device="cuda"), counts[s["used"]])
            s["place"] = torch.arange(rows, device="cuda") - offsets[s["used"]][s["expert"]]
        return s

    if op == "norm":
        dtype, tokens, hidden = _DTYPES[case["dtype"]], case["tokens"], case["hidden"]
        s["x"], s["residual"] = normal(tokens, hidden).to(dtype), activations(tokens, hidden).to(dtype)
        s["weight"] = (1 + 0.2 * normal(hidden)).to(dtype)
        if case["train"]:
            s["dy"], s["d_summed"] = normal(tokens, hidden).to(dtype), normal(tokens, hidden).to(dtype)
    elif op == "swiglu":
        dtype, rows, inner = _DTYPES[case["dtype"]], case["rows"], case["inner"]
        # some of the gates and ups lie past the limit
        s["h"] = (3 * normal(rows, 2 * inner)).to(dtype)
        if case["train"]:
            s["da"] = normal(rows, inner).to(dtype)
    else:
        tokens, experts = case["tokens"], case["experts"]
        s["logits"] = _logits(gen, tokens, experts, 0.3)
        s["ids"] = s["logits"].topk(min(case["top_k"], experts), dim=1).indices.to(torch.int32)
        # a padded batch: about a quarter of the tokens count for nothing
        s["mask"] = torch.rand(tokens, generator=gen, device="cuda") < 0.75 if case["masked"] else None
        s["d_loss"] = 0.01 + 0.01 * torch.rand((), generator=gen, device="cuda")
        # the gradient that reaches the logits through the routing weights
        s["d_logits"] = torch.zeros(tokens, experts, device="cuda").scatter_(
            1, s["ids"].long(), normal(*s["ids"].shape) * (0.01 / tokens))
    return s


# ------------------------------------------------------------ the plain forms

def _quantize(v):
    """32-bit rows as E4M3 codes and a scale for each 128 of a row (the last block may be shorter)."""
    rows, width = v.shape
    n = _blocks(width)
    v = torch.nn.functional.pad(v, (0, n * _BLOCK - width)).reshape(rows, n, _BLOCK)
    largest = v.abs().amax(2).clamp_min(_LEAST)
    codes = (v * (_LARGEST / largest)[..., None]).reshape(rows, -1)[:, :width].to(_E4M3)
    return codes, largest / _LARGEST


def _spread_scales(scales, width, dim=-1):
    return scales.repeat_interleave(_BLOCK, dim).narrow(dim, 0, width)


def _norm(s):
    case, w = s["case"], s["weight"].float()
    summed = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    h = summed.float()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + _EPS)
    normed = h * rstd
    y = normed * w
    if case["fp8"]:
        codes, scales = _quantize(y)
        out = {"codes": codes, "scales": scales, "summed": summed}
    else:
        out = {"y": y.to(summed.dtype), "summed": summed}
    if case["train"]:
        dy = s["dy"].float()
        g = dy * w
        dx = rstd * (g - normed * (g * normed).mean(1, keepdim=True)) + s["d_summed"].float()
        out.update(dx=dx.to(summed.dtype), d_weight=(dy * normed).sum(0))
    return out


def _halves(case, h):
    if case["split"]:
        return h[:, : case["inner"]], h[:, case["inner"]:]
    return h[:, 0::2], h[:, 1::2]


def _swiglu(s):
    case = s["case"]
    gate, up = _halves(case, s["h"].float())
    g, u = gate.clamp(max=_LIMIT), up.clamp(-_LIMIT, _LIMIT)
    sig = 1 / (1 + torch.exp(-_ALPHA * g))
    a = g * sig * (u + 1)
    out = dict(zip(("codes", "scales"), _quantize(a))) if case["fp8"] else {"a": a.to(s["h"].dtype)}
    if case["train"]:
        da = s["da"].float()
        dg = torch.where(gate <= _LIMIT, da * (u + 1) * sig * (1 + _ALPHA * g * (1 - sig)), 0.0)
        du = torch.where(up.abs() <= _LIMIT, da * g * sig, 0.0)
        both = torch.cat([dg, du], 1) if case["split"] else torch.stack([dg, du], 2).reshape(dg.shape[0], -1)
        out["dh"] = both.to(s["h"].dtype)
    return out


def _linear(s):
    """Rows times their expert's weights as one padded batched product (or one product, dense)."""
    case, forward = s["case"], s["case"]["op"] == "linear"
    x = s["rows"].float()
    if forward:
        codes, scales = _quantize(x) if case["quantize"] else (s["rows"], s["row_scales"])
        x = codes.float() * _spread_scales(scales, case["k"])
    w, scales, bias = s["weight"], s["weight_scales"], s["bias"]
    if case["experts"]:
        # (the used experts' codes as bytes: their numbers alone are looked up)
        w, scales = w.view(torch.uint8)[s["used"]].view(_E4M3), scales[s["used"]]
    w = w.float() * _spread_scales(_spread_scales(scales, case["k"]), case["n"], -2)
    if not case["experts"]:
        y = x @ (w.t() if forward else w)
        return (y + bias.float() if bias is not None else y).bfloat16()
    e, i = s["expert"], s["place"]
    padded = torch.zeros(len(s["used"]), s["capacity"], x.shape[1], device="cuda")
    padded[e, i] = x
    y = torch.bmm(padded, w.transpose(1, 2) if forward else w)[e, i]
    return (y + bias[s["used"]].float()[e] if bias is not None else y).bfloat16()


def _balance(s):
    logits, ids, experts = s["logits"], s["ids"].long(), s["case"]["experts"]
    live = s["mask"] if s["mask"] is not None else torch.ones(len(logits), dtype=torch.bool, device="cuda")
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = torch.where(live[:, None], p / p.sum(1, keepdim=True), 0.0)
    counts = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    flat = torch.where(live[:, None], ids, experts).reshape(-1)
    counts = counts.scatter_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))[:-1]
    tokens = live.sum().clamp_min(1).float()
    density = experts * (counts.float() / counts.sum().clamp_min(1)) / tokens
    loss = (density * p.sum(0)).sum()
    d = s["d_loss"] * p * (density - (p * density).sum(1, keepdim=True))
    return {"loss": loss, "counts": counts, "d_logits": s["d_logits"] + d}


def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        return {"norm": _norm, "swiglu": _swiglu, "balance": _balance}.get(op, _linear)(s)

    from mxfp4_quantized_expert_amd import binding

    if op == "norm":
        if case["fp8"]:
            codes, scales, summed, rstd = binding.moe_rms_norm_fp8(s["x"], s["weight"], s["residual"], _EPS)
            out = {"codes": codes, "scales": scales, "summed": summed}
        else:
            y, summed, rstd = binding.moe_rms_norm(s["x"], s["weight"], s["residual"], _EPS)
            out = {"y": y, "summed": summed}
        if case["train"]:
            out["dx"], out["d_weight"] = binding.moe_rms_norm_backward(s["dy"], summed, s["weight"], rstd,
                                                                       s["d_summed"])
        return out
    if op == "swiglu":
        if case["fp8"]:
            out = dict(zip(("codes", "scales"), binding.moe_swiglu_fp8(s["h"], case["split"])))
        else:
            out = {"a": binding.moe_swiglu(s["h"], case["split"])}
        if case["train"]:
            out["dh"] = binding.moe_swiglu_backward(s["da"], s["h"], case["split"])
        return out
    if op == "balance":
        loss, counts, density = binding.moe_balance_loss(s["logits"], s["ids"], s["mask"])
        return {"loss": loss, "counts": counts,
                "d_logits": binding.moe_balance_loss_backward(s["logits"], density, s["d_loss"], s["mask"],
                                                              s["d_logits"])}
    if op == "linear":
        codes, scales = binding.moe_fp8_quantize(s["rows"]) if case["quantize"] else (s["rows"], s["row_scales"])
        return binding.moe_fp8_linear(codes, scales, s["weight"], s["weight_scales"], s["bias"], s["offsets"])
    return binding.moe_fp8_linear_backward(s["rows"], s["weight"], s["weight_scales"], s["offsets"])


# -------------------------------------------------------------------- the work

def work(case):
    op = case["op"]
    if op in ("linear", "linear_grad"):
        rows, n, k, experts = case["tokens"] * case["top_k"], case["n"], case["k"], case["experts"]
        # experts that a batch of evenly routed tokens reaches
        used = experts * (1 - (1 - case["top_k"] / experts) ** case["tokens"]) if experts else 1
        weight = n * k + 4 * _blocks(n) * _blocks(k) + (2 * n if case["bias"] else 0)
        row = 2 * n + (2 * k if op == "linear_grad" or case["quantize"] else k + 4 * _blocks(k))
        return {"bytes": used * weight + rows * row, "flops": 2 * rows * n * k}
    if op == "balance":
        # the logits are read for the loss, and again with the gradient that it adds to
        tokens, experts = case["tokens"], case["experts"]
        return {"bytes": tokens * (12 * experts + 4 * min(case["top_k"], experts) + (1 if case["masked"] else 0)),
                "flops": 12 * tokens * experts}
    size = 4 if case["dtype"] == "f32" else 2
    if op == "norm":
        rows, width = case["tokens"], case["hidden"]
        moved = 3 * width * size + (width + 4 * _blocks(width) if case["fp8"] else width * size)
        if case["train"]:  # dy, the stream's gradient and the sum in, dx out
            moved += 4 * width * size
        return {"bytes": rows * moved + width * size + (4 * width if case["train"] else 0),
                "flops": rows * width * (16 if case["train"] else 6)}
    rows, width = case["rows"], case["inner"]
    moved = 2 * width * size + (width + 4 * _blocks(width) if case["fp8"] else width * size)
    if case["train"]:
        moved += 5 * width * size
    return {"bytes": rows * moved, "flops": rows * width * (24 if case["train"] else 10)}


# ------------------------------------------------------------- in 64 bits, apart

def _exact_quantized(v):
    """The quotients that the codes round, and the scales, block by block."""
    parts = torch.split(v, _BLOCK, dim=1)
    scales = [torch.linalg.vector_norm(p, math.inf, dim=1).clamp_min(_LEAST) / _LARGEST for p in parts]
    return torch.cat([p / q[:, None] for p, q in zip(parts, scales)], 1), torch.stack(scales, 1)


def _exact_linear(s):
    case, forward = s["case"], s["case"]["op"] == "linear"
    n, k = case["n"], case["k"]
    x, row_scales = s["rows"].double(), None
    if forward:
        row_scales = s["row_scales"].double() if not case["quantize"] else None
        if case["quantize"]:
            x, row_scales = _exact_quantized(x)
            x = x.float().to(_E4M3).double()
        x = torch.cat([p * row_scales[:, j: j + 1] for j, p in enumerate(torch.split(x, _BLOCK, dim=1))], 1)
    bounds = [0, x.shape[0]] if s["offsets"] is None else s["offsets"].tolist()
    weight = s["weight"].reshape(-1, n, k)
    scales = s["weight_scales"].reshape(-1, _blocks(n), _blocks(k)).double()
    row = torch.arange(n, device="cuda") // _BLOCK
    col = torch.arange(k, device="cuda") // _BLOCK
    out = torch.zeros(x.shape[0], n if forward else k, dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if a == b:
            continue
        w = weight[e].double() * scales[e][row][:, col]
        out[a:b] = torch.mm(x[a:b], w.t() if forward else w)
        if s["bias"] is not None:
            out[a:b] += s["bias"].reshape(-1, n)[e].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "linear_grad"):
        return _exact_linear(s)

    if op == "norm":
        summed = s["x"].double() + s["residual"].double()
        # what follows reads the sum as it was stored
        h, w = summed.to(s["x"].dtype).double(), s["weight"].double()
        size = torch.linalg.vecdot(h, h) / case["hidden"] + _EPS
        y = h * w / size.sqrt()[:, None]
        out = dict(zip(("codes", "scales"), _exact_quantized(y))) if case["fp8"] else {"y": y}
        out["summed"] = summed
        if case["train"]:
            dy = s["dy"].double()
            # d/dh of h_i (m + eps)^(-1/2), m = sum h^2 / H
            along = torch.linalg.vecdot(dy * w, h)[:, None] * h / case["hidden"]
            out["dx"] = dy * w * size[:, None] ** -0.5 - along * size[:, None] ** -1.5 + s["d_summed"].double()
            out["d_weight"] = torch.linalg.vecdot(dy.t(), (h * size[:, None] ** -0.5).t())
        return out

    if op == "swiglu":
        h = s["h"].double()
        pairs = h.reshape(-1, 2, case["inner"]).transpose(1, 2) if case["split"] else h.reshape(-1, case["inner"], 2)
        gate, up = pairs.unbind(2)
        g, u = torch.minimum(gate, gate.new_tensor(_LIMIT)), up.clamp(-_LIMIT, _LIMIT)
        a = g * torch.sigmoid(_ALPHA * g) * (u + 1)
        out = dict(zip(("codes", "scales"), _exact_quantized(a))) if case["fp8"] else {"a": a}
        if case["train"]:
            da, sig = s["da"].double(), torch.sigmoid(_ALPHA * g)
            slope = sig + _ALPHA * g * sig * torch.sigmoid(-_ALPHA * g)
            dg = da * (u + 1) * slope * (gate <= _LIMIT)
            du = da * g * sig * ((up <= _LIMIT) & (up >= -_LIMIT))
            both = torch.stack([dg, du], 1 if case["split"] else 2)
            out["dh"] = both.reshape(h.shape)
        return out

    logits, ids, experts = s["logits"].double(), s["ids"].long(), case["experts"]
    rows = torch.arange(len(logits), device="cuda") if s["mask"] is None else torch.nonzero(s["mask"]).reshape(-1)
    d_logits = s["d_logits"].double()
    if not len(rows):
        return {"loss": torch.zeros((), dtype=torch.float64, device="cuda"), "counts": None, "d_logits": d_logits}
    p = torch.softmax(logits[rows], 1)
    share = torch.bincount(ids[rows].reshape(-1), minlength=experts).double() / (len(rows) * ids.shape[1])
    loss = experts * torch.dot(share, p.mean(0))
    # the softmax's Jacobian applied to the gradient that every token's probabilities get
    g = s["d_loss"].double() * experts * share / len(rows)
    d_logits[rows] += p * g - p * torch.mv(p, g)[:, None]
    return {"loss": loss, "counts": None, "d_logits": d_logits}
