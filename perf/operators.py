"""Cases and plain forms of the expert layer's separate operators.

The operators: token rows sorted by expert (``permute``) and summed back with the
routing weights (``unpermute``), each with its gradient; the gradient of the routing
softmax (``route_grad``); rows times 4-bit weights with group scales, dense or per
expert (``linear``), and the gradient to those rows (``linear_grad``).

``run`` computes a case in plain 32-bit torch operations, or, with ``own`` set, through
the library's entry points.  ``exact`` computes it in 64 bits.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_MAGNITUDE = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the sorted copy of a 20b decode batch: four tokens, latency alone counts
        {"name": "permute_decode", "op": "permute", "tokens": 4, "hidden": 2880, "experts": 32, "local": 32,
         "top_k": 4, "dtype": "bf16", "train": False},
        # a 120b long prefill batch in a training step: the sorted copy, then its gradient
        {"name": "permute_train_prefill", "op": "permute", "tokens": 4096, "hidden": 2880, "experts": 128,
         "local": 128, "top_k": 4, "dtype": "bf16", "train": True},
        # the end of a decode step: one token's expert outputs
        {"name": "unpermute_one_token", "op": "unpermute", "tokens": 1, "hidden": 2880, "experts": 32, "local": 32,
         "top_k": 4, "dtype": "bf16", "train": False},
        # an expert-parallel rank that owns 5 of 8 experts (tokens without a local expert among
        # them), float32 rows of an odd width, with the gradients
        {"name": "unpermute_train_share", "op": "unpermute", "tokens": 777, "hidden": 1001, "experts": 8, "local": 5,
         "top_k": 2, "dtype": "f32", "train": True},
        # the 120b long prefill's weighted sum and its gradients
        {"name": "unpermute_train_prefill", "op": "unpermute", "tokens": 4096, "hidden": 2880, "experts": 128,
         "local": 128, "top_k": 4, "dtype": "bf16", "train": True},
        # routing gradients: a 20b prefill batch, and a long batch over 120b's experts
        {"name": "route_grad_256", "op": "route_grad", "tokens": 256, "experts": 32, "top_k": 4},
        {"name": "route_grad_long", "op": "route_grad", "tokens": 32768, "experts": 128, "top_k": 4},
        # one token through a dense 4-bit projection
        {"name": "linear_one_token", "op": "linear", "format": "mxfp4", "tokens": 1, "top_k": 1, "experts": 0,
         "n": 2880, "k": 4096, "bias": True, "skew": 0.0},
        # a decode batch of 20b through its experts' gate and up rows, NVFP4
        {"name": "linear_decode_experts", "op": "linear", "format": "nvfp4", "tokens": 4, "top_k": 4, "experts": 32,
         "n": 5760, "k": 2880, "bias": True, "skew": 0.0},
        # the 120b long prefill through its experts' gate and up rows
        {"name": "linear_prefill_experts", "op": "linear", "format": "mxfp4", "tokens": 4096, "top_k": 4,
         "experts": 128, "n": 5760, "k": 2880, "bias": True, "skew": 0.2},
        # a small fine-tuning batch over few experts with ragged sizes, NVFP4
        {"name": "linear_grad_ragged", "op": "linear_grad", "format": "nvfp4", "tokens": 150, "top_k": 2,
         "experts": 8, "n": 1000, "k": 736, "bias": False, "skew": 0.0},
        # fine-tuning through the frozen down projections of the 120b long prefill
        {"name": "linear_grad_prefill_experts", "op": "linear_grad", "format": "mxfp4", "tokens": 4096, "top_k": 4,
         "experts": 128, "n": 2880, "k": 2880, "bias": False, "skew": 0.2},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute", "unpermute", "route_grad", "linear", "linear", "linear_grad"])
    if op in ("permute", "unpermute"):
        experts, tokens = _spread(rng, 4, 128), _spread(rng, 1, 4096)
        # a rank's share: at least a quarter of the experts, for batches that surely reach it
        share = tokens >= 64 and rng.random() < 0.5
        return {"op": op, "tokens": tokens, "hidden": _spread(rng, 64, 2880), "experts": experts,
                "local": rng.randint((experts + 3) // 4, experts) if share else experts, "top_k": rng.randint(1, 4),
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "train": rng.random() < 0.6}
    if op == "route_grad":
        experts = _spread(rng, 8, 128)
        return {"op": op, "tokens": _spread(rng, 1, 32768), "experts": experts, "top_k": rng.randint(2, 8)}
    dense = rng.random() < 0.4
    experts = 0 if dense else _spread(rng, 2, 128)
    return {"op": op, "format": rng.choice(["mxfp4", "nvfp4"]), "tokens": _spread(rng, 1, 4096),
            "top_k": 1 if dense else rng.randint(1, min(4, experts)), "experts": experts, "n": _spread(rng, 64, 2880),
            "k": 32 * _spread(rng, 2, 90), "bias": op == "linear" and rng.random() < 0.5,
            "skew": 0.0 if dense else 0.1 * rng.randint(0, 2)}


# ----------------------------------------------------------------- the inputs

def _routing(gen, tokens, experts, top_k, skew=0.0):
    """A batch's routing: ids and weights of its top_k experts, pairs ordered by (expert, pair), offsets."""
    rank = torch.arange(1, experts + 1, device="cuda", dtype=torch.float32)
    logits = torch.randn((tokens, experts), generator=gen, device="cuda") - skew * rank.log()
    top, ids = logits.topk(top_k, dim=1)
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.bincount(flat, minlength=experts).cumsum(0)
    return ids, torch.softmax(top, 1), order, offsets


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    s = {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    op = case["op"]
    if op in ("linear", "linear_grad"):
        tokens, top_k, experts, n, k = (case[q] for q in ("tokens", "top_k", "experts", "n", "k"))
        group = 32 if case["format"] == "mxfp4" else 16
        rows, lead = tokens * top_k, (experts,) if experts else ()
        s["blocks"] = torch.randint(0, 256, lead + (n, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
        lo, hi = (118, 132) if group == 32 else (0x30, 0x48)
        s["scales"] = torch.randint(lo, hi + 1, lead + (n, k // group), generator=gen, device="cuda",
                                    dtype=torch.uint8)
        s["scale2"] = None
        if group == 16:
            s["scale2"] = torch.rand(max(experts, 1), generator=gen, device="cuda") * (3 / 16) + 1 / 16
        s["bias"] = (normal(*lead, n) * 0.02).bfloat16() if case["bias"] else None
        s["rows"] = normal(rows, k if op == "linear" else n).bfloat16()
        s["offsets"] = None
        if experts:
            offsets = _routing(gen, tokens, experts, top_k, case["skew"])[3]
            s["offsets"] = offsets.to(torch.int32)
            # the plan of a padded batched product over the experts that hold rows: every row's expert
            # among those, and its place there
            counts = offsets[1:] - offsets[:-1]
            s["capacity"], s["used"] = int(counts.max()), torch.nonzero(counts).reshape(-1)
            s["expert"] = torch.repeat_interleave(torch.arange(len(s["used"]), device="cuda"), counts[s["used"]])
            s["place"] = torch.arange(rows, device="cuda") - offsets[s["used"]][s["expert"]]
        return s

    tokens, experts, top_k = case["tokens"], case["experts"], min(case["top_k"], case["experts"])
    ids, weights, order, offsets = _routing(gen, tokens, experts, top_k)
    s["top_k"] = top_k
    if op == "route_grad":
        s["ids"], s["weights"] = ids.to(torch.int32), weights
        s["d_weights"] = normal(tokens, top_k)
        return s
    # experts below `local` are this rank's: their pairs first, then empty rows
    here = ids.reshape(-1)[order] < case["local"]
    s["sorted_pairs"] = torch.where(here, order, -torch.ones_like(order)).to(torch.int32)
    place = torch.full((tokens * top_k,), -1, dtype=torch.int32, device="cuda")
    place[order[here]] = torch.nonzero(here).reshape(-1).to(torch.int32)
    dtype = _DTYPES[case["dtype"]]
    if op == "permute":
        s["x"] = normal(tokens, case["hidden"]).to(dtype)
        s["d_rows"] = normal(tokens * top_k, case["hidden"]).to(dtype)
    else:
        s["pair_rows"] = place
        s["weights"] = weights
        s["rows"] = normal(tokens * top_k, case["hidden"]).to(dtype)
        s["dy"] = normal(tokens, case["hidden"]).to(dtype)
    return s


# ------------------------------------------------------------ the plain forms

def _weights(s, dtype):
    """The weights that the codes and group scales stand for, [..., N, K] (of the experts that hold rows)."""
    case, blocks, scales = s["case"], s["blocks"], s["scales"]
    if case["experts"]:
        blocks, scales = blocks[s["used"]], scales[s["used"]]
    value = torch.tensor(_MAGNITUDE + [-m for m in _MAGNITUDE], dtype=dtype, device="cuda")
    byte = torch.arange(256, device="cuda")
    w = torch.stack([value[byte & 15], value[byte >> 4]], 1)[blocks.to(torch.int32)]
    if case["format"] == "mxfp4":
        scale = torch.exp2(scales.to(dtype) - 127)
    else:
        scale = scales.view(torch.float8_e4m3fn).to(dtype)
    return (w.reshape(*scale.shape, -1) * scale[..., None]).reshape(*blocks.shape[:-1], -1)


def _linear(s):
    """Rows times their expert's weights as one padded batched product (or one product, dense)."""
    case, x = s["case"], s["rows"].float()
    w, scale2, bias = _weights(s, torch.float32), s["scale2"], s["bias"]
    forward = case["op"] == "linear"
    if not case["experts"]:
        y = x @ (w.t() if forward else w)
        y = y * scale2 if scale2 is not None else y
        return (y + bias.float() if bias is not None else y).bfloat16()
    e, i = s["expert"], s["place"]
    padded = torch.zeros(len(s["used"]), s["capacity"], x.shape[1], device="cuda")
    padded[e, i] = x
    y = torch.bmm(padded, w.transpose(1, 2) if forward else w)[e, i]
    y = y * scale2[s["used"]][e, None] if scale2 is not None else y
    return (y + bias[s["used"]].float()[e] if bias is not None else y).bfloat16()


def _permute(s):
    case, x, pairs, k = s["case"], s["x"], s["sorted_pairs"].long(), s["top_k"]
    rows = torch.where(pairs[:, None] >= 0, x[pairs.clamp_min(0) // k], torch.zeros((), dtype=x.dtype, device="cuda"))
    # the row of every pair; empty rows write to a place behind the last pair
    pair_rows = torch.full((pairs.numel() + 1,), -1, dtype=torch.int32, device="cuda")
    pair_rows[torch.where(pairs >= 0, pairs, pairs.numel())] = torch.arange(pairs.numel(), dtype=torch.int32,
                                                                            device="cuda")
    pair_rows = pair_rows[:-1]
    if not case["train"]:
        return {"rows": rows, "pair_rows": pair_rows}
    back = s["d_rows"].float()[pair_rows.clamp_min(0)] * (pair_rows >= 0)[:, None]
    return {"rows": rows, "pair_rows": pair_rows, "dx": back.reshape(-1, k, x.shape[1]).sum(1).to(x.dtype)}


def _unpermute(s):
    case, z, w, k = s["case"], s["rows"], s["weights"], s["top_k"]
    at, there = s["pair_rows"].clamp_min(0), s["pair_rows"] >= 0
    taken = torch.where(there[:, None], z[at].float(), 0.0).reshape(-1, k, z.shape[1])
    y = (w[..., None] * taken).sum(1).to(z.dtype)
    if not case["train"]:
        return {"y": y}
    dy = s["dy"].float()
    d_weights = (taken * dy[:, None]).sum(2)
    pairs = s["sorted_pairs"].long()
    scaled = w.reshape(-1)[pairs.clamp_min(0), None] * dy[pairs.clamp_min(0) // k]
    return {"y": y, "d_rows": torch.where(pairs[:, None] >= 0, scaled, 0.0).to(z.dtype), "d_weights": d_weights}


def _route_grad(s):
    w, dw = s["weights"], s["d_weights"]
    g = w * (dw - (w * dw).sum(1, keepdim=True))
    out = torch.zeros(w.shape[0], s["case"]["experts"], device="cuda")
    return out.scatter_(1, s["ids"].long(), g)


def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        if op == "permute":
            return _permute(s)
        if op == "unpermute":
            return _unpermute(s)
        return _route_grad(s) if op == "route_grad" else _linear(s)

    from mxfp4_quantized_expert_amd import binding

    if op == "permute":
        rows, pair_rows = binding.moe_permute(s["x"], s["sorted_pairs"], s["top_k"])
        if not case["train"]:
            return {"rows": rows, "pair_rows": pair_rows}
        return {"rows": rows, "pair_rows": pair_rows,
                "dx": binding.moe_permute_backward(s["d_rows"], pair_rows, s["top_k"])}
    if op == "unpermute":
        y = binding.moe_unpermute(s["rows"], s["pair_rows"], s["weights"])
        if not case["train"]:
            return {"y": y}
        d_rows, d_weights = binding.moe_unpermute_backward(s["dy"], s["rows"], s["sorted_pairs"], s["pair_rows"],
                                                           s["weights"])
        return {"y": y, "d_rows": d_rows, "d_weights": d_weights}
    if op == "route_grad":
        return binding.moe_route_backward(s["ids"], s["weights"], s["d_weights"], case["experts"])
    if op == "linear":
        if case["format"] == "mxfp4":
            return binding.moe_mxfp4_linear(s["rows"], s["blocks"], s["scales"], s["bias"], s["offsets"])
        return binding.moe_nvfp4_linear(s["rows"], s["blocks"], s["scales"], s["scale2"], s["bias"], s["offsets"])
    if case["format"] == "mxfp4":
        return binding.moe_mxfp4_linear_backward(s["rows"], s["blocks"], s["scales"], s["offsets"])
    return binding.moe_nvfp4_linear_backward(s["rows"], s["blocks"], s["scales"], s["scale2"], s["offsets"])


# -------------------------------------------------------------------- the work

def work(case):
    op = case["op"]
    if op in ("linear", "linear_grad"):
        rows, n, k, experts = case["tokens"] * case["top_k"], case["n"], case["k"], case["experts"]
        # experts that a batch of evenly routed tokens reaches
        used = experts * (1 - (1 - case["top_k"] / experts) ** case["tokens"]) if experts else 1
        weight = n * k * (0.5 + (1 / 32 if case["format"] == "mxfp4" else 1 / 16))
        return {"bytes": used * (weight + (2 * n if case["bias"] else 0)) + 2 * rows * (n + k),
                "flops": 2 * rows * n * k}
    tokens, top_k = case["tokens"], min(case["top_k"], case["experts"])
    pairs = tokens * top_k
    if op == "route_grad":
        return {"bytes": pairs * 12 + 4 * tokens * case["experts"], "flops": 5 * pairs}
    row = case["hidden"] * (4 if case["dtype"] == "f32" else 2)
    held = pairs * case["local"] / case["experts"]  # rows that hold a pair
    if op == "permute":  # every row is written, the gradient reads those that hold a pair
        moved = (tokens + pairs) * row + 8 * pairs
        return {"bytes": moved + ((held + tokens) * row + 4 * pairs if case["train"] else 0),
                "flops": held * case["hidden"] if case["train"] else 0}
    moved = (held + tokens) * row + 8 * pairs
    if case["train"]:
        moved += (tokens + held + pairs) * row + 16 * pairs
    return {"bytes": moved, "flops": held * case["hidden"] * (5 if case["train"] else 2)}


# ------------------------------------------------------------- in 64 bits, apart

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route_grad":
        # the Jacobian of the softmax over the picks, diag(w) - w w^T, applied to each token's gradient
        w, dw = s["weights"].double(), s["d_weights"].double()
        g = torch.matmul(torch.diag_embed(w) - w[:, :, None] * w[:, None, :], dw[:, :, None])[..., 0]
        one_hot = s["ids"].long()[..., None] == torch.arange(case["experts"], device="cuda")
        return torch.stack([(one_hot[:, j] * g[:, j, None]) for j in range(w.shape[1])]).sum(0)

    if op in ("linear", "linear_grad"):
        x, forward = s["rows"].double(), op == "linear"
        out = torch.zeros(x.shape[0], case["n"] if forward else case["k"], dtype=torch.float64, device="cuda")
        bounds = [0, x.shape[0]] if s["offsets"] is None else s["offsets"].tolist()
        blocks, scales = (s[q].reshape(-1, *s[q].shape[-2:]) for q in ("blocks", "scales"))
        magnitude = torch.tensor(_MAGNITUDE, dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
            if a == b:
                continue
            code = torch.stack([blocks[e] & 15, blocks[e] >> 4], -1).reshape(case["n"], case["k"]).long()
            w = torch.where(code >= 8, -1.0, 1.0) * magnitude[code & 7]
            byte = scales[e].long()
            if case["format"] == "mxfp4":
                scale = torch.ldexp(torch.ones_like(byte, dtype=torch.float64), byte - 127)
            else:  # four exponent bits (bias 7) over three mantissa bits
                exponent, mantissa = (byte >> 3) & 15, (byte & 7).double()
                scale = torch.where(exponent > 0, (8 + mantissa) * torch.exp2(exponent.double() - 10),
                                    mantissa * 2.0 ** -9) * torch.where(byte >= 128, -1.0, 1.0)
                scale = scale * s["scale2"][e].double()
            w = w * scale.repeat_interleave(case["k"] // scale.shape[1], 1)
            out[a:b] = torch.mm(x[a:b], w.t() if forward else w)
            if s["bias"] is not None:
                out[a:b] += s["bias"].reshape(-1, case["n"])[e].double()
        return out

    # the pairs' places as a sorted list, without those of other ranks
    k, tokens = s["top_k"], case["tokens"]
    row = torch.nonzero(s["sorted_pairs"] >= 0).reshape(-1)
    pair = s["sorted_pairs"].long()[row]
    token = torch.div(pair, k, rounding_mode="floor")
    if op == "permute":
        rows = torch.zeros(tokens * k, case["hidden"], dtype=torch.float64, device="cuda")
        rows[row] = s["x"].double()[token]
        got = {"rows": rows, "pair_rows": None}
        if case["train"]:
            dx = torch.zeros(tokens, case["hidden"], dtype=torch.float64, device="cuda")
            got["dx"] = dx.index_add_(0, token, s["d_rows"].double()[row])
        return got
    w, z, dy = s["weights"].double().reshape(-1)[pair], s["rows"].double()[row], s["dy"].double()[token]
    y = torch.zeros(tokens, case["hidden"], dtype=torch.float64, device="cuda").index_add_(0, token, w[:, None] * z)
    got = {"y": y}
    if case["train"]:
        d_rows = torch.zeros(tokens * k, case["hidden"], dtype=torch.float64, device="cuda")
        d_rows[row] = w[:, None] * dy
        d_weights = torch.zeros(tokens * k, dtype=torch.float64, device="cuda")
        d_weights[pair] = torch.linalg.vecdot(dy, z)
        got.update(d_rows=d_rows, d_weights=d_weights.reshape(tokens, k))
    return got
