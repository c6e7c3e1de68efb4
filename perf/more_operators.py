"""Cases of the experts' operators: the router with its balance loss, and the
layers' products in 8-bit floating point with a scale for each block of 128.

The operators (E experts; F8 = a pair of 8-bit floats q, rows x cols, and scales,
ceil(cols / 128) x rows for blocks of 1 x 128 or ceil(cols / 128) x
ceil(rows / 128) for blocks of 128 x 128, standing for q times its block's scale):

  quantize    X to F8 and back, X^T to F8 and back, or both: s = max |x| / top of
              a block in fp32, at least 2^-126 (pow2: the smallest power of two
              >= max |x| / top, kept in 8 bits), q = x / s rounded to the nearest
              8-bit float, ties to even; top = 448 (e4m3) or 57344 (e5m2)
  matmul      C <- beta C + A B^T, A and B both F8
  route       p = softmax of a token's logits, its top_k experts (ties to the
              lowest index; an expert of logit -inf is none, index -1), their
              weights p, or p / sum of the chosen p, the tokens per expert c_e,
              P_e = sum of p_e over the n tokens that have an expert, and the
              balance loss E sum_e (c_e / sum c) (P_e / n)
  route_grad  the logits' gradient from those of the weights and of the loss

`run` computes them in plain form, or with `own` through
newton_schulz_04_amd. Weights are those of the library's workloads:
8192 x 6144, experts of 2048 x 6144 and 512 x 10240; counts of tokens and of
experts are generic.
"""
import math
import random

import numpy
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# (bits of the significand, exponent of the smallest normal number, largest number)
SHAPES = {"e4m3": (4, -6, 448.0), "e5m2": (3, -14, 57344.0)}
# the largest products, copies and routers listed, which no drawn case exceeds
MOST_FLOPS = 2 * 4096 * 8192 * 6144
MOST_VALUES = 8192 * 6144
MOST_LOGITS = 32768 * 256


def listed():
    return [
        # the inputs of a few tokens before the product that serves them: latency
        {"name": "quantize_decode", "op": "quantize", "mats": 1, "rows": 4, "cols": 6144, "square": False,
         "form": "rows", "pow2": True, "format": "e4m3", "dtype": "bf16"},
        # a dense layer's input for its forward product and, transposed, for its weight gradient
        {"name": "quantize_dense_both", "op": "quantize", "mats": 1, "rows": 8192, "cols": 6144, "square": False,
         "form": "both", "pow2": True, "format": "e4m3", "dtype": "bf16"},
        # fp32 weights of experts after an optimizer step, odd sizes, for both directions
        {"name": "quantize_weights_fp32", "op": "quantize", "mats": 4, "rows": 4 * 2043, "cols": 6101, "square": True,
         "form": "both", "pow2": False, "format": "e4m3", "dtype": "fp32"},
        # one token through a dense layer: the weights are read once
        {"name": "matmul_one_token", "op": "matmul", "items": 1, "m": 1, "n": 8192, "k": 6144, "ragged": "m",
         "square": True, "pow2": True, "format": "e4m3", "dtype": "bf16", "beta": 0.0},
        # a training batch through a dense layer
        {"name": "matmul_dense", "op": "matmul", "items": 1, "m": 4096, "n": 8192, "k": 6144, "ragged": "m",
         "square": True, "pow2": True, "format": "e4m3", "dtype": "bf16", "beta": 0.0},
        # sixteen experts with ragged token counts, one of them without tokens
        {"name": "matmul_experts", "op": "matmul", "items": 16, "m": 3001, "n": 2048, "k": 6144, "ragged": "m",
         "square": True, "pow2": True, "format": "e4m3", "dtype": "bf16", "beta": 0.0},
        # experts whose weights come with fp32 scales
        {"name": "matmul_fp32_scales", "op": "matmul", "items": 4, "m": 1999, "n": 2048, "k": 6144, "ragged": "m",
         "square": True, "pow2": False, "format": "e4m3", "dtype": "bf16", "beta": 0.0},
        # a dense layer's weight gradient, summed over an odd count of tokens, into an fp32 buffer
        {"name": "grad_weight_dense", "op": "matmul", "items": 1, "m": 8192, "n": 6144, "k": 4001, "ragged": "k",
         "square": False, "pow2": True, "format": "e5m2", "dtype": "fp32", "beta": 1.0},
        # the router of a few tokens: latency
        {"name": "route_decode", "op": "route", "tokens": 8, "experts": 16, "top_k": 2, "normalize": True,
         "masked": False, "dtype": "bf16"},
        # a training batch's
        {"name": "route_train", "op": "route", "tokens": 32768, "experts": 256, "top_k": 8, "normalize": True,
         "masked": False, "dtype": "fp32"},
        # the gradient of the same router
        {"name": "route_grad_train", "op": "route_grad", "tokens": 32768, "experts": 256, "top_k": 8,
         "normalize": True, "masked": False, "dtype": "fp32"},
        # a padded batch of odd sizes
        {"name": "route_grad_padded", "op": "route_grad", "tokens": 4001, "experts": 47, "top_k": 3,
         "normalize": False, "masked": True, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _width(rng, lo, hi):
    """A layer's width: mostly a multiple of 16, now and then any number."""
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.25 else max(16, n // 16 * 16)


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "route", "route_grad"])
    dtype = rng.choice(["bf16", "fp32"])
    if op in ("route", "route_grad"):
        experts = _log_int(rng, 2, 512)
        tokens = min(_log_int(rng, 1, 32768), MOST_LOGITS // experts)
        return {"op": op, "tokens": tokens, "experts": experts, "top_k": rng.randint(1, min(8, experts)),
                "normalize": rng.random() < 0.5, "masked": rng.random() < 0.5, "dtype": dtype}
    kind = {"pow2": rng.random() < 0.7, "format": rng.choice(["e4m3", "e4m3", "e5m2"]), "dtype": dtype}
    if op == "quantize":
        cols = _width(rng, 24, 10240)
        rows = max(1, min(_log_int(rng, 1, 8192), MOST_VALUES // cols))
        return {"op": op, "mats": min(rows, rng.choice([1, 1, 2, 5, 16])), "rows": rows, "cols": cols,
                "square": rng.random() < 0.3, "form": rng.choice(["rows", "transposed", "both"]), **kind}
    items = rng.choice([1, 1, 1, 2, 5, 16])
    if rng.random() < 0.6:
        # a layer's tokens, forward or backward
        n, k, m = _width(rng, 16, 10240), _width(rng, 24, 10240), _log_int(rng, 1, 8192)
        m = max(1, min(m, MOST_FLOPS // (2 * n * k)))
        while items > 1 and items * n * k > 16 * 2048 * 6144:
            items //= 2
        return {"op": op, "items": items, "m": m, "n": n, "k": k, "ragged": "m", "square": rng.random() < 0.8,
                **kind, "beta": 0.0}
    # a layer's weights, summed over its tokens
    m, n, k = _width(rng, 16, 10240), _width(rng, 24, 10240), _log_int(rng, 1, 8192)
    k = max(1, min(k, MOST_FLOPS // (2 * m * n)))
    while items > 1 and items * m * n > 8 * 2048 * 6144:
        items //= 2
    return {"op": op, "items": items, "m": m, "n": n, "k": k, "ragged": "k", "square": False, **kind,
            "beta": rng.choice([0.0, 0.9375, 1.0])}


def shares(case):
    """Tokens of each item of a case: ragged, the third one without any
    (quantize: as even as they come)."""
    if case["op"] == "quantize":
        n, total = case["mats"], case["rows"]
        return [total // n + (i < total % n) for i in range(n)]
    n, total = case["items"], case[case["ragged"]]
    if n == 1:
        return [total]
    rng = random.Random(1000 * n + total)
    w = [0.0 if i == 2 else rng.random() ** 2 + 0.05 for i in range(n)]
    counts = [int(total * v / sum(w)) for v in w]
    counts[0] += total - sum(counts)
    return counts


def sizes(case):
    """(m, n, k) of each product of a case."""
    return [(t, case["n"], case["k"]) if case["ragged"] == "m" else (case["m"], case["n"], t) for t in shares(case)]


def _blocks(x, square):
    """The largest magnitude of each block, and each value's, in 64 bits."""
    rows, cols = x.shape
    tall = 128 if square else 1
    nr, nc = -(-rows // tall), -(-cols // 128)
    wide = x.new_zeros((nr * tall, nc * 128), dtype=torch.float64)
    wide[:rows, :cols] = x.abs()
    top = wide.view(nr, tall, nc, 128).amax((1, 3))
    return top, lambda v: v.repeat_interleave(tall, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def _power(e):
    """2^e of normal numbers, from their bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _scales(top, largest, pow2):
    if not pow2:
        return (top / largest).float().clamp_min(2.0 ** -126).double()
    m, e = torch.frexp(top / largest)
    return _power(torch.where(m > 0.5, e, e - 1).clamp_min(-126))


def _round8(y, shape):
    """y to the nearest 8-bit float, ties to even, in 64 bits: a quotient next to
    a border must not be rounded twice."""
    bits, least, largest = shape
    e = torch.frexp(y)[1].clamp_min(least + 1)
    step = _power(e - bits)
    return ((y / step).round() * step).clamp(-largest, largest)


def _f8(x, square, pow2, format):
    """F8 of x as the library's quantiser lays it out: q at a pitch of a multiple
    of 16 bytes, scales block by block at a pitch of a multiple of 16."""
    rows, cols = x.shape
    top, spread = _blocks(x, square)
    s = _scales(top, SHAPES[format][2], pow2)
    v = _round8(x.double() / spread(s), SHAPES[format]).float()
    q = torch.empty((rows, -(-cols // 16) * 16), dtype=FORMATS[format], device=x.device)[:, :cols]
    q.copy_(v)
    kept = torch.float8_e8m0fnu if pow2 else torch.float32
    scale = torch.empty((s.shape[1], -(-s.shape[0] // 16) * 16), dtype=kept, device=x.device)[:, :s.shape[0]]
    scale.copy_(s.T.float())
    return q, scale


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    state = {"case": case, "dtype": dtype}
    if op in ("route", "route_grad"):
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        # experts of unlike popularity
        state["logits"] = (2 * normal(t, e) + normal(e)).to(dtype)
        # the last tenth of a padded batch, and single tokens before it
        state["mask"] = (uniform(t) < 0.95) & (torch.arange(t, device=dev) < t - t // 10) if case["masked"] else None
        if op == "route_grad":
            state["dweights"], state["dloss"] = normal(t, k), 0.01 * uniform(1)[0]
            experts, _, _, n = _plain_route(state["logits"], state["mask"], k, case["normalize"])
            # as a run of `route` leaves them
            state["experts"], state["tokens"] = experts, n
            state["counts"] = _counts(experts, e)
        return state
    if op == "quantize":
        # a few channels are an order of magnitude larger, as in a transformer's residual stream
        width = torch.where(uniform(case["cols"]) < 0.01, 10.0, 1.0)
        state["x"] = [(normal(r, case["cols"]) * width).to(dtype) for r in shares(case)]
        return state

    def operand(rows, cols, square, format):
        return _f8(normal(rows, cols) * torch.exp(normal(rows, 1)), square, case["pow2"], format)

    # (gradients in e5m2 meet weights and inputs in e4m3)
    state["a"] = [operand(m, k, False, case["format"]) for m, n, k in sizes(case)]
    state["b"] = [operand(n, k, case["square"], "e4m3") for m, n, k in sizes(case)]
    state["c"] = [normal(m, n).to(dtype) for m, n, _ in sizes(case)] if case["beta"] else None
    return state


def _plain_round_trip(x, case, dtype):
    """Rounded in 64 bits, then read back in 32."""
    top, spread = _blocks(x, case["square"])
    s = spread(_scales(top, SHAPES[case["format"]][2], case["pow2"]))
    return (_round8(x.double() / s, SHAPES[case["format"]]).float() * s.float()).to(dtype)


def _values(q, scale):
    """What an F8 pair stands for, in 32 bits."""
    rows, cols = q.shape
    s = scale.float().repeat_interleave(128, 0)[:cols].T
    return q.float() * (s if s.shape[0] == rows else s.repeat_interleave(128, 0)[:rows])


def _counts(experts, n):
    """Tokens per expert."""
    return torch.zeros(n + 1, dtype=torch.int32, device=experts.device).index_add_(
        0, experts.flatten() + 1, torch.ones_like(experts).flatten())[1:]


def _plain_route(logits, mask, top_k, normalize):
    """experts, their weights, p (0 for tokens that do not count), n"""
    x = logits.float()
    p = torch.exp(x - x.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    experts = x.sort(dim=1, descending=True, stable=True).indices[:, :top_k].int()
    weights = p.gather(1, experts.long())
    if normalize:
        weights = weights / weights.sum(1, keepdim=True)
    if mask is not None:
        experts = torch.where(mask[:, None], experts, -1)
        weights, p = weights * mask[:, None], p * mask[:, None]
        n = mask.sum(dtype=torch.int32)
    else:
        n = torch.full((), x.shape[0], dtype=torch.int32, device=x.device)
    return experts, weights, p, n


def run(state):
    case, dtype = state["case"], state["dtype"]
    op = case["op"]
    if own:
        import newton_schulz_04_amd as ns
        if op == "quantize":
            kept = ns.f8_quantize(state["x"], form=case["form"], square=case["square"], pow2=case["pow2"],
                                  dtype=FORMATS[case["format"]])
            if case["form"] == "both":
                kept = [half for pair in kept for half in pair]
            return ns.f8_dequantize(kept, dtype=dtype)
        if op == "matmul":
            return ns.f8_matmul(state["a"], state["b"], dtype=dtype, out=state["c"], beta=case["beta"])
        if op == "route":
            r = ns.route_experts(state["logits"], case["top_k"], normalize=case["normalize"], mask=state["mask"])
            return {"experts": r.experts, "weights": r.weights, "counts": r.counts, "probs": r.probs,
                    "loss": r.loss}
        return ns.route_experts_grad(state["logits"], state["experts"], state["counts"], state["tokens"],
                                     dweights=state["dweights"], dloss=state["dloss"], normalize=case["normalize"])
    if op == "quantize":
        forms = {"rows": (False,), "transposed": (True,), "both": (False, True)}[case["form"]]
        return [_plain_round_trip(x.T if turned else x, case, dtype) for x in state["x"] for turned in forms]
    if op == "matmul":
        sums = [_values(*a) @ _values(*b).T for a, b in zip(state["a"], state["b"])]
        if state["c"] is None:
            return [s.to(dtype) for s in sums]
        return [c.copy_(case["beta"] * c.float() + s) for c, s in zip(state["c"], sums)]
    e = case["experts"]
    if op == "route":
        experts, weights, p, n = _plain_route(state["logits"], state["mask"], case["top_k"], case["normalize"])
        counts, probs = _counts(experts, e), p.sum(0)
        loss = e * (counts.float() / counts.sum().clamp_min(1) * (probs / n.clamp_min(1))).sum()
        return {"experts": experts, "weights": weights, "counts": counts, "probs": probs, "loss": loss}
    x, experts = state["logits"].float(), state["experts"].long()
    live = experts >= 0
    p = torch.exp(x - x.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    h = state["dweights"] * live
    if case["normalize"]:
        chosen = p.gather(1, experts.clamp_min(0)) * live
        total = chosen.sum(1, keepdim=True).clamp_min(2.0 ** -126)
        # (one expert has the weight 1, and no gradient)
        h = (h - (h * (chosen / total)).sum(1, keepdim=True)) / total * live
    share = state["counts"].float() / state["counts"].sum().clamp_min(1)
    g = (state["dloss"] * e / state["tokens"].clamp_min(1)) * share.expand_as(x)
    g = g.scatter_add(1, experts.clamp_min(0), h)
    return (p * (g - (g * p).sum(1, keepdim=True)) * live[:, :1]).to(dtype)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "quantize":
        ways = 2 if case["form"] == "both" else 1
        values = case["rows"] * case["cols"]
        # values in; int8 written and read, and values back out, for each form
        return {"bytes": values * (size + ways * (2 + size)), "flops": 4 * ways * values}
    if case["op"] == "matmul":
        moved = flops = 0
        for m, n, k in sizes(case):
            passes = 2 if case["beta"] else 1
            # an item without rows or without a sum reads nothing
            live = 1 if m * n * k else 0
            moved += live * (m + n) * k + passes * size * m * n
            flops += 2 * m * n * k
        return {"bytes": moved, "flops": flops}
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    if case["op"] == "route":
        return {"bytes": t * (e * size + 8 * k) + 8 * e, "flops": t * e * (6 + k)}
    return {"bytes": t * (2 * e * size + 8 * k) + 4 * e, "flops": t * (9 * e + 4 * k)}


def _exact_scale(top, largest, pow2):
    s = (top / largest).astype(numpy.float32).astype(numpy.float64)
    if pow2:
        # from a power of two below, up
        s = 2.0 ** (numpy.floor(numpy.log2(numpy.maximum(top, 2.0 ** -110) / largest)) - 1)
        for _ in range(2):
            s = numpy.where(largest * s < top, 2 * s, s)
    return numpy.maximum(s, 2.0 ** -126)


def _exact_block(v, case):
    """The values of one block of a matrix, from its definition."""
    bits, least, largest = SHAPES[case["format"]]
    s = _exact_scale(numpy.abs(v).max(axis=-1, keepdims=True), largest, case["pow2"])
    r = numpy.abs(v / s)
    unit = 2.0 ** (numpy.floor(numpy.log2(numpy.maximum(r, 2.0 ** least))) - (bits - 1))
    low = numpy.floor(r / unit)
    part = r / unit - low
    up = (part > 0.5) | ((part == 0.5) & (low % 2 == 1))
    return numpy.sign(v) * numpy.minimum((low + up) * unit, largest) * s


def _exact_quantize(x, case):
    rows, cols = x.shape
    out = numpy.empty((rows, cols))
    for c in range(0, cols, 128):
        piece = x[:, c:c + 128]
        if not case["square"]:
            out[:, c:c + 128] = _exact_block(piece, case)
            continue
        for r in range(0, rows, 128):
            part = piece[r:r + 128]
            out[r:r + 128, c:c + 128] = _exact_block(part.reshape(1, -1), case).reshape(part.shape)
    return out


def exact(case, seed):
    """The definitions in 64 bits."""
    op = case["op"]
    if op == "quantize":
        if case["rows"] * case["cols"] > 1 << 23:
            return None   # (more than 20 seconds)
        state, out = prepare(case, seed), []
        for x in state["x"]:
            v = x.double().cpu().numpy()
            if case["form"] != "transposed":
                out.append(_exact_quantize(v, case))
            if case["form"] != "rows":
                out.append(_exact_quantize(numpy.ascontiguousarray(v.T), case))
        return out
    state = prepare(case, seed)
    if op == "matmul":
        out = []
        for i, ((qa, sa), (qb, sb)) in enumerate(zip(state["a"], state["b"])):
            (m, k), n = qa.shape, qb.shape[0]
            c = torch.zeros((m, n), dtype=torch.float64, device=qa.device)
            if state["c"] is not None:
                c += case["beta"] * state["c"][i].double()
            # block by block, as the definition reads
            for b in range(-(-k // 128)):
                a8, b8 = (q[:, 128 * b:128 * b + 128].double() for q in (qa, qb))
                wb = sb[b].double()
                if wb.shape[0] != n:
                    wb = wb[torch.arange(n, device=wb.device) // 128]
                c += sa[b].double()[:, None] * torch.matmul(a8, b8.T.contiguous()) * wb
            out.append(c)
        return out
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    x = state["logits"].double().cpu().numpy()
    live = numpy.ones(t, bool) if state["mask"] is None else state["mask"].cpu().numpy()
    p = numpy.exp(x - x.max(1, keepdims=True))
    p = p / p.sum(1, keepdims=True) * live[:, None]
    chosen = numpy.argsort(-x, axis=1, kind="stable")[:, :k]
    picked = numpy.take_along_axis(p, chosen, 1)
    total = numpy.where(live, picked.sum(1), 1.0)[:, None]
    counts = numpy.bincount(chosen[live].reshape(-1), minlength=e)
    n = max(1, int(live.sum()))
    if op == "route":
        return {"experts": numpy.where(live[:, None], chosen, -1).astype(numpy.int32),
                "weights": picked / total if case["normalize"] else picked, "counts": counts.astype(numpy.int32),
                "probs": p.sum(0), "loss": e * float((counts / max(1, counts.sum()) * p.sum(0)).sum()) / n}
    dw = state["dweights"].double().cpu().numpy() * live[:, None]
    if case["normalize"]:
        dw = (dw - (dw * (picked / total)).sum(1, keepdims=True)) / total * live[:, None]
    g = numpy.tile(float(state["dloss"]) * e / n * counts / max(1, counts.sum()), (t, 1))
    rows = numpy.arange(t)[:, None]
    g[rows, chosen] += dw
    return p * (g - (g * p).sum(1, keepdims=True))
