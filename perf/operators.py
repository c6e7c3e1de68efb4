"""Cases of the 8-bit linear-layer operators: what is computed, on which
inputs, in plain torch operations and through the library.

The operators (T tokens, `out` x `inp` weights, one scale per row of a
quantised matrix, Q8 = a pair of int8 values q and row scales s, standing for q s):

  checkpoint   rows of X to Q8 and back: s = max |x| / 127 per row in fp32, at
               least 2^-126 (pow2: the smallest power of two >= max |x| / 127),
               q = x / s rounded to the nearest integer, ties to even;
               read back as q s
  matmul       Y = Xq Wq^T, both Q8 (token scales, channel scales)
  grad_input   dX = dY Wq, Wq Q8 with channel scales
  grad_weight  G <- beta G + dY^T Xq, Xq the Q8 checkpoint of the layer's input

Each takes a list of layers (or experts) of any shapes in one call.
`run` computes them in plain form, or with `own` through
newton_schulz_04_amd. Sizes are those of the library's workloads: weights of
8192 x 6144, experts of 2048 x 6144 and 512 x 10240, attention gates of
18 x 2304, 64 x 32 for the smallest; token counts are generic.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# the largest products and copies listed, which no drawn case exceeds
MOST_FLOPS = 2 * 4096 * 8192 * 6144
MOST_VALUES = 8192 * 6144


def listed():
    return [
        # a training step keeps the input of a dense layer for the backward pass
        {"name": "checkpoint_dense", "op": "checkpoint", "layers": 1, "tokens": 8192, "inp": 6144,
         "pow2": True, "dtype": "bf16"},
        # the inputs of a few tokens, quantised before the product that serves them: latency
        {"name": "checkpoint_decode", "op": "checkpoint", "layers": 1, "tokens": 4, "inp": 6144,
         "pow2": False, "dtype": "bf16"},
        # fp32 weights of 24 experts, quantised per channel after an optimizer step, odd sizes
        {"name": "checkpoint_weights_fp32", "op": "checkpoint", "layers": 24, "tokens": 1531 * 24, "inp": 1027,
         "pow2": False, "dtype": "fp32"},
        # one token through a dense layer: the weights are read once
        {"name": "matmul_one_token", "op": "matmul", "layers": 1, "tokens": 1, "out": 8192, "inp": 6144,
         "dtype": "bf16"},
        # four small layers, a few tokens: latency
        {"name": "matmul_tiny_fp32", "op": "matmul", "layers": 4, "tokens": 28, "out": 64, "inp": 32,
         "dtype": "fp32"},
        # a training batch through a dense layer
        {"name": "matmul_dense", "op": "matmul", "layers": 1, "tokens": 4096, "out": 8192, "inp": 6144,
         "dtype": "bf16"},
        # sixteen experts with ragged token counts, one of them without tokens
        {"name": "matmul_experts", "op": "matmul", "layers": 16, "tokens": 3001, "out": 2048, "inp": 6144,
         "dtype": "bf16"},
        # the gradient of a dense layer's input
        {"name": "grad_input_dense", "op": "grad_input", "layers": 1, "tokens": 4096, "out": 8192, "inp": 6144,
         "dtype": "bf16", "slice": False},
        # the same for experts, dY a slice of a wider gradient
        {"name": "grad_input_experts", "op": "grad_input", "layers": 8, "tokens": 1999, "out": 512, "inp": 10240,
         "dtype": "bf16", "slice": True},
        # the gradient of a dense layer's weights, added to an fp32 buffer over micro-batches
        {"name": "grad_weight_dense", "op": "grad_weight", "layers": 1, "tokens": 4096, "out": 8192, "inp": 6144,
         "dtype": "fp32", "pow2": True, "beta": 1.0, "slice": False},
        # experts' gradients straight into bf16 momentum, ready to be orthogonalised
        {"name": "grad_weight_experts", "op": "grad_weight", "layers": 16, "tokens": 3001, "out": 2048, "inp": 6144,
         "dtype": "bf16", "pow2": False, "beta": 0.9375, "slice": False},
        # attention gates: small gradients summed over many tokens
        {"name": "grad_weight_gates", "op": "grad_weight", "layers": 4, "tokens": 4 * 4096, "out": 18, "inp": 2304,
         "dtype": "bf16", "pow2": False, "beta": 0.0, "slice": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _width(rng, lo, hi):
    """A layer's width: mostly a multiple of 16, now and then any number."""
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.25 else max(16, n // 16 * 16)


def draw(rng):
    op = rng.choice(["checkpoint", "matmul", "grad_input", "grad_weight"])
    layers = rng.choice([1, 1, 1, 2, 5, 16])
    inp, out = _width(rng, 24, 10240), _width(rng, 16, 10240)
    tokens = _log_int(rng, 1, 8192)
    if rng.random() < 0.5:
        tokens |= 1
    if op == "checkpoint":
        tokens = max(1, min(tokens, MOST_VALUES // inp))
        return {"op": op, "layers": min(layers, tokens), "tokens": tokens, "inp": inp,
                "pow2": rng.random() < 0.5, "dtype": rng.choice(["bf16", "fp32"])}
    tokens = max(1, min(tokens, MOST_FLOPS // (2 * out * inp)))
    while layers > 1 and layers * out * inp > 16 * 2048 * 6144:
        layers //= 2
    case = {"op": op, "layers": layers, "tokens": tokens, "out": out, "inp": inp,
            "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "grad_input":
        # the gradient of an activation, in the activations' type
        case.update(dtype="bf16", slice=rng.random() < 0.5)
    if op == "grad_weight":
        # fp32 buffers go with the checkpoints whose scales are powers of two
        case.update(pow2=case["dtype"] == "fp32" or rng.random() < 0.5,
                    beta=rng.choice([0.0, 0.9375, 1.0]), slice=rng.random() < 0.5)
    return case


def shares(case):
    """Token counts of a case's layers: ragged, the third one without any
    (checkpoint: as even as they come)."""
    n, total = case["layers"], case["tokens"]
    if n == 1:
        return [total]
    if case["op"] == "checkpoint":
        return [total // n + (i < total % n) for i in range(n)]
    rng = random.Random(1000 * n + total)
    w = [0.0 if i == 2 else rng.random() ** 2 + 0.05 for i in range(n)]
    counts = [int(total * v / sum(w)) for v in w]
    counts[0] += total - sum(counts)
    return counts


def _int8(x, pow2=False):
    """Q8 of the rows of x as the library's quantiser lays it out: rows at a
    pitch of a multiple of 16."""
    amax = x.abs().amax(1).double()
    s = (amax / 127).float().clamp_min(2.0 ** -126)
    if pow2:
        m, e = torch.frexp(amax / 127)
        s = torch.ldexp(torch.ones_like(m), torch.where(m > 0.5, e, e - 1).clamp_min(-126)).float()
    q = torch.empty((x.shape[0], -(-x.shape[1] // 16) * 16), dtype=torch.int8, device=x.device)[:, :x.shape[1]]
    q.copy_((x.double() / s.double()[:, None]).round())
    return q, s


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, inp, counts = case["op"], case["inp"], shares(case)
    out = case.get("out", 0)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def activations(t):
        # a few channels are an order of magnitude larger, as in a
        # transformer's residual stream
        width = torch.where(torch.rand(inp, generator=gen, device=dev) < 0.01, 10.0, 1.0)
        return normal(t, inp) * width

    def gradient(t):
        # tokens weigh differently, and those that the loss masks have none
        g = 1e-3 * normal(t, out) * torch.exp(normal(t, 1))
        g = torch.where(torch.rand((t, 1), generator=gen, device=dev) < 0.1, torch.zeros_like(g), g)
        if not case["slice"]:
            return g.to(torch.bfloat16)
        pad = -(-out // 8) * 8
        wide = normal(t, 2 * pad).to(torch.bfloat16)
        wide[:, pad:pad + out] = g.to(torch.bfloat16)
        return wide[:, pad:pad + out]

    state = {"case": case, "dtype": dtype}
    if op == "checkpoint":
        state["x"] = [activations(t).to(dtype) for t in counts]
        return state
    if op in ("matmul", "grad_weight"):
        state["x"] = [_int8(activations(t).bfloat16(), case.get("pow2", False)) for t in counts]
    if op in ("matmul", "grad_input"):
        state["w"] = [_int8(normal(out, inp) / inp ** 0.5) for _ in counts]
    if op in ("grad_input", "grad_weight"):
        state["dy"] = [gradient(t) for t in counts]
    if op == "grad_weight":
        state["g"] = [(1e-2 * normal(out, inp)).to(dtype) for _ in counts]
    return state


def _plain_round_trip(x, pow2, dtype):
    amax = x.abs().amax(1, keepdim=True).double()
    if pow2:
        m, e = torch.frexp(amax / 127)
        s = torch.ldexp(torch.ones_like(m), torch.where(m > 0.5, e, e - 1).clamp_min(-126)).float()
    else:
        s = (amax / 127).float().clamp_min(2.0 ** -126)
    # in 64 bits: a quotient next to a half must not be rounded twice
    q = (x.double() / s.double()).round().clamp(-127, 127)
    return (q.float() * s).to(dtype), s[:, 0]


def run(state):
    case, dtype = state["case"], state["dtype"]
    op = case["op"]
    if own:
        import newton_schulz_04_amd as ns
        if op == "checkpoint":
            kept = ns.quantize_rows(state["x"], pow2=case["pow2"])
            return {"x": ns.dequantize_rows(kept, dtype=dtype), "scale": [scale for _, scale in kept]}
        if op == "matmul":
            return ns.q8_matmul(state["x"], state["w"], dtype=dtype)
        if op == "grad_input":
            return ns.q8_grad_input(state["dy"], state["w"])
        return ns.q8_grad_weight(state["dy"], state["x"], state["g"], beta=case["beta"])
    if op == "checkpoint":
        pairs = [_plain_round_trip(x, case["pow2"], dtype) for x in state["x"]]
        return {"x": [p[0] for p in pairs], "scale": [p[1] for p in pairs]}
    if op == "matmul":
        return [((xq.float() @ wq.float().T) * xs[:, None] * ws).to(dtype)
                for (xq, xs), (wq, ws) in zip(state["x"], state["w"])]
    if op == "grad_input":
        return [(dy.float() @ (wq.float() * ws[:, None])).to(dtype)
                for dy, (wq, ws) in zip(state["dy"], state["w"])]
    beta = case["beta"]
    return [g.copy_((beta * g.float() if beta else 0.0) + dy.float().T @ (xq.float() * xs[:, None]))
            for dy, (xq, xs), g in zip(state["dy"], state["x"], state["g"])]


def work(case):
    counts, inp, n = shares(case), case["inp"], case["layers"]
    total, size = sum(counts), 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "checkpoint":
        # values in and back out, int8 written and read, scales written and read
        return {"bytes": total * (inp * (2 * size + 2) + 8), "flops": 4 * total * inp}
    out, live = case["out"], sum(t > 0 for t in counts)
    x8, y = total * (inp + 4), total * out
    w8 = live * out * (inp + 4)
    if case["op"] == "matmul":
        moved = x8 + w8 + size * y
    elif case["op"] == "grad_input":
        moved = 2 * y + w8 + size * total * inp
    else:
        passes = 2 if case["beta"] else 1
        # a layer without tokens still scales its buffer
        moved = 2 * y + x8 + passes * size * n * out * inp
    return {"bytes": moved, "flops": 2 * total * out * inp}


def exact(case, seed):
    """The definition in 64 bits."""
    state = prepare(case, seed)
    op = case["op"]

    def values(pair):
        return pair[0].to(torch.float64) * pair[1].to(torch.float64).unsqueeze(1)

    if op == "checkpoint":
        xs, scales = [], []
        for x in state["x"]:
            v = x.to(torch.float64)
            top = torch.maximum(v.max(1).values, -v.min(1).values)
            s = (top / 127).to(torch.float32).to(torch.float64)
            if case["pow2"]:
                # from a power of two below (made exact by the cast), up
                s = torch.pow(2.0, torch.floor(torch.log2(torch.clamp(top, min=2.0 ** -120) / 127)) - 1)
                s = s.to(torch.float32).to(torch.float64)
                for _ in range(2):
                    s = torch.where(127 * s < top, 2 * s, s)
            s = torch.clamp(s, min=2.0 ** -126).unsqueeze(1)
            r = v / s
            low = torch.floor(r)
            up = (r - low > 0.5) | ((r - low == 0.5) & (torch.remainder(low, 2) == 1))
            xs.append((low + up) * s)
            scales.append(s.squeeze(1))
        return {"x": xs, "scale": scales}
    if op == "matmul":
        return [torch.matmul(values(x), values(w).transpose(0, 1).contiguous())
                for x, w in zip(state["x"], state["w"])]
    if op == "grad_input":
        return [torch.matmul(dy.to(torch.float64), values(w)) for dy, w in zip(state["dy"], state["w"])]
    return [case["beta"] * g.to(torch.float64) + torch.matmul(dy.to(torch.float64).transpose(0, 1).contiguous(), values(x))
            for dy, x, g in zip(state["dy"], state["x"], state["g"])]
