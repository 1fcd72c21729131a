"""The MXFP4 operators as they are measured: the cases, their inputs, their plain forms and the
framework's calls.

MXFP4 (microscaled 4-bit floating point): a row of K values is cut into blocks of 32; a block has
one scale byte e (the factor 2^(e - 127)) and 32 codes of 4 bits (sign, two exponent bits, one
mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two per byte, the lower index in the low half.

Operators (``op`` of a case):
    quantize            x -> codes and scales -> the values they stand for
    linear              y = x W^T, bf16 activations, MXFP4 weights
    linear_backward     dx = dy W
    a4_linear           y = Q(x) W^T, the activations quantized to MXFP4 in the call
    gate_up             h = silu(x Wg^T) * (x Wu^T)
    gate_up_backward    dx, and the gradients of the two projections, from x and dh

Sizes: hidden 2560, MLP 9728, 4096 query columns and a vocabulary of 151936 columns are the layer
shapes of this repository's benchmark.
"""

import math

import torch

own = False

DEV = "cuda"
BLOCK = 32
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LARGEST = 4096 * 9728 * 2560


def listed():
    return [
        # the activations of a short ragged batch before a product: a call that is all latency
        {"name": "quantize_33x2560", "op": "quantize", "m": 33, "k": 2560, "type": "bf16"},
        # a float32 projection of a checkpoint on its way to 4 bits
        {"name": "quantize_9728x2560_fp32", "op": "quantize", "m": 9728, "k": 2560, "type": "fp32"},
        # one token of one sequence through the up projection
        {"name": "linear_1x9728x2560", "op": "linear", "m": 1, "n": 9728, "k": 2560},
        # the vocabulary head for the last tokens of five sequences
        {"name": "linear_5x151936x2560", "op": "linear", "m": 5, "n": 151936, "k": 2560},
        # a prompt of 509 tokens through the down projection: a long sum, an odd row count
        {"name": "linear_509x2560x9728", "op": "linear", "m": 509, "n": 2560, "k": 9728},
        # the query projection's input gradient while adapters are trained on 2048 tokens
        {"name": "linear_backward_2048x4096x2560", "op": "linear_backward", "m": 2048, "n": 4096, "k": 2560},
        # one token of each of four sequences through the down projection, 4-bit activations
        {"name": "a4_linear_4x2560x9728", "op": "a4_linear", "m": 4, "n": 2560, "k": 9728},
        # a long prompt through the up projection, 4-bit activations
        {"name": "a4_linear_4096x9728x2560", "op": "a4_linear", "m": 4096, "n": 9728, "k": 2560},
        # one token through the gated half of the feed-forward block
        {"name": "gate_up_1x9728x2560", "op": "gate_up", "m": 1, "n": 9728, "k": 2560},
        # a prompt of 512 tokens through it
        {"name": "gate_up_512x9728x2560", "op": "gate_up", "m": 512, "n": 9728, "k": 2560},
        # a small ragged training step: widths that fill no tile
        {"name": "gate_up_backward_130x1000x416", "op": "gate_up_backward", "m": 130, "n": 1000, "k": 416},
        # a training step on 4096 tokens
        {"name": "gate_up_backward_4096x9728x2560", "op": "gate_up_backward", "m": 4096, "n": 9728, "k": 2560},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], evenly over the logarithm."""
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear_backward", "a4_linear", "gate_up", "gate_up_backward"])
    # decode rows half of the time where decoding meets the operator, prompts and batches else
    serving = op in ("linear", "a4_linear", "gate_up")
    m = _spread(rng, 1, 16) if serving and rng.random() < 0.5 else _spread(rng, 1, 4096)
    k = BLOCK * _spread(rng, 2, 304)
    if op == "quantize":
        return {"op": op, "m": _spread(rng, 1, 9728), "k": k, "type": rng.choice(["bf16", "fp32"])}
    n = _spread(rng, 16, 16384)
    if op == "gate_up_backward":
        n = max(8, n // 8 * 8)          # rows of whole 16 bytes
    while m * n * k > LARGEST:
        m = (m + 1) // 2
    return {"op": op, "m": m, "n": n, "k": k}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(rows, cols, dtype, scale=1.0):
        return (torch.randn(rows, cols, generator=g, device=DEV) * scale).to(dtype)

    def weight(n, k):
        """Codes and scales of an N(0, 0.02) weight matrix, in pieces of bounded memory."""
        parts = [_quantized(normal(min(16384, n - r), k, torch.float32, 0.02)) for r in range(0, n, 16384)]
        return (torch.cat([p[0] for p in parts]).contiguous(), torch.cat([p[1] for p in parts]).contiguous())

    op, m, k = case["op"], case["m"], case["k"]
    if op == "quantize":
        return {"op": op, "x": normal(m, k, torch.float32 if case["type"] == "fp32" else torch.bfloat16)}
    n = case["n"]
    if op == "linear_backward":
        return {"op": op, "dy": normal(m, n, torch.bfloat16), "w": weight(n, k)}
    state = {"op": op, "x": normal(m, k, torch.bfloat16), "w": weight(n, k)}
    if op.startswith("gate_up"):
        state["w2"] = weight(n, k)
    if op == "gate_up_backward":
        state["dh"] = normal(m, n, torch.bfloat16)
    return state


def run(state):
    op = state["op"]
    if own:
        import w4a16_group_quantized_qmv_amd as w4
        if op == "quantize":
            return w4.mxfp4_dequantize_rows(*w4.mxfp4_quantize_rows(state["x"]))
        if op == "linear":
            return w4.mxfp4_linear(state["x"], *state["w"])
        if op == "linear_backward":
            return w4.mxfp4_linear_backward(state["dy"], *state["w"])
        if op == "a4_linear":
            return w4.mxfp4a4_linear(state["x"], *state["w"])
        if op == "gate_up":
            return w4.mxfp4_gate_up_swiglu(state["x"], state["w"], state["w2"])
        return w4.mxfp4_gate_up_swiglu_backward(state["x"], state["w"], state["w2"], state["dh"])
    if op == "quantize":
        return _values(*_quantized(state["x"])).to(torch.bfloat16)
    if op == "linear":
        return (state["x"].float() @ _values(*state["w"]).t()).to(torch.bfloat16)
    if op == "linear_backward":
        return (state["dy"].float() @ _values(*state["w"])).to(torch.bfloat16)
    if op == "a4_linear":
        return (_values(*_quantized(state["x"])) @ _values(*state["w"]).t()).to(torch.bfloat16)
    x, wg, wu = state["x"].float(), _values(*state["w"]), _values(*state["w2"])
    gate, up = x @ wg.t(), x @ wu.t()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    if op == "gate_up":
        return (gate * sig * up).to(torch.bfloat16)
    dh = state["dh"].float()
    dgate, dup = dh * up * sig * (1.0 + gate * (1.0 - sig)), dh * gate * sig
    return tuple(t.to(torch.bfloat16) for t in (dgate @ wg + dup @ wu, dgate, dup))


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    packed = k // 2 + k // BLOCK                      # bytes of one row in MXFP4
    if op == "quantize":                              # x read, codes and scales written and read, values written
        return {"bytes": m * (k * (4 if case["type"] == "fp32" else 2) + 2 * packed + 2 * k), "flops": 2 * m * k}
    n = case["n"]
    product = 2 * m * n * k
    if op in ("linear", "a4_linear", "linear_backward"):
        return {"bytes": n * packed + 2 * m * (n + k), "flops": product}
    if op == "gate_up":
        return {"bytes": 2 * n * packed + 2 * m * (n + k), "flops": 2 * product}
    # x and dh read, dx and both projections' gradients written; both projections, and both of their transposes
    return {"bytes": 2 * n * packed + 2 * m * (2 * k + 3 * n), "flops": 4 * product}


# ---- the plain form: 32 bits, elementary operations


def _quantized(x):
    """Codes [rows, K/2] and scales [rows, K/32] of the rows of x (all values finite)."""
    rows, k = x.shape
    blocks = x.float().reshape(rows, k // BLOCK, BLOCK)
    top = blocks.abs().amax(dim=2)
    exponent = torch.where(top > 0, torch.frexp(top)[1] - 1, torch.full_like(top, -127, dtype=torch.int32))
    shift = (exponent - 2).clamp(-127, 127)           # floor(log2(largest)) less the exponent of 4
    # two exact steps: 2^-shift itself may be as large as 2^127
    scaled = torch.ldexp(torch.ldexp(blocks.abs(), -(shift // 2)[..., None]), -(shift - shift // 2)[..., None])
    # the number of borders below a value is its code; a border goes to the code whose mantissa bit is 0
    above = torch.tensor((0.25, 1.25, 2.5, 5.0), device=x.device)
    from_ = torch.tensor((0.75, 1.75, 3.5), device=x.device)
    code = (scaled[..., None] > above).sum(-1, dtype=torch.uint8) + (scaled[..., None] >= from_).sum(-1, dtype=torch.uint8)
    code += 8 * torch.signbit(blocks).to(torch.uint8)
    code = code.reshape(rows, k // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (shift + 127).to(torch.uint8)


def _values(codes, scales):
    """float32 values of MXFP4 rows."""
    rows, half = codes.shape
    table = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), dtype=torch.float32, device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), dim=2).reshape(rows, half // 16, BLOCK)
    factor = torch.ldexp(torch.ones((), device=codes.device), scales.to(torch.int32) - 127)
    return (table[both.int()] * factor[..., None]).reshape(rows, 2 * half)


# ---- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]

    def decode(codes, scales):
        c = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
        for half in (0, 1):
            q = (codes >> (4 * half)) & 15
            e, f = ((q >> 1) & 3).double(), (q & 1).double()
            v = torch.where(e > 0, (1 + f / 2) * torch.exp2(e - 1), f / 2)
            c[:, half::2] = torch.where(q > 7, -v, v)
        return c * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, dim=1)

    def nearest(x):
        """x rounded to its blocks' grids: steps of 2^(exponent - 1) above 1, of 1/2 below, at most 6."""
        b = x.double().reshape(x.shape[0], -1, BLOCK)
        top = b.abs().amax(2, keepdim=True)
        unit = torch.exp2(torch.where(top > 0, torch.frexp(top)[1].double() - 3, -127.0).clamp(min=-127))
        r = b.abs() / unit
        step = torch.exp2(torch.frexp(r.clamp(min=1.0))[1].double() - 2)
        r = (torch.round(r / step) * step).clamp(max=6.0)
        return (torch.copysign(r, b) * unit).reshape(x.shape)

    if op == "quantize":
        return nearest(s["x"])
    w = decode(*s["w"])
    if op == "linear":
        return s["x"].double() @ w.t()
    if op == "linear_backward":
        return s["dy"].double() @ w
    if op == "a4_linear":
        return nearest(s["x"]) @ w.t()
    w2, x = decode(*s["w2"]), s["x"].double()
    a, b = x @ w.t(), x @ w2.t()
    if op == "gate_up":
        return a / (1 + torch.exp(-a)) * b
    dh, t = s["dh"].double(), torch.exp(-a)
    da = dh * b * (1 + t + a * t) / (1 + t) ** 2
    db = dh * a / (1 + t)
    return da @ w + db @ w2, da, db
