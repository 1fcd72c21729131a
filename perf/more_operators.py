"""The 8-bit products and the operators of mixtures of experts as they are measured: the cases, their
inputs, their plain forms and the framework's calls.

An int8 matrix [N, K] has one float32 scale a row; it stands for scale * code.  Activations are quantized
row by row (token by token) in a call, all in float32:

    a = max |x|,   inv = 127 / a,   scale = a / 127,   code = rint(x * inv)   (ties to even)

Operators (``op`` of a case):
    linear              y = Q(x) W^T, Q the quantization of the activations to 8 bits
    linear_backward     dx = dy W  (the quantization passes gradients on)
    route               the top_k largest logits of each token, their softmax, and the (token, expert) pairs in
                        order of the expert; with "train" the gradient of the logits as well
    gate_up             expert by expert h = silu(Q(x) Wg^T) * (Q(x) Wu^T) over the rows of the tokens it got
    experts             gate_up, then y = Q(h) Wd^T by the same experts
    experts_linear_backward   dh = dy Wd, expert by expert
    gate_up_backward    a row's gradient of x, and the gradients of the two projections
    combine             out[t] = sum_j weight[t, j] * y[row of the j-th expert of t]; with "train" the gradients of
                        y and of the weights as well

Pairs of a token and an expert are rows: first all rows of expert 0 by token, then those of expert 1, and so on.
``offsets`` [E + 1] are the experts' first rows, ``tokens`` [rows] the rows' tokens, ``positions``
[tokens, top_k] the rows of a token's experts.

Sizes: hidden 2560, MLP 9728, 4096 query columns are the layer shapes of this repository's benchmark; the
experts' widths are generic (1216 is an eighth of the MLP).
"""

import math

import torch

own = False

DEV = "cuda"
LARGEST = 32768 * 1216 * 2560            # rows x expert columns x values of the largest listed case
WEIGHTS = 64 * 1216 * 2560               # weights of one projection of all experts


def listed():
    return [
        # one token of one sequence through the up projection
        {"name": "linear_1x9728x2560", "op": "linear", "m": 1, "n": 9728, "k": 2560},
        # a prompt of 509 tokens through the down projection: a long sum, an odd row count
        {"name": "linear_509x2560x9728", "op": "linear", "m": 509, "n": 2560, "k": 9728},
        # a long prompt through the up projection
        {"name": "linear_4096x9728x2560", "op": "linear", "m": 4096, "n": 9728, "k": 2560},
        # the query projection's input gradient while adapters are trained on 2048 tokens
        {"name": "linear_backward_2048x4096x2560", "op": "linear_backward", "m": 2048, "n": 4096, "k": 2560},
        # the router of a decode step of five sequences: a call that is all latency
        {"name": "route_5x60_top4", "op": "route", "t": 5, "e": 60, "top": 4, "type": "fp32", "train": False},
        # the router of a training step, with its gradient; bf16 logits tie often
        {"name": "route_train_32767x256_top8", "op": "route", "t": 32767, "e": 256, "top": 8, "type": "bf16", "train": True},
        # one token of each of four sequences through the experts' gated halves
        {"name": "gate_up_4_64x1216x2560_top8", "op": "gate_up", "t": 4, "e": 64, "top": 8, "n": 1216, "k": 2560},
        # a prompt of 509 tokens through both halves of the experts
        {"name": "experts_509_64x1216x2560_top4", "op": "experts", "t": 509, "e": 64, "top": 4, "n": 1216, "k": 2560},
        # a training step on 4096 tokens: the down projections' input gradient
        {"name": "experts_linear_backward_4096_64x1216x2560_top8", "op": "experts_linear_backward", "t": 4096, "e": 64,
         "top": 8, "n": 1216, "k": 2560},
        # the same step's gated halves
        {"name": "gate_up_backward_4096_64x1216x2560_top8", "op": "gate_up_backward", "t": 4096, "e": 64, "top": 8,
         "n": 1216, "k": 2560},
        # the end of a decode step's block, five sequences
        {"name": "combine_5x2560_top4", "op": "combine", "t": 5, "e": 60, "top": 4, "k": 2560, "train": False},
        # the end of a training step's block and its gradients
        {"name": "combine_train_8191x2560_top8", "op": "combine", "t": 8191, "e": 64, "top": 8, "k": 2560, "train": True},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], evenly over the logarithm."""
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "route", "gate_up", "experts", "experts_linear_backward",
                     "gate_up_backward", "combine"])
    # decode rows half of the time where decoding meets the operator, prompts and batches else
    few = op in ("linear", "gate_up", "experts", "combine", "route") and rng.random() < 0.5
    k = 16 * _spread(rng, 4, 608)
    if op in ("linear", "linear_backward"):
        m, n = _spread(rng, 1, 16) if few else _spread(rng, 1, 4096), _spread(rng, 16, 16384)
        while m * n * k > LARGEST:
            m = (m + 1) // 2
        return {"op": op, "m": m, "n": n, "k": k}
    e = _spread(rng, 4, 256)
    top = rng.randint(1, min(8, e))
    t = _spread(rng, 1, 16) if few else _spread(rng, 1, 4096)
    if op == "route":
        if not few:
            t = _spread(rng, 1, 32768)
        return {"op": op, "t": t, "e": e, "top": top, "type": rng.choice(["bf16", "fp32"]), "train": rng.random() < 0.5}
    if op == "combine":
        return {"op": op, "t": t, "e": e, "top": top, "k": k, "train": not few}
    k = 16 * _spread(rng, 8, 256)
    n = 16 * _spread(rng, 4, 128)
    while e * n * k > WEIGHTS:
        e, n = max(e // 2, 4), max(n // 32 * 16, 64)
    top = min(top, e)
    while t * top * n * k > LARGEST:
        t = (t + 1) // 2
    return {"op": op, "t": t, "e": e, "top": top, "n": n, "k": k}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]

    def normal(rows, cols, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(rows, cols, generator=g, device=DEV) * scale).to(dtype)

    def weight(n, k):
        """Codes and scales of an N(0, 0.02) weight matrix."""
        codes, scales = _quantized(normal(n, k, torch.float32, 0.02))
        return codes.to(torch.int8), scales

    def stacked(e, n, k):
        parts = [weight(n, k) for _ in range(e)]
        return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])

    if op == "linear":
        return {"op": op, "x": normal(case["m"], case["k"]), "w": weight(case["n"], case["k"])}
    if op == "linear_backward":
        return {"op": op, "dy": normal(case["m"], case["n"]), "w": weight(case["n"], case["k"])}
    t, e, top = case["t"], case["e"], case["top"]
    # experts differ in how often they are chosen, more so where many tokens are routed
    popular = torch.randn(e, generator=g, device=DEV) * (0.5 if t > 64 else 0.0)
    logits = torch.randn(t, e, generator=g, device=DEV) + popular
    if op == "route":
        state = {"op": op, "logits": logits.to(torch.bfloat16 if case["type"] == "bf16" else torch.float32), "top": top}
        if case["train"]:
            state["dweights"] = normal(t, top, torch.float32)
        return state
    weights, _, positions, tokens, offsets = _routed(logits, top)
    state = {"op": op, "positions": positions, "tokens": tokens, "offsets": offsets}
    if op == "combine":
        state.update(y=normal(t * top, case["k"]), weights=weights)
        if case["train"]:
            state["dout"] = normal(t, case["k"])
        return state
    n, k = case["n"], case["k"]
    if op == "experts_linear_backward":
        state.update(dy=normal(t * top, k), down=stacked(e, k, n))
        return state
    state.update(x=normal(t, k), gate=stacked(e, n, k), up=stacked(e, n, k))
    if op == "experts":
        state["down"] = stacked(e, k, n)
    if op == "gate_up_backward":
        state["dh"] = normal(t * top, n)
    return state


def run(state):
    op = state["op"]
    if own:
        import w4a16_group_quantized_qmv_amd as w4
        if op == "linear":
            return w4.w8a8_linear(state["x"], *state["w"])
        if op == "linear_backward":
            return w4.w8a8_linear_backward(state["dy"], *state["w"])
        if op == "route":
            routed = w4.experts_route(state["logits"], state["top"])
            if "dweights" not in state:
                return routed
            return (*routed, w4.experts_route_backward(state["logits"], routed[1], state["dweights"]))
        if op == "combine":
            out = w4.experts_combine(state["y"], state["positions"], state["weights"])
            if "dout" not in state:
                return out
            return (out, *w4.experts_combine_backward(state["dout"], state["y"], state["positions"], state["weights"]))
        offsets = state["offsets"]
        if op == "experts_linear_backward":
            return w4.w8a8_experts_linear_backward(state["dy"], *state["down"], offsets)
        if op == "gate_up_backward":
            return w4.w8a8_experts_gate_up_swiglu_backward(state["x"], state["gate"], state["up"], state["dh"], offsets,
                                                           state["tokens"])
        h = w4.w8a8_experts_gate_up_swiglu(state["x"], state["gate"], state["up"], offsets, state["tokens"])
        return h if op == "gate_up" else w4.w8a8_experts_linear(h, *state["down"], offsets)

    if op == "linear":
        return _product(*_quantized(state["x"]), *state["w"]).to(torch.bfloat16)
    if op == "linear_backward":
        return (state["dy"].float() @ _values(*state["w"])).to(torch.bfloat16)
    if op == "route":
        logits = state["logits"].float()
        weights, experts, positions, tokens, offsets = _routed(logits, state["top"])
        if "dweights" not in state:
            return weights, experts, positions, tokens, offsets
        d = weights * (state["dweights"] - (weights * state["dweights"]).sum(1, keepdim=True))
        dlogits = torch.zeros_like(logits).scatter(1, experts.long(), d)
        return weights, experts, positions, tokens, offsets, dlogits.to(state["logits"].dtype)
    if op == "combine":
        y, at, weights = state["y"].float(), state["positions"].long(), state["weights"]
        rows = y[at]                                                         # [tokens, top_k, k]
        out = (rows * weights[..., None]).sum(1).to(torch.bfloat16)
        if "dout" not in state:
            return out
        dout = state["dout"].float()
        dy = torch.empty_like(y)
        dy[at.reshape(-1)] = (weights[..., None] * dout[:, None, :]).reshape(-1, y.shape[1])
        return out, dy.to(torch.bfloat16), (rows * dout[:, None, :]).sum(2)
    bounds = state["offsets"].tolist()
    spans = [(i, slice(a, b)) for i, (a, b) in enumerate(zip(bounds, bounds[1:])) if b > a]
    if op == "experts_linear_backward":
        dy, down = state["dy"], state["down"]
        return torch.cat([(dy[s].float() @ _values(down[0][i], down[1][i])).to(torch.bfloat16) for i, s in spans])
    tokens, gate, up = state["tokens"].long(), state["gate"], state["up"]
    codes, scales = _quantized(state["x"])
    parts = []
    for i, s in spans:
        a, f = codes[tokens[s]], scales[tokens[s]]
        g, u = _product(a, f, gate[0][i], gate[1][i]), _product(a, f, up[0][i], up[1][i])
        sig = 1.0 / (1.0 + torch.exp(-g))
        if op == "gate_up_backward":
            dh = state["dh"][s].float()
            dg, du = dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig
            dx = dg @ _values(gate[0][i], gate[1][i]) + du @ _values(up[0][i], up[1][i])
            parts.append(tuple(v.to(torch.bfloat16) for v in (dx, dg, du)))
        else:
            parts.append((g * sig * u).to(torch.bfloat16))
    if op == "gate_up_backward":
        return tuple(torch.cat(p) for p in zip(*parts))
    h = torch.cat(parts)
    if op == "gate_up":
        return h
    codes, scales = _quantized(h)
    down = state["down"]
    return torch.cat([_product(codes[s], scales[s], down[0][i], down[1][i]).to(torch.bfloat16) for i, s in spans])


def work(case):
    op = case["op"]
    if op in ("linear", "linear_backward"):
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * (k + 4) + 2 * m * (n + k), "flops": 2 * m * n * k}
    t, e, top = case["t"], case["e"], case["top"]
    rows = t * top
    if op == "route":
        size = 2 if case["type"] == "bf16" else 4
        forward = t * e * size + rows * 16 + 4 * (e + 1)          # weights, experts, positions and tokens written
        back = rows * 4 + t * e * size if case["train"] else 0    # their gradient read, the logits' written
        return {"bytes": forward + back, "flops": t * e * (4 if case["train"] else 2)}
    if op == "combine":
        k = case["k"]
        forward = 2 * rows * k + 8 * rows + 2 * t * k
        back = 2 * t * k + 2 * rows * k + 4 * rows if case["train"] else 0
        return {"bytes": forward + back, "flops": rows * k * (5 if case["train"] else 2)}
    n, k = case["n"], case["k"]
    used = e * (1.0 - (1.0 - top / e) ** t)                       # experts that some token reaches, evenly routed
    ids = 4 * (e + 1) + 4 * rows
    matrix = used * n * k
    if op == "experts_linear_backward":
        return {"bytes": int(matrix + 4 * used * k) + ids + 2 * rows * (n + k), "flops": 2 * rows * n * k}
    gated = 2 * int(matrix + 4 * used * n) + ids + 2 * t * k
    if op == "gate_up":
        return {"bytes": gated + 2 * rows * n, "flops": 4 * rows * n * k}
    if op == "experts":                                           # h written and read
        return {"bytes": gated + 4 * rows * n + int(matrix + 4 * used * k) + 2 * rows * k, "flops": 6 * rows * n * k}
    # dh read, both projections' gradients and the rows of dx written
    return {"bytes": gated + 6 * rows * n + 2 * rows * k, "flops": 8 * rows * n * k}


# ---- the plain form: 32 bits, elementary operations


def _quantized(x):
    """Codes (as float32) and scales of the rows of x, all values finite."""
    x = x.float()
    top = x.abs().amax(dim=1)
    inverse = torch.where(top > 0, 127.0 / top, torch.zeros_like(top))
    return torch.round(x * inverse[:, None]).clamp(-127, 127), top / 127.0


def _values(codes, scales):
    return codes.float() * scales[:, None]


def _product(codes, scales, w, w_scales):
    return (codes @ w.float().t()) * w_scales[None, :] * scales[:, None]


def _routed(logits, top):
    """Weights, experts, positions, tokens and offsets of float32 logits; equal logits go to the lowest expert."""
    t, e = logits.shape
    chosen, experts = torch.sort(logits, dim=1, descending=True, stable=True)
    chosen, experts = chosen[:, :top], experts[:, :top]
    weights = torch.exp(chosen - chosen[:, :1])
    weights = weights / weights.sum(1, keepdim=True)
    flat = experts.reshape(-1)
    order = torch.argsort(flat, stable=True)                      # rows by expert, then by token
    positions = torch.empty_like(order)
    positions[order] = torch.arange(t * top, device=logits.device)
    counts = torch.zeros(e, dtype=torch.int64, device=logits.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    as_int = [v.to(torch.int32).contiguous() for v in (experts, positions.reshape(t, top), order // top, offsets)]
    return (weights.contiguous(), *as_int)


# ---- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]

    def nearest(x):
        """The values that the rows of x are quantized to (the code is the rounding of a float32 product)."""
        v = x.double()
        a = v.abs().max(dim=1, keepdim=True).values
        inverse = (127.0 / a).float().double()
        return torch.round((v * inverse).float()).double() * (a / 127.0).float().double()

    def decode(w, i=None):
        codes, scales = w if i is None else (w[0][i], w[1][i])
        return codes.double() * scales.double().unsqueeze(1)

    if op == "linear":
        return nearest(s["x"]) @ decode(s["w"]).t()
    if op == "linear_backward":
        return s["dy"].double() @ decode(s["w"])
    if op == "route":
        l, top = s["logits"].double(), s["top"]
        # selection by counting: an expert's place is the number of experts before it in (logit, index)
        place = torch.empty(l.shape, dtype=torch.int64, device=l.device)
        index = torch.arange(l.shape[1], device=l.device)
        for i in range(0, l.shape[0], 1024):
            b = l[i:i + 1024]
            ahead = (b[:, None, :] > b[:, :, None]) | ((b[:, None, :] == b[:, :, None]) & (index[None, :] < index[:, None]))
            place[i:i + 1024] = ahead.sum(2)
        inside = place < top
        p = torch.where(inside, torch.exp(l - l.max(1, keepdim=True).values), 0.0)
        p = p / p.sum(1, keepdim=True)
        at = torch.argsort(place, dim=1)[:, :top]
        weights = p.gather(1, at)
        if "dweights" not in s:
            return weights, None, None, None, None
        d = torch.zeros_like(l).scatter(1, at, s["dweights"].double())
        return weights, None, None, None, None, p * (d - (p * d).sum(1, keepdim=True))
    if op == "combine":
        at, w, y = s["positions"].long(), s["weights"].double(), s["y"].double()
        out = sum(w[:, j:j + 1] * y[at[:, j]] for j in range(at.shape[1]))
        if "dout" not in s:
            return out
        d = s["dout"].double()
        dy = torch.zeros_like(y)
        for j in range(at.shape[1]):
            dy[at[:, j]] = w[:, j:j + 1] * d
        dw = torch.stack([(d * y[at[:, j]]).sum(1) for j in range(at.shape[1])], dim=1)
        return out, dy, dw
    first = s["offsets"].cpu().numpy()
    spans = [(i, int(first[i]), int(first[i + 1])) for i in range(len(first) - 1)]
    if op == "experts_linear_backward":
        return torch.cat([s["dy"][a:b].double() @ decode(s["down"], i) for i, a, b in spans])
    x, tokens = nearest(s["x"]), s["tokens"].long()
    hs, grads = [], []
    for i, a, b in spans:
        rows, wg, wu = x[tokens[a:b]], decode(s["gate"], i), decode(s["up"], i)
        g, u = rows @ wg.t(), rows @ wu.t()
        t = torch.exp(-g)
        hs.append(g * u / (1 + t))
        if op == "gate_up_backward":
            dh = s["dh"][a:b].double()
            dg, du = dh * u * (1 + t + g * t) / (1 + t) ** 2, dh * g / (1 + t)
            grads.append((dg @ wg + du @ wu, dg, du))
    if op == "gate_up_backward":
        return tuple(torch.cat(v) for v in zip(*grads))
    if op == "gate_up":
        return torch.cat(hs)
    h = torch.cat(hs).float().to(torch.bfloat16)        # h is an output of the first call: bf16, then 8 bits
    h = nearest(h) if h.shape[0] else h.double()
    return torch.cat([h[a:b] @ decode(s["down"], i).t() for i, a, b in spans])
