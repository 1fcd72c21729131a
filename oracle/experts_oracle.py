"""CPU oracle of the int8 products and of the experts' operators: numpy, 64 bits, loops where they are plainest.

Each function returns float64 values and, beside them, how far a result may be off them.  The bounds count:
 * H = 2^-8, half a step of bf16 relative to the value, at every rounding to bf16 (an output, or an operand of a
   16-bit matrix product);
 * F = 2^-24, half a step of fp32, at every fp32 operation; a sum of n fp32 terms in any order is off by at most
   n F times the sum of their magnitudes;
 * integer sums of codes are exact;
 * TINY = 2^-126 for results that fp32 or bf16 cannot hold as normal numbers;
 * the sigmoid of the kernels: relative (4 + |z|) 2^-23, absolute 2^-126.
"""

from __future__ import annotations

import numpy as np

__all__ = ["w8_quantize", "w8_product", "w8_linear", "w8_linear_backward", "w8_gate_up", "w8_gate_up_backward", "route_reference",
           "route_backward_reference", "combine_reference", "combine_backward_reference", "within"]

H, F, TINY = 2.0 ** -8, 2.0 ** -24, 2.0 ** -126

NAN_ROW = -2 ** 31       # the position of a slot without an expert whose token's logits hold a NaN


def w8_quantize(x):
    """Codes (int8) and scales (float32) of rows of float values: every step in fp32, as the format is defined."""
    x = np.asarray(x, dtype=np.float32)
    codes, scales = np.zeros(x.shape, np.int8), np.zeros(x.shape[0], np.float32)
    for i, row in enumerate(x):
        if not np.isfinite(row).all():
            scales[i] = np.nan
            continue
        a = np.abs(row).max()
        if a < np.float32(2.0 ** -110):
            continue
        scales[i] = a / np.float32(127)
        codes[i] = np.clip(np.rint(row * (np.float32(127) / a)), -127, 127).astype(np.int8)
    return codes, scales


def w8_product(xq, xs, wq, ws):
    """P[m, n] xs[m] ws[n] in 64 bits (integers below 2^53: P is exact), and the error of fp32 before the output's
    rounding: the conversion of P and two products."""
    with np.errstate(invalid="ignore"):
        d = (xq.astype(np.float64) @ wq.astype(np.float64).T) * xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]
        return d, np.abs(d) * 3.01 * F


def _rounded(value, error):
    """The bound after the output's rounding to bf16."""
    return value, error + (np.abs(value) + error) * H + TINY


def w8_linear(xq, xs, wq, ws):
    return _rounded(*w8_product(xq, xs, wq, ws))


def w8_linear_backward(dy, wq, ws):
    """dx = dy W; each weight is rounded to bf16 (and once in fp32), the products are exact in fp32 but for their sum."""
    w = wq.astype(np.float64) * ws.astype(np.float64)[:, None]
    dx, mass = dy @ w, np.abs(dy) @ np.abs(w)
    return _rounded(dx, mass * (H + (w.shape[0] + 4) * F * (1 + H)) + TINY)


def _gated(xq, xs, gate, up):
    g, eg = w8_product(xq, xs, *gate)
    u, eu = w8_product(xq, xs, *up)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return g, eg, u, eu, s, s * (4 + np.abs(g)) * 2 * F + TINY + s * (1 - s) * eg


def w8_gate_up(xq, xs, gate, up):
    """h = g s u.  With the errors eg, eu, es of its factors (es holds that of g, through the sigmoid, as well) and two
    products in fp32."""
    g, eg, u, eu, s, es = _gated(xq, xs, gate, up)
    h = g * s * u
    error = eg * s * np.abs(u) + es * np.abs(g * u) + eu * np.abs(g * s) + np.abs(h) * 2 * F
    return _rounded(h, error * 1.01 + TINY)


def w8_gate_up_backward(xq, xs, gate, up, dh):
    """((dx, bound), (dgate, bound), (dup, bound)).

    dup = dh g s: as h above.  dgate = dh u s f with f = 1 + g (1 - s): f is off by |g| (es + F (1 - s)) for 1 - s and
    the factor, eg (1 - s), F |g (1 - s)| for the product and F |f| for the sum; dh u s by its factors and two
    products; one more product.  dx = (dgate ws_g) . Cg + (dup ws_u) . Cu: each gradient times its scale is one fp32
    product and one rounding to bf16, the codes are exact, the sum has 2 N terms."""
    g, eg, u, eu, s, es = _gated(xq, xs, gate, up)
    dup = dh * g * s
    e_up = 1.01 * np.abs(dh) * (eg * s + es * np.abs(g)) + np.abs(dup) * 2.1 * F + TINY
    f = 1 + g * (1 - s)
    ef = np.abs(g) * (es + F * (1 - s)) + eg * (1 - s) + F * np.abs(g * (1 - s)) + F * np.abs(f)
    c = dh * u * s
    ec = np.abs(dh) * (eu * s + es * np.abs(u)) + np.abs(c) * 2.1 * F
    dgate = c * f
    e_gate = 1.01 * (ec * np.abs(f) + ef * np.abs(c)) + np.abs(dgate) * 1.1 * F + TINY
    dx, error = 0.0, 0.0
    for d, e, (wq, ws) in ((dgate, e_gate, gate), (dup, e_up, up)):
        w = wq.astype(np.float64) * ws.astype(np.float64)[:, None]
        dx = dx + d @ w
        error = error + (e + (np.abs(d) + e) * (H + 2 * F)) @ np.abs(w) + ((np.abs(d) + e) @ np.abs(w)) * (2 * w.shape[0] + 4) * F
        error = error + TINY * np.abs(wq.astype(np.float64)).sum(0)[None, :]
    return _rounded(dx, error), _rounded(dgate, e_gate), _rounded(dup, e_up)


def route_reference(logits, top_k, renormalize=True):
    """(weights, bound), experts, positions, tokens, offsets by sorting each token's experts in Python."""
    T, E = logits.shape
    weights, experts = np.zeros((T, top_k)), np.full((T, top_k), -1, np.int32)
    positions = np.full((T, top_k), -1, np.int32)
    for t in range(T):
        row = [float(v) for v in logits[t]]
        chosen = sorted((e for e in range(E) if row[e] > -np.inf), key=lambda e: (-row[e], e))[:top_k]
        experts[t, :len(chosen)] = chosen
        if any(v != v for v in row):
            weights[t], positions[t] = np.nan, NAN_ROW
        elif chosen:
            over = chosen if renormalize else [e for e in range(E) if row[e] > -np.inf]
            with np.errstate(invalid="ignore"):
                p = {e: np.exp(np.float64(row[e]) - row[chosen[0]]) for e in over}
            weights[t, :len(chosen)] = [p[e] / sum(p.values()) for e in chosen]
    tokens, offsets = np.full(T * top_k, -1, np.int32), [0]
    row = 0
    for e in range(E):
        for t in range(T):
            for j in range(top_k):
                if experts[t, j] == e:
                    positions[t, j], tokens[row] = row, t
                    row += 1
        offsets.append(row)
    # exponentials of differences: the difference rounds once (F of it), expf is off by at most 2 steps; the sum has
    # up to E terms; one division
    spread = np.zeros((T, 1))
    for t in range(T):
        finite = logits[t][np.isfinite(logits[t])]
        spread[t] = finite.max() - finite.min() if len(finite) else 0.0
    bound = np.abs(weights) * (2 * spread + E + 12) * F + TINY
    return (weights, bound), experts, positions, tokens, np.array(offsets, np.int32)


def route_backward_reference(logits, experts, dweights, renormalize=True):
    """dlogits and the fp32 error before the output's rounding."""
    T, E = logits.shape
    d, error = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if np.isnan(logits[t]).any():
            d[t] = np.nan
            continue
        mine = [e for e in experts[t] if e >= 0]
        if not mine:
            continue
        over = np.array(mine if renormalize else [e for e in range(E) if logits[t, e] > -np.inf])
        p = np.exp(logits[t, over] - logits[t, over].max())
        p /= p.sum()
        dw = np.zeros(E)
        dw[mine] = dweights[t, :len(mine)]
        c = (p * dw[over]).sum()
        d[t, over] = p * (dw[over] - c)
        ep = (2 * np.ptp(logits[t, over]) + E + 12) * F           # relative, of each p
        mass = (p * np.abs(dw[over])).sum()
        error[t, over] = p * (np.abs(dw[over] - c) * (ep + 2 * F) + mass * (ep + (E + 2) * F)) + TINY
    return d, error


def combine_reference(y, positions, weights=None):
    T, top_k = positions.shape
    out, mass = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(top_k):
            if 0 <= positions[t, j] < len(y):
                term = (1.0 if weights is None else float(weights[t, j])) * y[positions[t, j]]
                out[t] += term
                mass[t] += np.abs(term)
            elif positions[t, j] == NAN_ROW:
                out[t] = np.nan
    return _rounded(out, mass * (top_k + 1) * F + TINY)


def combine_backward_reference(dout, y, positions, weights):
    """(dy, bound) with NaN in rows at no position, (dweights, bound)."""
    T, top_k = positions.shape
    dy, dw, mass = np.full(y.shape, np.nan), np.zeros((T, top_k)), np.zeros((T, top_k))
    for t in range(T):
        for j in range(top_k):
            r = positions[t, j]
            if 0 <= r < len(y):
                dy[r] = float(weights[t, j]) * dout[t]
                dw[t, j] = (dout[t] * y[r]).sum()
                mass[t, j] = np.abs(dout[t] * y[r]).sum()
            elif r == NAN_ROW:
                dw[t, j] = np.nan
    return _rounded(dy, np.abs(dy) * F), (dw, mass * (y.shape[1] + 1) * F + TINY)


def within(got, expected):
    """None, or what is wrong: NaN where the reference has NaN, infinities alike, else within the bound."""
    value, bound = expected
    got = np.asarray(got, dtype=np.float64)
    if got.shape != np.shape(value):
        return f"shape {got.shape}, expected {np.shape(value)}"
    nan = np.isnan(value)
    same = np.where(np.isinf(value), got == value, True)
    with np.errstate(invalid="ignore"):
        near = np.where(np.isfinite(value), np.abs(got - value) <= bound, True)
    bad = np.where(nan, ~np.isnan(got), ~(same & near & ~np.isnan(got)))
    if not bad.any():
        return None
    at = tuple(int(i) for i in np.argwhere(bad)[0])
    return f"{int(bad.sum())} of {bad.size} wrong, first at {at}: {got[at]!r}, expected {value[at]!r} within {np.broadcast_to(bound, got.shape)[at]!r}"
