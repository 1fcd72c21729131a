"""Plain CPU oracle for the MXFP4 operators: quantization, products, the gated feed-forward block.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): the product path never imports this module.

MXFP4: a row of K values in blocks of 32; a block has a scale byte e (the factor ``2**(e - 127)``,
255 is NaN) and 32 codes of 4 bits, sign / two exponent bits / one mantissa bit.  Codes are packed two
per byte, the lower index in the low half.

Each matrix-valued function returns, next to the value, a bound on how far an implementation may be
off that takes exact products of the stored operands, sums them in fp32 in any order and rounds the
result to bf16 once:

* a sum of n terms in fp32: at most ``n 2^-24 / (1 - n 2^-24)`` times the sum of the terms'
  magnitudes; ``(n + 8) 2^-24`` covers that for every n used here;
* rounding to bf16: half a step, ``2^-8`` of the value (and ``2^-134`` near zero).
"""

import numpy as np

__all__ = ["MX_BLOCK", "MX_VALUES", "mx_pack", "mx_unpack", "mx_scale_values", "mx_decode", "mx_encode",
           "mx_linear", "mx_linear_backward", "mx_gate_up", "mx_gate_up_backward", "mx_check"]

MX_BLOCK = 32
_POSITIVE = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MX_VALUES = np.concatenate([_POSITIVE, -_POSITIVE])

_U32 = 2.0 ** -24          # half a step of fp32, relative
_U16 = 2.0 ** -8           # half a step of bf16, relative
_TINY = 2.0 ** -134        # half of bf16's smallest subnormal


def mx_pack(codes):
    """Codes ``[R, K]`` (0..15) -> bytes ``[R, K/2]``."""
    c = np.asarray(codes, dtype=np.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def mx_unpack(packed):
    p = np.asarray(packed, dtype=np.uint8)
    out = np.empty((p.shape[0], 2 * p.shape[1]), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = p & 15, p >> 4
    return out


def mx_scale_values(scales):
    s = np.asarray(scales).astype(np.int64)
    return np.where(s == 255, np.nan, np.ldexp(1.0, np.where(s == 255, 0, s - 127)))


def mx_decode(packed, scales):
    """float64 values of packed rows."""
    return MX_VALUES[mx_unpack(packed)] * np.repeat(mx_scale_values(scales), MX_BLOCK, axis=1)


def mx_encode(x):
    """(packed, scales) of the rows of x: nearest value by comparing all eight, ties to even codes."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    b = x.reshape(R, K // MX_BLOCK, MX_BLOCK)
    scales = np.zeros(b.shape[:2], dtype=np.uint8)
    codes = np.zeros(b.shape, dtype=np.uint8)
    for r in range(b.shape[0]):
        for g in range(b.shape[1]):
            v = b[r, g]
            if not np.all(np.isfinite(v)):
                scales[r, g] = 255
                continue
            a = np.max(np.abs(v))
            e = max(int(np.frexp(a)[1]) - 1 - 2, -127) if a > 0 else -127
            scales[r, g] = e + 127
            far = np.abs(np.abs(np.ldexp(v, -e))[:, None] - _POSITIVE[None, :])
            best = far.min(axis=1, keepdims=True)
            near = far == best                                   # one code, or two beside a tie
            even = near & (np.arange(8) % 2 == 0)
            pick = np.where(near.sum(1) > 1, even.argmax(1), near.argmax(1))
            codes[r, g] = pick + 8 * np.signbit(v)
    return mx_pack(codes.reshape(R, K)), scales


def _sum_bound(n, magnitude):
    return (n + 8) * _U32 * magnitude


def _rounded(value, before):
    """Bound after rounding a value known to +-before to bf16."""
    return before + _U16 * (np.abs(value) + before) + _TINY


def mx_linear(x, w):
    """(x w^T, bound): x float64 [M, K], w float64 [N, K]."""
    y = x @ w.T
    return y, _rounded(y, _sum_bound(x.shape[1], np.abs(x) @ np.abs(w).T))


def mx_linear_backward(dy, w):
    """(dy w, bound)."""
    dx = dy @ w
    return dx, _rounded(dx, _sum_bound(w.shape[0], np.abs(dy) @ np.abs(w)))


def _sigmoid(g):
    return 1.0 / (1.0 + np.exp(-g))


def _projections(x, wg, wu):
    g, u = x @ wg.T, x @ wu.T
    n = x.shape[1]
    return g, u, _sum_bound(n, np.abs(x) @ np.abs(wg).T), _sum_bound(n, np.abs(x) @ np.abs(wu).T)


def mx_gate_up(x, wg, wu):
    """(silu(g) u, bound).  silu has a slope of at most 1.1; exp, the quotient and the products are
    within 16 steps of fp32 of their values, and e^-g of an fp32 argument adds |g| steps."""
    with np.errstate(over="ignore"):
        g, u, dg, du = _projections(x, wg, wu)
        s = g * _sigmoid(g)
    h = s * u
    before = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + (16 + np.abs(g)) * _U32 * np.abs(h)
    return h, _rounded(h, before)


def mx_gate_up_backward(x, wg, wu, dh):
    """((dx, bound), (dgate, bound), (dup, bound)).

    dup = dh silu(g); dgate = dh u t(g) with t = s (1 + g (1 - s)), |t| <= 1.1 and |t'| <= 0.5.  In
    fp32 t is off by at most (16 + |g|) steps of s (1 + |g| (1 - s)).  dx takes the gradients within
    their bounds, so its bound has theirs through the weights, and its own sum of 2 N terms.
    """
    with np.errstate(over="ignore"):
        g, u, eg, eu = _projections(x, wg, wu)
        s = _sigmoid(g)
        rest = _sigmoid(-g)
    silu, t = g * s, s * (1.0 + g * rest)
    dup = dh * silu
    bup = _rounded(dup, np.abs(dh) * 1.1 * eg + (16 + np.abs(g)) * _U32 * np.abs(dup))
    dgate = dh * u * t
    wide = s * (1.0 + np.abs(g) * rest)
    bgate = _rounded(dgate, np.abs(dh) * ((1.1 + 0.5 * eg) * eu + 0.5 * np.abs(u) * eg
                                          + (16 + np.abs(g)) * _U32 * wide * np.abs(u)))
    dx = dgate @ wg + dup @ wu
    before = bgate @ np.abs(wg) + bup @ np.abs(wu)
    before += _sum_bound(2 * wg.shape[0], (np.abs(dgate) + bgate) @ np.abs(wg) + (np.abs(dup) + bup) @ np.abs(wu))
    return (dx, _rounded(dx, before)), (dgate, bgate), (dup, bup)


def mx_check(got, value, bound):
    """None, or what is wrong: the worst element beyond its bound.  NaN and infinities have to be where they are
    in value (their bounds do not matter), and every finite value needs a finite bound."""
    got = np.asarray(got, dtype=np.float64)
    if got.shape != value.shape:
        return f"shape {got.shape}, not {value.shape}"
    nan = np.isnan(value)
    if not np.array_equal(np.isnan(got), nan):
        i = np.argwhere(np.isnan(got) != nan)[0]
        return f"NaN differs at {tuple(i)}: got {got[tuple(i)]}, {value[tuple(i)]} expected"
    unbounded = np.isfinite(value) & ~np.isfinite(bound)
    if unbounded.any():
        i = tuple(map(int, np.argwhere(unbounded)[0]))
        return f"no finite bound at {i}: {value[i]} +- {bound[i]}"
    # an infinity has to be met exactly; NaN elsewhere cannot arise, so a comparison decides every element
    exact = nan | (np.isinf(value) & (got == value))
    with np.errstate(invalid="ignore"):
        off = np.where(exact, 0.0, np.abs(got - value) - np.where(np.isfinite(bound), bound, 0.0))
    wrong = ~(off <= 0)
    if wrong.any():
        i = tuple(map(int, np.unravel_index(np.where(wrong, off, -np.inf).argmax(), off.shape)))
        return (f"{int(wrong.sum())} of {off.size} beyond the bound, worst at {i}: got {got[i]}, "
                f"{value[i]} +- {bound[i]} expected")
    return None
