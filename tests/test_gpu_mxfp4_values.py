"""MXFP4 on the GPU at the ends of its values: what decode rows quantize on the way, NaN and infinities,
the smallest and largest scales, gates where the sigmoid vanishes, the longest contraction."""

import numpy as np
import pytest

import oracle as O

from gpu_helpers import announce
from test_gpu_mxfp4 import bf16, bf16_values, check, to_gpu, values, weight

pytestmark = pytest.mark.gpu

DECODE_ROWS = [1, 2, 3, 4, 5, 8, 9, 16]


def one_hot(N, K, scale):
    """Weight rows n < K with one 1.0 (code 2) at k = n, all others zero; one scale byte."""
    import torch
    codes = np.zeros((N, K), np.uint8)
    n = np.arange(min(N, K))
    codes[n, n] = 2
    return to_gpu(O.mx_pack(codes), torch.uint8), torch.full((N, K // 32), scale, dtype=torch.uint8, device="cuda:0")


def special_blocks():
    """(name, weight scale byte, float32 blocks [n, 32]): every finite bf16 value under three tops and as its
    block's top, the borders between codes, zeros of both signs."""
    every = (np.arange(65536, dtype=np.uint32) << 16).view(np.float32)
    out = []
    for name, top, scale in (("one", 1.0, 127), ("smallest", 2.0 ** -126, 187), ("large", 2.0 ** 100, 127)):
        x = every.reshape(-1, 16).copy()
        x[~np.isfinite(x) | (np.abs(x) >= np.float32(8 * top))] = 0
        rows = np.zeros((x.shape[0], 32), np.float32)
        rows[:, :16], rows[:, 31] = x, 6 * top
        out.append((name, scale, rows))
    finite = every[np.isfinite(every)]
    small, rest = finite[np.abs(finite) < 1], finite[np.abs(finite) >= 1]
    for name, tops, scale in (("small tops", small, 187), ("tops", rest, 67)):
        rows = np.zeros((tops.size, 32), np.float32)
        rows[np.arange(tops.size), np.arange(tops.size) % 32] = tops
        out.append((name, scale, rows))
    borders = np.array([0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.5, 7.0, 7.5], np.float32)
    near = np.concatenate([borders * np.float32(f) for f in (1 - 2.0 ** -7, 1.0, 1 + 2.0 ** -7)])
    near = np.asarray(bf16_values(near[near < 8]), np.float32)
    for name, scale, exponents in (("small borders", 187, (-127, -126, -125, -60)), ("borders", 67, (0, 60))):
        rows = []
        for e in exponents:
            block = np.zeros((near.size, 32), np.float32)
            block[:, 5], block[:, 6] = np.ldexp(near, e), -np.ldexp(near, e)
            block[:, 31], block[:, 0] = np.ldexp(np.float32(4), e), -0.0
            rows.append(block)
        out.append((name, scale, np.asarray(bf16_values(np.concatenate(rows)), np.float32)))
    return out


def quantized_on_the_way(lib, x, N, scale, M):
    """mxfp4a4_linear of M rows at a time against one-hot weights: the value each element was rounded to."""
    import torch
    K = x.shape[1]
    w = one_hot(N, K, scale)
    t = bf16(x)
    assert np.array_equal(values(t), x.astype(np.float64))
    got = torch.cat([lib.mxfp4a4_linear(t[r:r + M].contiguous(), *w)[:, :K] for r in range(0, x.shape[0], M)])
    steps = torch.cat([lib.qmm_mxfp4a4(*lib.mxfp4_quantize_rows(t[r:r + M].contiguous()), *w)[:, :K]
                       for r in range(0, x.shape[0], M)])
    assert torch.equal(got.view(torch.int16), steps.view(torch.int16))
    factor = 2.0 ** (scale - 127)
    expected = O.mx_decode(*O.mx_encode(x)) * factor
    wrong = np.argwhere(values(got) != expected)
    assert not wrong.size, [(tuple(i), x[tuple(i)], values(got)[tuple(i)], expected[tuple(i)]) for i in wrong[:4]]


@pytest.mark.parametrize("M", DECODE_ROWS)
def test_decode_rows_quantize_every_value(lib, M):
    """Up to 16 rows mxfp4a4_linear quantizes in the product's kernel: the same rule, value by value."""
    K = 512 if M > 4 else 1056                         # whole windows, and a ragged last unit
    for name, scale, blocks in special_blocks():
        announce(f"mxfp4a4_linear quantizing M={M} {name}")
        blocks = blocks if M in (1, 16) else blocks[::7]
        per_row = K // 32
        rows = -(-blocks.shape[0] // per_row)
        x = np.zeros((rows * per_row, 32), np.float32)
        x[:blocks.shape[0]] = blocks
        quantized_on_the_way(lib, x.reshape(rows, K), K, scale, M)


@pytest.mark.parametrize("M,N", [(1, 20500), (5, 12300), (16, 12300)])
def test_wide_decode_rows_quantize_every_value(lib, M, N):
    K = 512
    assert lib.mxfp4_plan(lib.MXFP4A4_LINEAR, M, N, K)["variant"] == 0
    for name, scale, blocks in special_blocks():
        announce(f"mxfp4a4_linear wide quantizing M={M} {name}")
        blocks = blocks[::5]
        rows = -(-blocks.shape[0] // 16)
        x = np.zeros((rows * 16, 32), np.float32)
        x[:blocks.shape[0]] = blocks
        quantized_on_the_way(lib, x.reshape(rows, K), N, scale, M)


SHAPES = [(M, 136, 288) for M in DECODE_ROWS] + [(40, 136, 288), (1, 20500, 512), (5, 12300, 512), (16, 12300, 512)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_invalid_values_stay_in_their_rows_and_columns(lib, M, N, K, bad):
    """Decode rows, the wide form and tiles: an invalid activation reaches its own row, a NaN scale its own
    column, in the projections and the gated pair."""
    import torch
    announce(f"mxfp4 invalid values M={M} N={N} K={K} {bad}")
    rng = np.random.default_rng(M + N)
    (codes, scales), _ = weight(rng, N, K, 118, 124)
    up, uv = weight(rng, N, K, 118, 124)
    x = bf16_values(rng.standard_normal((M, K)))
    stored = O.mx_unpack(codes.cpu().numpy())
    stored[stored % 8 == 0] = 1                        # (an infinity times a zero weight would be NaN)
    codes = to_gpu(O.mx_pack(stored), torch.uint8)
    bad_scales = scales.clone()
    bad_scales[N // 3, 2] = 255
    wv = O.mx_decode(codes.cpu().numpy(), bad_scales.cpu().numpy())
    row = M - 1
    x[row, 70] = np.nan if bad == "nan" else -np.inf
    t = bf16(np.where(np.isfinite(x), x, 0))
    t[row, 70] = float("nan") if bad == "nan" else float("-inf")
    with np.errstate(invalid="ignore"):
        expected = O.mx_linear(x, wv)
        check(lib.mxfp4_linear(t, codes, bad_scales), expected)
        xq = lib.mxfp4_quantize_rows(t)
        xv = O.mx_decode(*(q.cpu().numpy() for q in xq))
        assert np.isnan(xv[row, 64:96]).all() and np.isfinite(xv).sum() == xv.size - 32
        four = O.mx_linear(xv, wv)
        check(lib.qmm_mxfp4a4(*xq, codes, bad_scales), four)
        check(lib.mxfp4a4_linear(t, codes, bad_scales), four)
        if N > 1000:
            return
        # the gated pair; an infinite gate or up leaves nothing finite (silu(-inf) is -inf 0)
        h = values(lib.mxfp4_gate_up_swiglu(t, (codes, bad_scales), up))
        dh = bf16_values(rng.standard_normal((M, N)))
        dx, dgate, dup = (values(v) for v in lib.mxfp4_gate_up_swiglu_backward(t, (codes, bad_scales), up, bf16(dh)))
    keep_r, keep_c = np.arange(M) != row, np.arange(N) != N // 3
    xs, gs, us = x[keep_r], wv[keep_c], uv[keep_c]
    if M > 1:
        check(torch.from_numpy(h[keep_r][:, keep_c]), O.mx_gate_up(xs, gs, us))
        (_, _), eg, eu = O.mx_gate_up_backward(xs, gs, us, dh[keep_r][:, keep_c])
        check(torch.from_numpy(dgate[keep_r][:, keep_c]), eg)
        check(torch.from_numpy(dup[keep_r][:, keep_c]), eu)
        # that column's gradients are NaN, and its weights spread them over the rows' dx
        assert np.isnan(dx[keep_r]).all()
    for v in (h, dgate, dup):
        assert np.isnan(v[:, N // 3]).all() and not np.isfinite(v[row]).any()


@pytest.mark.parametrize("M", [1, 4, 16, 20, 200])
def test_extreme_scales(lib, M):
    """The smallest scales, alone too, and the largest that bf16 holds, in both directions of the product;
    subnormal activations."""
    announce(f"mxfp4 extreme scales M={M}")
    rng = np.random.default_rng(M)
    for low, high, size in ((0, 1, 2.0 ** 100), (0, 4, 2.0 ** 100), (248, 253, 2.0 ** -100), (220, 224, 2.0 ** -131)):
        w, wv = weight(rng, 136, 320, low, high)
        x = bf16_values(rng.standard_normal((M, 320)) * size)
        dy = bf16_values(rng.standard_normal((M, 136)) * size)
        check(lib.mxfp4_linear(bf16(x), *w), O.mx_linear(x, wv))
        check(lib.mxfp4_linear_backward(bf16(dy), *w), O.mx_linear_backward(dy, wv))
        xq = lib.mxfp4_quantize_rows(bf16(x))
        check(lib.qmm_mxfp4a4(*xq, *w), O.mx_linear(O.mx_decode(*(t.cpu().numpy() for t in xq)), wv))
        check(lib.mxfp4a4_linear(bf16(x), *w), O.mx_linear(O.mx_decode(*(t.cpu().numpy() for t in xq)), wv))


def test_dequantize_the_two_largest_scales(lib):
    """Scale bytes 253 and 254: 2^128 and above is past bf16 and decodes to an infinity of its sign."""
    import torch
    announce("mxfp4_dequantize_rows scales 253 and 254")
    codes = np.tile(O.mx_pack(np.arange(32).reshape(1, 32) % 16), (2, 1))
    scales = np.array([[253], [254]], np.uint8)
    ref = O.mx_decode(codes, scales)
    ref = np.where(np.abs(ref) >= 2.0 ** 128, np.copysign(np.inf, ref), ref)
    assert np.isinf(ref).sum(1).tolist() == [8, 16]
    got = values(lib.mxfp4_dequantize_rows(to_gpu(codes, torch.uint8), to_gpu(scales, torch.uint8)))
    assert np.array_equal(got, ref) and np.array_equal(np.signbit(got), np.signbit(ref))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products_with_the_two_largest_scales(lib, M, N, K):
    """Weight-only products take such weights as infinities; 4-bit products scale in the matrix core and
    stay exact up to fp32's range."""
    import torch
    announce(f"mxfp4 products with scales 253 and 254 M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + 1)
    (codes, _), _ = weight(rng, N, K)
    # in every third block of every third weight row, so that finite outputs are left in both directions
    s = np.full((N, K // 32), 252, np.uint8)
    s[::3, ::3] = rng.integers(253, 255, s[::3, ::3].shape)
    w, wv = (codes, to_gpu(s, torch.uint8)), O.mx_decode(codes.cpu().numpy(), s)
    x, xv = weight(rng, M, K, 60, 64)
    check(lib.qmm_mxfp4a4(*x, *w), O.mx_linear(xv, wv))
    check(lib.mxfp4a4_linear(lib.mxfp4_dequantize_rows(*x), *w),
          O.mx_linear(O.mx_decode(*O.mx_encode(xv)), wv))

    def activations(shape):                            # no zeros: an infinity times zero would be NaN
        return bf16_values(np.where(rng.random(shape) < 0.5, -1, 1) * rng.uniform(1, 2, shape) * 2.0 ** -60)
    held = np.where(np.abs(wv) >= 2.0 ** 128, np.copysign(np.inf, wv), wv)
    assert np.isinf(held).any()
    with np.errstate(invalid="ignore"):
        xb = activations((M, K))
        check(lib.mxfp4_linear(bf16(xb), *w), O.mx_linear(xb, held))
        if N < 1000:
            dy = activations((M, N))
            check(lib.mxfp4_linear_backward(bf16(dy), *w), O.mx_linear_backward(dy, held))


@pytest.mark.parametrize("M", [1, 8, 40])
def test_gates_where_the_sigmoid_vanishes(lib, M):
    """Gates of +-60 .. 96, exact in fp32, beside up = 1 .. 2^40.  The sigmoid is within (4 + |g|) 2^-23 of its
    value, or 0 where that is below 2^-126 (off by less than 2^-126 then); the products add a few steps of
    fp32, of both terms where 1 + g (1 - s) has two, and the rounding to bf16 2^-8."""
    import torch
    announce(f"mxfp4 gates where the sigmoid vanishes M={M}")
    N, K = 144, 64
    codes = np.zeros((2, N, K), np.uint8)
    codes[0, :, :2] = codes[1, :, 33:34] = 2           # 1.0: the gate is x[:, 0] + x[:, 1], up takes x[:, 33] = 1
    exps = np.full((2, N, 2), 127, np.uint8)
    exps[1, :, 1] += (np.arange(N) % 41).astype(np.uint8)
    gate, up = ((to_gpu(O.mx_pack(codes[i]), torch.uint8), to_gpu(exps[i], torch.uint8)) for i in range(2))
    uv = np.ldexp(1.0, np.arange(N) % 41)[None, :]
    every = np.arange(60, 96, 0.25)
    every = np.concatenate([-every, every])
    for first in range(0, every.size, M):
        x = np.zeros((M, K))
        gv = np.resize(every[first:first + M], M)[:, None]
        x[:, :1], x[:, 1:2], x[:, 33] = np.trunc(gv), gv - np.trunc(gv), 1
        assert np.array_equal(bf16_values(x), x)
        h = lib.mxfp4_gate_up_swiglu(bf16(x), gate, up)
        _, dg, du = lib.mxfp4_gate_up_swiglu_backward(bf16(x), gate, up, bf16(np.ones((M, N))))
        s, rest = 1 / (1 + np.exp(-gv)), 1 / (1 + np.exp(gv))
        off = s * (4 + np.abs(gv)) * 2.0 ** -23 + np.where(s < 2.0 ** -125, 2.0 ** -126, 0)
        for got, value, slope, terms in ((h, gv * s * uv, gv * uv, 0), (du, gv * s + 0 * uv, gv + 0 * uv, 0),
                                         (dg, uv * s * (1 + gv * rest), uv * (1 + np.abs(gv)), uv * s * (1 + np.abs(gv)))):
            before = np.abs(slope) * off + 2.0 ** -22 * (np.abs(value) + terms)
            check(got, (value, before + 2.0 ** -8 * (np.abs(value) + before) + 2.0 ** -134))


@pytest.mark.parametrize("M,N", [(2, 37), (16, 20), (20, 70)])
def test_the_longest_contraction(lib, M, N):
    """2^20 values of a weight row, and 2^20 weight rows of the transposed product."""
    import torch
    announce(f"mxfp4 longest contraction M={M} N={N}")
    L = 1 << 20
    rng = np.random.default_rng(M)
    w, wv = weight(rng, N, L, 118, 124)
    x = bf16(rng.standard_normal((M, L)).astype(np.float32))
    check(lib.mxfp4_linear(x, *w), O.mx_linear(values(x), wv))
    xq = lib.mxfp4_quantize_rows(x)
    xv = O.mx_decode(*(t.cpu().numpy() for t in xq))
    expected = O.mx_linear(xv, wv)
    check(lib.qmm_mxfp4a4(*xq, *w), expected)
    check(lib.mxfp4a4_linear(x, *w), expected)
    del wv, xv
    wt, tv = weight(rng, L, 64, 118, 124)
    check(lib.mxfp4_linear_backward(x, *wt), O.mx_linear_backward(values(x), tv))
