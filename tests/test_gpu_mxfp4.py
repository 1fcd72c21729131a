"""GPU parity of the MXFP4 operators against the 64-bit CPU oracle.

Quantization and dequantization are compared bit for bit.  Products are held to the oracle's bounds:
exact products summed in fp32 in any order, one rounding to bf16 (see ``oracle/mxfp4_oracle.py``).
"""

import numpy as np
import pytest

import oracle as O
from w4a16_group_quantized_qmv_amd import synth

from gpu_helpers import announce

pytestmark = pytest.mark.gpu


def bf16_values(a):
    """float array rounded to bf16, as float64."""
    return O.bf16_to_f64(synth.to_bf16_bits(np.asarray(a, dtype=np.float32)))


def to_gpu(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0").to(dtype)


def bf16(a):
    import torch
    return to_gpu(np.asarray(a, dtype=np.float32), torch.bfloat16)


def values(t):
    return t.float().cpu().numpy().astype(np.float64)


def weight(rng, N, K, low=110, high=130):
    """Random codes and scales, on the GPU and as float64 values."""
    import torch
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    scales = rng.integers(low, high, (N, K // 32)).astype(np.uint8)
    return (to_gpu(codes, torch.uint8), to_gpu(scales, torch.uint8)), O.mx_decode(codes, scales)


def guarded(M, N, offset=0, dtype=None):
    """A bf16 output [M, N] inside a larger buffer, and a check that its surroundings stay."""
    import torch
    buf = torch.full((M * N + 512,), -77.0, dtype=torch.bfloat16, device="cuda:0")
    y = buf[256 + offset:256 + offset + M * N].view(M, N)

    def untouched():
        return bool((buf[:256 + offset] == -77).all()) and bool((buf[256 + offset + M * N:] == -77).all())
    return y, untouched


def check(got, expected):
    problem = O.mx_check(values(got), *expected)
    assert problem is None, problem


# ---------------------------------------------------------------------------- rows

def check_quantizer(lib, x, dtype):
    import torch
    t = to_gpu(x.astype(np.float32), dtype)
    codes, scales = lib.mxfp4_quantize_rows(t)
    torch.cuda.synchronize()
    ref_codes, ref_scales = O.mx_encode(t.float().cpu().numpy().astype(np.float64))
    assert np.array_equal(scales.cpu().numpy(), ref_scales)
    got = codes.cpu().numpy()
    assert np.array_equal(got, ref_codes), np.argwhere(got != ref_codes)[:4]
    back = values(lib.mxfp4_dequantize_rows(codes, scales))
    with np.errstate(invalid="ignore"):
        assert np.array_equal(back, O.mx_decode(ref_codes, ref_scales), equal_nan=True)


@pytest.mark.parametrize("R,K", [(1, 32), (3, 32), (33, 2560), (7, 96), (130, 416), (1, 9728)])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_quantize_random_rows(lib, R, K, kind):
    import torch
    announce(f"mxfp4_quantize_rows R={R} K={K} {kind}")
    rng = np.random.default_rng(R * 1000 + K)
    x = rng.standard_normal((R, K)) * np.exp(rng.uniform(-30, 30, (R, 1)))
    check_quantizer(lib, x, torch.bfloat16 if kind == "bf16" else torch.float32)


def test_quantize_every_bf16_value(lib):
    """All 65536 bit patterns, each in a block with a fixed top, and each as the top of its block."""
    import torch
    announce("mxfp4_quantize_rows every bf16 value")
    bits = np.arange(65536, dtype=np.uint32)
    every = (bits << 16).view(np.float32)
    for top in (1.0, 2.0 ** -126, 2.0 ** 100):
        x = every.reshape(-1, 16).copy()
        x[~np.isfinite(x) | (np.abs(x) >= np.float32(8 * top))] = 0
        rows = np.zeros((x.shape[0], 32), np.float32)
        rows[:, :16] = x
        rows[:, 31] = 6 * top
        check_quantizer(lib, rows, torch.bfloat16)
    rows = np.zeros((65536, 32), np.float32)
    rows[np.arange(65536), np.arange(65536) % 32] = every
    check_quantizer(lib, rows, torch.bfloat16)


def test_quantize_borders_in_fp32(lib):
    """The values at and one step beside every border, at small, ordinary and large scales."""
    import torch
    announce("mxfp4_quantize_rows borders")
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], dtype=np.float32)
    near = np.stack([np.nextafter(borders, np.float32(0)), borders, np.nextafter(borders, np.float32(8))], 1).ravel()
    rows = []
    for e in (-120, -20, 0, 20, 120):
        row = np.zeros(64, np.float32)
        row[:near.size] = np.ldexp(near, e)
        row[32:32 + near.size] = -np.ldexp(near, e)
        row[31] = row[63] = np.ldexp(np.float32(4), e)
        rows.append(row)
    check_quantizer(lib, np.stack(rows), torch.float32)


def test_quantize_invalid_zero_and_tiny_blocks(lib):
    import torch
    announce("mxfp4_quantize_rows invalid blocks")
    x = np.zeros((6, 96), np.float32)
    x[0, 3], x[1, 40], x[2, 95], x[3, 0] = np.inf, -np.inf, np.nan, -0.0
    x[4, 5], x[4, 50] = 1e-45, -1.2e-38
    x[5, 7] = 3.4e38
    for dtype in (torch.bfloat16, torch.float32):
        check_quantizer(lib, x, dtype)


def test_dequantize_every_code_and_scale(lib):
    import torch
    announce("mxfp4_dequantize_rows every code and scale")
    scales = np.arange(253, dtype=np.uint8).reshape(-1, 1)
    scales = np.concatenate([scales, [[255]]]).astype(np.uint8)
    codes = np.tile(O.mx_pack(np.arange(32).reshape(1, 32) % 16), (scales.shape[0], 1))
    got = values(lib.mxfp4_dequantize_rows(to_gpu(codes, torch.uint8), to_gpu(scales, torch.uint8)))
    ref = O.mx_decode(codes, scales)
    assert np.array_equal(got, ref, equal_nan=True)
    assert np.array_equal(np.signbit(got[:-1]), np.signbit(ref[:-1]))


# ---------------------------------------------------------------------------- products

# rows, weight rows, values: single rows and columns, widths that fill no tile, a tail of one block,
# tails of a half and of a whole step, and shapes with a policy split
SIZES = [(1, 1, 32), (1, 7, 64), (2, 33, 96), (3, 130, 160), (5, 100, 544), (8, 257, 512), (9, 64, 1120),
         (16, 300, 416), (17, 129, 1056), (31, 72, 2560), (33, 500, 288), (64, 64, 64), (127, 130, 608),
         (129, 127, 320), (130, 1000, 416), (300, 264, 736), (109, 1485, 2592), (35, 112, 1312), (1, 2560, 9728), (4, 1024, 2560)]
BACK_SIZES = SIZES[:-2] + [(1, 1000, 2560), (130, 1003, 416)]


@pytest.mark.parametrize("split", [0, 1, 3])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(lib, M, N, K, split):
    announce(f"mxfp4_linear M={M} N={N} K={K} split={split}")
    rng = np.random.default_rng(M + N + K)
    w, wv = weight(rng, N, K)
    x = bf16_values(rng.standard_normal((M, K)))
    y, untouched = guarded(M, N, offset=M % 2)             # rows at 2-byte alignment too
    assert lib.mxfp4_linear(bf16(x), *w, y=y, split_k=split) is y
    check(y, O.mx_linear(x, wv))
    assert untouched()


@pytest.mark.parametrize("split", [0, 1, 2])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_of_codes(lib, M, N, K, split):
    announce(f"qmm_mxfp4a4 M={M} N={N} K={K} split={split}")
    rng = np.random.default_rng(M + N + K + 1)
    w, wv = weight(rng, N, K)
    x, xv = weight(rng, M, K)
    y, untouched = guarded(M, N, offset=M % 2)
    lib.qmm_mxfp4a4(*x, *w, y=y, split_k=split)
    check(y, O.mx_linear(xv, wv))
    assert untouched()


@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_with_4_bit_activations(lib, M, N, K):
    """One call equals its two steps bit for bit."""
    import torch
    announce(f"mxfp4a4_linear M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K + 2)
    w, wv = weight(rng, N, K)
    x = bf16_values(rng.standard_normal((M, K)))
    y = lib.mxfp4a4_linear(bf16(x), *w)
    check(y, O.mx_linear(O.mx_decode(*O.mx_encode(x)), wv))
    again = lib.qmm_mxfp4a4(*lib.mxfp4_quantize_rows(bf16(x)), *w)
    assert torch.equal(y, again)


@pytest.mark.parametrize("split", [0, 1, 3])
@pytest.mark.parametrize("M,N,K", BACK_SIZES)
def test_linear_backward(lib, M, N, K, split):
    announce(f"mxfp4_linear_backward M={M} N={N} K={K} split={split}")
    rng = np.random.default_rng(M + N + K + 3)
    w, wv = weight(rng, N, K)
    dy = bf16_values(rng.standard_normal((M, N)))
    dx, untouched = guarded(M, K, offset=M % 2)
    lib.mxfp4_linear_backward(bf16(dy), *w, dx=dx, split_k=split)
    check(dx, O.mx_linear_backward(dy, wv))
    assert untouched()


# many columns: the wide decode form, with ragged last blocks, and the grids of the large tiles
WIDE_SIZES = [(1, 20500, 512), (3, 20007, 1536), (5, 12391, 1024), (16, 16384, 512), (16, 12300, 4608)]
LARGE_SIZES = [(773, 13176, 96), (522, 13265, 96), (961, 10881, 544), (300, 17001, 160),
               (770, 5999, 4928)]
LARGE_BACK_SIZES = [(2323, 72, 4928), (1298, 72, 5952), (321, 75, 5408), (771, 140, 4928)]
LARGE_GATED_SIZES = [(390, 11227, 96), (257, 10998, 96), (2325, 72, 4896), (1422, 75, 5408), (201, 2000, 1376),
                     (513, 3999, 416), (771, 75, 4928)]


# long contractions at decode rows: shares of one and two batches a wave, whole and ragged, one
# workgroup a compute unit and more
@pytest.mark.parametrize("M,N,K", [(1, 1500, 8192), (2, 1029, 9728), (3, 1100, 14336), (4, 500, 9728), (6, 2100, 8224),
                                   (7, 2070, 9728), (8, 2051, 16416), (8, 2100, 32768), (16, 70, 9728), (13, 33, 16384)])
def test_long_contractions_at_decode_rows(lib, M, N, K):
    import torch
    announce(f"mxfp4 long decode M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K + 8)
    w, wv = weight(rng, N, K)
    x = bf16_values(rng.standard_normal((M, K)))
    y, untouched = guarded(M, N, offset=1)
    lib.mxfp4_linear(bf16(x), *w, y=y)
    check(y, O.mx_linear(x, wv))
    xq = lib.mxfp4_quantize_rows(bf16(x))
    z = lib.qmm_mxfp4a4(*xq, *w)
    check(z, O.mx_linear(O.mx_decode(*(t.cpu().numpy() for t in xq)), wv))
    assert torch.equal(z, lib.mxfp4a4_linear(bf16(x), *w)) and untouched()
    check(lib.mxfp4_gate_up_swiglu(bf16(x), w, (w[0].flip(0), w[1].flip(0))), O.mx_gate_up(x, wv, wv[::-1]))


@pytest.mark.parametrize("M,N,K", WIDE_SIZES)
def test_many_columns_at_decode_rows(lib, M, N, K):
    import torch
    announce(f"mxfp4 wide decode M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K + 6)
    w, wv = weight(rng, N, K)
    x = bf16_values(rng.standard_normal((M, K)))
    for op in (lib.MXFP4_LINEAR, lib.MXFP4_QMM_A4, lib.MXFP4A4_LINEAR):
        p = lib.mxfp4_plan(op, M, N, K)
        assert (p["path"], p["variant"]) == (lib.PATH_MXFP4_QMV, 0)
    y, untouched = guarded(M, N, offset=1)
    lib.mxfp4_linear(bf16(x), *w, y=y)
    check(y, O.mx_linear(x, wv))
    xq = lib.mxfp4_quantize_rows(bf16(x))
    z = lib.qmm_mxfp4a4(*xq, *w)
    check(z, O.mx_linear(O.mx_decode(*(t.cpu().numpy() for t in xq)), wv))
    assert torch.equal(z, lib.mxfp4a4_linear(bf16(x), *w)) and untouched()
    # scale rows that start at an odd address: the other form, the same products
    odd = torch.cat([w[1].view(-1)[:1], w[1].view(-1)])[1:].view(w[1].shape)
    check(lib.mxfp4_linear(bf16(x), w[0], odd), O.mx_linear(x, wv))
    check(lib.qmm_mxfp4a4(*xq, w[0], odd), O.mx_linear(O.mx_decode(*(t.cpu().numpy() for t in xq)), wv))


@pytest.mark.parametrize("M,N,K", LARGE_SIZES)
def test_large_grids(lib, M, N, K):
    announce(f"mxfp4 large grids M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K + 7)
    w, wv = weight(rng, N, K)
    x = bf16_values(rng.standard_normal((M, K)))
    y, untouched = guarded(M, N)
    check(lib.mxfp4_linear(bf16(x), *w, y=y), O.mx_linear(x, wv))
    xq = lib.mxfp4_quantize_rows(bf16(x))
    lib.qmm_mxfp4a4(*xq, *w, y=y)
    check(y, O.mx_linear(O.mx_decode(*(t.cpu().numpy() for t in xq)), wv))
    assert untouched()


@pytest.mark.parametrize("M,N,K", LARGE_BACK_SIZES)
def test_large_grids_backward(lib, M, N, K):
    announce(f"mxfp4 large backward grids M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K + 8)
    w, wv = weight(rng, N, K)
    dy = bf16_values(rng.standard_normal((M, N)))
    dx, untouched = guarded(M, K)
    check(lib.mxfp4_linear_backward(bf16(dy), *w, dx=dx), O.mx_linear_backward(dy, wv))
    assert untouched()


@pytest.mark.parametrize("M,N,K", LARGE_GATED_SIZES)
def test_large_grids_gated(lib, M, N, K):
    announce(f"mxfp4 large gated grids M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K + 9)
    x, gate, gv, up, uv = gated(rng, M, N, K)
    h, untouched = guarded(M, N)
    check(lib.mxfp4_gate_up_swiglu(bf16(x), gate, up, h=h), O.mx_gate_up(x, gv, uv))
    dh = bf16_values(rng.standard_normal((M, N)))
    got = lib.mxfp4_gate_up_swiglu_backward(bf16(x), gate, up, bf16(dh))
    for g, expected in zip(got, O.mx_gate_up_backward(x, gv, uv, dh)):
        check(g, expected)
    assert untouched()


@pytest.mark.parametrize("op,sizes", [
    ("MXFP4_LINEAR", "SIZES LARGE_SIZES"), ("MXFP4_QMM_A4", "SIZES LARGE_SIZES"),
    ("MXFP4_GATE_UP", "SIZES LARGE_GATED_SIZES"), ("MXFP4_LINEAR_BACKWARD", "BACK_SIZES LARGE_BACK_SIZES"),
    ("MXFP4_GATE_UP_BACKWARD", "BACK_SIZES LARGE_GATED_SIZES")])
def test_sizes_reach_every_tile(lib, op, sizes):
    """The size lists above cover the five tile shapes, split and not, of every operator's policy."""
    plans = [lib.mxfp4_plan(getattr(lib, op), *s) for name in sizes.split() for s in globals()[name]]
    tiles = {p["variant"] for p in plans if p["path"] == lib.PATH_MXFP4}
    splits = {p["split_k"] > 1 for p in plans if p["path"] == lib.PATH_MXFP4}
    assert tiles == {0, 1, 2, 3, 4} and splits == {False, True}, (tiles, splits)


def gated(rng, M, N, K):
    """Inputs whose gate values reach both ends of the sigmoid."""
    gate, gv = weight(rng, N, K, 118, 124)
    up, uv = weight(rng, N, K, 118, 124)
    return bf16_values(rng.standard_normal((M, K))), gate, gv, up, uv


@pytest.mark.parametrize("split", [0, 1, 2])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gate_up(lib, M, N, K, split):
    announce(f"mxfp4_gate_up_swiglu M={M} N={N} K={K} split={split}")
    x, gate, gv, up, uv = gated(np.random.default_rng(M + N + K + 4), M, N, K)
    h, untouched = guarded(M, N, offset=M % 2)
    lib.mxfp4_gate_up_swiglu(bf16(x), gate, up, h=h, split_k=split)
    check(h, O.mx_gate_up(x, gv, uv))
    assert untouched()


@pytest.mark.parametrize("split", [0, 1, 3])
@pytest.mark.parametrize("M,N,K", BACK_SIZES)
def test_gate_up_backward(lib, M, N, K, split):
    announce(f"mxfp4_gate_up_swiglu_backward M={M} N={N} K={K} split={split}")
    rng = np.random.default_rng(M + N + K + 5)
    x, gate, gv, up, uv = gated(rng, M, N, K)
    dh = bf16_values(rng.standard_normal((M, N)))
    d = to_gpu(np.zeros((M, N + 1)), bf16(0).dtype).view(-1)[M % 2:M % 2 + M * N].view(M, N)   # dh at 2 bytes
    d.copy_(bf16(dh))
    dx, untouched = guarded(M, K, offset=M % 2)
    _, dgate, dup = lib.mxfp4_gate_up_swiglu_backward(bf16(x), gate, up, d, dx=dx, split_k=split)
    for got, expected in zip((dx, dgate, dup), O.mx_gate_up_backward(x, gv, uv, dh)):
        check(got, expected)
    assert untouched()
    # and closely: dx from the gradients that the call returned
    both = np.concatenate([values(dgate), values(dup)], 1)
    check(dx, O.mx_linear_backward(both, np.concatenate([gv, uv])))


def test_gate_up_backward_against_differences(lib):
    """The returned gradient, element by element, against differences of the 64-bit forward pass."""
    announce("mxfp4_gate_up_swiglu_backward differences")
    M, N, K = 3, 40, 64
    rng = np.random.default_rng(77)
    x, gate, gv, up, uv = gated(rng, M, N, K)
    dh = bf16_values(rng.standard_normal((M, N)))
    dx, _, _ = lib.mxfp4_gate_up_swiglu_backward(bf16(x), gate, up, bf16(dh))

    def loss(v):
        g, u = v @ gv.T, v @ uv.T
        return np.sum(dh * g / (1 + np.exp(-g)) * u)

    (ref, bound), _, _ = O.mx_gate_up_backward(x, gv, uv, dh)
    got = values(dx)
    for i in np.ndindex(M, K):
        d = np.zeros((M, K))
        d[i] = 2.0 ** -14
        slope = (loss(x + d) - loss(x - d)) / 2.0 ** -13
        # the difference itself is off by the third derivative times eps^2 / 6 and by rounding: both far
        # below a thousandth of the gradients' own bound here
        assert abs(slope - got[i]) <= 1.001 * bound[i] + 1e-5, i


# ---------------------------------------------------------------------------- values outside the ordinary

def test_invalid_values_stay_in_their_rows_and_columns(lib):
    """A NaN scale reaches its own output column, an invalid activation its own row."""
    import torch
    announce("mxfp4 invalid values")
    M, N, K = 40, 136, 288
    rng = np.random.default_rng(8)
    (codes, scales), wv = weight(rng, N, K)
    x = bf16_values(rng.standard_normal((M, K)))
    bad_scales = scales.clone()
    bad_scales[5, 3] = 255
    wv_bad = wv.copy()
    wv_bad[5, 96:128] = np.nan
    x_bad = bf16(x)
    x_bad[7, 100] = float("nan")
    xv_bad = x.copy()
    xv_bad[7, 100] = np.nan

    def expect(value, bound):
        return value, np.where(np.isnan(bound), 0, bound)

    check(lib.mxfp4_linear(x_bad, codes, bad_scales), expect(*O.mx_linear(xv_bad, wv_bad)))
    qc, qs = lib.mxfp4_quantize_rows(x_bad)
    xq = O.mx_decode(qc.cpu().numpy(), qs.cpu().numpy())
    check(lib.qmm_mxfp4a4(qc, qs, codes, bad_scales), expect(*O.mx_linear(xq, wv_bad)))
    dy = bf16_values(rng.standard_normal((M, N)))
    got = values(lib.mxfp4_linear_backward(bf16(dy), codes, bad_scales))
    assert np.isnan(got[:, 96:128]).all() and not np.isnan(got[:, :96]).any() and not np.isnan(got[:, 128:]).any()


def test_small_and_large_scales(lib):
    """Weights down to the smallest scale and up to the largest that bf16 holds."""
    announce("mxfp4 extreme scales")
    rng = np.random.default_rng(9)
    for low, high, size in ((0, 4, 2.0 ** 100), (248, 253, 2.0 ** -100)):
        w, wv = weight(rng, 72, 320, low, high)
        x = bf16_values(rng.standard_normal((20, 320)) * size)
        check(lib.mxfp4_linear(bf16(x), *w), O.mx_linear(x, wv))
        xq = lib.mxfp4_quantize_rows(bf16(x))
        check(lib.qmm_mxfp4a4(*xq, *w), O.mx_linear(O.mx_decode(*(t.cpu().numpy() for t in xq)), wv))


def test_large_gates(lib):
    """Gates where e^-g overflows or vanishes: finite results at both ends."""
    announce("mxfp4 large gates")
    M, N, K = 9, 40, 96
    rng = np.random.default_rng(10)
    gate, gv = weight(rng, N, K, 128, 134)
    up, uv = weight(rng, N, K, 118, 124)
    x = bf16_values(rng.standard_normal((M, K)))
    assert np.abs(x @ gv.T).max() > 200
    check(lib.mxfp4_gate_up_swiglu(bf16(x), gate, up), O.mx_gate_up(x, gv, uv))
    dh = bf16_values(rng.standard_normal((M, N)))
    got = lib.mxfp4_gate_up_swiglu_backward(bf16(x), gate, up, bf16(dh))
    for g, expected in zip(got, O.mx_gate_up_backward(x, gv, uv, dh)):
        check(g, expected)


# ---------------------------------------------------------------------------- as they are used

def test_feed_forward_block_and_its_backward(lib):
    """Checkpoint weights quantized, a block forward and backward, decode and prompt rows."""
    import torch
    rng = np.random.default_rng(11)
    H, F = 416, 608
    host = [rng.standard_normal(s) * 0.05 for s in ((F, H), (F, H), (H, F))]
    w = [lib.mxfp4_quantize_rows(to_gpu(m, torch.float32)) for m in host]
    v = [O.mx_decode(*(t.cpu().numpy() for t in pair)) for pair in w]
    for M in (1, 5, 70):
        announce(f"mxfp4 feed-forward block M={M}")
        x = bf16_values(rng.standard_normal((M, H)))
        h = lib.mxfp4_gate_up_swiglu(bf16(x), w[0], w[1])
        y = lib.mxfp4_linear(h, *w[2])
        check(h, O.mx_gate_up(x, v[0], v[1]))
        check(y, O.mx_linear(values(h), v[2]))
        dy = bf16_values(rng.standard_normal((M, H)))
        dh = lib.mxfp4_linear_backward(bf16(dy), *w[2])
        check(dh, O.mx_linear_backward(dy, v[2]))
        grads = lib.mxfp4_gate_up_swiglu_backward(bf16(x), w[0], w[1], dh)
        for got, expected in zip(grads, O.mx_gate_up_backward(x, v[0], v[1], values(dh))):
            check(got, expected)


def _calls(lib, M=40, N=136, K=1056, seed=12):
    """Every operator as a function of nothing, with its tensors kept."""
    rng = np.random.default_rng(seed)
    a, _ = weight(rng, N, K)
    b, _ = weight(rng, N, K, 118, 122)
    x, dh = bf16(rng.standard_normal((M, K))), bf16(rng.standard_normal((M, N)))
    xq = lib.mxfp4_quantize_rows(x)
    return {
        "quantize": lambda: lib.mxfp4_quantize_rows(x), "dequantize": lambda: (lib.mxfp4_dequantize_rows(*xq),),
        "linear": lambda: (lib.mxfp4_linear(x, *a, split_k=3),),
        "linear_backward": lambda: (lib.mxfp4_linear_backward(dh, *a, split_k=2),),
        "qmm_a4": lambda: (lib.qmm_mxfp4a4(*xq, *a, split_k=2),), "a4_linear": lambda: (lib.mxfp4a4_linear(x, *a),),
        "gate_up": lambda: (lib.mxfp4_gate_up_swiglu(x, a, b, split_k=2),),
        "gate_up_backward": lambda: lib.mxfp4_gate_up_swiglu_backward(x, a, b, dh, split_k=2),
    }


def _equal(a, b):
    import torch
    return len(a) == len(b) and all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("M", [1, 6, 40])
def test_calls_repeat_bit_for_bit_and_on_two_streams_at_once(lib, M):
    import torch
    calls = _calls(lib, M)
    first = {n: [t.clone() for t in f()] for n, f in calls.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = {n: [] for n in calls}
    for n, f in calls.items():
        announce(f"mxfp4 {n} M={M} on two streams at once")
        for s in streams:
            with torch.cuda.stream(s):
                got[n].append(f())
    torch.cuda.synchronize()
    for n in calls:
        for outputs in got[n]:
            assert _equal(first[n], outputs), n


@pytest.mark.parametrize("M", [1, 6, 40])
def test_calls_replay_in_two_graphs(lib, M):
    """Two captured graphs, replayed in turns with eager work between: each replay equals the eager result."""
    import torch
    calls = _calls(lib, M)
    eager = {n: [t.clone() for t in f()] for n, f in calls.items()}
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = {n: f() for n, f in calls.items()}
        graphs.append((g, out))
    for turn in range(3):
        for g, out in graphs:
            announce(f"mxfp4 graph replay M={M} turn {turn}")
            for ts in out.values():
                for t in ts:
                    t.zero_()
            g.replay()
            again = {n: f() for n, f in calls.items()}
            torch.cuda.synchronize()
            for n in calls:
                assert _equal(eager[n], out[n]) and _equal(eager[n], again[n]), (n, turn)


def test_stream_argument(lib):
    """A call given a stream runs there; what it allocates outlives the call's references."""
    import torch
    announce("mxfp4 stream argument")
    rng = np.random.default_rng(13)
    w, wv = weight(rng, 200, 1056)
    x = bf16_values(rng.standard_normal((50, 1056)))
    xt = bf16(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = lib.mxfp4_linear(xt, *w, split_k=4, stream=s)
    z = lib.mxfp4a4_linear(xt, *w, stream=s.cuda_stream)
    s.synchronize()
    check(y, O.mx_linear(x, wv))
    check(z, O.mx_linear(O.mx_decode(*O.mx_encode(x)), wv))


def test_workspaces(lib):
    """A given workspace serves; a short one drops a policy split and refuses a forced one."""
    import torch
    announce("mxfp4 workspaces")
    M, N, K = 40, 136, 2560
    rng = np.random.default_rng(14)
    w, wv = weight(rng, N, K)
    x = bf16_values(rng.standard_normal((M, K)))
    expected = O.mx_linear(x, wv)
    need = lib.mxfp4_plan(lib.MXFP4_LINEAR, M, N, K, 4)["workspace_bytes"]
    assert need == 4 * M * N * 4
    ws = torch.full((need // 4,), float("nan"), device="cuda:0")
    check(lib.mxfp4_linear(bf16(x), *w, split_k=4, workspace=ws), expected)
    short = torch.empty(4, device="cuda:0")
    check(lib.mxfp4_linear(bf16(x), *w, workspace=short), expected)
    with pytest.raises(ValueError, match="WORKSPACE"):
        lib.mxfp4_linear(bf16(x), *w, split_k=4, workspace=short)
    with pytest.raises(ValueError, match="WORKSPACE"):
        lib.mxfp4a4_linear(bf16(x), *w, workspace=short)
    few = bf16(x)[:3]                                      # decode rows need none
    check(lib.mxfp4a4_linear(few, *w, workspace=short), O.mx_linear(O.mx_decode(*O.mx_encode(x[:3])), wv))
    with pytest.raises(ValueError, match="ALIGN"):
        lib.mxfp4_linear(bf16(x), *w, split_k=4, workspace=torch.empty(need // 4 + 1, device="cuda:0")[1:])


def test_refused_tensors(lib):
    """Shapes, strides, types and overlaps, by the errors of the binding and of the library."""
    import torch
    rng = np.random.default_rng(15)
    (codes, scales), _ = weight(rng, 64, 96)
    x = bf16(rng.standard_normal((8, 96)))
    with pytest.raises(ValueError, match="shape"):
        lib.mxfp4_linear(x[:, :64].contiguous(), codes, scales)
    with pytest.raises(ValueError, match="contiguous"):
        lib.mxfp4_linear(bf16(rng.standard_normal((96, 8))).t(), codes, scales)
    with pytest.raises(TypeError):
        lib.mxfp4_linear(x.float(), codes, scales)
    with pytest.raises(ValueError, match="shape"):
        lib.mxfp4_linear(x, codes, scales[:, :2].contiguous())
    with pytest.raises(ValueError, match="GPU"):
        lib.mxfp4_linear(x, codes.cpu(), scales.cpu())
    with pytest.raises(ValueError, match="OVERLAP"):
        lib.mxfp4_linear(x, codes, scales, y=x.view(-1)[:8 * 64].view(8, 64))
    with pytest.raises(ValueError, match="ALIGN"):
        lib.mxfp4_linear(bf16(rng.standard_normal(8 * 96 + 1)).view(-1)[1:].view(8, 96), codes, scales)
    with pytest.raises(ValueError, match="WORKSPACE"):
        lib.mxfp4_linear_backward(bf16(rng.standard_normal((8, 60))), codes[:60], scales[:60],
                                  workspace=torch.empty(16, device="cuda:0"))
    with pytest.raises(ValueError):
        lib.mxfp4_linear(x[:0], codes, scales)
    with pytest.raises(ValueError, match="must be"):
        lib.mxfp4_gate_up_swiglu(x, (codes, scales), (codes[:32], scales[:32]))
    with pytest.raises(ValueError, match="negative"):
        lib.mxfp4_linear(x, codes, scales, split_k=-1)


def test_scales_at_odd_addresses_and_tiles(lib):
    """Scale rows may start anywhere: the tiles' word and 16-byte loads give way to bytes."""
    import torch
    announce("mxfp4 odd scale addresses")
    M, N, K = 40, 136, 1024
    rng = np.random.default_rng(16)
    (codes, scales), wv = weight(rng, N, K)
    (up_codes, up_scales), uv = weight(rng, N, K, 118, 124)

    def odd(s):
        return torch.cat([s.view(-1)[:1], s.view(-1)])[1:].view(s.shape)
    x = bf16_values(rng.standard_normal((M, K)))
    check(lib.mxfp4_linear(bf16(x), codes, odd(scales)), O.mx_linear(x, wv))
    xq = lib.mxfp4_quantize_rows(bf16(x))
    xv = O.mx_decode(*(t.cpu().numpy() for t in xq))
    check(lib.qmm_mxfp4a4(xq[0], odd(xq[1]), codes, scales), O.mx_linear(xv, wv))
    check(lib.qmm_mxfp4a4(*xq, codes, odd(scales)), O.mx_linear(xv, wv))
    check(lib.mxfp4_linear_backward(bf16(x[:, :N]), codes, odd(scales)), O.mx_linear_backward(x[:, :N], wv))
    g = (up_codes, up_scales)
    check(lib.mxfp4_gate_up_swiglu(bf16(x), g, (up_codes, odd(up_scales))), O.mx_gate_up(x, uv, uv))


def test_prepared_calls(lib):
    """Prepared calls equal the functions, launch after launch, on new contents of their tensors."""
    import torch
    announce("mxfp4 prepared calls")
    rng = np.random.default_rng(17)
    for M in (1, 12, 50):
        w, _ = weight(rng, 136, 1056)
        u, _ = weight(rng, 136, 1056, 118, 122)
        x = bf16(rng.standard_normal((M, 1056)))
        prepared = [lib.PreparedMxfp4Linear(x, *w, split_k=0), lib.PreparedMxfp4Linear(x, *w, split_k=3),
                    lib.PreparedMxfp4Linear(x, *w, four_bit_activations=True), lib.PreparedMxfp4GateUp(x, w, u)]
        for _ in range(2):
            x.copy_(bf16(rng.standard_normal((M, 1056))))
            expected = [lib.mxfp4_linear(x, *w), lib.mxfp4_linear(x, *w, split_k=3), lib.mxfp4a4_linear(x, *w),
                        lib.mxfp4_gate_up_swiglu(x, w, u)]
            for p, e in zip(prepared, expected):
                assert torch.equal(p(), e)
    with pytest.raises(ValueError, match="shape"):
        lib.PreparedMxfp4Linear(x[:, :512].contiguous(), *w)
    with pytest.raises(ValueError, match="WORKSPACE"):
        lib.PreparedMxfp4Linear(x, *w, split_k=3, workspace=torch.empty(4, device="cuda:0"))()
    room = torch.empty(1 << 20)
    with pytest.raises(ValueError, match="workspace"):
        lib.PreparedMxfp4Linear(x, *w, split_k=3, workspace=room)
    with pytest.raises(ValueError, match="workspace"):
        lib.PreparedMxfp4GateUp(x, w, u, split_k=2, workspace=room.cuda()[::2])


def test_timing_request_takes_the_product(lib):
    """w4a16_time_next_launch times the product's kernel, not the quantization before it."""
    import torch
    announce("mxfp4 kernel timestamps")
    rng = np.random.default_rng(18)
    w, _ = weight(rng, 600, 1024)
    x = bf16(rng.standard_normal((100, 1024)))
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record(), stop.record()
    lib.w4a16_time_next_launch(start, stop)
    y = lib.mxfp4a4_linear(x, *w)
    torch.cuda.synchronize()
    assert 0 < start.elapsed_time(stop) < 100
    assert torch.equal(y, lib.mxfp4a4_linear(x, *w))


# ---------------------------------------------------------------------------- offsets beyond 32 bits

def _sampled(rows):
    return sorted({0, 1, rows // 2, rows - 2, rows - 1})


def test_outputs_beyond_two_to_the_31(lib):
    """More than 2^31 output elements: rows and columns at both ends."""
    import torch
    M, N, K = 16400, 131100, 32
    announce(f"mxfp4_linear M={M} N={N}: {M * N} outputs")
    assert M * N > 2 ** 31
    g = torch.Generator(device="cuda:0").manual_seed(1)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda:0", generator=g)
    scales = torch.randint(118, 124, (N, K // 32), dtype=torch.uint8, device="cuda:0", generator=g)
    x = torch.randn(M, K, device="cuda:0", generator=g).to(torch.bfloat16)
    y = lib.mxfp4_linear(x, codes, scales)
    rows, cols = _sampled(M), _sampled(N)
    wv = O.mx_decode(codes[cols].cpu().numpy(), scales[cols].cpu().numpy())
    check(y[rows][:, cols], O.mx_linear(values(x[rows]), wv))


@pytest.mark.parametrize("M", [2, 40])
def test_weights_beyond_four_gib(lib, M):
    """More than 2^32 bytes of codes: the last weight rows, and the transposed product over all rows."""
    import torch
    N, K = 300000, 32768
    announce(f"mxfp4_linear M={M}: {N * K // 2} bytes of codes")
    assert N * K // 2 > 2 ** 32
    g = torch.Generator(device="cuda:0").manual_seed(2)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda:0", generator=g)
    scales = torch.randint(118, 124, (N, K // 32), dtype=torch.uint8, device="cuda:0", generator=g)
    x = torch.randn(M, K, device="cuda:0", generator=g).to(torch.bfloat16)
    cols = _sampled(N)
    wv = O.mx_decode(codes[cols].cpu().numpy(), scales[cols].cpu().numpy())
    check(lib.mxfp4_linear(x, codes, scales)[:, cols], O.mx_linear(values(x), wv))
    xq = lib.mxfp4_quantize_rows(x)
    check(lib.qmm_mxfp4a4(*xq, codes, scales)[:, cols], O.mx_linear(O.mx_decode(*(t.cpu().numpy() for t in xq)), wv))
    # gradients of zero but in the sampled weight rows
    dy = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda:0")
    dy[:, cols] = torch.randn(M, len(cols), device="cuda:0", generator=g).to(torch.bfloat16)
    check(lib.mxfp4_linear_backward(dy, codes, scales), O.mx_linear_backward(values(dy[:, cols]), wv))


def test_rows_beyond_two_to_the_31(lib):
    import torch
    R, K = 66000, 32768
    announce(f"mxfp4_quantize_rows {R * K} values")
    assert R * K > 2 ** 31
    g = torch.Generator(device="cuda:0").manual_seed(3)
    x = torch.randn(R, K, device="cuda:0", generator=g, dtype=torch.bfloat16)
    codes, scales = lib.mxfp4_quantize_rows(x)
    back = lib.mxfp4_dequantize_rows(codes, scales)
    for r in (0, R // 2, R - 1):
        ref = O.mx_encode(values(x[r:r + 1]))
        assert np.array_equal(codes[r:r + 1].cpu().numpy(), ref[0]) and np.array_equal(scales[r:r + 1].cpu().numpy(), ref[1])
        assert np.array_equal(values(back[r:r + 1]), O.mx_decode(*ref))
