"""MXFP4 without a GPU: the oracle's pins, the launch policy, and every refusal of the entry points
(arguments that fail validation before any HIP call)."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest

import oracle as O
import w4a16_group_quantized_qmv_amd as w4

CUS = 256
OPS = {"linear": w4.MXFP4_LINEAR, "linear_backward": w4.MXFP4_LINEAR_BACKWARD, "qmm_a4": w4.MXFP4_QMM_A4,
       "a4_linear": w4.MXFP4A4_LINEAR, "gate_up": w4.MXFP4_GATE_UP, "gate_up_backward": w4.MXFP4_GATE_UP_BACKWARD}


# ---------------------------------------------------------------------------- the oracle's pins

def test_values_follow_the_bit_fields():
    for code in range(16):
        sign, exponent, mantissa = code >> 3, (code >> 1) & 3, code & 1
        v = Fraction(mantissa, 2) if exponent == 0 else Fraction(2 + mantissa, 2) * 2 ** (exponent - 1)
        assert Fraction(float(O.MX_VALUES[code])) == (-v if sign else v)
    assert np.signbit(O.MX_VALUES[8]) and not np.signbit(O.MX_VALUES[0])


def test_packing_low_half_first_and_back():
    codes = np.arange(64, dtype=np.uint8).reshape(2, 32) % 16
    packed = O.mx_pack(codes)
    assert packed[0, 0] == 0x10 and packed[0, 1] == 0x32
    assert np.array_equal(O.mx_unpack(packed), codes)


def test_scales_cover_the_exponent_range():
    v = O.mx_scale_values(np.array([0, 1, 126, 127, 128, 254, 255]))
    assert [float(t) for t in v[:-1]] == [2.0 ** -127, 2.0 ** -126, 0.5, 1.0, 2.0, 2.0 ** 127] and np.isnan(v[-1])


def test_encode_is_a_round_trip_on_the_grid():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, (5, 96)).astype(np.uint8)
    codes[:, ::32] = 7                              # each block holds its largest magnitude
    scales = rng.integers(0, 253, (5, 3)).astype(np.uint8)
    packed, s = O.mx_encode(O.mx_decode(O.mx_pack(codes), scales))
    assert np.array_equal(s, scales) and np.array_equal(O.mx_unpack(packed), codes)


@pytest.mark.parametrize("top", [4.0, 5.0, 6.0, 7.9])
def test_encode_ties_go_to_even_mantissas_and_large_values_saturate(top):
    ties = {0.25: 0.0, 0.75: 1.0, 1.25: 1.0, 1.75: 2.0, 2.5: 2.0, 3.5: 4.0, 5.0: 4.0, 6.5: 6.0, 7.5: 6.0}
    row = np.zeros((1, 32))
    row[0, 0] = top
    for i, t in enumerate(t for t in ties if t <= top):
        row[0, 2 * i + 1], row[0, 2 * i + 2] = t, -t
    packed, s = O.mx_encode(row)
    assert s[0, 0] == 127
    got = O.mx_decode(packed, s)[0]
    for i, t in enumerate(t for t in ties if t <= top):
        assert got[2 * i + 1] == ties[t] and got[2 * i + 2] == -ties[t]


def test_encode_error_is_within_half_a_step():
    """Nearest: |x - q| <= max(|x| / 4, 2^e / 4), except above 6 where the block's top is cut by at most 2."""
    x = np.random.default_rng(2).standard_normal((16, 320))
    packed, s = O.mx_encode(x)
    unit = np.repeat(O.mx_scale_values(s), 32, axis=1)
    off = np.abs(O.mx_decode(packed, s) - x) / unit
    r = np.abs(x) / unit
    assert np.all(r < 8)
    step = np.where(r < 2, 0.5, np.where(r < 4, 1.0, 2.0))
    assert np.all(off <= np.where(r > 6, 2.0, step / 2) + 1e-12)


def test_encode_zero_small_and_invalid_blocks():
    x = np.zeros((1, 32 * 5))
    x[0, 32] = 2.0 ** -149                       # below the smallest scale's grid
    x[0, 64] = 2.0 ** -126
    x[0, 96] = np.inf
    x[0, 128 + 7] = np.nan
    packed, s = O.mx_encode(x)
    assert s.tolist() == [[0, 0, 0, 255, 255]]
    v = O.mx_decode(packed, s)[0]
    assert v[32] == 0 and v[64] == 2.0 ** -126 and np.isnan(v[96:]).all()


def test_linear_against_fractions():
    rng = np.random.default_rng(3)
    x, w = rng.integers(-8, 9, (3, 32)) / 4.0, rng.integers(-8, 9, (2, 32)) / 8.0
    y, bound = O.mx_linear(x, w)
    for m in range(3):
        for n in range(2):
            assert Fraction(float(y[m, n])) == sum(Fraction(float(a)) * Fraction(float(b)) for a, b in zip(x[m], w[n]))
    dx, _ = O.mx_linear_backward(y, w)
    assert np.array_equal(dx, sum(y[:, n:n + 1] * w[n][None, :] for n in range(2)))
    assert np.all(bound >= 2.0 ** -8 * np.abs(y))


def test_gate_up_gradients_against_differences():
    rng = np.random.default_rng(4)
    x, wg, wu, dh = (rng.standard_normal(s) for s in ((3, 32), (5, 32), (5, 32), (3, 5)))

    def loss(x, g_add=0.0, u_add=0.0):
        g, u = x @ wg.T + g_add, x @ wu.T + u_add
        return np.sum(dh * g / (1 + np.exp(-g)) * u)

    (dx, _), (dgate, _), (dup, _) = O.mx_gate_up_backward(x, wg, wu, dh)
    eps = 1e-6
    for got, at in ((dx, lambda d: loss(x + d)), (dgate, lambda d: loss(x, g_add=d)), (dup, lambda d: loss(x, u_add=d))):
        for i in np.ndindex(got.shape):
            d = np.zeros(got.shape)
            d[i] = eps
            assert abs((at(d) - at(-d)) / (2 * eps) - got[i]) < 1e-6 * (1 + abs(got[i]))


def test_gate_up_limits():
    """silu at the ends: 0 for large negative g, g for large positive; the gradients follow."""
    wg, wu, x = np.eye(1, 32), 2 * np.eye(1, 32), np.zeros((3, 32))
    x[:, 0] = [-800.0, 0.0, 800.0]
    h, _ = O.mx_gate_up(x, wg, wu)
    assert h[:, 0].tolist() == [0.0, 0.0, 800.0 * 1600.0]
    (_, _), (dgate, _), (dup, _) = O.mx_gate_up_backward(x, wg, wu, np.ones((3, 1)))
    assert dgate[:, 0].tolist() == [0.0, 0.0, 1600.0] and dup[:, 0].tolist() == [0.0, 0.0, 800.0]


def test_check_finds_planted_mistakes():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 64))
    w = O.mx_decode(*O.mx_encode(rng.standard_normal((3, 64))))
    y, bound = O.mx_linear(x, w)
    assert O.mx_check(y, y, bound) is None
    dropped = x[:, 32:] @ w[:, 32:].T                    # one block left out
    swapped = x @ w[[1, 0, 2]].T                         # two columns exchanged
    for wrong in (dropped, swapped, y * (1 + 2.0 ** -6), np.where(np.arange(3) == 1, np.nan, y)):
        assert O.mx_check(wrong, y, bound) is not None


@pytest.mark.parametrize("place", ["bound_nan", "bound_inf", "both_inf", "other_inf", "inf_expected"])
def test_check_with_values_and_bounds_that_are_not_finite(place):
    """One odd element neither hides the others nor passes where it is wrong itself."""
    value, bound = np.ones((4, 3)), np.full((4, 3), 0.1)
    got = value.copy()
    if place.startswith("bound"):
        bound[1, 2] = np.nan if place == "bound_nan" else np.inf
        assert O.mx_check(got, value, bound) is not None           # no bound for a finite value
    elif place == "both_inf":
        got[1, 2] = value[1, 2] = -np.inf
        bound[1, 2] = np.nan                                       # (a bound relative to an infinity)
        assert O.mx_check(got, value, bound) is None
    else:
        (got if place == "other_inf" else value)[1, 2] = np.inf
        assert O.mx_check(got, value, bound) is not None
        value[1, 2], got[1, 2] = np.inf, -np.inf
        assert O.mx_check(got, value, bound) is not None
    assert O.mx_check(np.full((4, 3), 5.0), value, bound) is not None
    wrong = got.copy()
    wrong[3, 0] = 1.2
    assert "(3, 0)" in O.mx_check(wrong, np.where(np.isinf(value), got, value), np.where(np.isfinite(bound), bound, 0.1))


# ---------------------------------------------------------------------------- the policy

@pytest.mark.parametrize("op", list(OPS))
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 9728, 2560), (33, 1000, 416), (509, 2560, 9728), (4096, 9728, 2560),
                                   (5, 151936, 2560), (16, 151, 9728), (17, 4096, 2560), (130, 1000, 416)])
def test_plan_covers_the_output(op, M, N, K):
    p = w4.mxfp4_plan(OPS[op], M, N, K, 0, CUS)
    columns = K if "backward" in op else N
    assert p["path"] in (w4.PATH_MXFP4, w4.PATH_MXFP4_QMV) and p["num_cus"] == CUS
    assert p["grid_y"] * p["tile_m"] >= M > (p["grid_y"] - 1) * p["tile_m"]
    if p["path"] == w4.PATH_MXFP4_QMV and p["variant"] == 0:      # wide: workgroups take blocks in turn
        assert p["grid_x"] <= -(-columns // (p["tile_n"] * p["block_threads"] // 64)) and N > 16 * (3 * CUS - 1)
    else:
        assert p["grid_x"] * p["tile_n"] >= columns > (p["grid_x"] - 1) * p["tile_n"]
    assert p["block_threads"] % 64 == 0 and p["block_threads"] <= 1024
    partials = p["split_k"] * M * columns * 4 * (2 if op == "gate_up" else 1) if p["split_k"] > 1 else 0
    if op == "a4_linear" and M > 16:
        assert p["workspace_bytes"] >= M * K // 2 + M * K // 32 + partials
    else:
        # gradient rows that are no whole 16 bytes are copied
        pad = (2 if op == "gate_up_backward" else 1) * (-(-M * (-(-N // 8) * 8) * 2 // 256) * 256)
        assert p["workspace_bytes"] == partials + (pad if "backward" in op and N % 8 else 0)


@pytest.mark.parametrize("op", list(OPS))
def test_plan_split_is_clamped_to_the_steps(op):
    p = w4.mxfp4_plan(OPS[op], 200, 64, 64, 50, CUS)
    assert 1 <= p["split_k"] <= 2
    assert w4.mxfp4_plan(OPS[op], 200, 64, 64, 1, CUS)["split_k"] == 1


@pytest.mark.parametrize("M,N,K", [(58, 42636, 1216), (62, 33159, 1664), (24, 109405, 1120), (39, 71025, 1088)])
def test_code_tiles_that_fill_a_compute_unit_alone_are_counted_so(M, N, K):
    """64 x 128 tiles of codes hold 104 KB of LDS: with more of them than compute units the rest is another
    round, and the tiles of which two fit (128 x 128) are chosen."""
    tiles = -(-N // 128)
    assert tiles > CUS and w4.mxfp4_plan(w4.MXFP4_QMM_A4, M, N, K, 0, CUS)["variant"] == 0
    # one round of them: the smaller tile
    assert w4.mxfp4_plan(w4.MXFP4_QMM_A4, M, 9728, 2560, 0, CUS)["variant"] == 2


@pytest.mark.parametrize("args,error", [
    ((0, 0, 64, 64), ValueError), ((0, 8, 0, 64), ValueError), ((0, 8, 64, 0), ValueError),
    ((0, 8, 64, 48), ValueError), ((0, 8, 64, (1 << 20) + 32), ValueError), ((0, (1 << 30) + 1, 64, 64), ValueError),
    ((0, 8, (1 << 30) + 1, 64), ValueError), ((0, 8, 64, 64, -1), ValueError), ((6, 8, 64, 64), NotImplementedError),
    ((-1, 8, 64, 64), NotImplementedError),
    ((1, 8, (1 << 20) + 8, 64), ValueError), ((0, 1 << 30, 1 << 30, 32), ValueError)])
def test_plan_refusals(args, error):
    op, M, N, K, *split = args
    with pytest.raises(error):
        w4.mxfp4_plan(op, M, N, K, *(split or [0]), num_cus=CUS)


# ---------------------------------------------------------------------------- refusals of the calls

SHAPE, NULL, ALIGN, WORKSPACE, UNSUPPORTED, OVERLAP = 2, 1, 4, 5, 6, 9
BASE = 1 << 40                  # addresses that are never touched: every call below is refused first


def _buffers(M, N, K):
    """Distinct fake device addresses, 1 MiB and more apart."""
    names = ("x", "codes", "scales", "y", "codes2", "scales2", "dh", "dx", "dgate", "dup", "ws")
    return {n: BASE + (i << 32) for i, n in enumerate(names)}


CALLS = {
    "mxfp4_quantize_rows": lambda L, b, M, N, K: L.mxfp4_quantize_rows(b["x"], 0, b["codes"], b["scales"], M, K, None),
    "mxfp4_dequantize_rows": lambda L, b, M, N, K: L.mxfp4_dequantize_rows(b["codes"], b["scales"], b["y"], M, K, None),
    "mxfp4_linear": lambda L, b, M, N, K: L.mxfp4_linear(b["x"], b["codes"], b["scales"], b["y"], M, N, K, 0, b["ws"], 0, None),
    "mxfp4_linear_backward": lambda L, b, M, N, K: L.mxfp4_linear_backward(b["x"], b["codes"], b["scales"], b["y"], M, N, K, 0, b["ws"], 0, None),
    "qmm_mxfp4a4": lambda L, b, M, N, K: L.qmm_mxfp4a4(b["codes2"], b["scales2"], b["codes"], b["scales"], b["y"], M, N, K, 0, b["ws"], 0, None),
    "mxfp4a4_linear": lambda L, b, M, N, K: L.mxfp4a4_linear(b["x"], b["codes"], b["scales"], b["y"], M, N, K, 0, b["ws"], 1 << 20, None),
    "mxfp4_gate_up_swiglu": lambda L, b, M, N, K: L.mxfp4_gate_up_swiglu(b["x"], b["codes"], b["scales"], b["codes2"], b["scales2"], b["y"], M, N, K, 0, b["ws"], 0, None),
    "mxfp4_gate_up_swiglu_backward": lambda L, b, M, N, K: L.mxfp4_gate_up_swiglu_backward(
        b["x"], b["codes"], b["scales"], b["codes2"], b["scales2"], b["dh"], b["dx"], b["dgate"], b["dup"], M, N, K, 0, b["ws"], 0, None),
}
USED = {
    "mxfp4_quantize_rows": ("x", "codes", "scales"),
    "mxfp4_dequantize_rows": ("codes", "scales", "y"),
    "mxfp4_linear": ("x", "codes", "scales", "y"),
    "mxfp4_linear_backward": ("x", "codes", "scales", "y"),
    "qmm_mxfp4a4": ("codes", "scales", "codes2", "scales2", "y"),
    "mxfp4a4_linear": ("x", "codes", "scales", "y"),
    "mxfp4_gate_up_swiglu": ("x", "codes", "scales", "codes2", "scales2", "y"),
    "mxfp4_gate_up_swiglu_backward": ("x", "codes", "scales", "codes2", "scales2", "dh", "dx", "dgate", "dup"),
}
ALIGN16 = {"mxfp4_quantize_rows": ("x", "codes"), "mxfp4_dequantize_rows": ("codes", "y"),
           "mxfp4_linear": ("x", "codes"), "mxfp4_linear_backward": ("x", "codes"), "qmm_mxfp4a4": ("codes", "codes2"),
           "mxfp4a4_linear": ("x", "codes", "ws"), "mxfp4_gate_up_swiglu": ("x", "codes", "codes2"),
           "mxfp4_gate_up_swiglu_backward": ("x", "codes", "codes2", "dgate", "dup")}
OUTPUTS = {"mxfp4_quantize_rows": ("codes", "scales"), "mxfp4_gate_up_swiglu_backward": ("dx", "dgate", "dup")}


@pytest.mark.parametrize("name", list(CALLS))
def test_call_refusals(name):
    L, (M, N, K) = w4.load(), (40, 64, 96)
    call, good = CALLS[name], _buffers(M, N, K)
    for bad in ((0, N, K), (M, N, 0), (M, N, 80), (M, N, (1 << 20) + 32), ((1 << 30) + 1, N, K)):
        assert call(L, good, *bad) == SHAPE, bad
    if "quantize" not in name:
        assert call(L, good, M, 0, K) == SHAPE
    if "backward" in name:
        assert call(L, good, M, (1 << 20) + 1, K) == SHAPE
    for used in USED[name]:
        assert call(L, {**good, used: None}, M, N, K) == NULL, used
    for b in ALIGN16[name]:
        assert call(L, {**good, b: good[b] + 8}, M, N, K) == ALIGN, b
    outputs = OUTPUTS.get(name, ("y",))
    for o in outputs:
        if o not in ALIGN16[name] and o != "scales":
            assert call(L, {**good, o: good[o] + 1}, M, N, K) == ALIGN, o
        for other in USED[name]:
            if other != o and not (other == "scales" and o in ALIGN16[name]):
                assert call(L, {**good, o: good[other]}, M, N, K) == OVERLAP, (o, other)


def test_quantize_type_and_workspace_refusals():
    L, b = w4.load(), _buffers(8, 64, 96)
    assert L.mxfp4_quantize_rows(b["x"], 2, b["codes"], b["scales"], 8, 96, None) == UNSUPPORTED
    args = (b["x"], b["codes"], b["scales"], b["y"], 20, 64, 96, 0)
    assert L.mxfp4a4_linear(*args, None, 0, None) == WORKSPACE
    assert L.mxfp4a4_linear(*args, b["ws"], 20 * 48, None) == WORKSPACE
    assert L.mxfp4_linear(*args[:-1], -1, None, 0, None) == SHAPE


def test_python_refusals_without_a_gpu():
    import torch
    x, codes, scales = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        w4.mxfp4_linear(x, codes, scales)
    with pytest.raises(ValueError, match="GPU"):
        w4.mxfp4_quantize_rows(x)
    with pytest.raises(TypeError):
        w4.mxfp4_quantize_rows(x.to(torch.float16))
    with pytest.raises(ValueError, match="2-D"):
        w4.mxfp4_linear(x[0], codes, scales)
    with pytest.raises(ValueError, match="multiple"):
        w4.mxfp4_dequantize_rows(codes[:, :24].contiguous(), scales)
    with pytest.raises(TypeError):
        w4.mxfp4_linear(None, codes, scales)


def test_every_mxfp4_symbol_has_a_signature():
    L = w4.load()
    for name in w4.declared_symbols():
        if "mxfp4" in name:
            assert getattr(L, name).restype is ctypes.c_int and getattr(L, name).argtypes, name
            assert name in w4.__all__ and callable(getattr(w4, name))
