"""The int8 products' and the experts' operators without a GPU: pins of the oracle, plans, and every refusal."""

import ctypes
import gc
from fractions import Fraction

import numpy as np
import pytest

import oracle as O
import w4a16_group_quantized_qmv_amd as w4
from w4a16_group_quantized_qmv_amd import mxfp4, w8a8

from test_streams_cpu import CURRENT, SIDE, Model, Recorder

CUS = 256


# ---------------------------------------------------------------------------- the oracle

def nearest_even(q: Fraction) -> int:
    low = q.numerator // q.denominator
    rest = q - low
    return low + (rest > Fraction(1, 2) or (rest == Fraction(1, 2) and low % 2 == 1))


def fp32(q: Fraction) -> Fraction:
    """q rounded to 24 bits, ties to even (normal numbers)."""
    if q == 0:
        return q
    e = 0
    while abs(q) * Fraction(2) ** -e >= 2 ** 24:
        e += 1
    while abs(q) * Fraction(2) ** -e < 2 ** 23:
        e -= 1
    return nearest_even(abs(q) / Fraction(2) ** e) * Fraction(2) ** e * (1 if q > 0 else -1)


@pytest.mark.parametrize("seed", range(4))
def test_quantizer_in_fractions(seed):
    x = (np.random.default_rng(seed).standard_normal((3, 16)) * 10.0 ** (seed - 2)).astype(np.float32)
    codes, scales = O.w8_quantize(x)
    for row, c, s in zip(x, codes, scales):
        exact = [Fraction(float(v)) for v in row]
        a = max(abs(v) for v in exact)
        assert Fraction(float(s)) == fp32(a / 127)
        inv = fp32(Fraction(127) / a)
        assert [int(v) for v in c] == [max(-127, min(127, nearest_even(fp32(v * inv)))) for v in exact]


def test_quantizer_special_rows():
    x = np.zeros((6, 16), np.float32)
    x[1, 3] = np.inf
    x[2, 0] = np.nan
    x[3, 5] = 2.0 ** -111
    x[4, 5] = 2.0 ** -110
    x[5] = np.arange(16) - 8
    x[5, 0] = -127
    codes, scales = O.w8_quantize(x)
    assert scales[0] == 0 and np.isnan(scales[1]) and np.isnan(scales[2]) and scales[3] == 0 and not codes[:4].any()
    assert codes[4, 5] == 127 and scales[4] == np.float32(2.0 ** -110) / np.float32(127)
    assert scales[5] == 1 and np.array_equal(codes[5], x[5].astype(np.int8))


def _pair(rng, n, k):
    return rng.integers(-127, 128, (n, k)).astype(np.int8), (rng.random(n) * 0.02 + 1e-3).astype(np.float32)


def test_products_in_fractions():
    rng = np.random.default_rng(5)
    (xq, xs), (wq, ws) = _pair(rng, 3, 32), _pair(rng, 4, 32)
    value, bound = O.w8_linear(xq, xs, wq, ws)
    for m in range(3):
        for n in range(4):
            exact = sum(Fraction(int(a) * int(b)) for a, b in zip(xq[m], wq[n])) * Fraction(float(xs[m])) * Fraction(float(ws[n]))
            assert abs(float(exact) - value[m, n]) <= 1e-14 * abs(value[m, n]) and bound[m, n] >= abs(value[m, n]) * 2 ** -8


def gated(xv, gate, up):
    g, u = xv @ (gate[0] * gate[1][:, None].astype(float)).T, xv @ (up[0] * up[1][:, None].astype(float)).T
    return g / (1 + np.exp(-g)) * u


def test_gradients_against_differences():
    """The backward references are the derivatives of what the forward ones compute from unrounded activations."""
    rng = np.random.default_rng(6)
    gate, up = _pair(rng, 5, 16), _pair(rng, 5, 16)
    xq, xs = _pair(rng, 2, 16)
    xv, dh = xq * xs[:, None].astype(float), rng.standard_normal((2, 5))
    h, _ = O.w8_gate_up(xq, xs, gate, up)
    assert np.allclose(h, gated(xv, gate, up), rtol=1e-12)
    (dx, _), (dgate, _), (dup, _) = O.w8_gate_up_backward(xq, xs, gate, up, dh)
    step = 1e-6
    for m in range(2):
        for k in range(16):
            d = np.zeros_like(xv)
            d[m, k] = step
            diff = ((gated(xv + d, gate, up) - gated(xv - d, gate, up)) * dh).sum() / (2 * step)
            assert abs(diff - dx[m, k]) < 1e-7 * max(1, abs(dx[m, k]))
    assert np.allclose(dx, dgate @ (gate[0] * gate[1][:, None].astype(float)) + dup @ (up[0] * up[1][:, None].astype(float)))
    assert np.allclose(O.w8_linear_backward(dh, *gate)[0], dh @ (gate[0] * gate[1][:, None].astype(float)))


@pytest.mark.parametrize("renormalize", [True, False])
def test_router_gradient_against_differences(renormalize):
    rng = np.random.default_rng(7)
    logits, dw = rng.standard_normal((3, 9)), rng.standard_normal((3, 4))
    logits[1, 2] = -np.inf
    (_, _), experts, *_ = O.route_reference(logits, 4, renormalize)
    d, _ = O.route_backward_reference(logits, experts, dw, renormalize)
    for t in range(3):
        for e in range(9):
            if logits[t, e] == -np.inf:
                assert d[t, e] == 0
                continue
            up, down = logits.copy(), logits.copy()
            up[t, e] += 1e-6
            down[t, e] -= 1e-6
            diff = sum(((O.route_reference(v, 4, renormalize)[0][0]) * dw).sum() * s for v, s in ((up, 1), (down, -1))) / 2e-6
            assert abs(diff - d[t, e]) < 1e-8


def test_router_by_hand():
    logits = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4, [0.0, -0.0, 5.0, 0.0], [-np.inf, 2.0, -np.inf, -np.inf]])
    (w, _), experts, positions, tokens, offsets = O.route_reference(logits, 2)
    assert experts.tolist() == [[1, 2], [-1, -1], [2, 0], [1, -1]]
    assert offsets.tolist() == [0, 1, 3, 5, 5] and tokens.tolist() == [2, 0, 3, 0, 2, -1, -1, -1]
    assert positions.tolist() == [[1, 3], [-1, -1], [4, 0], [2, -1]]
    assert np.allclose(w, [[0.5, 0.5], [0, 0], [1 / (1 + np.exp(-5)), 1 / (1 + np.exp(5))], [1, 0]])


def test_combine_and_its_gradients_against_differences():
    rng = np.random.default_rng(8)
    y, w, dout = rng.standard_normal((5, 3)), rng.standard_normal((3, 2)), rng.standard_normal((3, 3))
    positions = np.array([[4, 0], [-1, 2], [1, 7]])
    out, _ = O.combine_reference(y, positions, w)
    assert np.allclose(out, [w[0, 0] * y[4] + w[0, 1] * y[0], w[1, 1] * y[2], w[2, 0] * y[1]])
    (dy, _), (dw, _) = O.combine_backward_reference(dout, y, positions, w)
    f = lambda y, w: (O.combine_reference(y, positions, w)[0] * dout).sum()
    for a, d, args in ((y, dy, lambda v: (v, w)), (w, dw, lambda v: (y, v))):
        for i in np.ndindex(a.shape):
            if np.isnan(d[i]):
                assert i[0] == 3
                continue
            p, m = a.copy(), a.copy()
            p[i] += 1e-6
            m[i] -= 1e-6
            assert abs((f(*args(p)) - f(*args(m))) / 2e-6 - d[i]) < 1e-8


PLANTED = {
    "scale of the next column": lambda xq, xs, wq, ws: O.w8_product(xq, xs, wq, np.roll(ws, 1))[0],
    "scale of the next row": lambda xq, xs, wq, ws: O.w8_product(xq, np.roll(xs, 1), wq, ws)[0],
    "last chunk left out": lambda xq, xs, wq, ws: O.w8_product(xq[:, :-16], xs, wq[:, :-16], ws)[0],
    "codes unsigned": lambda xq, xs, wq, ws: O.w8_product(xq, xs, wq.view(np.uint8).astype(np.int16), ws)[0],
    "two rows swapped": lambda xq, xs, wq, ws: O.w8_product(xq, xs, wq, ws)[0][[1, 0, 2]],
}


@pytest.mark.parametrize("name", list(PLANTED))
def test_the_bounds_find_planted_mistakes(name):
    rng = np.random.default_rng(9)
    (xq, xs), (wq, ws) = _pair(rng, 3, 64), _pair(rng, 4, 64)
    good = O.w8_linear(xq, xs, wq, ws)
    assert O.within(good[0] * (1 + 2.0 ** -9), good) is None
    assert O.within(PLANTED[name](xq, xs, wq, ws), good) is not None


# ---------------------------------------------------------------------------- the policy

DENSE = {"linear": w4.W8A8_LINEAR, "linear_backward": w4.W8A8_LINEAR_BACKWARD, "qmm": w4.W8A8_QMM}
EXPERTS = {"experts_linear": w4.W8A8_EXPERTS_LINEAR, "experts_linear_backward": w4.W8A8_EXPERTS_LINEAR_BACKWARD,
           "gate_up": w4.W8A8_EXPERTS_GATE_UP, "gate_up_backward": w4.W8A8_EXPERTS_GATE_UP_BACKWARD}


def r256(v):
    return -(-v // 256) * 256


@pytest.mark.parametrize("op", list(DENSE))
@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 9728, 2560), (4, 2560, 9728), (5, 151, 9728), (16, 100, 131056), (17, 4096, 2560),
                                   (33, 1000, 416), (509, 2560, 9728), (4096, 9728, 2560), (130, 1001, 400)])
def test_plan_covers_the_output(op, M, N, K):
    p = w4.w8a8_plan(DENSE[op], M, N, K, 0, CUS)
    columns = K if "backward" in op else N
    assert p["path"] == (w4.PATH_W8A8_QMV if M <= 16 and "backward" not in op else w4.PATH_W8A8) and p["num_cus"] == CUS
    assert p["grid_y"] * p["tile_m"] >= M > (p["grid_y"] - 1) * p["tile_m"]
    assert p["grid_x"] * p["tile_n"] >= columns > (p["grid_x"] - 1) * p["tile_n"]
    assert p["block_threads"] % 64 == 0 and p["block_threads"] <= 1024
    partials = p["split_k"] * M * columns * 4 if p["split_k"] > 1 else 0
    fixed = 0
    if op == "linear" and not (p["path"] == w4.PATH_W8A8_QMV and p["variant"] == 1):
        fixed = r256(M * K) + r256(4 * M)
    if op == "linear_backward" and N % 8:
        fixed = r256(M * (-(-N // 8) * 8) * 2)
    assert p["workspace_bytes"] == fixed + partials


@pytest.mark.parametrize("op", list(EXPERTS))
@pytest.mark.parametrize("E,T,R,N,K", [(1, 1, 1, 8, 16), (64, 4, 32, 1216, 2560), (64, 509, 2036, 1216, 2560), (1024, 3, 3, 16, 16),
                                       (64, 4096, 32768, 1216, 2560), (8, 100, 200, 1001, 400), (4, 40000, 40000, 64, 64)])
def test_experts_plan_has_room_for_every_split_of_the_rows(op, E, T, R, N, K):
    p = w4.w8a8_plan(EXPERTS[op], T, N, K, 0, CUS, E, R)
    columns = K if "backward" in op else N
    assert p["grid_x"] * p["tile_n"] >= columns and p["split_k"] == 1
    # the worst cases of R rows in E pieces: one row in each but one, all in one
    bm = p["tile_m"]
    used = min(E, R)
    assert p["grid_y"] >= used - 1 + -(-(R - used + 1) // bm) and p["grid_y"] >= -(-R // bm)
    fixed = r256(T * K) + r256(4 * T) if op != "experts_linear_backward" and not (
        p["path"] == w4.PATH_W8A8_QMV and p["variant"] == 1) else 0
    if op == "gate_up_backward":
        fixed += 2 * r256(R * (-(-N // 8) * 8) * 2)
    elif op == "experts_linear_backward" and N % 8:
        fixed += r256(R * (-(-N // 8) * 8) * 2)
    assert p["workspace_bytes"] == fixed


@pytest.mark.parametrize("op", list(DENSE))
def test_plan_split_is_clamped_to_the_steps(op):
    p = w4.w8a8_plan(DENSE[op], 200, 64, 128, 50, CUS)
    assert 1 <= p["split_k"] <= 2
    assert w4.w8a8_plan(DENSE[op], 200, 64, 128, 1, CUS)["split_k"] == 1


@pytest.mark.parametrize("args,error", [
    ((0, 0, 64, 64), ValueError), ((0, 8, 0, 64), ValueError), ((0, 8, 64, 0), ValueError), ((0, 8, 64, 24), ValueError),
    ((0, 8, 64, 131072), ValueError), ((0, (1 << 30) + 1, 64, 64), ValueError), ((0, 1 << 24, 64, 64), ValueError),
    ((0, 8, (1 << 30) + 1, 64), ValueError), ((0, 8, 64, 64, -1), ValueError), ((7, 8, 64, 64), NotImplementedError),
    ((-1, 8, 64, 64), NotImplementedError), ((1, 8, (1 << 20) + 8, 64), ValueError), ((0, (1 << 24) - 1, 1 << 30, 32), ValueError),
    ((0, 8, 64, 64, 0, CUS, 2), ValueError), ((0, 8, 64, 64, 0, CUS, 1, 9), ValueError), ((3, 8, 64, 64, 2, CUS, 2), NotImplementedError),
    ((3, 8, 64, 64, 0, CUS, 0), ValueError), ((3, 8, 64, 64, 0, CUS, 1025), ValueError), ((3, 8, 64, 64, 0, CUS, 2, 0), ValueError)])
def test_plan_refusals(args, error):
    op, M, N, K, *rest = args
    rest = rest + [0, CUS][len(rest):] if len(rest) < 2 else rest
    with pytest.raises(error):
        w4.w8a8_plan(op, M, N, K, *rest)


# ---------------------------------------------------------------------------- refusals of the calls

SHAPE, NULL, ALIGN, WORKSPACE, UNSUPPORTED, OVERLAP = 2, 1, 4, 5, 6, 9
BASE = 1 << 40                  # addresses that are never touched: every call below is refused first
NAMES = ("x", "codes", "scales", "y", "codes2", "scales2", "dh", "dx", "dgate", "dup", "offsets", "tokens", "weights", "experts",
         "positions", "logits", "dw", "ws")
GOOD = {n: BASE + (i << 32) for i, n in enumerate(NAMES)}
M_, N_, K_, E_, TOP = 40, 64, 96, 4, 2


def call(name, b, M=M_, N=N_, K=K_, E=E_, top=TOP, kind=0, split=0, ws=1 << 30):
    L = w4.load()
    w1, w2 = (b["codes"], b["scales"]), (b["codes2"], b["scales2"])
    R = M * top
    args = {
        "w8a8_quantize_rows": (b["x"], kind, b["codes"], b["scales"], M, K),
        "qmm_w8a8": (*w2, *w1, b["y"], M, N, K, split, b["ws"], ws),
        "w8a8_linear": (b["x"], *w1, b["y"], M, N, K, split, b["ws"], ws),
        "w8a8_linear_backward": (b["x"], *w1, b["y"], M, N, K, split, b["ws"], ws),
        "w8a8_experts_linear": (b["x"], *w1, b["offsets"], b["tokens"], b["y"], E, M, R, N, K, b["ws"], ws),
        "w8a8_experts_linear_backward": (b["x"], *w1, b["offsets"], b["y"], E, R, N, K, b["ws"], ws),
        "w8a8_experts_gate_up_swiglu": (b["x"], *w1, *w2, b["offsets"], b["tokens"], b["y"], E, M, R, N, K, b["ws"], ws),
        "w8a8_experts_gate_up_swiglu_backward": (b["x"], *w1, *w2, b["dh"], b["offsets"], b["tokens"], b["dx"], b["dgate"],
                                                 b["dup"], E, M, R, N, K, b["ws"], ws),
        "experts_route": (b["logits"], kind, b["weights"], b["experts"], b["positions"], b["tokens"], b["offsets"], M, E, top, 1,
                          b["ws"], ws),
        "experts_route_backward": (b["logits"], kind, b["experts"], b["dw"], b["y"], M, E, top, 1),
        "experts_combine": (b["x"], b["positions"], b["weights"], b["y"], M, top, R, N),
        "experts_combine_backward": (b["dh"], b["x"], b["positions"], b["weights"], b["y"], b["dw"], M, top, R, N),
    }[name]
    return getattr(L, name)(*args, None)


# inputs that must be there, and outputs, by call
USED = {
    "w8a8_quantize_rows": (("x",), ("codes", "scales")),
    "qmm_w8a8": (("codes", "scales", "codes2", "scales2"), ("y",)),
    "w8a8_linear": (("x", "codes", "scales"), ("y",)),
    "w8a8_linear_backward": (("x", "codes", "scales"), ("y",)),
    "w8a8_experts_linear": (("x", "codes", "scales", "offsets"), ("y",)),
    "w8a8_experts_linear_backward": (("x", "codes", "scales", "offsets"), ("y",)),
    "w8a8_experts_gate_up_swiglu": (("x", "codes", "scales", "codes2", "scales2", "offsets"), ("y",)),
    "w8a8_experts_gate_up_swiglu_backward": (("x", "codes", "scales", "codes2", "scales2", "dh", "offsets"), ("dx", "dgate", "dup")),
    "experts_route": (("logits",), ("weights", "experts", "positions", "tokens", "offsets")),
    "experts_route_backward": (("logits", "experts", "dw"), ("y",)),
    "experts_combine": (("x", "positions"), ("y",)),
    "experts_combine_backward": (("dh", "x", "positions", "weights"), ("y", "dw")),
}


@pytest.mark.parametrize("name", list(USED))
def test_call_refusals(name):
    inputs, outputs = USED[name]
    product = "w8a8" in name
    for bad in (dict(M=0), dict(M=-1), dict(M=(1 << 30) + 1)):
        assert call(name, GOOD, **bad) == SHAPE, bad
    if product:
        for bad in (dict(K=0), dict(K=8), dict(K=100), dict(K=131072)):
            assert call(name, GOOD, **bad) == SHAPE, bad
    if name != "w8a8_quantize_rows" and "route" not in name:
        assert call(name, GOOD, N=0) == SHAPE and call(name, GOOD, N=(1 << 30) + 1) == SHAPE
    if product and "backward" in name:
        assert call(name, GOOD, N=(1 << 20) + 1) == SHAPE
    if "experts" in name and "combine" not in name:
        assert call(name, GOOD, E=0) == SHAPE and call(name, GOOD, E=1025) == SHAPE
    if "route" in name or "combine" in name:
        assert call(name, GOOD, top=0) == SHAPE and call(name, GOOD, top=65, E=1024) == SHAPE
    if "route" in name:
        assert call(name, GOOD, top=5) == SHAPE and call(name, GOOD, kind=2) == UNSUPPORTED
    for used in inputs + outputs:
        assert call(name, {**GOOD, used: None}) == NULL, used
        assert call(name, {**GOOD, used: GOOD[used] + 1}) in ((0, 7) if used.startswith("codes") and not product else (ALIGN,)), used
    for b in inputs + outputs:
        if b.startswith("codes") or (b == "x" and product):
            assert call(name, {**GOOD, b: GOOD[b] + 8}) == ALIGN, b
    for o in outputs:
        for other in inputs + outputs:
            # (what a quantizer writes: its outputs' alignment is checked first where it differs)
            if other != o:
                assert call(name, {**GOOD, o: GOOD[other]}) == OVERLAP, (o, other)
    if "tokens" not in inputs + outputs and name in ("w8a8_experts_linear", "w8a8_experts_gate_up_swiglu",
                                                     "w8a8_experts_gate_up_swiglu_backward"):
        assert call(name, {**GOOD, "tokens": None}) == SHAPE          # T rows of x for R rows of y
        assert call(name, {**GOOD, "tokens": GOOD["tokens"] + 2}) == ALIGN
        assert call(name, {**GOOD, outputs[0]: GOOD["tokens"]}) == OVERLAP
        assert call(name, GOOD, M=1 << 23, K=1024) == SHAPE           # offsets of gathered rows pass 31 bits
    if name == "experts_combine":
        assert call(name, {**GOOD, "weights": GOOD["weights"] + 2}) == ALIGN
        assert call(name, {**GOOD, "y": GOOD["weights"]}) == OVERLAP


def test_type_split_and_workspace_refusals():
    assert call("w8a8_quantize_rows", GOOD, kind=2) == UNSUPPORTED
    for name in ("qmm_w8a8", "w8a8_linear", "w8a8_linear_backward"):
        assert call(name, GOOD, split=-1) == SHAPE
    assert call("experts_route", GOOD, M=65, ws=4 * 3 * E_ - 1) == WORKSPACE
    assert call("experts_route", {**GOOD, "ws": None}, M=65) == WORKSPACE
    assert call("experts_route", {**GOOD, "ws": GOOD["ws"] + 4}, M=65) == ALIGN
    assert w4.experts_route_workspace_bytes(64, E_) == 0 and w4.experts_route_workspace_bytes(65, E_) == 4 * 3 * E_
    assert w4.experts_route_workspace_bytes(0, E_) == 0 and w4.experts_route_workspace_bytes(65, 1025) == 0


def test_every_symbol_has_a_signature():
    L = w4.load()
    names = [n for n in w4.declared_symbols() if "w8a8" in n or n.startswith("experts")]
    assert len(names) == 14
    for name in names:
        assert getattr(L, name).restype in (ctypes.c_int, ctypes.c_uint64) and getattr(L, name).argtypes, name
        assert name in w4.__all__ and callable(getattr(w4, name))


def test_python_refusals_without_a_gpu():
    import torch
    x, codes, scales = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    stacked, offsets = (codes.reshape(2, 4, 64), scales.reshape(2, 4)), torch.zeros(3, dtype=torch.int32)
    for f in (lambda: w4.w8a8_linear(x, codes, scales), lambda: w4.w8a8_quantize_rows(x), lambda: w4.qmm_w8a8(codes, scales, codes, scales),
              lambda: w4.w8a8_experts_linear(x, *stacked, offsets), lambda: w4.experts_route(torch.zeros(4, 8), 2),
              lambda: w4.w8a8_experts_gate_up_swiglu(x, stacked, stacked, offsets),
              lambda: w4.experts_combine(x, torch.zeros(2, 2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(TypeError):
        w4.w8a8_quantize_rows(x.to(torch.float16))
    with pytest.raises(TypeError):
        w4.experts_route(x.to(torch.float64), 2)
    with pytest.raises(ValueError, match="multiple"):
        w4.w8a8_quantize_rows(x[:, :24].contiguous())
    with pytest.raises(ValueError, match="2-D"):
        w4.w8a8_linear(x[0], codes, scales)
    with pytest.raises(TypeError):
        w4.w8a8_linear(None, codes, scales)


# ---------------------------------------------------------------------------- memory of calls on streams

class Library(Recorder):
    def __getattr__(self, name):
        if name == "w8a8_plan":
            real = self.lib.w8a8_plan
            return lambda op, E, T, R, N, K, split, cus, out: real(op, E, T, R, N, K, split, cus or CUS, out)
        if name == "experts_route_workspace_bytes":
            return self.lib.experts_route_workspace_bytes
        return super().__getattr__(name)


@pytest.fixture
def model(monkeypatch):
    lib = w4.load()
    torch, recorder = Model(), Library(lib)
    for module in (w4, mxfp4, w8a8):
        monkeypatch.setattr(module, "_torch", lambda: torch)
    monkeypatch.setattr(w4, "_LIB", recorder)
    monkeypatch.setattr(w8a8, "load", lambda: recorder)
    for name in ("_T", "_BF16", "_FP32", "_U8", "_empty", "_raw_stream", "_current"):
        monkeypatch.setattr(mxfp4, name, None)
    for name in ("_BF16", "_FP32", "_I8", "_I32"):
        monkeypatch.setattr(w8a8, name, None)
    monkeypatch.setattr(mxfp4, "_FN", {})
    monkeypatch.setattr(w8a8, "_FN", {})
    w8a8._workspace_bytes.cache_clear()
    yield torch, recorder
    w8a8._workspace_bytes.cache_clear()


T, N, K, E = 200, 250, 1024, 4
PYTHON = {
    "w8a8_quantize_rows": lambda a, kw: w4.w8a8_quantize_rows(a["x"], **kw),
    "qmm_w8a8": lambda a, kw: (w4.qmm_w8a8(*a["q"], *a["w"], split_k=2, **kw),),
    "w8a8_linear": lambda a, kw: (w4.w8a8_linear(a["x"], *a["w"], **kw),),
    "w8a8_linear_backward": lambda a, kw: (w4.w8a8_linear_backward(a["dy"], *a["w"], **kw),),
    "w8a8_experts_linear": lambda a, kw: (w4.w8a8_experts_linear(a["x"], *a["e"], a["offsets"], a["tokens"], **kw),),
    "w8a8_experts_linear_backward": lambda a, kw: (w4.w8a8_experts_linear_backward(a["dr"], *a["e"], a["offsets"], **kw),),
    "w8a8_experts_gate_up_swiglu": lambda a, kw: (w4.w8a8_experts_gate_up_swiglu(
        a["x"], a["e"], a["e"], a["offsets"], a["tokens"], **kw),),
    "w8a8_experts_gate_up_swiglu_backward": lambda a, kw: w4.w8a8_experts_gate_up_swiglu_backward(
        a["x"], a["e"], a["e"], a["dr"], a["offsets"], a["tokens"], **kw),
    "experts_route": lambda a, kw: w4.experts_route(a["logits"], 2, **kw),
    "experts_route_backward": lambda a, kw: (w4.experts_route_backward(a["logits"], a["positions"], a["weights"], **kw),),
    "experts_combine": lambda a, kw: (w4.experts_combine(a["dr"], a["positions"], a["weights"], **kw),),
    "experts_combine_backward": lambda a, kw: w4.experts_combine_backward(a["dy"], a["dr"], a["positions"], a["weights"], **kw),
}


def arguments(t):
    new = t.Tensor
    return {"x": new((T, K), t.bfloat16), "dy": new((T, N), t.bfloat16), "dr": new((2 * T, N), t.bfloat16),
            "w": (new((N, K), t.int8), new((N,), t.float32)), "q": (new((T, K), t.int8), new((T,), t.float32)),
            "e": (new((E, N, K), t.int8), new((E, N), t.float32)), "offsets": new((E + 1,), t.int32),
            "tokens": new((2 * T,), t.int32), "logits": new((T, E), t.float32), "positions": new((T, 2), t.int32),
            "weights": new((T, 2), t.float32)}


@pytest.mark.parametrize("form", ["object", "handle", "default handle"])
@pytest.mark.parametrize("name", list(PYTHON))
def test_a_call_on_a_stream_takes_memory_of_that_stream(model, name, form):
    torch, recorder = model
    side = 0 if "default" in form else SIDE
    stream = torch.cuda.Stream(side) if "object" in form else side
    a = arguments(torch)
    known = set(torch.pools.owner)
    first = PYTHON[name](a, {})
    own = {p for p in recorder.calls[0][1] if p not in known}
    del first
    gc.collect()
    outputs = PYTHON[name](a, {"stream": stream})
    assert [c[2] for c in recorder.calls] == [CURRENT, side] and {c[0] for c in recorder.calls} == {name}
    mine = {p for p in recorder.calls[1][1] if p not in known}
    assert len(mine) == len(own) >= len(outputs) and not mine & own
    assert all(torch.pools.stream_of(p) == side for p in mine)
    assert all(CURRENT in t.recorded for t in outputs)


GRADIENTS = {"w8a8_quantize_rows": "x", "w8a8_linear": "x", "w8a8_linear_backward": "dy", "w8a8_experts_linear": "x",
             "w8a8_experts_linear_backward": "dr", "w8a8_experts_gate_up_swiglu": "x", "w8a8_experts_gate_up_swiglu_backward": "dr",
             "experts_route": "logits", "experts_route_backward": "weights", "experts_combine": "weights",
             "experts_combine_backward": "dy"}


@pytest.mark.parametrize("name", list(GRADIENTS))
def test_a_gradient_is_not_dropped_in_silence(model, name):
    torch, recorder = model
    a = arguments(torch)
    a[GRADIENTS[name]].requires_grad = True
    with pytest.raises(ValueError, match="requires a gradient"):
        PYTHON[name](a, {})
    assert not recorder.calls
    torch.is_grad_enabled = lambda: False
    PYTHON[name](a, {})
    assert len(recorder.calls) == 1


@pytest.mark.parametrize("workspace", [4096, "room"])
@pytest.mark.parametrize("name", [n for n in PYTHON if "quantize" not in n and "combine" not in n and n != "experts_route_backward"])
def test_a_workspace_that_is_no_tensor_is_refused(model, name, workspace):
    torch, recorder = model
    with pytest.raises(TypeError, match="workspace must be a torch.Tensor"):
        PYTHON[name](arguments(torch), {"workspace": workspace})
    assert not recorder.calls


@pytest.mark.parametrize("name,change", [
    ("w8a8_linear", dict(x=("x", (T, K - 16)))), ("w8a8_linear", dict(w=("wq", (N, K + 16)))),
    ("w8a8_experts_linear", dict(offsets=("offsets", (E,)))), ("w8a8_experts_linear", dict(e=("ws", (E, N + 1)))),
    ("w8a8_experts_gate_up_swiglu_backward", dict(dr=("dh", (2 * T, N + 1)))), ("experts_combine", dict(weights=("w", (T, 3)))),
    ("experts_route_backward", dict(weights=("dw", (T, 1)))), ("experts_combine_backward", dict(dy=("dout", (T + 1, N))))])
def test_shapes_that_do_not_fit_are_refused(model, name, change):
    torch, recorder = model
    a = arguments(torch)
    (key, (what, shape)), = change.items()
    if what == "wq":
        a[key] = (torch.Tensor(shape, torch.int8), a[key][1])
    elif what == "ws":
        a[key] = (a[key][0], torch.Tensor(shape, torch.float32))
    else:
        a[key] = torch.Tensor(shape, a[key].dtype)
    with pytest.raises(ValueError):
        PYTHON[name](a, {})
    assert not recorder.calls


@pytest.mark.parametrize("top_k", [-1, 0, E + 1, 65])
def test_more_experts_than_there_are_cannot_be_chosen(model, top_k):
    torch, recorder = model
    with pytest.raises(ValueError, match="top_k"):
        w4.experts_route(arguments(torch)["logits"], top_k)
    assert not recorder.calls
