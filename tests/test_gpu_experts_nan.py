"""GPU tests of tokens and weights that are not finite through the operators of mixtures of experts."""

import numpy as np
import pytest

import oracle as O

from gpu_helpers import announce
from test_gpu_experts import block_problem, compare, host, make_positions
from test_gpu_w8a8 import bf16, bf16_values, check, guarded, to_gpu, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T", [5, 130])
def test_a_token_of_nan_logits_stays_nan(lib, T, renormalize):
    """Tokens whose logits hold NaN, all of them or so many that experts are missing: their outputs and gradients are NaN,
    beside padding (all minus infinity), which gets zeros, and tokens whose results are as without them."""
    import torch
    announce(f"experts block, NaN logits, T={T} renormalize={renormalize}")
    _, x, logits, ((gate, _), (up, _), (down, _)), dout = block_problem(8, T, 48, 96, 7 * T)
    lost, padding = [1, T - 1], [2]
    real = np.setdiff1d(np.arange(T), lost + padding)

    def run(x, logits, dout):
        weights, experts, positions, tokens, offsets = lib.experts_route(to_gpu(logits), 3, renormalize)
        h = lib.w8a8_experts_gate_up_swiglu(bf16(x), gate, up, offsets, tokens)
        y = lib.w8a8_experts_linear(h, *down, offsets)
        dy, dweights = lib.experts_combine_backward(bf16(dout), y, positions, weights)
        dh = lib.w8a8_experts_linear_backward(dy, *down, offsets)
        rows, _, _ = lib.w8a8_experts_gate_up_swiglu_backward(bf16(x), gate, up, dh, offsets, tokens)
        return dict(weights=weights, out=lib.experts_combine(y, positions, weights), dx=lib.experts_combine(rows, positions),
                    dlogits=lib.experts_route_backward(to_gpu(logits), experts, dweights, renormalize),
                    dweights=dweights, experts=experts, positions=positions)
    alone = run(x[real], logits[real], dout[real])
    logits[padding] = -np.inf
    logits[1] = np.nan
    logits[T - 1, :7] = [np.nan, -np.inf, np.nan, np.nan, -np.inf, np.nan, np.nan]      # expert 7 alone is left
    r = run(x, logits, dout)
    for n in ("weights", "out", "dx", "dlogits"):
        assert bool(r[n][lost].isnan().all()), n
    for n in ("weights", "out", "dx", "dlogits", "dweights"):
        assert bool((r[n][padding] == 0).all()), n
        assert torch.equal(r[n][to_gpu(real)], alone[n]), n
    assert bool(r["dweights"][1].isnan().all()) and bool(r["dweights"][T - 1, 1:].isnan().all())
    none = lib.EXPERTS_NAN_ROW
    assert host(r["experts"])[[1, T - 1, 2]].tolist() == [[-1] * 3, [7, -1, -1], [-1] * 3]
    assert host(r["positions"])[[1, 2]].tolist() == [[none] * 3, [-1] * 3] and host(r["positions"])[T - 1, 1:].tolist() == [none] * 2


@pytest.mark.parametrize("N", [8, 40, 41])
@pytest.mark.parametrize("top", [1, 3, 4, 20])
def test_the_mark_of_nan_logits_reaches_the_combination(lib, top, N):
    """At any slot, with and without weights, whatever the weight there; no row is read or written for it."""
    announce(f"experts_combine, mark of NaN, top={top} N={N}")
    rng = np.random.default_rng(top)
    T, R = 24, 24 * top
    y, dout = bf16_values(rng.standard_normal((R, N))), bf16_values(rng.standard_normal((T, N)))
    w, positions = rng.random((T, top)).astype(np.float32), make_positions(rng, T, top, R)
    for t in range(0, T, 2):
        positions[t, t % top] = lib.EXPERTS_NAN_ROW
        w[t, t % top] = (0.0, 1.0, np.nan)[t % 3]
    for weights in (w, None):
        want = O.combine_reference(y, positions, weights)
        assert np.isnan(want[0][::2]).all() and not np.isnan(want[0][1::2]).any()
        check(lib.experts_combine(bf16(y), to_gpu(positions), None if weights is None else to_gpu(weights)), want)
    dy, untouched = guarded(R, N, 0)
    dy.fill_(-77)
    _, dw = lib.experts_combine_backward(bf16(dout), bf16(y), to_gpu(positions), to_gpu(w), dy=dy)
    (want, bound), (want_dw, bound_dw) = O.combine_backward_reference(dout, y, positions, w)
    reached = ~np.isnan(want).any(1)
    check(dy, (want, bound), reached)
    assert (values(dy)[~reached] == -77).all() and untouched()
    assert (np.isnan(want_dw) == (positions == lib.EXPERTS_NAN_ROW)).all()
    compare(dw, want_dw, bound_dw)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("E", [16, 20, 64, 300, 1000])
def test_the_gradient_of_infinite_logits(lib, E, kind):
    """Beside an infinite logit the softmax over all experts is NaN for each of them, and so are their gradients; masked
    ones (minus infinity) and other tokens are as without it."""
    announce(f"experts_route_backward, infinite logits, E={E} {kind}")
    rng = np.random.default_rng(E)
    T, top = 21, 3
    logits = bf16_values(rng.standard_normal((T, E))).astype(np.float32)
    logits[rng.random((T, E)) < 0.2] = -np.inf
    logits[3, E // 2], logits[T - 1, [0, E - 1]] = np.inf, np.inf
    logits[5] = -np.inf
    t = bf16(logits) if kind == "bf16" else to_gpu(logits)
    dw = rng.standard_normal((T, top)).astype(np.float32)
    for renormalize in (True, False):
        experts = lib.experts_route(t, top, renormalize)[1]
        d = lib.experts_route_backward(t, experts, to_gpu(dw), renormalize)
        with np.errstate(invalid="ignore"):
            want, bound = O.route_backward_reference(logits.astype(np.float64), host(experts), dw.astype(np.float64), renormalize)
        if not renormalize:
            assert (np.isnan(want[[3, T - 1]]) == (logits[[3, T - 1]] > -np.inf)).all()
        if kind == "bf16":
            bound = bound + (np.abs(want) + bound) * 2.0 ** -8
        compare(d.float(), want, bound)
