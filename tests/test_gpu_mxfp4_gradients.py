"""MXFP4 calls and autograd: a gradient is never dropped in silence, and the backward calls serve an
autograd function that a user writes."""

import numpy as np
import pytest

import oracle as O

from gpu_helpers import announce
from test_gpu_mxfp4 import bf16, bf16_values, check, gated, values

pytestmark = pytest.mark.gpu


def _problem(M, N=136, K=96):
    rng = np.random.default_rng(M)
    x, gate, gv, up, uv = gated(rng, M, N, K)
    return x, gate, gv, up, uv, bf16_values(rng.standard_normal((M, N)))


@pytest.mark.parametrize("M", [3, 40])
def test_a_tensor_that_requires_a_gradient_is_refused(lib, M):
    import torch
    announce(f"mxfp4 gradients refused M={M}")
    x, gate, _, up, _, dh = _problem(M)
    x, dh = bf16(x), bf16(dh)
    xr, dr = x.clone().requires_grad_(), dh.clone().requires_grad_()
    y = torch.empty_like(dh).requires_grad_()
    refused = [
        lambda: lib.mxfp4_linear(xr, *gate), lambda: lib.mxfp4a4_linear(xr, *gate),
        lambda: lib.mxfp4_linear_backward(dr, *gate), lambda: lib.mxfp4_gate_up_swiglu(xr, gate, up),
        lambda: lib.mxfp4_gate_up_swiglu_backward(xr, gate, up, dh),
        lambda: lib.mxfp4_gate_up_swiglu_backward(x, gate, up, dr),
        lambda: lib.PreparedMxfp4Linear(xr, *gate), lambda: lib.PreparedMxfp4GateUp(xr, gate, up),
        lambda: lib.mxfp4_linear(x, *gate, y=y),
    ]
    for call in refused:
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
    # nothing is lost where no history is recorded, and quantizing a parameter has no gradient to lose
    expected = [lib.mxfp4_linear(x, *gate), lib.mxfp4_gate_up_swiglu(x, gate, up)]
    with torch.no_grad():
        assert torch.equal(lib.mxfp4_linear(xr, *gate), expected[0])
        assert torch.equal(lib.mxfp4_gate_up_swiglu(xr, gate, up), expected[1])
        assert torch.equal(lib.PreparedMxfp4Linear(xr, *gate)(), expected[0])
    assert torch.equal(lib.mxfp4_linear(xr.detach(), *gate), expected[0])
    a, b = lib.mxfp4_quantize_rows(torch.nn.Parameter(x)), lib.mxfp4_quantize_rows(x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("M", [3, 40])
def test_the_calls_inside_an_autograd_function(lib, M):
    import torch
    announce(f"mxfp4 autograd function M={M}")
    x, gate, gv, up, uv, dh = _problem(M)

    class GateUp(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            ctx.save_for_backward(x)
            return lib.mxfp4_gate_up_swiglu(x, gate, up)

        @staticmethod
        def backward(ctx, dh):
            return lib.mxfp4_gate_up_swiglu_backward(ctx.saved_tensors[0], gate, up, dh.contiguous())[0]

    leaf = bf16(x).requires_grad_()
    h = GateUp.apply(leaf)
    h.backward(bf16(dh))
    check(h.detach(), O.mx_gate_up(x, gv, uv))
    check(leaf.grad, O.mx_gate_up_backward(x, gv, uv, dh)[0])
    assert np.isfinite(values(leaf.grad)).all()
