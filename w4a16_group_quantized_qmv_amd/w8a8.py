"""Int8 products and mixtures of experts of ``libw4a16.so``: quantization, projections and their input
gradients, one matrix or one per expert, the router and the combination of the experts' outputs.

The functions have the names of the C ABI and only marshal arguments, as the rest of the package.

Tensor conventions (all on the GPU, contiguous):
    x, dy, y, h, ...   torch.bfloat16 [rows, columns]
    codes              torch.int8     [N, K], for experts [E, N, K]; K % 16 == 0
    scales             torch.float32  [N], for experts [E, N]: a row stands for scale * code
    offsets            torch.int32    [E + 1]      expert e has rows offsets[e] .. offsets[e + 1] - 1
    tokens             torch.int32    [R]          the rows' tokens
    positions          torch.int32    [T, top_k]   the rows of a token's experts, -1 for none; EXPERTS_NAN_ROW for none
                                                   of a token whose logits hold a NaN, which makes its sums NaN
A weight matrix is its ``(codes, scales)`` pair.  Rows behind ``offsets[E]`` are left as they were in every output.

A block of a mixture of experts, forward and backward with frozen weights:

    weights, experts, positions, tokens, offsets = experts_route(logits, top_k)
    h = w8a8_experts_gate_up_swiglu(x, gate, up, offsets, tokens)
    y = w8a8_experts_linear(h, *down, offsets)
    out = experts_combine(y, positions, weights)

    dy, dweights = experts_combine_backward(dout, y, positions, weights)
    dlogits = experts_route_backward(logits, experts, dweights)
    dh = w8a8_experts_linear_backward(dy, *down, offsets)
    dx_rows, dgate, dup = w8a8_experts_gate_up_swiglu_backward(x, gate, up, dh, offsets, tokens)
    dx = experts_combine(dx_rows, positions)

The calls record nothing for autograd: a gradient is the matching ``..._backward`` call.  While gradients are
recorded, a tensor that requires one is refused rather than cut off from its history.
"""

from __future__ import annotations

import ctypes
import functools

from . import _empty_for, _raise_for, _stream_handle, _torch, Plan, load
from . import mxfp4 as _mx
from .mxfp4 import _check_workspace, _matrix, _no_history, _output, _tensor

__all__ = [
    "W8A8_CHUNK", "EXPERTS_MAX_TOP_K", "EXPERTS_NAN_ROW", "W8A8_LINEAR", "W8A8_LINEAR_BACKWARD", "W8A8_QMM",
    "W8A8_EXPERTS_LINEAR", "W8A8_EXPERTS_LINEAR_BACKWARD", "W8A8_EXPERTS_GATE_UP", "W8A8_EXPERTS_GATE_UP_BACKWARD", "PATH_W8A8",
    "PATH_W8A8_QMV", "w8a8_plan", "w8a8_quantize_rows", "qmm_w8a8", "w8a8_linear", "w8a8_linear_backward",
    "w8a8_experts_linear", "w8a8_experts_linear_backward", "w8a8_experts_gate_up_swiglu",
    "w8a8_experts_gate_up_swiglu_backward", "experts_route_workspace_bytes", "experts_route",
    "experts_route_backward", "experts_combine", "experts_combine_backward",
]

W8A8_CHUNK = 16
EXPERTS_MAX_TOP_K = 64
EXPERTS_NAN_ROW = -2 ** 31
(W8A8_LINEAR, W8A8_LINEAR_BACKWARD, W8A8_QMM, W8A8_EXPERTS_LINEAR, W8A8_EXPERTS_LINEAR_BACKWARD, W8A8_EXPERTS_GATE_UP,
 W8A8_EXPERTS_GATE_UP_BACKWARD) = range(7)
PATH_W8A8, PATH_W8A8_QMV = 10, 11


def w8a8_plan(op: int, M: int, N: int, K: int, split_k: int = 0, num_cus: int = 0, experts: int = 1, rows=None) -> dict:
    """Launch plan of a W8A8 operator (``W8A8_LINEAR`` and so on): ``M`` activation rows, and for experts
    their number and the ``rows`` of the outputs (None: M)."""
    p = Plan()
    _raise_for(load().w8a8_plan(op, experts, M, M if rows is None else rows, N, K, split_k, num_cus, ctypes.byref(p)),
               "w8a8_plan")
    return p.as_dict()


def experts_route_workspace_bytes(T: int, E: int) -> int:
    """Workspace bytes of ``experts_route``."""
    return int(load().experts_route_workspace_bytes(T, E))


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(op, M, N, K, split_k, experts, rows, device):
    """The plan's workspace bytes on this (current) device; the plan depends on nothing else."""
    return int(w8a8_plan(op, M, N, K, split_k, 0, experts, rows)["workspace_bytes"])


# The library's functions and torch's types, looked up once.  The table is what a call looks at, so it comes last
# and whole: another thread in its first call finds all of it or looks everything up for itself.
_FN = {}
_BF16 = _FP32 = _I8 = _I32 = None


def _bind():
    global _FN, _BF16, _FP32, _I8, _I32
    if _mx._T is None:
        _mx._bind()
    torch, lib = _torch(), load()
    _BF16, _FP32, _I8, _I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32
    _FN = {n: getattr(lib, n) for n in __all__ if hasattr(lib, n)}


def _rows(t, name):
    """Shape of a matrix; the first check of every call."""
    if not _FN:
        _bind()
    return _matrix(t, name)


def _weights(codes, scales, name, index, experts=False, like=None):
    """Checks codes and scales; returns their shape, (N, K) or (E, N, K)."""
    T = _mx._T
    if not isinstance(codes, T):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = tuple(codes.shape)
    if len(shape) != (3 if experts else 2):
        raise ValueError(f"{name} must be {3 if experts else 2}-D, got {len(shape)} dimensions")
    if shape[-1] == 0 or shape[-1] % W8A8_CHUNK:
        raise ValueError(f"{name}: K={shape[-1]} must be a positive multiple of {W8A8_CHUNK}")
    if like is not None and shape != like:
        raise ValueError(f"{name} must be {list(like)}, got {list(shape)}")
    _tensor(codes, name, _I8, shape, index)
    _tensor(scales, f"{name} scales", _FP32, shape[:-1], index)
    _no_history(scales, f"{name} scales")
    return shape


def _gpu(index, name):
    if index < 0:
        raise ValueError(f"{name} must be on the GPU")


def _memory(nbytes, workspace, index, stream):
    """Pointer and size of a call's workspace, allocated where the caller gave none; the tensor keeps it alive."""
    if workspace is not None:
        _check_workspace(workspace, index)
    elif nbytes:
        where = f"cuda:{index}"
        workspace = (_mx._empty(nbytes, dtype=_mx._U8, device=where) if stream is None else
                     _empty_for(stream, nbytes, _mx._U8, where, output=False))
    if workspace is None or not nbytes:
        return workspace, (None, 0)
    return workspace, (workspace.data_ptr(), workspace.numel() * workspace.element_size())


def _launch(name, index, stream, args, plan=None, split_k=0, workspace=None, nbytes=None):
    """One C-ABI call on GPU ``index``.  ``plan``: (op, M, N, K, experts, rows) of a call with a workspace, ``args``
    without it; or its bytes in ``nbytes``."""
    if index != _mx._current():
        with _torch().cuda.device(index):
            return _launch(name, index, stream, args, plan, split_k, workspace, nbytes)
    if plan is not None:
        if split_k < 0:
            raise ValueError(f"split_k={split_k} must not be negative")
        op, M, N, K, experts, rows = plan
        nbytes = _workspace_bytes(op, M, N, K, split_k, experts, rows, index)
    if nbytes is not None:
        workspace, memory = _memory(nbytes, workspace, index, stream)
        args += memory
    status = _FN[name](*args, _mx._raw_stream(index) if stream is None else _stream_handle(stream))
    if status:
        _raise_for(status, name)


def w8a8_quantize_rows(x, codes=None, scales=None, stream=None):
    """Int8 codes and fp32 scales of the rows of ``x`` (bf16 or fp32 ``[R, K]``); returns ``(codes, scales)``."""
    R, K = _rows(x, "x")
    if x.dtype is not _BF16 and x.dtype is not _FP32:
        raise TypeError(f"x must be torch.bfloat16 or torch.float32, got {x.dtype}")
    if K == 0 or K % W8A8_CHUNK:
        raise ValueError(f"K={K} must be a positive multiple of {W8A8_CHUNK}")
    _tensor(x, "x", x.dtype, (R, K))
    _no_history(x, "x")
    codes = _output(codes, "codes", (R, K), x, _I8, stream)
    scales = _output(scales, "scales", (R,), x, _FP32, stream)
    _launch("w8a8_quantize_rows", x.get_device(), stream,
            (x.data_ptr(), int(x.dtype is _FP32), codes.data_ptr(), scales.data_ptr(), R, K))
    return codes, scales


def qmm_w8a8(xq, xs, codes, scales, y=None, split_k: int = 0, workspace=None, stream=None):
    """``y = X . W^T`` of two quantized operands (``xq``, ``xs`` from ``w8a8_quantize_rows``)."""
    M, _ = _rows(xq, "xq")
    index = xq.get_device()
    _gpu(index, "xq")
    N, K = _weights(codes, scales, "weight", index)
    _weights(xq, xs, "x", index, like=(M, K))
    y = _output(y, "y", (M, N), xq, _BF16, stream)
    _launch("qmm_w8a8", index, stream,
            (xq.data_ptr(), xs.data_ptr(), codes.data_ptr(), scales.data_ptr(), y.data_ptr(), M, N, K, split_k),
            (W8A8_QMM, M, N, K, 1, M), split_k, workspace)
    return y


def _projection(name, op, x, codes, scales, y, split_k, workspace, stream):
    M, _ = _rows(x, "x")
    index = x.get_device()
    _gpu(index, "x")
    N, K = _weights(codes, scales, "weight", index)
    back = op == W8A8_LINEAR_BACKWARD
    _tensor(x, "dy" if back else "x", _BF16, (M, N if back else K))
    _no_history(x, "dy" if back else "x")
    y = _output(y, "dx" if back else "y", (M, K if back else N), x, _BF16, stream)
    _launch(name, index, stream,
            (x.data_ptr(), codes.data_ptr(), scales.data_ptr(), y.data_ptr(), M, N, K, split_k),
            (op, M, N, K, 1, M), split_k, workspace)
    return y


def w8a8_linear(x, codes, scales, y=None, split_k: int = 0, workspace=None, stream=None):
    """Projection ``y = Q(x) . W^T`` of bf16 ``x [M, K]``, whose rows are quantized to int8 in the call; split_k as for
    ``qmm_w4a16``."""
    return _projection("w8a8_linear", W8A8_LINEAR, x, codes, scales, y, split_k, workspace, stream)


def w8a8_linear_backward(dy, codes, scales, dx=None, split_k: int = 0, workspace=None, stream=None):
    """Gradient of ``w8a8_linear``'s input, ``dx = dy . W``; the quantization of x passes gradients on, the weights are
    frozen."""
    return _projection("w8a8_linear_backward", W8A8_LINEAR_BACKWARD, dy, codes, scales, dx, split_k, workspace, stream)


def _routing(offsets, tokens, E, T, index):
    """Checks offsets and tokens; returns the number of rows."""
    _tensor(offsets, "offsets", _I32, (E + 1,), index)
    if tokens is None:
        return T
    if not isinstance(tokens, _mx._T):
        raise TypeError("tokens must be a torch.Tensor")
    _tensor(tokens, "tokens", _I32, (tokens.numel(),), index)
    return tokens.numel()


def w8a8_experts_linear(x, codes, scales, offsets, tokens=None, y=None, workspace=None, stream=None):
    """Projection by experts: row r of expert e is ``Q(x[tokens[r]]) . W_e^T``; without ``tokens`` the rows of ``x``
    are the experts' rows.  Returns y ``[R, N]``."""
    T, _ = _rows(x, "x")
    index = x.get_device()
    _gpu(index, "x")
    E, N, K = _weights(codes, scales, "weight", index, experts=True)
    _tensor(x, "x", _BF16, (T, K))
    _no_history(x, "x")
    R = _routing(offsets, tokens, E, T, index)
    y = _output(y, "y", (R, N), x, _BF16, stream)
    _launch("w8a8_experts_linear", index, stream,
            (x.data_ptr(), codes.data_ptr(), scales.data_ptr(), offsets.data_ptr(),
             None if tokens is None else tokens.data_ptr(), y.data_ptr(), E, T, R, N, K),
            (W8A8_EXPERTS_LINEAR, T, N, K, E, R), 0, workspace)
    return y


def w8a8_experts_linear_backward(dy, codes, scales, offsets, dx=None, workspace=None, stream=None):
    """Gradient of the rows of ``w8a8_experts_linear``: ``dx[r] = dy[r] . W_e`` (``experts_combine`` without weights
    adds up those of a token)."""
    R, _ = _rows(dy, "dy")
    index = dy.get_device()
    _gpu(index, "dy")
    E, N, K = _weights(codes, scales, "weight", index, experts=True)
    _tensor(dy, "dy", _BF16, (R, N))
    _no_history(dy, "dy")
    _routing(offsets, None, E, R, index)
    dx = _output(dx, "dx", (R, K), dy, _BF16, stream)
    _launch("w8a8_experts_linear_backward", index, stream,
            (dy.data_ptr(), codes.data_ptr(), scales.data_ptr(), offsets.data_ptr(), dx.data_ptr(), E, R, N, K),
            (W8A8_EXPERTS_LINEAR_BACKWARD, R, N, K, E, R), 0, workspace)
    return dx


def _gated(x, gate, up, offsets, tokens):
    """Checks of the gated calls; returns sizes and device."""
    T, _ = _rows(x, "x")
    index = x.get_device()
    _gpu(index, "x")
    E, N, K = _weights(*gate, "gate", index, experts=True)
    _weights(*up, "up", index, experts=True, like=(E, N, K))
    _tensor(x, "x", _BF16, (T, K))
    _no_history(x, "x")
    return E, T, _routing(offsets, tokens, E, T, index), N, K, index


def w8a8_experts_gate_up_swiglu(x, gate, up, offsets, tokens=None, h=None, workspace=None, stream=None):
    """``h[r] = silu(Q(x) . Wg_e^T) * (Q(x) . Wu_e^T)`` over the experts' rows, in one kernel; ``gate`` and ``up`` are
    ``(codes, scales)`` pairs of one shape.  Returns h ``[R, N]``."""
    E, T, R, N, K, index = _gated(x, gate, up, offsets, tokens)
    h = _output(h, "h", (R, N), x, _BF16, stream)
    _launch("w8a8_experts_gate_up_swiglu", index, stream,
            (x.data_ptr(), gate[0].data_ptr(), gate[1].data_ptr(), up[0].data_ptr(), up[1].data_ptr(), offsets.data_ptr(),
             None if tokens is None else tokens.data_ptr(), h.data_ptr(), E, T, R, N, K),
            (W8A8_EXPERTS_GATE_UP, T, N, K, E, R), 0, workspace)
    return h


def w8a8_experts_gate_up_swiglu_backward(x, gate, up, dh, offsets, tokens=None, dx=None, dgate=None, dup=None,
                                         workspace=None, stream=None):
    """Backward pass of ``w8a8_experts_gate_up_swiglu`` from ``x`` and ``dh``; returns ``(dx, dgate, dup)``: the rows'
    gradients of x (``experts_combine`` without weights adds up those of a token), and of both projections' outputs."""
    E, T, R, N, K, index = _gated(x, gate, up, offsets, tokens)
    _tensor(dh, "dh", _BF16, (R, N), index)
    _no_history(dh, "dh")
    dx = _output(dx, "dx", (R, K), x, _BF16, stream)
    dgate = _output(dgate, "dgate", (R, N), x, _BF16, stream)
    dup = _output(dup, "dup", (R, N), x, _BF16, stream)
    _launch("w8a8_experts_gate_up_swiglu_backward", index, stream,
            (x.data_ptr(), gate[0].data_ptr(), gate[1].data_ptr(), up[0].data_ptr(), up[1].data_ptr(), dh.data_ptr(),
             offsets.data_ptr(), None if tokens is None else tokens.data_ptr(), dx.data_ptr(), dgate.data_ptr(),
             dup.data_ptr(), E, T, R, N, K),
            (W8A8_EXPERTS_GATE_UP_BACKWARD, T, N, K, E, R), 0, workspace)
    return dx, dgate, dup


def _logits(logits):
    T, E = _rows(logits, "logits")
    if logits.dtype is not _BF16 and logits.dtype is not _FP32:
        raise TypeError(f"logits must be torch.bfloat16 or torch.float32, got {logits.dtype}")
    _tensor(logits, "logits", logits.dtype, (T, E))
    _no_history(logits, "logits")
    return T, E, logits.get_device()


def experts_route(logits, top_k: int, renormalize: bool = True, weights=None, experts=None, positions=None, tokens=None,
                  offsets=None, workspace=None, stream=None):
    """The ``top_k`` experts of each token by ``logits`` (bf16 or fp32 ``[T, E]``) and the rows' order; returns
    ``(weights, experts, positions, tokens, offsets)``.  The weights are the softmax over the chosen experts, or with
    ``renormalize=False`` their part of the softmax over all of them.  Logits of minus infinity are never chosen: expert
    and position are -1 there and the weight 0.  Logits that hold a NaN give NaN weights, and the position
    ``EXPERTS_NAN_ROW`` where no expert is chosen, so that the token's results are NaN."""
    T, E, index = _logits(logits)
    if not 1 <= top_k <= min(E, EXPERTS_MAX_TOP_K):
        raise ValueError(f"top_k={top_k} must be 1 .. {min(E, EXPERTS_MAX_TOP_K)} for {E} experts")
    weights = _output(weights, "weights", (T, top_k), logits, _FP32, stream)
    experts = _output(experts, "experts", (T, top_k), logits, _I32, stream)
    positions = _output(positions, "positions", (T, top_k), logits, _I32, stream)
    tokens = _output(tokens, "tokens", (T * top_k,), logits, _I32, stream)
    offsets = _output(offsets, "offsets", (E + 1,), logits, _I32, stream)
    _launch("experts_route", index, stream,
            (logits.data_ptr(), int(logits.dtype is _FP32), weights.data_ptr(), experts.data_ptr(), positions.data_ptr(),
             tokens.data_ptr(), offsets.data_ptr(), T, E, top_k, int(renormalize)),
            None, 0, workspace, experts_route_workspace_bytes(T, E))
    return weights, experts, positions, tokens, offsets


def experts_route_backward(logits, experts, dweights, renormalize: bool = True, dlogits=None, stream=None):
    """Gradient of the logits from that of the weights; ``experts`` from ``experts_route``."""
    T, E, index = _logits(logits)
    _, top_k = _matrix(experts, "experts")
    _tensor(experts, "experts", _I32, (T, top_k), index)
    _tensor(dweights, "dweights", _FP32, (T, top_k), index)
    _no_history(dweights, "dweights")
    dlogits = _output(dlogits, "dlogits", (T, E), logits, logits.dtype, stream)
    _launch("experts_route_backward", index, stream,
            (logits.data_ptr(), int(logits.dtype is _FP32), experts.data_ptr(), dweights.data_ptr(), dlogits.data_ptr(),
             T, E, top_k, int(renormalize)))
    return dlogits


def _pairs(y, positions, weights):
    R, N = _rows(y, "y")
    T, top_k = _matrix(positions, "positions")
    index = y.get_device()
    _gpu(index, "y")
    _tensor(y, "y", _BF16, (R, N))
    _no_history(y, "y")
    _tensor(positions, "positions", _I32, (T, top_k), index)
    if weights is not None:
        _tensor(weights, "weights", _FP32, (T, top_k), index)
        _no_history(weights, "weights")
    return T, top_k, R, N, index


def experts_combine(y, positions, weights=None, out=None, stream=None):
    """``out[t] = sum_j weights[t, j] * y[positions[t, j]]`` (without ``weights``: their sum); returns out ``[T, N]``."""
    T, top_k, R, N, index = _pairs(y, positions, weights)
    out = _output(out, "out", (T, N), y, _BF16, stream)
    _launch("experts_combine", index, stream,
            (y.data_ptr(), positions.data_ptr(), None if weights is None else weights.data_ptr(), out.data_ptr(), T, top_k,
             R, N))
    return out


def experts_combine_backward(dout, y, positions, weights, dy=None, dweights=None, stream=None):
    """Gradients of ``experts_combine``; returns ``(dy, dweights)``.  A row is at one position at most.  Rows of ``dy`` at
    no position are left as they were (a new ``dy`` holds no values there)."""
    if weights is None:
        raise TypeError("weights must be a torch.Tensor")
    T, top_k, R, N, index = _pairs(y, positions, weights)
    _tensor(dout, "dout", _BF16, (T, N), index)
    _no_history(dout, "dout")
    dy = _output(dy, "dy", (R, N), y, _BF16, stream)
    dweights = _output(dweights, "dweights", (T, top_k), y, _FP32, stream)
    _launch("experts_combine_backward", index, stream,
            (dout.data_ptr(), y.data_ptr(), positions.data_ptr(), weights.data_ptr(), dy.data_ptr(), dweights.data_ptr(), T,
             top_k, R, N))
    return dy, dweights
