"""MXFP4 operators of ``libw4a16.so``: quantization, products, and the gated feed-forward block.

The functions have the names of the C ABI and only marshal arguments, as the rest of the package.

Tensor conventions (all on the GPU, contiguous):
    x, dy, y, h, ...   torch.bfloat16 [rows, columns]
    codes              torch.uint8    [R, K/2]    two codes per byte, the lower index in the low half
    scales             torch.uint8    [R, K/32]   the factor 2^(byte - 127) of 32 values; 255 is NaN
A weight matrix is its ``(codes, scales)`` pair with R = N output columns; K % 32 == 0.

The calls record nothing for autograd: a gradient is the matching ``..._backward`` call, as in the
``backward`` of a ``torch.autograd.Function``.  While gradients are recorded, a tensor that requires one
is refused rather than cut off from its history.
"""

from __future__ import annotations

import ctypes
import functools

from . import _empty_for, _raise_for, _stream_handle, _torch, Plan, load

__all__ = [
    "MXFP4_BLOCK", "MXFP4_LINEAR", "MXFP4_LINEAR_BACKWARD", "MXFP4_QMM_A4", "MXFP4A4_LINEAR", "MXFP4_GATE_UP",
    "MXFP4_GATE_UP_BACKWARD", "PATH_MXFP4", "PATH_MXFP4_QMV", "mxfp4_plan", "mxfp4_quantize_rows", "mxfp4_dequantize_rows",
    "mxfp4_linear", "mxfp4_linear_backward", "qmm_mxfp4a4", "mxfp4a4_linear", "mxfp4_gate_up_swiglu",
    "mxfp4_gate_up_swiglu_backward", "PreparedMxfp4Linear", "PreparedMxfp4GateUp",
]

MXFP4_BLOCK = 32
(MXFP4_LINEAR, MXFP4_LINEAR_BACKWARD, MXFP4_QMM_A4, MXFP4A4_LINEAR, MXFP4_GATE_UP,
 MXFP4_GATE_UP_BACKWARD) = range(6)
PATH_MXFP4, PATH_MXFP4_QMV = 8, 9


def mxfp4_plan(op: int, M: int, N: int, K: int, split_k: int = 0, num_cus: int = 0) -> dict:
    """Launch plan of an MXFP4 operator (``MXFP4_LINEAR`` and so on)."""
    p = Plan()
    _raise_for(load().mxfp4_plan(op, M, N, K, split_k, num_cus, ctypes.byref(p)), "mxfp4_plan")
    return p.as_dict()


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(op, M, N, K, split_k, device):
    """The plan's workspace bytes on this (current) device; the plan depends on nothing else."""
    return int(mxfp4_plan(op, M, N, K, split_k)["workspace_bytes"])


# What every call needs, looked up once by _bind: torch, its types and queries, the library's functions.
_T = _BF16 = _FP32 = _U8 = _empty = _raw_stream = _current = None
_FN = {}


def _bind():
    global _T, _BF16, _FP32, _U8, _empty, _raw_stream, _current
    torch = _torch()
    lib = load()
    _FN.update((n, getattr(lib, n)) for n in __all__ if hasattr(lib, n))
    _BF16, _FP32, _U8, _empty = torch.bfloat16, torch.float32, torch.uint8, torch.empty
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if _raw_stream is None:
        def _raw_stream(index):
            return torch.cuda.current_stream(index).cuda_stream
    _current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _T = torch.Tensor


def _tensor(t, name, dtype, shape, index=None):
    """Checks a tensor, on GPU ``index`` if that is given; every condition in one expression for the
    calls that are right."""
    if (t.__class__ is _T and t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous()
            and (index is None or t.get_device() == index)):
        return
    if not isinstance(t, _T):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if index is not None and t.get_device() != index:
        where = f"cuda:{index}" if index >= 0 else "the CPU"
        raise ValueError(f"all tensors must be on one device: {name} is on {t.device}, another on {where}")


def _no_history(t, name):
    """Refuses a tensor whose gradient this call would drop."""
    if t.requires_grad and _torch().is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which this call does not record: call it under torch.no_grad() "
                         "(or on a detached tensor) and the matching _backward function for the gradient")


def _matrix(t, name):
    if _T is None:
        _bind()
    if not isinstance(t, _T):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got {len(shape)} dimensions")
    return shape


def _weights(codes, scales, name, index, like=None):
    """Checks codes and scales; returns (N, K).  What is right takes the first expression."""
    if (codes.__class__ is _T and scales.__class__ is _T and codes.dtype is _U8 and scales.dtype is _U8
            and 0 <= index == codes.get_device() == scales.get_device()
            and codes.is_contiguous() and scales.is_contiguous()):
        shape = codes.shape
        if len(shape) == 2:
            N, half = shape
            if half and not half % 16 and scales.shape == (N, half // 16) and (like is None or (N, 2 * half) == like):
                return N, 2 * half
    N, half = _matrix(codes, name)
    K = 2 * half
    if K == 0 or K % MXFP4_BLOCK:
        raise ValueError(f"{name}: K={K} must be a positive multiple of {MXFP4_BLOCK}")
    if like is not None and (N, K) != like:
        raise ValueError(f"{name} must be [{like[0]}, {like[1]}], got [{N}, {K}]")
    _tensor(codes, name, _U8, (N, half), index)
    _tensor(scales, name, _U8, (N, K // MXFP4_BLOCK), index)
    return N, K


def _output(t, name, shape, x, dtype, stream=None):
    """An output beside ``x``: allocated for ``stream``, or checked if it is given."""
    if t is None:
        if stream is not None:
            return _empty_for(stream, shape, dtype, x.device)
        return x.new_empty(shape) if x.dtype is dtype else x.new_empty(shape, dtype=dtype)
    _tensor(t, name, dtype, shape, x.get_device())
    _no_history(t, name)
    return t


def _check_workspace(workspace, index):
    if not isinstance(workspace, _T):
        raise TypeError("workspace must be a torch.Tensor")
    if not workspace.is_cuda or not workspace.is_contiguous() or workspace.get_device() != index:
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{index}")


def _call(name, op, dims, index, stream, workspace, args, split_k=0):
    """One C-ABI call on GPU ``index``: its workspace (allocated where the caller gave none), the stream,
    the status."""
    if index != _current():
        with _torch().cuda.device(index):
            return _call(name, op, dims, index, stream, workspace, args, split_k)
    if op is None:
        args += dims
    else:
        if split_k < 0:
            raise ValueError(f"split_k={split_k} must not be negative")
        need = _workspace_bytes(op, *dims, split_k, index)
        if not need:
            args += (*dims, split_k, None, 0)
        else:
            if workspace is None:
                where = f"cuda:{index}"
                workspace = (_empty(need, dtype=_U8, device=where) if stream is None else
                             _empty_for(stream, need, _U8, where, output=False))
            else:
                _check_workspace(workspace, index)
            args += (*dims, split_k, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    if stream is None:
        status = _FN[name](*args, _raw_stream(index))
    else:
        status = _FN[name](*args, _stream_handle(stream))
    if status:
        _raise_for(status, name)


def mxfp4_quantize_rows(x, codes=None, scales=None, stream=None):
    """MXFP4 codes and scales of the rows of ``x`` (bf16 or fp32 ``[R, K]``); returns
    ``(codes, scales)``.  A block holding an infinity or a NaN decodes to NaN."""
    R, K = _matrix(x, "x")
    if x.dtype is not _BF16 and x.dtype is not _FP32:
        raise TypeError(f"x must be torch.bfloat16 or torch.float32, got {x.dtype}")
    if K == 0 or K % MXFP4_BLOCK:
        raise ValueError(f"K={K} must be a positive multiple of {MXFP4_BLOCK}")
    _tensor(x, "x", x.dtype, (R, K))
    codes = _output(codes, "codes", (R, K // 2), x, _U8, stream)
    scales = _output(scales, "scales", (R, K // MXFP4_BLOCK), x, _U8, stream)
    _call("mxfp4_quantize_rows", None, (R, K), x.get_device(), stream, None,
          (x.data_ptr(), int(x.dtype is _FP32), codes.data_ptr(), scales.data_ptr()))
    return codes, scales


def mxfp4_dequantize_rows(codes, scales, y=None, stream=None):
    """The values of MXFP4 rows as bf16 ``[R, K]`` (exact; 2^128 and above, which only scale bytes 253 and
    254 reach, as infinities); returns y."""
    _matrix(codes, "codes")
    index = codes.get_device()
    R, K = _weights(codes, scales, "rows", index)
    y = _output(y, "y", (R, K), codes, _BF16, stream)
    _call("mxfp4_dequantize_rows", None, (R, K), index, stream, None,
          (codes.data_ptr(), scales.data_ptr(), y.data_ptr()))
    return y


def _projection(name, op, x, codes, scales, y, split_k, workspace, stream):
    M, _ = _matrix(x, "x")
    index = x.get_device()
    N, K = _weights(codes, scales, "weight", index)
    back = op == MXFP4_LINEAR_BACKWARD
    _tensor(x, "dy" if back else "x", _BF16, (M, N if back else K))
    _no_history(x, "dy" if back else "x")
    y = _output(y, "dx" if back else "y", (M, K if back else N), x, _BF16, stream)
    _call(name, op, (M, N, K), index, stream, workspace,
          (x.data_ptr(), codes.data_ptr(), scales.data_ptr(), y.data_ptr()), split_k)
    return y


def mxfp4_linear(x, codes, scales, y=None, split_k: int = 0, workspace=None, stream=None):
    """Weight-only projection ``y = x . W^T`` of bf16 ``x [M, K]``; split_k as for ``qmm_w4a16``."""
    return _projection("mxfp4_linear", MXFP4_LINEAR, x, codes, scales, y, split_k, workspace, stream)


def mxfp4_linear_backward(dy, codes, scales, dx=None, split_k: int = 0, workspace=None, stream=None):
    """Gradient of ``mxfp4_linear``'s input, ``dx = dy . W``; the weights are frozen."""
    return _projection("mxfp4_linear_backward", MXFP4_LINEAR_BACKWARD, dy, codes, scales, dx, split_k, workspace,
                       stream)


def mxfp4a4_linear(x, codes, scales, y=None, split_k: int = 0, workspace=None, stream=None):
    """Projection with 4-bit activations: ``x`` is quantized to MXFP4 in the call's workspace, the
    product runs on the scaled matrix cores.  Returns y."""
    return _projection("mxfp4a4_linear", MXFP4A4_LINEAR, x, codes, scales, y, split_k, workspace, stream)


def qmm_mxfp4a4(xq, xs, codes, scales, y=None, split_k: int = 0, workspace=None, stream=None):
    """``y = X . W^T`` of two MXFP4 operands (``xq``, ``xs`` from ``mxfp4_quantize_rows``)."""
    M, _ = _matrix(xq, "xq")
    index = xq.get_device()
    N, K = _weights(codes, scales, "weight", index)
    _weights(xq, xs, "x", index, (M, K))
    y = _output(y, "y", (M, N), xq, _BF16, stream)
    _call("qmm_mxfp4a4", MXFP4_QMM_A4, (M, N, K), index, stream, workspace,
          (xq.data_ptr(), xs.data_ptr(), codes.data_ptr(), scales.data_ptr(), y.data_ptr()), split_k)
    return y


def mxfp4_gate_up_swiglu(x, gate, up, h=None, split_k: int = 0, workspace=None, stream=None):
    """``h = silu(x . Wg^T) * (x . Wu^T)`` in one kernel; ``gate`` and ``up`` are ``(codes, scales)``
    pairs of one shape.  Returns h."""
    M, _ = _matrix(x, "x")
    index = x.get_device()
    N, K = _weights(*gate, "gate", index)
    _weights(*up, "up", index, (N, K))
    _tensor(x, "x", _BF16, (M, K))
    _no_history(x, "x")
    h = _output(h, "h", (M, N), x, _BF16, stream)
    _call("mxfp4_gate_up_swiglu", MXFP4_GATE_UP, (M, N, K), index, stream, workspace,
          (x.data_ptr(), gate[0].data_ptr(), gate[1].data_ptr(), up[0].data_ptr(), up[1].data_ptr(), h.data_ptr()),
          split_k)
    return h


def mxfp4_gate_up_swiglu_backward(x, gate, up, dh, dx=None, dgate=None, dup=None, split_k: int = 0, workspace=None,
                                  stream=None):
    """Backward pass of ``mxfp4_gate_up_swiglu`` from ``x`` and ``dh``; returns ``(dx, dgate, dup)``,
    the last two the gradients of both projections' outputs.  The weights are frozen."""
    M, _ = _matrix(x, "x")
    index = x.get_device()
    N, K = _weights(*gate, "gate", index)
    _weights(*up, "up", index, (N, K))
    _tensor(x, "x", _BF16, (M, K))
    _tensor(dh, "dh", _BF16, (M, N), index)
    _no_history(x, "x")
    _no_history(dh, "dh")
    dx = _output(dx, "dx", (M, K), x, _BF16, stream)
    dgate = _output(dgate, "dgate", (M, N), x, _BF16, stream)
    dup = _output(dup, "dup", (M, N), x, _BF16, stream)
    _call("mxfp4_gate_up_swiglu_backward", MXFP4_GATE_UP_BACKWARD, (M, N, K), index, stream, workspace,
          (x.data_ptr(), gate[0].data_ptr(), gate[1].data_ptr(), up[0].data_ptr(), up[1].data_ptr(), dh.data_ptr(),
           dx.data_ptr(), dgate.data_ptr(), dup.data_ptr()), split_k)
    return dx, dgate, dup


class _Prepared:
    """A call with fixed tensors, validated once; ``plan`` is its launch plan and ``workspace`` what it
    needs of that.  ``__call__`` issues one C-ABI call on the stream current at construction."""

    def _prepare(self, name, op, dims, index, args, split_k, workspace):
        with _torch().cuda.device(index):
            self.plan = mxfp4_plan(op, *dims, split_k)
        need = self.plan["workspace_bytes"]
        if workspace is None and need:
            workspace = _empty(need, dtype=_U8, device=f"cuda:{index}")
        elif workspace is not None:
            _check_workspace(workspace, index)
        self.workspace = workspace
        ptr, nbytes = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                           workspace.numel() * workspace.element_size())
        self._name, self._fn, self._device = name, _FN[name], index
        self._args = (*args, *dims, split_k, ptr, nbytes, _raw_stream(index))

    def _run(self):
        if self._device != _current():
            with _torch().cuda.device(self._device):
                status = self._fn(*self._args)
        else:
            status = self._fn(*self._args)
        if status:
            _raise_for(status, self._name)


class PreparedMxfp4Linear(_Prepared):
    """One projection with fixed tensors (see ``PreparedLinear``): ``mxfp4_linear``, or with
    ``four_bit_activations`` ``mxfp4a4_linear``.  Calling it returns ``y``."""

    def __init__(self, x, codes, scales, y=None, four_bit_activations: bool = False, split_k: int = 0, workspace=None):
        M, _ = _matrix(x, "x")
        N, K = _weights(codes, scales, "weight", x.get_device())
        _tensor(x, "x", _BF16, (M, K))
        _no_history(x, "x")
        self.M, self.N, self.K, self.y = M, N, K, _output(y, "y", (M, N), x, _BF16)
        self._keep = (x, codes, scales)
        name, op = (("mxfp4a4_linear", MXFP4A4_LINEAR) if four_bit_activations else ("mxfp4_linear", MXFP4_LINEAR))
        self._prepare(name, op, (M, N, K), x.get_device(),
                      (x.data_ptr(), codes.data_ptr(), scales.data_ptr(), self.y.data_ptr()), split_k, workspace)

    def __call__(self):
        self._run()
        return self.y


class PreparedMxfp4GateUp(_Prepared):
    """``mxfp4_gate_up_swiglu`` with fixed tensors (see ``PreparedGateUp``).  Calling it returns ``h``."""

    def __init__(self, x, gate, up, h=None, split_k: int = 0, workspace=None):
        M, _ = _matrix(x, "x")
        N, K = _weights(*gate, "gate", x.get_device())
        _weights(*up, "up", x.get_device(), (N, K))
        _tensor(x, "x", _BF16, (M, K))
        _no_history(x, "x")
        self.M, self.N, self.K, self.h = M, N, K, _output(h, "h", (M, N), x, _BF16)
        self._keep = (x, *gate, *up)
        self._prepare("mxfp4_gate_up_swiglu", MXFP4_GATE_UP, (M, N, K), x.get_device(),
                      (x.data_ptr(), gate[0].data_ptr(), gate[1].data_ptr(), up[0].data_ptr(), up[1].data_ptr(),
                       self.h.data_ptr()), split_k, workspace)

    def __call__(self):
        self._run()
        return self.h
