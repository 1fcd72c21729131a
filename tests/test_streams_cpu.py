"""Where calls with a ``stream`` argument take their memory from, and what they refuse, without a GPU.

torch's allocator keeps one pool per stream and hands a freed block out again in that stream's order.
A model of torch with such an allocator stands in for it here, and the library's functions are
replaced by a recorder of the pointers and the stream that they are given.  What a call allocates has
to come from the pool of the stream that its kernels run on: a block of another stream's pool can
still be in use there.
"""

import contextlib
import gc
import types

import pytest

import w4a16_group_quantized_qmv_amd as w4
from w4a16_group_quantized_qmv_amd import mxfp4

CURRENT, SIDE = 0x100, 0x200          # stream handles


class Pools:
    """Blocks by stream; a block freed with another stream recorded on it is not handed out again."""

    def __init__(self):
        self.current, self.next, self.free, self.owner = CURRENT, 1 << 40, [], {}

    def take(self, nbytes):
        size = -(-max(nbytes, 1) // 512) * 512
        for block in self.free:
            if block[0] == self.current and block[1] == size:
                self.free.remove(block)
                return block
        self.next += size
        self.owner[self.next - size] = (self.current, size)
        return (self.current, size, self.next - size)

    def stream_of(self, ptr):
        return next((s for base, (s, size) in self.owner.items() if base <= ptr < base + size), None)


class Model:
    """The parts of torch that the binding uses."""

    def __init__(self):
        pools = self.pools = Pools()
        sizes = {"bfloat16": 2, "float32": 4, "uint8": 1, "int8": 1, "int32": 4}

        class Tensor:
            is_cuda = True
            device = "cuda:0"
            requires_grad = False

            def __init__(self, shape, dtype):
                self.shape, self.dtype = tuple(shape), dtype
                self.block, self.recorded = pools.take(self.numel() * sizes[dtype]), []

            def __del__(self):
                if not [s for s in self.recorded if s != self.block[0]]:
                    pools.free.append(self.block)

            def numel(self):
                n = 1
                for s in self.shape:
                    n *= s
                return n

            def dim(self):
                return len(self.shape)

            def element_size(self):
                return sizes[self.dtype]

            def is_contiguous(self):
                return True

            def get_device(self):
                return 0

            def data_ptr(self):
                return self.block[2]

            def new_empty(self, shape, dtype=None):
                return Tensor(shape, dtype or self.dtype)

            def record_stream(self, s):
                self.recorded.append(s.cuda_stream)

        class Stream:
            def __init__(self, handle, device=None):
                self.cuda_stream = int(handle)

        def external(handle, device=None):
            return Stream(handle or 0x900)             # (a null handle gives one of torch's own streams)

        @contextlib.contextmanager
        def stream(s):
            before, pools.current = pools.current, s.cuda_stream
            try:
                yield
            finally:
                pools.current = before

        def empty(shape, dtype=None, device=None):
            return Tensor((shape,) if isinstance(shape, int) else shape, dtype)

        self.Tensor, self.empty = Tensor, empty
        for name in sizes:
            setattr(self, name, name)
        self.is_grad_enabled = lambda: True
        self._C = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda index: pools.current, _cuda_getDevice=lambda: 0)
        self.cuda = types.SimpleNamespace(Stream=Stream, ExternalStream=external, stream=stream,
                                          default_stream=lambda device=None: Stream(0),
                                          device=lambda index: contextlib.nullcontext(),
                                          current_device=lambda: 0,
                                          current_stream=lambda device=None: Stream(pools.current))


class Recorder:
    """The library: plans and sizes are its own (256 compute units), compute calls are recorded."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        real = getattr(self.lib, name)
        if name in ("w4a8_xsum_cols", "w4a16_status_string"):
            return real
        if name == "mxfp4_plan":
            return lambda op, M, N, K, split, cus, out: real(op, M, N, K, split, cus or 256, out)
        if name in ("w4a16_plan",):
            return lambda M, N, K, g, path, split, cus, out: real(M, N, K, g, path, split, cus or 256, out)
        if name in ("w4a16_gate_up_plan", "w4a8_plan"):
            return lambda M, N, K, g, split, cus, out: real(M, N, K, g, split, cus or 256, out)
        if name in ("w4a16_workspace_bytes", "w4a8_linear_workspace_bytes"):
            return lambda M, N, K, g, cus: real(M, N, K, g, cus or 256)
        if name == "w4a16_grouped_plan":
            return lambda count, n, M, K, g, cus, out: real(count, n, M, K, g, cus or 256, out)

        def call(*args):
            pointers = []
            for a in args[:-1]:
                for v in (a if hasattr(a, "__len__") else (a,)):
                    v = getattr(v, "value", v)
                    if isinstance(v, int) and v >= 1 << 40:
                        pointers.append(v)
            stream = args[-1]
            self.calls.append((name, pointers, getattr(stream, "value", stream) or 0))
            return 0
        return call


@pytest.fixture
def model(monkeypatch):
    lib = w4.load()
    torch, recorder = Model(), Recorder(lib)
    for module in (w4, mxfp4):
        monkeypatch.setattr(module, "_torch", lambda: torch)
    monkeypatch.setattr(w4, "_LIB", recorder)
    for name in ("_T", "_BF16", "_FP32", "_U8", "_empty", "_raw_stream", "_current"):
        monkeypatch.setattr(mxfp4, name, None)
    monkeypatch.setattr(mxfp4, "_FN", {})
    mxfp4._workspace_bytes.cache_clear()
    yield torch, recorder
    mxfp4._workspace_bytes.cache_clear()


M, N, K = 40, 256, 1024
CALLS = {
    "mxfp4_quantize_rows": lambda t, a, kw: w4.mxfp4_quantize_rows(a["x"], **kw),
    "mxfp4_dequantize_rows": lambda t, a, kw: (w4.mxfp4_dequantize_rows(*a["w"], **kw),),
    "mxfp4_linear": lambda t, a, kw: (w4.mxfp4_linear(a["x"], *a["w"], split_k=4, **kw),),
    "mxfp4_linear_backward": lambda t, a, kw: (w4.mxfp4_linear_backward(a["dy"], *a["w"], split_k=2, **kw),),
    "mxfp4a4_linear": lambda t, a, kw: (w4.mxfp4a4_linear(a["x"], *a["w"], **kw),),
    "qmm_mxfp4a4": lambda t, a, kw: (w4.qmm_mxfp4a4(*a["q"], *a["w"], split_k=2, **kw),),
    "mxfp4_gate_up_swiglu": lambda t, a, kw: (w4.mxfp4_gate_up_swiglu(a["x"], a["w"], a["w"], split_k=2, **kw),),
    "mxfp4_gate_up_swiglu_backward": lambda t, a, kw: w4.mxfp4_gate_up_swiglu_backward(
        a["x"], a["w"], a["w"], a["dy"], split_k=2, **kw),
    "qmv_w4a16": lambda t, a, kw: (w4.qmv_w4a16(a["few"], *a["a4"], **kw),),
    "qmv_affine": lambda t, a, kw: (w4.qmv_affine(a["few"], *a["a4"], bits=4, **kw),),
    "qmm_w4a16": lambda t, a, kw: (w4.qmm_w4a16(a["x"], *a["a4"], split_k=2, **kw),),
    "w4a16_linear": lambda t, a, kw: (w4.w4a16_linear(a["x"], *a["a4"], **kw),),
    "w4a16_gate_up_swiglu": lambda t, a, kw: (w4.w4a16_gate_up_swiglu(a["x"], a["a4"], a["a4"], split_k=2, **kw),),
    "w4a8_quantize_rows": lambda t, a, kw: w4.w4a8_quantize_rows(a["x"], **kw),
    "qmm_w4a8": lambda t, a, kw: (w4.qmm_w4a8(*a["q8"], *a["a4"], split_k=2, **kw),),
    "w4a8_linear": lambda t, a, kw: (w4.w4a8_linear(a["x"], *a["a4"], **kw),),
    "w4a16_linear_grouped": lambda t, a, kw: w4.w4a16_linear_grouped(a["x"], [a["a4"], a["a4"]], **kw),
}


def arguments(t):
    new = t.Tensor
    return {"x": new((M, K), t.bfloat16), "few": new((4, K), t.bfloat16), "dy": new((M, N), t.bfloat16),
            "w": (new((N, K // 2), t.uint8), new((N, K // 32), t.uint8)),
            "q": (new((M, K // 2), t.uint8), new((M, K // 32), t.uint8)),
            "a4": (new((N, K // 8), t.int32), new((N, K // 128), t.bfloat16), new((N, K // 128), t.bfloat16)),
            "q8": (new((M, K), t.int8), new((M,), t.float32), new((M, w4.w4a8_xsum_cols(K)), t.bfloat16))}


@pytest.mark.parametrize("form", ["object", "handle", "default object", "default handle"])
@pytest.mark.parametrize("name", list(CALLS))
def test_a_call_on_a_stream_takes_memory_of_that_stream(model, name, form):
    torch, recorder = model
    side = 0 if "default" in form else SIDE
    stream = torch.cuda.Stream(side) if "object" in form else side
    a = arguments(torch)
    known = set(torch.pools.owner)
    # queued on the current stream; the workspace returns to the current stream's pool at once
    first = CALLS[name](torch, a, {})
    own = {p for p in recorder.calls[0][1] if p not in known}
    del first
    gc.collect()
    # the same on the side stream, which does not wait for the current one
    outputs = CALLS[name](torch, a, {"stream": stream})
    assert [c[2] for c in recorder.calls] == [CURRENT, side] and {c[0] for c in recorder.calls} == {name}
    mine = {p for p in recorder.calls[1][1] if p not in known}
    assert len(mine) == len(own) >= len(outputs)
    assert not mine & own, "memory of a call that is still queued on the current stream"
    for p in mine:
        assert torch.pools.stream_of(p) == side, "memory of another stream's pool"
    # outputs are read elsewhere: the current stream keeps them from the side stream's next call
    kept = {t.data_ptr() for t in outputs}
    assert all(CURRENT in t.recorded for t in outputs)
    del outputs
    gc.collect()
    again = CALLS[name](torch, a, {"stream": stream})
    assert not kept & {t.data_ptr() for t in again}
    # and without the argument everything is the current stream's
    results = CALLS[name](torch, a, {})
    assert all(torch.pools.stream_of(t.data_ptr()) == CURRENT and not t.recorded for t in results)


@pytest.mark.parametrize("name", ["mxfp4_linear", "mxfp4_linear_backward", "mxfp4a4_linear", "mxfp4_gate_up_swiglu",
                                  "mxfp4_gate_up_swiglu_backward"])
def test_a_gradient_is_not_dropped_in_silence(model, name):
    torch, recorder = model
    a = arguments(torch)
    a["x"].requires_grad = a["dy"].requires_grad = True
    with pytest.raises(ValueError, match="requires a gradient"):
        CALLS[name](torch, a, {})
    assert not recorder.calls
    torch.is_grad_enabled = lambda: False
    CALLS[name](torch, a, {})
    assert len(recorder.calls) == 1


@pytest.mark.parametrize("workspace", [4096, "room", b"room"])
@pytest.mark.parametrize("name", ["mxfp4_linear", "mxfp4_linear_backward", "mxfp4a4_linear", "qmm_mxfp4a4",
                                  "mxfp4_gate_up_swiglu", "mxfp4_gate_up_swiglu_backward", "qmm_w4a16",
                                  "w4a16_gate_up_swiglu", "qmm_w4a8", "w4a8_linear"])
def test_a_workspace_that_is_no_tensor_is_refused(model, name, workspace):
    torch, recorder = model
    a = arguments(torch)
    with pytest.raises(TypeError, match="workspace must be a torch.Tensor"):
        CALLS[name](torch, a, {"workspace": workspace})
    if name == "mxfp4_linear":
        with pytest.raises(TypeError, match="workspace must be a torch.Tensor"):
            w4.PreparedMxfp4Linear(a["x"], *a["w"], split_k=2, workspace=workspace)
    assert not recorder.calls
