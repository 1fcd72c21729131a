"""Calls with a ``stream`` argument on the GPU: whose memory they use, and what stands queued around them."""

import pytest

from gpu_helpers import announce

pytestmark = pytest.mark.gpu

M, N, K, SPLIT = 64, 2000, 4096, 4


def _random(shape, seed, scale=1.0):
    import torch
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    return (torch.randn(shape, device="cuda:0", generator=g) * scale).to(torch.bfloat16)


def _calls(lib):
    """Split products and the gated pair with its backward, as functions of their input and ``stream``."""
    import torch
    g = torch.Generator(device="cuda:0").manual_seed(1)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda:0", generator=g)
    exps = torch.randint(118, 122, (N, K // 32), dtype=torch.uint8, device="cuda:0", generator=g)
    wq = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), dtype=torch.int64, device="cuda:0", generator=g).to(torch.int32)
    s, b = _random((N, K // 128), 2, 0.01), _random((N, K // 128), 3, 0.01)
    dh = _random((M, N), 4)
    return {
        "mxfp4_linear": lambda x, **kw: (lib.mxfp4_linear(x, codes, exps, split_k=SPLIT, **kw),),
        "mxfp4a4_linear": lambda x, **kw: (lib.mxfp4a4_linear(x, codes, exps, split_k=SPLIT, **kw),),
        "mxfp4_gate_up_swiglu_backward": lambda x, **kw: lib.mxfp4_gate_up_swiglu_backward(
            x, (codes, exps), (codes, exps), dh, split_k=SPLIT, **kw),
        "qmm_w4a16": lambda x, **kw: (lib.qmm_w4a16(x, wq, s, b, split_k=SPLIT, **kw),),
    }


def _pool_of(ptr):
    """The stream whose pool of torch's allocator holds an address."""
    import torch
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= ptr < segment["address"] + segment["total_size"]:
            return segment["stream"]
    return None


@pytest.mark.parametrize("name", ["mxfp4_linear", "mxfp4a4_linear", "mxfp4_gate_up_swiglu_backward", "qmm_w4a16"])
def test_memory_and_order_of_a_call_on_a_side_stream(lib, name):
    """The current stream is busy and a split call is queued behind that; the same call on an idle side
    stream runs at once, beside it.  Both give what they give alone, with the references dropped and the
    memory asked for again before anything has ended."""
    import torch
    call = _calls(lib)[name]
    x1, x2 = _random((M, K), 5), _random((M, K), 6)
    alone = [[t.clone() for t in call(x)] for x in (x1, x2)]
    busy = _random((4096, 4096), 7, 1 / 64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        announce(f"{name} on a side stream beside a queued one, as {type(stream).__name__}")
        out = busy
        for _ in range(40):
            out = out @ busy
        first = call(x1)
        second = call(x2, stream=stream)
        assert all(_pool_of(t.data_ptr()) == side.cuda_stream for t in second)
        kept = [t.data_ptr() for t in second]
        # outputs are read on the current stream, queued behind what keeps it busy, and dropped
        torch.cuda.current_stream().wait_stream(side)
        copies = [t.clone() for t in second]
        del second
        third = call(x1, stream=stream)
        assert not set(kept) & {t.data_ptr() for t in third}
        torch.cuda.synchronize()
        for got, want in ((first, alone[0]), (copies, alone[1]), (third, alone[0])):
            assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_a_captured_call_on_a_side_stream(lib):
    """Captured on a side stream that forks from the capture and joins it: every replay equals the eager
    result, with eager calls between."""
    import torch
    calls = _calls(lib)
    x = _random((M, K), 8)
    eager = {n: [t.clone() for t in f(x)] for n, f in calls.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    announce("captured calls on a side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = {n: f(x, stream=side) for n, f in calls.items()}
        torch.cuda.current_stream().wait_stream(side)
    for turn in range(3):
        for ts in out.values():
            for t in ts:
                t.zero_()
        graph.replay()
        again = {n: f(x, stream=side) for n, f in calls.items()}
        torch.cuda.synchronize()
        for n in calls:
            assert all(torch.equal(a, b) for a, b in zip(out[n], eager[n])), (n, turn)
            assert all(torch.equal(a, b) for a, b in zip(again[n], eager[n])), (n, turn)


@pytest.mark.parametrize("form", ["object", "handle"])
def test_the_default_stream_given_from_another(lib, form):
    """The default stream, whose handle is 0, given while another one is current."""
    import torch
    call = _calls(lib)["mxfp4_linear"]
    x = _random((M, K), 9)
    alone = call(x)[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    default = torch.cuda.default_stream()
    announce(f"mxfp4_linear on the default stream from another, {form}")
    with torch.cuda.stream(side):
        got, = call(x, stream=default if form == "object" else 0)
        assert _pool_of(got.data_ptr()) == default.cuda_stream == 0
        assert torch.cuda.current_stream() == side
        side.wait_stream(default)
        copy = got.clone()
    torch.cuda.synchronize()
    assert torch.equal(copy, alone)
