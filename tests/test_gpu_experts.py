"""GPU parity of the router and the combination of experts against the 64-bit CPU oracle, and a whole block of a
mixture of experts, forward and backward.

Experts, positions, tokens and offsets are compared exactly; weights and gradients within the oracle's bounds.
"""

import numpy as np
import pytest

import oracle as O

from gpu_helpers import announce
from test_gpu_w8a8 import bf16, bf16_values, check, guarded, spans, to_gpu, values, weight

pytestmark = pytest.mark.gpu


def host(t):
    return t.cpu().numpy()


def make_logits(rng, T, E, kind):
    logits = rng.standard_normal((T, E)).astype(np.float32)
    if kind == "ties":
        logits = np.round(logits)
        logits[logits == 0] *= rng.choice([-1.0, 1.0], (logits == 0).sum())     # zeros of both signs
    elif kind == "masked":
        logits[rng.random((T, E)) < 0.7] = -np.inf
        logits[T // 2] = -np.inf
    elif kind == "wide":
        logits *= 60
    elif kind == "close":                                     # apart in the lowest bits alone, some rows only at the border
        logits[::2] = 1 + rng.integers(0, 300, logits[::2].shape) * np.float32(2.0 ** -23)
        logits[1::2] = np.float32(-3) - np.argsort(rng.random(logits[1::2].shape), 1) * np.float32(2.0 ** -16)
    elif kind == "bf16":
        logits = bf16_values(logits).astype(np.float32)
    return logits


def compare(got, want, bound):
    problem = O.within(host(got).astype(np.float64), (want, bound))
    assert problem is None, problem


ROUTES = [(1, 1, 1, "plain"), (1, 60, 4, "plain"), (5, 60, 4, "bf16"), (3, 8, 8, "masked"), (64, 64, 6, "ties"), (65, 64, 2, "masked"),
          (63, 65, 8, "bf16"), (130, 128, 1, "plain"), (300, 256, 8, "ties"), (1000, 5, 3, "masked"), (257, 512, 10, "wide"),
          (100, 1000, 8, "bf16"), (70, 1024, 64, "plain"), (2100, 3, 2, "ties"), (4161, 40, 8, "bf16"),
          (75, 1024, 10, "bf16"), (9, 1000, 5, "ties"), (80, 600, 16, "masked"), (66, 200, 40, "close"), (66, 700, 33, "bf16"),
          (90, 256, 8, "close"), (20, 16, 16, "close"), (70, 1024, 9, "close"), (33, 100, 3, "close")]


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,top,kind", ROUTES)
def test_route_and_its_gradient(lib, T, E, top, kind, renormalize):
    import torch
    announce(f"experts_route {T}x{E} top {top} {kind} renormalize={renormalize}")
    rng = np.random.default_rng(T + E)
    logits = make_logits(rng, T, E, kind)
    t = bf16(logits) if kind == "bf16" else to_gpu(logits)
    weights, experts, positions, tokens, offsets = lib.experts_route(t, top, renormalize)
    torch.cuda.synchronize()
    (w, wb), e, p, k, o = O.route_reference(logits.astype(np.float64), top, renormalize)
    assert np.array_equal(host(experts), e)
    assert np.array_equal(host(offsets), o)
    assert np.array_equal(host(tokens), k)
    assert np.array_equal(host(positions), p)
    compare(weights, w, wb)
    dw = rng.standard_normal((T, top)).astype(np.float32)
    d = lib.experts_route_backward(t, experts, to_gpu(dw), renormalize)
    want, bound = O.route_backward_reference(logits.astype(np.float64), e, dw.astype(np.float64), renormalize)
    if kind == "bf16":
        bound = bound + (np.abs(want) + bound) * 2.0 ** -8
    compare(d.float(), want, bound)


def test_route_of_logits_that_are_not_finite(lib):
    """NaN is never chosen and makes the token's weights NaN; an infinity is chosen first."""
    import torch
    announce("experts_route, not finite")
    logits = np.random.default_rng(1).standard_normal((70, 20)).astype(np.float32)
    logits[3, 4] = np.nan
    logits[5] = np.nan
    logits[7, 11] = np.inf
    logits[9, :18] = -np.inf
    logits[66, 2] = np.nan
    for T in (20, 70):
        for renormalize in (True, False):
            w, e, p, k, o = lib.experts_route(to_gpu(logits[:T]), 4, renormalize)
            (want, bound), we, wp, wk, wo = O.route_reference(logits[:T].astype(np.float64), 4, renormalize)
            for got, ref in ((e, we), (p, wp), (k, wk), (o, wo)):
                assert np.array_equal(host(got), ref)
            finite = [t for t in range(T) if t != 7]
            compare(w[finite], want[finite], bound[finite])
            assert host(e)[7, 0] == 11 and np.isnan(host(w)[7, 0]) and host(e)[5].tolist() == [-1] * 4
            d = host(lib.experts_route_backward(to_gpu(logits[:T]), e, torch.ones_like(w), renormalize))
            assert np.isnan(d[3]).all() and np.isnan(d[5]).all() and (d[9, :18] == 0).all()


def test_route_writes_nothing_outside(lib):
    import torch
    announce("experts_route, surroundings")
    for T, E, top in ((5, 9, 3), (200, 65, 7)):
        logits = to_gpu(np.random.default_rng(T).standard_normal((T, E)).astype(np.float32))
        sizes = {"weights": (T, top), "experts": (T, top), "positions": (T, top), "tokens": (T * top,), "offsets": (E + 1,)}
        buffers, views = {}, {}
        for n, shape in sizes.items():
            dtype = torch.float32 if n == "weights" else torch.int32
            count = int(np.prod(shape))
            buffers[n] = torch.full((count + 9,), -77, dtype=dtype, device="cuda")
            views[n] = buffers[n][4:4 + count].view(shape)
        lib.experts_route(logits, top, **views)
        for got, want in zip(views.values(), lib.experts_route(logits, top)):
            assert torch.equal(got, want)
        for n, b in buffers.items():
            assert bool((b[:4] == -77).all()) and bool((b[4 + views[n].numel():] == -77).all()), n


def make_positions(rng, T, top, R):
    """Distinct rows in random order, some missing, some out of range."""
    flat = np.full(T * top, -1, np.int32)
    count = min(T * top, R)
    flat[rng.permutation(T * top)[:count]] = rng.permutation(R)[:count]
    flat[rng.random(T * top) < 0.1] = -1
    flat[rng.random(T * top) < 0.05] = R
    return flat.reshape(T, top)


@pytest.mark.parametrize("T,top,R,N", [(1, 1, 1, 1), (5, 4, 20, 2560), (3, 2, 9, 13), (64, 8, 512, 128), (200, 3, 640, 1001), (7, 64, 448, 72),
                                       (1030, 2, 2060, 8)])
def test_combine_and_its_gradients(lib, T, top, R, N):
    import torch
    announce(f"experts_combine T={T} top={top} R={R} N={N}")
    rng = np.random.default_rng(T + N)
    y, dout = bf16_values(rng.standard_normal((R, N))), bf16_values(rng.standard_normal((T, N)))
    w, positions = rng.random((T, top)).astype(np.float32), make_positions(rng, T, top, R)
    for offset in (0, 1):                                     # rows of whole 16 bytes, and others
        out, untouched = guarded(T, N, offset)
        lib.experts_combine(bf16(y), to_gpu(positions), to_gpu(w), out=out)
        check(out, O.combine_reference(y, positions, w))
        assert untouched()
        lib.experts_combine(bf16(y), to_gpu(positions), out=out)
        check(out, O.combine_reference(y, positions))
        dy, untouched = guarded(R, N, offset)
        dy.fill_(-77)
        _, dw = lib.experts_combine_backward(bf16(dout), bf16(y), to_gpu(positions), to_gpu(w), dy=dy)
        (want, bound), (want_dw, bound_dw) = O.combine_backward_reference(dout, y, positions, w)
        reached = ~np.isnan(want).any(1)
        check(dy, (want, bound), reached)
        assert (values(dy)[~reached] == -77).all() and untouched()
        compare(dw, want_dw, bound_dw)


def test_rows_of_no_token_do_not_reach_the_sum(lib):
    """NaN and infinities in rows at no position, and a token with no rows."""
    import torch
    announce("experts_combine, rows of no token")
    y = torch.full((6, 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    y[2], y[4] = 1.0, 2.0
    positions = to_gpu(np.array([[2, -1], [-1, -1], [4, 6], [-5, 2]], np.int32))
    out = values(lib.experts_combine(y, positions))
    assert np.array_equal(out, np.repeat([[1.0], [0.0], [2.0], [1.0]], 40, 1))
    weights = torch.full((4, 2), float("nan"), device="cuda")
    weights[0, 0] = weights[2, 0] = weights[3, 1] = 3.0
    assert np.array_equal(values(lib.experts_combine(y, positions, weights))[:, 0], [3.0, 0.0, 6.0, 3.0])


def block(lib, x, logits, gate, up, down, top, dout=None):
    """A block of a mixture of experts as a user writes it, and its backward pass."""
    weights, experts, positions, tokens, offsets = lib.experts_route(logits, top)
    h = lib.w8a8_experts_gate_up_swiglu(x, gate, up, offsets, tokens)
    y = lib.w8a8_experts_linear(h, *down, offsets)
    out = lib.experts_combine(y, positions, weights)
    if dout is None:
        return out
    dy, dweights = lib.experts_combine_backward(dout, y, positions, weights)
    dlogits = lib.experts_route_backward(logits, experts, dweights)
    dh = lib.w8a8_experts_linear_backward(dy, *down, offsets)
    rows, dgate, dup = lib.w8a8_experts_gate_up_swiglu_backward(x, gate, up, dh, offsets, tokens)
    dx = lib.experts_combine(rows, positions)
    return dict(weights=weights, experts=experts, positions=positions, tokens=tokens, offsets=offsets, h=h, y=y, out=out, dy=dy,
                dweights=dweights, dlogits=dlogits, dh=dh, rows=rows, dgate=dgate, dup=dup, dx=dx)


def block_problem(E, T, F, K, seed):
    rng = np.random.default_rng(seed)
    x, logits = bf16_values(rng.standard_normal((T, K))), rng.standard_normal((T, E)).astype(np.float32)
    weights = [weight(rng, E, F, K), weight(rng, E, F, K), weight(rng, E, K, F)]
    return rng, x, logits, weights, bf16_values(rng.standard_normal((T, K)))


@pytest.mark.parametrize("E,T,F,K,top", [(4, 3, 32, 64, 2), (8, 1, 80, 96, 8), (16, 100, 208, 144, 4), (6, 700, 96, 272, 2)])
def test_a_block_forward_and_backward(lib, E, T, F, K, top):
    """Each step against the oracle on what the step before it gave."""
    import torch
    announce(f"experts block E={E} T={T} F={F} K={K} top={top}")
    rng, x, logits, ((gate, hg), (up, hu), (down, hd)), dout = block_problem(E, T, F, K, E + T)
    r = block(lib, bf16(x), to_gpu(logits), gate, up, down, top, bf16(dout))
    torch.cuda.synchronize()
    positions, tokens, offsets = host(r["positions"]), host(r["tokens"]), host(r["offsets"])
    assert offsets[-1] == T * top
    xq, xs = (v[tokens] for v in O.w8_quantize(x))
    hq, hs = O.w8_quantize(values(r["h"]))
    v = {n: values(t) for n, t in r.items()}
    for e, s in spans(offsets):
        g, u, d = (hg[0][e], hg[1][e]), (hu[0][e], hu[1][e]), (hd[0][e], hd[1][e])
        check(r["h"][s], O.w8_gate_up(xq[s], xs[s], g, u))
        check(r["y"][s], O.w8_linear(hq[s], hs[s], *d))
        check(r["dh"][s], O.w8_linear_backward(v["dy"][s], *d))
        for n, want in zip(("rows", "dgate", "dup"), O.w8_gate_up_backward(xq[s], xs[s], g, u, v["dh"][s])):
            check(r[n][s], want)
    check(r["out"], O.combine_reference(v["y"], positions, v["weights"]))
    dy, dw = O.combine_backward_reference(dout, v["y"], positions, v["weights"])
    check(r["dy"], dy)
    compare(r["dweights"], *dw)
    compare(r["dlogits"], *O.route_backward_reference(logits.astype(np.float64), host(r["experts"]), v["dweights"]))
    check(r["dx"], O.combine_reference(v["rows"], positions))


@pytest.mark.parametrize("T", [6, 200])
def test_a_padded_batch(lib, T):
    """Tokens of padding, all logits minus infinity and x and dout NaN, reach no expert: the others' results are those of a
    batch without them, theirs zeros."""
    import torch
    announce(f"experts block, padded, T={T}")
    _, x, logits, ((gate, _), (up, _), (down, _)), dout = block_problem(8, T, 48, 96, 3 * T)
    real = np.flatnonzero(np.arange(T) % 3 != 1)
    padding = np.setdiff1d(np.arange(T), real)
    alone = block(lib, bf16(x[real]), to_gpu(logits[real]), gate, up, down, 2, bf16(dout[real]))
    x[padding] = dout[padding] = np.nan
    logits[padding] = -np.inf
    r = block(lib, bf16(x), to_gpu(logits), gate, up, down, 2, bf16(dout))
    rows = len(real) * 2
    assert int(r["offsets"][-1]) == rows and (host(r["experts"])[padding] == -1).all()
    for n in ("h", "y", "dy", "dh", "rows", "dgate", "dup"):
        assert torch.equal(r[n][:rows], alone[n]), n
    for n in ("out", "dx", "weights", "dlogits", "dweights"):
        assert torch.equal(r[n][to_gpu(real)], alone[n]), n
        assert bool((r[n][to_gpu(padding)] == 0).all()), n


@pytest.mark.parametrize("kind", ["plain", "bf16"])
@pytest.mark.parametrize("E", [16, 64, 256])
def test_logits_at_any_alignment(lib, E, kind):
    """Logits and their gradient one value behind a whole 16 bytes, against the same at the start of an allocation."""
    import torch
    announce(f"experts_route alignment E={E} {kind}")
    T, top = 100, 5
    values = torch.from_numpy(np.random.default_rng(E).standard_normal(T * E + 1).astype(np.float32)).cuda()
    values = values.to(torch.bfloat16) if kind == "bf16" else values
    shifted, whole = values[1:].view(T, E), values[1:].clone().view(T, E)
    for renormalize in (True, False):
        want = lib.experts_route(whole, top, renormalize)
        for got, ref in zip(lib.experts_route(shifted, top, renormalize), want):
            if ref.dtype is torch.float32:
                # (the sums of the softmax in another order: 256 terms)
                assert torch.allclose(got, ref, rtol=260 * 2.0 ** -24, atol=0)
            else:
                assert torch.equal(got, ref)
        dw = torch.rand(T, top, device="cuda")
        out = torch.full((T * E + 9,), -77.0, dtype=values.dtype, device="cuda")
        lib.experts_route_backward(shifted, want[1], dw, renormalize, dlogits=out[1:1 + T * E].view(T, E))
        assert bool((out[:1] == -77).all()) and bool((out[1 + T * E:] == -77).all())
        reference, bound = O.route_backward_reference(whole.double().cpu().numpy(), host(want[1]), dw.double().cpu().numpy(), renormalize)
        if kind == "bf16":
            bound = bound + (np.abs(reference) + bound) * 2.0 ** -8
        compare(out[1:1 + T * E].view(T, E).float(), reference, bound)


def test_a_block_in_an_autograd_function(lib):
    """The block as a torch.autograd.Function: its gradients are the calls', eager and captured, forward and backward."""
    import torch
    announce("experts block, autograd")
    _, x, logits, ((gate, _), (up, _), (down, _)), dout = block_problem(8, 90, 64, 96, 5)

    class Block(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, logits):
            ctx.save_for_backward(x, logits)
            return block(lib, x, logits, gate, up, down, 2)

        @staticmethod
        def backward(ctx, dout):
            r = block(lib, *ctx.saved_tensors, gate, up, down, 2, dout.contiguous())
            return r["dx"], r["dlogits"]

    x, logits, dout = bf16(x), to_gpu(logits), bf16(dout)
    want = block(lib, x, logits, gate, up, down, 2, dout)
    for leaf in ((x, logits), (x.clone(), logits.clone())):
        a, b = (t.detach().clone().requires_grad_() for t in leaf)
        out = Block.apply(a, b)
        assert torch.equal(out, want["out"])
        out.backward(dout)
        assert torch.equal(a.grad, want["dx"]) and torch.equal(b.grad, want["dlogits"])
    with pytest.raises(ValueError, match="requires a gradient"):
        lib.experts_route(logits.clone().requires_grad_(), 2)
    del a, b, out

    # captured: leaves of its own, that no eager graph holds
    leaves = [t.clone().requires_grad_() for t in (x, logits)]

    def step():
        result = Block.apply(*leaves)
        return (result.detach(), *torch.autograd.grad(result, leaves, dout))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    g = torch.Generator(device="cuda").manual_seed(6)
    for _ in range(3):
        with torch.no_grad():
            for t in leaves:
                t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        graph.replay()
        want = block(lib, *(t.detach() for t in leaves), gate, up, down, 2, dout)
        torch.cuda.synchronize()
        for got, n in zip(captured, ("out", "dx", "dlogits")):
            assert torch.equal(got, want[n]), n


def test_a_block_captured_and_replayed_with_new_inputs(lib):
    """Routing is made on the device, so a captured block follows its inputs: every replay equals the eager block."""
    import torch
    announce("experts block, captured")
    for T in (4, 150):
        _, x, logits, ((gate, _), (up, _), (down, _)), dout = block_problem(8, T, 64, 96, T)
        x, logits, dout = bf16(x), to_gpu(logits), bf16(dout)
        block(lib, x, logits, gate, up, down, 2, dout)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = block(lib, x, logits, gate, up, down, 2, dout)
        g = torch.Generator(device="cuda").manual_seed(T)
        for turn in range(3):
            x.copy_(torch.randn(x.shape, device="cuda", generator=g))
            logits.copy_(torch.randn(logits.shape, device="cuda", generator=g))
            if turn == 1:
                logits[:, 5] += 20.0                          # nearly everything to one expert
            graph.replay()
            want = block(lib, x, logits, gate, up, down, 2, dout)
            torch.cuda.synchronize()
            for n in want:
                assert torch.equal(out[n], want[n]), (n, turn)


def test_a_call_repeats_bit_for_bit(lib):
    import torch
    announce("experts block, repeated")
    _, x, logits, ((gate, _), (up, _), (down, _)), dout = block_problem(16, 300, 96, 128, 9)
    x, logits, dout = bf16(x), to_gpu(logits), bf16(dout)
    first = block(lib, x, logits, gate, up, down, 4, dout)
    for _ in range(3):
        again = block(lib, x, logits, gate, up, down, 4, dout)
        assert all(torch.equal(first[n], again[n]) for n in first)
