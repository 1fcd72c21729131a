"""GPU parity of the int8 products, of one matrix and by experts, against the 64-bit CPU oracle.

Quantization is compared bit for bit.  Products are held to the oracle's bounds (``oracle/experts_oracle.py``): exact
integer sums, fp32 scaling and one rounding to bf16; the transposed products with one rounding of an operand to bf16.
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


def to_gpu(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")
    return t if dtype is None else t.to(dtype)


def bf16(a):
    import torch
    return to_gpu(np.asarray(a, dtype=np.float32), torch.bfloat16)


def values(t):
    return t.float().cpu().numpy().astype(np.float64)


def weight(rng, *shape):
    """Random codes and scales, on the GPU and on the host."""
    codes = rng.integers(-128, 128, shape).astype(np.int8)
    scales = (rng.random(shape[:-1]) * 0.02 + 1e-3).astype(np.float32)
    return (to_gpu(codes), to_gpu(scales)), (codes, scales)


def guarded(M, N, offset=0):
    """A bf16 output [M, N] inside a larger buffer, and a check that its surroundings stay."""
    import torch
    buf = torch.full((M * N + 512,), -77.0, dtype=torch.bfloat16, device="cuda:0")
    y = buf[256 + offset:256 + offset + M * N].view(M, N)

    def untouched():
        return bool((buf[:256 + offset] == -77).all()) and bool((buf[256 + offset + M * N:] == -77).all())
    return y, untouched


def check(got, expected, rows=slice(None)):
    problem = O.within(values(got)[rows], tuple(e[rows] for e in expected))
    assert problem is None, problem


# ---------------------------------------------------------------------------- rows

def check_quantizer(lib, x, kind):
    import torch
    t = to_gpu(x.astype(np.float32), torch.bfloat16 if kind == "bf16" else torch.float32)
    codes, scales = lib.w8a8_quantize_rows(t)
    torch.cuda.synchronize()
    want, want_scales = O.w8_quantize(t.float().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_scales, equal_nan=True)
    got = codes.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:4]


@pytest.mark.parametrize("R,K", [(1, 16), (3, 48), (33, 2560), (130, 400), (2, 9728), (1, 131056)])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_quantize_random_rows(lib, R, K, kind):
    announce(f"w8a8 quantize {R}x{K} {kind}")
    rng = np.random.default_rng(R * K)
    check_quantizer(lib, rng.standard_normal((R, K)) * 10.0 ** rng.integers(-30, 30, (R, 1)), kind)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_quantize_special_rows(lib, kind):
    """Ties, zeros, the smallest and largest rows, infinities and NaN."""
    announce(f"w8a8 quantize special rows {kind}")
    rows = [np.zeros(32), -np.zeros(32), np.full(32, np.inf), np.full(32, np.nan), np.full(32, 2.0 ** -110), np.full(32, 2.0 ** -111),
            np.full(32, -2.0 ** -149), np.full(32, 3.38e38), np.concatenate([[127], np.arange(31) + 0.5]),
            np.concatenate([[-127], -np.arange(31) - 0.5]), np.concatenate([[1e-3, np.inf], np.ones(30)]),
            np.concatenate([np.ones(31), [-np.inf]]), np.concatenate([np.ones(31), [np.nan]]), np.concatenate([[2.0 ** -126], np.zeros(31)])]
    check_quantizer(lib, np.array(rows), kind)


def test_every_bf16_value_quantizes_as_the_format_says(lib):
    announce("w8a8 quantize all bf16 values")
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint32) << 16
    x = bits.view(np.float32).reshape(-1, 16)
    check_quantizer(lib, x, "bf16")


# ---------------------------------------------------------------------------- one matrix

SHAPES = [(1, 8, 16), (1, 151, 2576), (2, 100, 131056), (4, 2560, 9728), (5, 96, 400), (7, 1000, 4096), (16, 4097, 2560), (17, 33, 48),
          (33, 1000, 416), (64, 128, 2560), (100, 3001, 528), (130, 260, 9728), (509, 640, 2560), (600, 2560, 512), (1100, 2400, 272),
          (2048, 4096, 256)]
# reach the other tiles, heights, splits and pieces
FORWARD = [(1000, 4100, 16), (8200, 1000, 16), (3000, 4100, 16), (1000, 4100, 528), (8200, 130, 2576), (8200, 130, 5008),
           (4100, 4100, 16), (4100, 9001, 272)]
BACKWARD = [(513, 2056, 5008), (4100, 33, 1040), (3000, 3001, 144), (8200, 33, 528), (4100, 3001, 144), (3000, 33, 2576),
            (6000, 9001, 16), (8200, 2056, 16), (3000, 33, 5008), (6000, 33, 2576)]


def problem(rng, M, N, K):
    x = rng.standard_normal((M, K)).astype(np.float32)
    w, host = weight(rng, N, K)
    return bf16(x), w, host


@pytest.mark.parametrize("M,N,K", SHAPES + FORWARD)
def test_linear(lib, M, N, K):
    import torch
    announce(f"w8a8_linear {M}x{N}x{K}")
    x, w, host = problem(np.random.default_rng(M + N), M, N, K)
    xq, xs = O.w8_quantize(x.float().cpu().numpy())
    want = O.w8_linear(xq, xs, *host)
    y, untouched = guarded(M, N, 1)
    lib.w8a8_linear(x, *w, y=y)
    torch.cuda.synchronize()
    check(y, want)
    assert untouched()
    # the two calls that it stands for, bit for bit, and an aligned output
    again = lib.qmm_w8a8(*lib.w8a8_quantize_rows(x), *w)
    assert torch.equal(again, y)


@pytest.mark.parametrize("split", [1, 2, 3, 7])
@pytest.mark.parametrize("M,N,K", [(3, 130, 2576), (40, 97, 1040), (300, 512, 400)])
def test_split_products_are_the_same(lib, M, N, K, split):
    import torch
    announce(f"w8a8 split {M}x{N}x{K} S={split}")
    x, w, host = problem(np.random.default_rng(split), M, N, K)
    whole = lib.w8a8_linear(x, *w)
    assert torch.equal(lib.w8a8_linear(x, *w, split_k=split), whole)
    dy = bf16(np.random.default_rng(split + 1).standard_normal((M, N)))
    want = O.w8_linear_backward(values(dy), *host)
    dx = lib.w8a8_linear_backward(dy, *w, split_k=split)
    check(dx, want)
    assert torch.equal(lib.w8a8_linear_backward(dy, *w, split_k=split), dx)


@pytest.mark.parametrize("M,N,K", [s for s in SHAPES if s[2] < 131056] + [(1, 1, 16), (3, 20000, 64)] + BACKWARD)
def test_linear_backward(lib, M, N, K):
    import torch
    announce(f"w8a8_linear_backward {M}x{N}x{K}")
    rng = np.random.default_rng(M * 3 + N)
    w, host = weight(rng, N, K)
    dy = bf16(rng.standard_normal((M, N)))
    dx, untouched = guarded(M, K, 3)
    lib.w8a8_linear_backward(dy, *w, dx=dx)
    torch.cuda.synchronize()
    check(dx, O.w8_linear_backward(values(dy), *host))
    assert untouched()
    assert torch.equal(lib.w8a8_linear_backward(dy, *w), dx)


def test_the_shapes_reach_every_form(lib):
    def forms(op, shapes):
        plans = [lib.w8a8_plan(op, *s) for s in shapes]
        return plans, {(p["variant"], p["tile_m"]) for p in plans if p["path"] == lib.PATH_W8A8}

    plans, forward = forms(lib.W8A8_LINEAR, SHAPES + FORWARD)
    assert {p["variant"] for p in plans if p["path"] == lib.PATH_W8A8_QMV} == {0, 1}
    assert {(0, 128), (1, 192), (1, 256), (2, 64), (3, 128), (5, 128), (10, 128), (11, 256)} <= forward
    assert {2, 3} <= {p["variant"] for p in plans if p["split_k"] > 1 and p["path"] == lib.PATH_W8A8}
    plans, back = forms(lib.W8A8_LINEAR_BACKWARD, SHAPES + BACKWARD)
    assert {(0, 64), (1, 64), (1, 96), (1, 128), (2, 192), (2, 256), (12, 256)} <= back
    assert {p["variant"] for p in plans if p["split_k"] > 1} == {0, 1, 2}


def test_integer_cases_are_exact(lib):
    """Scales of one and sums below 256: every output is exact, in both directions."""
    import torch
    announce("w8a8 integer cases")
    rng = np.random.default_rng(3)
    for M, N, K in ((4, 40, 64), (40, 200, 64), (300, 300, 64)):
        codes = np.zeros((N, K), np.int8)
        codes[np.arange(N), np.arange(N) % K] = rng.integers(-127, 128, N)
        x = np.zeros((M, K), np.float32)
        x[np.arange(M), (np.arange(M) * 7) % K] = 127.0                # scale 1, codes 0 and 127
        y = lib.w8a8_linear(bf16(x), to_gpu(codes), torch.full((N,), 1 / 127, device="cuda"))
        want = x.astype(np.float64) @ codes.T.astype(np.float64)
        assert np.abs(values(y) - want / 127).max() <= 2.0 ** -8 * 127 * 1.001
        dy = np.zeros((M, N), np.float32)
        dy[np.arange(M), (np.arange(M) * 5) % N] = 1.0
        dx = lib.w8a8_linear_backward(bf16(dy), to_gpu(codes), torch.ones(N, device="cuda"))
        assert np.array_equal(values(dx), dy.astype(np.float64) @ codes)


@pytest.mark.parametrize("M", [2, 9, 50])
def test_values_that_are_not_finite_stay_in_their_rows(lib, M):
    """A row with an infinity or NaN gives NaN, a column with such a scale too; all others are as without them."""
    import torch
    announce(f"w8a8 not finite M={M}")
    x, (codes, scales), host = problem(np.random.default_rng(M), M, 70, 96)
    plain = lib.w8a8_linear(x, codes, scales)
    x[1, 5] = float("inf")
    scales = scales.clone()
    scales[69] = float("nan")
    y = lib.w8a8_linear(x, codes, scales)
    assert bool(y[1].isnan().all()) and bool(y[:, 69].isnan().all())
    keep = [m for m in range(M) if m != 1]
    assert torch.equal(y[keep, :69], plain[keep, :69])
    dy = torch.ones(M, 70, dtype=torch.bfloat16, device="cuda")
    clean = lib.w8a8_linear_backward(dy, codes, to_gpu(host[1]))
    dy[1, 3] = float("nan")
    dx = lib.w8a8_linear_backward(dy, codes, to_gpu(host[1]))
    assert bool(dx[1].isnan().all()) and torch.equal(dx[keep], clean[keep])


@pytest.mark.parametrize("M", [1, 20])
def test_the_largest_sums_fit(lib, M):
    """All codes at their ends over the longest contraction: the sum is 128 * 128 * 131056, just below 2^31."""
    import torch
    announce(f"w8a8 largest sums M={M}")
    K = 131056
    xq = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    wq[1] = 127
    wq[2, ::2] = 127
    one = lambda n: torch.ones(n, device="cuda")
    y = values(lib.qmm_w8a8(xq, one(M), wq, one(3)))
    want = np.array([128 * 128 * K, -128 * 127 * K, 64 * K], dtype=np.float64)
    assert (np.abs(y - want) <= want * np.sign(want) * 2.0 ** -8).all()


# ---------------------------------------------------------------------------- experts

def ragged(rng, E, R, kind):
    """Rows of each expert: kinds of raggedness."""
    if kind == "one":
        counts = np.zeros(E, int)
        counts[E // 2] = R
    elif kind == "each":
        counts = np.full(E, R // E)
    elif kind == "gaps":                                     # rows before the first and behind the last stay
        counts = rng.multinomial(R * 3 // 4, rng.dirichlet(np.full(E, 0.3)))
        return np.concatenate([[R // 8], R // 8 + np.cumsum(counts)]).astype(np.int32)
    elif kind == "none":
        counts = np.zeros(E, int)
    else:
        counts = rng.multinomial(R, rng.dirichlet(np.full(E, 0.5)))
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


EXPERTS = [(1, 5, 24, 48, 64, "random"), (4, 7, 14, 100, 96, "random"), (8, 200, 400, 136, 272, "random"), (3, 100, 300, 257, 400, "gaps"),
           (16, 16, 16, 64, 2560, "random"), (64, 3, 24, 1216, 256, "random"), (70, 40, 90, 50, 80, "gaps"), (5, 900, 900, 72, 528, "one"),
           (6, 1300, 2600, 300, 144, "random"), (1000, 30, 60, 24, 32, "random"), (4, 3000, 6000, 520, 64, "each"),
           (2, 40, 40, 33, 16, "none"), (9, 2, 18, 48, 4112, "each"), (128, 60, 240, 80, 9728, "random"),
           (5, 3000, 6000, 520, 1040, "random"), (3, 2100, 4200, 1000, 528, "gaps"), (64, 6000, 12000, 264, 144, "random"),
           (64, 3000, 6000, 1000, 144, "gaps"), (64, 20, 40, 1000, 144, "random"), (64, 3000, 6000, 130, 80, "random"),
           (64, 150, 300, 33, 528, "random"), (64, 3000, 6000, 33, 528, "each")]


def expert_problem(E, T, R, N, K, kind, gather):
    rng = np.random.default_rng(E * 1000 + R)
    offsets = ragged(rng, E, R, kind)
    tokens = rng.integers(0, T, R).astype(np.int32) if gather else None
    if gather and R > 8:
        tokens[[2, 5]] = -1, T                               # no such tokens: activations of zeros
    x = bf16_values(rng.standard_normal((T if gather else R, K)))
    xq, xs = O.w8_quantize(x)
    source = np.arange(R) if tokens is None else tokens
    ok = (source >= 0) & (source < len(x))
    at = np.where(ok, source, 0)
    xq, xs = xq[at] * ok[:, None].astype(np.int8), np.where(ok, xs[at], 0).astype(np.float32)
    return rng, offsets, tokens, bf16(x), xq, xs


def spans(offsets):
    return [(e, slice(int(a), int(b))) for e, (a, b) in enumerate(zip(offsets, offsets[1:])) if b > a]


def per_expert(offsets, R, columns, f):
    """(value, bound) [R, columns] with NaN where no expert has the row."""
    value, bound = np.full((R, columns), np.nan), np.zeros((R, columns))
    for e, s in spans(offsets):
        value[s], bound[s] = f(e, s)
    return value, bound


def check_rows(got, want, offsets, untouched):
    """The experts' rows within their bounds, all others as they were."""
    first, last = int(offsets[0]), int(offsets[-1])
    check(got, want, slice(first, last))
    v = values(got)
    assert (v[:first] == -77).all() and (v[last:] == -77).all() and untouched()


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E,T,R,N,K,kind", EXPERTS)
def test_experts_linear(lib, E, T, R, N, K, kind, gather):
    import torch
    announce(f"w8a8_experts_linear E={E} T={T} R={R} {N}x{K} {kind} gather={gather}")
    rng, offsets, tokens, x, xq, xs = expert_problem(E, T, R, N, K, kind, gather)
    w, (codes, scales) = weight(rng, E, N, K)
    y, untouched = guarded(R, N, 1)
    o, t = to_gpu(offsets), None if tokens is None else to_gpu(tokens)
    y.fill_(-77)
    lib.w8a8_experts_linear(x, *w, o, t, y=y)
    torch.cuda.synchronize()
    check_rows(y, per_expert(offsets, R, N, lambda e, s: O.w8_linear(xq[s], xs[s], codes[e], scales[e])), offsets, untouched)
    dy = bf16(rng.standard_normal((R, N)))
    dx, untouched = guarded(R, K, 1)
    lib.w8a8_experts_linear_backward(dy, *w, o, dx=dx)
    torch.cuda.synchronize()
    check_rows(dx, per_expert(offsets, R, K, lambda e, s: O.w8_linear_backward(values(dy)[s], codes[e], scales[e])), offsets, untouched)


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E,T,R,N,K,kind", EXPERTS)
def test_experts_gate_up(lib, E, T, R, N, K, kind, gather):
    import torch
    announce(f"w8a8_experts_gate_up E={E} T={T} R={R} {N}x{K} {kind} gather={gather}")
    rng, offsets, tokens, x, xq, xs = expert_problem(E, T, R, N, K, kind, gather)
    (gate, hg), (up, hu) = weight(rng, E, N, K), weight(rng, E, N, K)
    o, t = to_gpu(offsets), None if tokens is None else to_gpu(tokens)
    pick = lambda e: ((hg[0][e], hg[1][e]), (hu[0][e], hu[1][e]))
    h, untouched = guarded(R, N, 1)
    lib.w8a8_experts_gate_up_swiglu(x, gate, up, o, t, h=h)
    torch.cuda.synchronize()
    check_rows(h, per_expert(offsets, R, N, lambda e, s: O.w8_gate_up(xq[s], xs[s], *pick(e))), offsets, untouched)
    dh = bf16(rng.standard_normal((R, N)))
    outs = [guarded(R, c, off) for c, off in ((K, 3), (N, 5), (N, 2))]
    lib.w8a8_experts_gate_up_swiglu_backward(x, gate, up, dh, o, t, *(y for y, _ in outs))
    torch.cuda.synchronize()
    for i, ((got, untouched), columns) in enumerate(zip(outs, (K, N, N))):
        want = per_expert(offsets, R, columns, lambda e, s: O.w8_gate_up_backward(xq[s], xs[s], *pick(e), values(dh)[s])[i])
        check_rows(got, want, offsets, untouched)


def test_the_experts_shapes_reach_every_form(lib):
    reached = {"W8A8_EXPERTS_LINEAR": {1, 2, 3, 4, 5}, "W8A8_EXPERTS_LINEAR_BACKWARD": {0, 1, 2}, "W8A8_EXPERTS_GATE_UP": {0, 1, 2, 3, 4},
               "W8A8_EXPERTS_GATE_UP_BACKWARD": {0, 1, 2}}
    for op, forms in reached.items():
        plans = [lib.w8a8_plan(getattr(lib, op), T, N, K, 0, 0, E, R) for E, T, R, N, K, _ in EXPERTS]
        assert all(p["path"] == lib.PATH_W8A8 for p in plans)
        assert forms <= {p["variant"] for p in plans}, op


@pytest.mark.parametrize("R", [12, 600])
def test_offsets_that_make_no_sense_stay_inside_the_buffers(lib, R):
    """Offsets below 0, above R, falling: nothing outside the outputs is written, what is well-formed is right."""
    import torch
    announce(f"w8a8 experts, senseless offsets, R={R}")
    rng = np.random.default_rng(R)
    w, (codes, scales) = weight(rng, 4, 40, 64)
    x = bf16(rng.standard_normal((R, 64)))
    xq, xs = O.w8_quantize(x.float().cpu().numpy())
    offsets = to_gpu(np.array([-5, R // 2, R // 4, R // 4, R + 1000], np.int32))
    y, untouched = guarded(R, 40, 1)
    lib.w8a8_experts_linear(x, *w, offsets, y=y)
    dx, untouched_dx = guarded(R, 64, 1)
    lib.w8a8_experts_linear_backward(y.contiguous().clone(), *w, offsets, dx=dx)
    h, untouched_h = guarded(R, 40, 1)
    lib.w8a8_experts_gate_up_swiglu(x, w, w, offsets, h=h)
    torch.cuda.synchronize()
    assert untouched() and untouched_dx() and untouched_h()
    check(y, O.w8_linear(xq, xs, codes[0], scales[0]), slice(0, R // 4))
    check(y, O.w8_linear(xq, xs, codes[3], scales[3]), slice(R // 2, R))


def test_offsets_whose_tiles_pass_31_bits(lib):
    """Falling offsets give 512 experts 2^28 rows each, 2^31 tiles of 64 rows: only as many as the grid holds are taken."""
    import torch
    announce("w8a8 experts, tiles past 31 bits")
    E, R, K = 1024, 1 << 28, 16
    w, _ = weight(np.random.default_rng(8), 1, K)
    x = bf16(np.random.default_rng(9).standard_normal((1, K)))
    tokens = torch.zeros(R, dtype=torch.int32, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1::2] = R
    y, untouched = guarded(R, 1)
    lib.w8a8_experts_linear(x, w[0].expand(E, 1, K).contiguous(), w[1].expand(E, 1).contiguous(), offsets, tokens, y=y)
    torch.cuda.synchronize()
    assert bool((y == lib.w8a8_linear(x, *w)).all()) and untouched()


def test_weights_past_four_gigabytes(lib):
    """The last of 130 experts starts beyond 2^32 bytes."""
    import torch
    announce("w8a8 experts past 4 GiB")
    E, N, K, R = 130, 4096, 8192, 40
    codes = torch.zeros(E, N, K, dtype=torch.int8, device="cuda")
    rng = np.random.default_rng(4)
    w, host = weight(rng, N, K)
    codes[-1] = w[0]
    scales = torch.ones(E, N, device="cuda")
    scales[-1] = w[1]
    x = bf16(rng.standard_normal((R, K)))
    xq, xs = O.w8_quantize(x.float().cpu().numpy())
    for rows in (R, 3):
        offsets = to_gpu(np.array([0] * E + [rows], np.int32))
        y = lib.w8a8_experts_linear(x[:rows].contiguous(), codes, scales, offsets)
        check(y, O.w8_linear(xq[:rows], xs[:rows], *host))
    dy = bf16(rng.standard_normal((R, N)))
    dx = lib.w8a8_experts_linear_backward(dy, codes, scales, to_gpu(np.array([0] * E + [R], np.int32)))
    check(dx, O.w8_linear_backward(values(dy), *host))


def test_outputs_past_two_to_the_31(lib):
    """y of 36864 x 60000 has 2.2e9 elements; rows beyond 2^31 elements against rows alone."""
    import torch
    announce("w8a8 outputs past 2^31")
    M, N, K = 36864, 60000, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    w = lib.w8a8_quantize_rows(torch.randn(N, K, device="cuda", generator=g))
    y = lib.w8a8_linear(x, *w)
    assert torch.equal(y[-40:], lib.w8a8_linear(x[-40:].contiguous(), *w))
    offsets = torch.tensor([0, 36000, M], dtype=torch.int32, device="cuda")
    two = (torch.stack([w[0], w[0]]), torch.stack([w[1], w[1]]))
    again = lib.w8a8_experts_linear(x, *two, offsets)
    assert torch.equal(again[-40:], y[-40:])


# ---------------------------------------------------------------------------- gradients, streams, graphs

def test_gradients_against_differences(lib):
    """On activations that are codes exactly (scale 1), y is linear: y(x + d) - y(x) = dx's row times d."""
    import torch
    announce("w8a8 gradients against differences")
    rng = np.random.default_rng(12)
    N, K = 24, 64
    (codes, scales), host = weight(rng, N, K)
    base = rng.integers(-100, 100, K).astype(np.float32)
    base[0] = 127.0                                          # the row's scale stays 1
    x = np.tile(base, (K, 1))
    x[np.arange(1, K), np.arange(1, K)] += 8.0
    y = values(lib.w8a8_linear(bf16(x), codes, scales))
    v = bf16_values(rng.standard_normal((1, N)))
    dx = values(lib.w8a8_linear_backward(bf16(v), codes, scales))[0]
    w = host[0] * host[1][:, None].astype(np.float64)
    error = O.w8_linear_backward(v, *host)[1][0]
    for k in range(1, K):
        diff = ((y[k] - y[0]) * v[0]).sum() / 8.0
        # each y is off by half a step of bf16
        slack = (np.abs(v[0]) * (np.abs(y[k]) + np.abs(y[0]))).sum() * 2.0 ** -8 / 8.0 * 1.01
        assert abs(diff - dx[k]) <= slack + error[k]
        assert abs((v @ w)[0, k] - dx[k]) <= error[k]


def _calls(lib):
    """Every call with its inputs, as functions of ``kw``."""
    rng = np.random.default_rng(20)
    E, T, R, N, K = 6, 150, 300, 200, 528
    _, offsets, tokens, x, _, _ = expert_problem(E, T, R, N, K, "random", True)
    o, t = to_gpu(offsets), to_gpu(tokens)
    gate, up, one = weight(rng, E, N, K)[0], weight(rng, E, N, K)[0], weight(rng, N, K)[0]
    dh, dy = bf16(rng.standard_normal((R, N))), bf16(rng.standard_normal((T, N)))
    few = x[:3].contiguous()
    logits = bf16(rng.standard_normal((T, 40)))
    chosen = lib.experts_route(logits, 3)
    rows = bf16(rng.standard_normal((3 * T, N)))
    return {
        "route": lambda **kw: lib.experts_route(logits, 3, **kw),
        "route backward": lambda **kw: (lib.experts_route_backward(logits, chosen[1], chosen[0], **kw),),
        "combine": lambda **kw: (lib.experts_combine(rows, chosen[2], chosen[0], **kw),),
        "combine backward": lambda **kw: lib.experts_combine_backward(dy, rows, chosen[2], chosen[0], **kw),
        "quantize": lambda **kw: lib.w8a8_quantize_rows(x, **kw),
        "linear": lambda **kw: (lib.w8a8_linear(x, *one, **kw),),
        "linear few": lambda **kw: (lib.w8a8_linear(few, *one, **kw),),
        "linear split": lambda **kw: (lib.w8a8_linear(x, *one, split_k=3, **kw),),
        "backward": lambda **kw: (lib.w8a8_linear_backward(dy, *one, split_k=2, **kw),),
        "experts": lambda **kw: (lib.w8a8_experts_linear(x, *gate, o, t, **kw)[:int(offsets[-1])],),
        "experts backward": lambda **kw: (lib.w8a8_experts_linear_backward(dh, *gate, o, **kw)[:int(offsets[-1])],),
        "gate_up": lambda **kw: (lib.w8a8_experts_gate_up_swiglu(x, gate, up, o, t, **kw)[:int(offsets[-1])],),
        "gate_up backward": lambda **kw: [v[:int(offsets[-1])] for v in lib.w8a8_experts_gate_up_swiglu_backward(
            x, gate, up, dh, o, t, **kw)],
    }


def test_captured_calls_replay(lib):
    """Two graphs of every call replayed in turn with eager calls between: each replay equals the eager result."""
    import torch
    calls = _calls(lib)
    eager = {n: [t.clone() for t in f()] for n, f in calls.items()}
    torch.cuda.synchronize()
    announce("w8a8 captured calls")
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = {n: f() for n, f in calls.items()}
        graphs.append((g, out))
    for turn in range(4):
        g, out = graphs[turn % 2]
        for ts in out.values():
            for t in ts:
                t.zero_()
        g.replay()
        again = {n: f() for n, f in calls.items()}
        torch.cuda.synchronize()
        for n in calls:
            assert all(torch.equal(a, b) for a, b in zip(out[n], eager[n])), (n, turn)
            assert all(torch.equal(a, b) for a, b in zip(again[n], eager[n])), (n, turn)


def test_calls_on_two_streams_at_once(lib):
    import torch
    calls = _calls(lib)
    alone = {n: [t.clone() for t in f()] for n, f in calls.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    announce("w8a8 two streams")
    for _ in range(3):
        first = {n: f() for n, f in calls.items()}
        second = {n: f(stream=side) for n, f in calls.items()}
        torch.cuda.synchronize()
        for n in calls:
            assert all(torch.equal(a, b) for a, b in zip(first[n], alone[n])), n
            assert all(torch.equal(a, b) for a, b in zip(second[n], alone[n])), n


def test_given_workspaces(lib):
    """A given workspace is used; a short one drops a policy split or is refused, before any launch."""
    import torch
    announce("w8a8 workspaces")
    rng = np.random.default_rng(30)
    x, w, _ = problem(rng, 130, 260, 9728)
    plan = lib.w8a8_plan(lib.W8A8_LINEAR, 130, 260, 9728)
    assert plan["split_k"] > 1
    whole = lib.w8a8_linear(x, *w)
    fixed = lib.w8a8_plan(lib.W8A8_LINEAR, 130, 260, 9728, 1)["workspace_bytes"]
    for nbytes in (plan["workspace_bytes"], plan["workspace_bytes"] - 16, fixed):
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        assert torch.equal(lib.w8a8_linear(x, *w, workspace=ws), whole)
    with pytest.raises(ValueError):
        lib.w8a8_linear(x, *w, workspace=torch.empty(fixed - 16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        lib.w8a8_linear(x, *w, split_k=2, workspace=torch.empty(fixed, dtype=torch.uint8, device="cuda"))
