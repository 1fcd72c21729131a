"""GPU tests of sizes at the limits of the int8 and experts' operators: rows that repeat, against the same rows alone."""

import numpy as np
import pytest

from gpu_helpers import announce
from test_gpu_w8a8 import bf16, to_gpu, weight

pytestmark = pytest.mark.gpu

ROWS = (1 << 24) + 40          # three launches of the quantizer, the last one of 40 rows


def repeated(block, rows):
    """``rows`` rows: the block's over and over."""
    return block.repeat(-(-rows // len(block)), 1)[:rows].contiguous()


def same(got, block):
    """Whole blocks are equal, and what is left is the block's beginning."""
    import torch
    n = len(got) // len(block)
    whole = got[:n * len(block)].view(n, *block.shape)
    return torch.equal(whole, block.expand_as(whole)) and torch.equal(got[n * len(block):], block[:len(got) - n * len(block)])


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_rows_past_two_to_the_24_are_quantized(lib, kind):
    announce(f"w8a8_quantize_rows, 2^24 rows, {kind}")
    block = to_gpu(np.random.default_rng(1).standard_normal((1000, 16)).astype(np.float32))
    block = bf16(block.cpu().numpy()) if kind == "bf16" else block
    codes, scales = lib.w8a8_quantize_rows(block)
    got = lib.w8a8_quantize_rows(repeated(block, ROWS))
    assert same(got[0], codes) and same(got[1].view(-1, 1), scales.view(-1, 1))


def test_products_of_rows_past_two_to_the_24(lib):
    """One expert after the other, forward and backward, and the product of codes and the gradient of one matrix."""
    import torch
    announce("w8a8 products, 2^24 rows")
    rng = np.random.default_rng(2)
    N, K = 8, 16
    w, _ = weight(rng, N, K)
    x, dy = bf16(rng.standard_normal((1000, K))), bf16(rng.standard_normal((1000, N)))
    y, dx = lib.w8a8_linear(x, *w), lib.w8a8_linear_backward(dy, *w)
    many, many_dy = repeated(x, ROWS), repeated(dy, ROWS)
    two = torch.stack([w[0], w[0]]), torch.stack([w[1], w[1]])
    offsets = to_gpu(np.array([0, 1 << 23, ROWS], np.int32))
    assert same(lib.w8a8_experts_linear(many, *two, offsets), y)
    assert same(lib.w8a8_experts_linear_backward(many_dy, *two, offsets), dx)
    assert same(lib.w8a8_linear_backward(many_dy, *w), dx)
    assert same(lib.qmm_w8a8(*lib.w8a8_quantize_rows(many), *w), y)
    h, alone = lib.w8a8_experts_gate_up_swiglu(many, two, two, offsets), to_gpu(np.array([0, 0, 1000], np.int32))
    assert same(h, lib.w8a8_experts_gate_up_swiglu(x, two, two, alone))
    for got, want in zip(lib.w8a8_experts_gate_up_swiglu_backward(many, two, two, many_dy, offsets),
                         lib.w8a8_experts_gate_up_swiglu_backward(x, two, two, dy, alone)):
        assert same(got, want)


def test_a_combination_of_two_to_the_26_pairs(lib):
    announce("experts_combine, 2^26 pairs")
    rng = np.random.default_rng(3)
    T, top = (1 << 23) + 11, 8
    for N in (8, 3):
        y = bf16(rng.standard_normal((500, N)))
        positions, weights = to_gpu(rng.integers(-1, 500, (1000, top)).astype(np.int32)), to_gpu(rng.random((1000, top)).astype(np.float32))
        out = lib.experts_combine(y, repeated(positions, T), repeated(weights, T))
        assert same(out, lib.experts_combine(y, positions, weights))


def test_the_largest_gradient_of_a_combination(lib):
    import torch
    announce("experts_combine_backward, 2^26 - 8 pairs")
    rng = np.random.default_rng(4)
    T, top, N = (1 << 23) - 1, 8, 8
    y, dout, weights = bf16(rng.standard_normal((8000, N))), bf16(rng.standard_normal((1000, N))), to_gpu(rng.random((1000, top)).astype(np.float32))
    positions = torch.arange(T * top, dtype=torch.int32, device="cuda").view(T, top)
    dy, dweights = lib.experts_combine_backward(repeated(dout, T), repeated(y, T * top), positions, repeated(weights, T))
    want_dy, want_dweights = lib.experts_combine_backward(dout, y, positions[:1000], weights)
    assert same(dy, want_dy) and same(dweights, want_dweights)
