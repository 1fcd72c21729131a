"""Sizes at the limits of the int8 and experts' operators, without a GPU."""

import pytest

import w4a16_group_quantized_qmv_amd as w4

from test_w8a8_cpu import GOOD, NULL, SHAPE, call

CUS = 256


def test_the_plan_of_the_gated_backward_knows_both_launches():
    """1024 x 2^20 outputs of 1024 experts: dx has few tiles, both projections 2^24 of 256 threads, which one launch
    cannot have.  The plan refuses what the call does."""
    sizes = (1024, 1 << 20, 16, 0, CUS, 1024, 1024)
    with pytest.raises(ValueError):
        w4.w8a8_plan(w4.W8A8_EXPERTS_GATE_UP, *sizes)
    with pytest.raises(ValueError):
        w4.w8a8_plan(w4.W8A8_EXPERTS_GATE_UP_BACKWARD, *sizes)
    assert w4.w8a8_plan(w4.W8A8_EXPERTS_GATE_UP_BACKWARD, 1000, 1 << 19, 16, 0, CUS, 1000, 1000)["path"] == w4.PATH_W8A8


ROWS = (1 << 24) + 40


@pytest.mark.parametrize("op,experts", [(w4.W8A8_QMM, 1), (w4.W8A8_LINEAR_BACKWARD, 1), (w4.W8A8_EXPERTS_LINEAR, 8),
                                        (w4.W8A8_EXPERTS_LINEAR_BACKWARD, 8), (w4.W8A8_EXPERTS_GATE_UP, 8),
                                        (w4.W8A8_EXPERTS_GATE_UP_BACKWARD, 8)])
def test_rows_past_two_to_the_24_are_planned(op, experts):
    """As many rows as the router makes of 2^24 tokens and fewer, where no call quantizes them in one launch."""
    for rows in (1 << 24, ROWS):
        assert w4.w8a8_plan(op, rows, 64, 64, 0, CUS, experts)["path"] == w4.PATH_W8A8
    if experts > 1:
        assert w4.w8a8_plan(op, 1 << 24, 64, 64, 0, CUS, experts, 1 << 25)["path"] == w4.PATH_W8A8


def test_quantized_rows_past_two_to_the_24():
    """The sizes pass: what is refused is the pointer that is missing."""
    assert call("w8a8_quantize_rows", {**GOOD, "codes": None}, M=ROWS, K=16) == NULL
    assert call("w8a8_quantize_rows", {**GOOD, "codes": None}, M=1 << 30, K=16) == NULL
    assert call("w8a8_quantize_rows", {**GOOD, "codes": None}, M=(1 << 30) + 1, K=16) == SHAPE


def test_limits_of_the_combination():
    """Forward a thread for eight columns, backward a wave for a pair; where the sizes pass, the missing pointer is refused."""
    def forward(T, top, N):
        return call("experts_combine", {**GOOD, "y": None}, M=T, top=top, N=N)

    def backward(T, top, N):
        return call("experts_combine_backward", {**GOOD, "dw": None}, M=T, top=top, N=N)
    assert forward(1 << 24, 8, 8) == forward(1 << 24, 64, 2040) == forward(1 << 21, 8, 16376) == forward((1 << 24) - 1, 8, 2048) == NULL
    assert forward((1 << 24) + 1, 1, 8) == forward(1 << 24, 1, 2041) == forward(1 << 21, 8, 16384) == SHAPE
    assert backward((1 << 23) - 1, 8, 16384) == backward((1 << 20) - 1, 64, 8) == backward(1 << 24, 3, 1 << 14) == NULL
    assert backward(1 << 23, 8, 8) == backward(1 << 20, 64, 8) == backward(1 << 24, 4, 8) == SHAPE
