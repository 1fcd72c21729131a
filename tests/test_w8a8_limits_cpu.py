"""Sizes at the limits of the int8 and experts' operators, without a GPU."""

import pytest

import w4a16_group_quantized_qmv_amd as w4

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
