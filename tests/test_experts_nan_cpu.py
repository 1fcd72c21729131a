"""The oracle of the experts' operators on logits that hold NaN."""

import numpy as np

import oracle as O
import w4a16_group_quantized_qmv_amd as w4


def test_nan_logits_by_hand():
    """A slot without an expert is marked where the token's logits hold a NaN, and the mark makes sums NaN."""
    nan, inf, mark = np.nan, np.inf, w4.EXPERTS_NAN_ROW
    logits = np.array([[1.0, 3.0, nan], [nan] * 3, [-inf] * 3, [nan, -inf, 2.0], [0.0, 1.0, -inf]])
    (w, _), experts, positions, tokens, offsets = O.route_reference(logits, 2)
    assert experts.tolist() == [[1, 0], [-1, -1], [-1, -1], [2, -1], [1, 0]]
    assert offsets.tolist() == [0, 2, 4, 5] and tokens.tolist() == [0, 4, 0, 4, 3] + [-1] * 5
    assert positions.tolist() == [[2, 0], [mark, mark], [-1, -1], [4, mark], [3, 1]] and mark == -2 ** 31
    assert np.isnan(w[[0, 1, 3]]).all() and not w[2].any()
    y, dout = np.ones((10, 4)), np.ones((5, 4))
    for weights in (w, None):
        out, _ = O.combine_reference(y, positions, weights)
        expected = [True, True, False, True, False] if weights is not None else [False, True, False, True, False]
        assert np.isnan(out).all(1).tolist() == expected == np.isnan(out).any(1).tolist()
    (dy, _), (dw, _) = O.combine_backward_reference(dout, y, positions, w)
    assert np.isnan(dy[:, 0]).tolist() == [True, False, True, False] + [True] * 6
    assert np.isnan(dw).tolist() == [[False, False], [True, True], [False, False], [False, True], [False, False]]
    d, _ = O.route_backward_reference(logits, experts, np.ones((5, 2)))
    assert np.isnan(d).all(1).tolist() == [True, True, False, True, False] and not d[[2, 4]].any()
