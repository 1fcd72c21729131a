"""GPU tests of int8 weights that are not finite in split products."""

import numpy as np
import pytest

from gpu_helpers import announce
from test_gpu_w8a8 import bf16, to_gpu, values, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("split", [1, 2, 3, 7])
@pytest.mark.parametrize("M,N,K", [(40, 97, 1040), (40, 130, 272), (300, 512, 400), (600, 700, 528)])
def test_infinite_weights_in_a_split_gradient(lib, M, N, K, split):
    """An infinite scale makes dx infinite where its code is not zero, with the sign of gradient and code, in whichever
    slice its row lies, and NaN where it is."""
    announce(f"w8a8_linear_backward, infinite scale, {M}x{N}x{K} S={split}")
    rng = np.random.default_rng(N)
    (codes, scales), host = weight(rng, N, K)
    dy = rng.standard_normal((M, N))
    dy[dy == 0] = 1
    for n in {0, 64, 65, N // 2, N - 1}:
        s = host[1].copy()
        s[n] = np.inf
        dx = values(lib.w8a8_linear_backward(bf16(dy), codes, to_gpu(s), split_k=split))
        sign = np.sign(dy[:, n])[:, None] * np.sign(host[0][n].astype(np.float64))[None, :]
        want = np.select([sign > 0, sign < 0], [np.inf, -np.inf], np.nan)
        assert np.array_equal(dx, want, equal_nan=True), (n, np.argwhere(~((dx == want) | (np.isnan(dx) & np.isnan(want))))[:3])
