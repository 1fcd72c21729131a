"""GPU tests of the int8 products at sizes that make the launch policy choose every tile, height, split and number of
pieces that it has (``test_w8a8_forms_cpu.py`` compares them with the policy's choices)."""

import pytest

import test_gpu_experts as experts
import test_gpu_w8a8 as products

pytestmark = pytest.mark.gpu

# (rows, weight rows, contraction) that the sizes of the other tests leave out
LINEAR = [(2770, 778, 8000), (2297, 7965, 2528), (1871, 1422, 9920), (5828, 2945, 1392), (2365, 1758, 6688), (3772, 4876, 944),
          (1174, 3313, 4384), (407, 3009, 9664), (795, 1181, 7744), (509, 2560, 9728)]
BACKWARD = [(795, 15080, 400), (3337, 431, 4752), (1325, 8, 13968)]
EXPERTS = [(251, 3246, 22722, 26, 48, "random"), (251, 2255, 9020, 24, 64, "random"), (248, 2786, 13930, 35, 48, "random"),
           (132, 2108, 14756, 443, 48, "random"), (121, 1588, 11116, 203, 64, "random"), (75, 1545, 9270, 533, 64, "random"),
           (16, 3634, 29072, 550, 80, "random"), (36, 736, 4416, 787, 336, "random")]
# experts, tokens, their width, the tokens', chosen
BLOCKS = [(16, 3000, 560, 272, 4), (251, 3246, 48, 96, 7)]


@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(lib, M, N, K):
    products.test_linear(lib, M, N, K)


@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_linear_backward(lib, M, N, K):
    products.test_linear_backward(lib, M, N, K)


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E,T,R,N,K,kind", EXPERTS)
def test_experts_linear(lib, E, T, R, N, K, kind, gather):
    products.test_experts_linear(lib, E, T, R, N, K, kind, gather)


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E,T,R,N,K,kind", EXPERTS)
def test_experts_gate_up(lib, E, T, R, N, K, kind, gather):
    products.test_experts_gate_up(lib, E, T, R, N, K, kind, gather)


@pytest.mark.parametrize("E,T,F,K,top", BLOCKS)
def test_a_block(lib, E, T, F, K, top):
    experts.test_a_block_forward_and_backward(lib, E, T, F, K, top)
