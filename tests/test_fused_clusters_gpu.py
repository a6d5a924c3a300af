"""The fused products' split-K over every cluster size: those that divide the work unevenly (3, 5, 6 and 7; 7 fills the
receive buffer to the last row that it is sized for) and those that the planner takes for wide weights (4 to 8
CTAs by the number of weight tiles). References and bounds as in the other tests of these products."""
import pytest
import torch

from fused_refs import ACTS, DTYPES
from test_fused_products_gpu import Product, glu_case, grad_case, linear_case, quant_case

pytestmark = pytest.mark.gpu

K = 2048


@pytest.mark.parametrize("cluster", [4, 6, 7])
@pytest.mark.parametrize("M", [1, 16, 17, 33, 64])
def test_few_tokens(cuda_device, M, cluster):
    plan = {"cluster": cluster}
    p = Product(cuda_device, M, 328, K, 1100 + M)
    for i, dtype in enumerate(DTYPES):
        linear_case(p, dtype, ACTS[(M + i) % 6], bias=True, residual=i != 1, plan=plan)
    p = Product(cuda_device, M, 2 * 192, K, 1200 + M, gated=True)
    for i, dtype in enumerate(DTYPES):
        glu_case(p, dtype, ACTS[(M + i) % 6], plan)
        grad_case(p, dtype, ACTS[(M + i + 2) % 6], plan)
    quant_case(p, "silu", plan, tiled=True)
    quant_case(p, "gelu", plan, tiled=False)


@pytest.mark.parametrize("cluster", [2, 4, 5, 6, 7])
@pytest.mark.parametrize("M", [65, 300])
def test_many_tokens(cuda_device, M, cluster):
    plan = {"bn": 128, "cluster": cluster}
    p = Product(cuda_device, M, 264, K, 1300 + M)
    for i, dtype in enumerate(DTYPES):
        linear_case(p, dtype, ACTS[(M + i) % 6], bias=i != 1, residual=i != 2, plan=plan)
    p = Product(cuda_device, M, 2 * 192, K, 1400 + M, gated=True)
    for i, dtype in enumerate(DTYPES):
        glu_case(p, dtype, ACTS[(M + i) % 6], plan)
        grad_case(p, dtype, ACTS[(M + i + 2) % 6], plan)
    quant_case(p, "silu", plan, tiled=True)
    quant_case(p, "gelu_tanh", plan, tiled=False)


@pytest.mark.parametrize("M,I", [(16, 1344), (16, 1504), (16, 2048), (50, 2048), (3, 2368)])
def test_planner_clusters_of_wide_weights(cuda_device, M, I):
    """21, 24, 32 and 37 weight tiles: the planner's own clusters of 7, 6, 4 and 4 CTAs on 148 SMs, where they fit."""
    p = Product(cuda_device, M, 2 * I, K, 1500 + I, gated=True)
    glu_case(p, torch.bfloat16, "silu", {})
    grad_case(p, torch.float32, "gelu", {})
    quant_case(p, "silu", {}, tiled=I % 64 == 0)
    linear_case(Product(cuda_device, M, 2 * I, K, 1600 + I), torch.float16, "gelu_tanh", True, True, {})
