"""The products and the weight gradient at sizes that take each tile (64, 128 and 256
results to a side), ragged on both sides, every operand pair and result type, and
uneven experts whose average is few rows: against the float64 oracle."""
import pytest
import torch

from tests.test_gpu_gemm import check_product
from tests.test_gpu_wgrad import check_wgrad

pytestmark = pytest.mark.gpu

PAIRS = [("44", 640), ("44", 288), ("44", 96), ("84", 384), ("88", 640), ("88", 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,k", PAIRS)
@pytest.mark.parametrize("m,n", [(130, 1100), (700, 4200)])
def test_products(m, n, fmt, k, dtype):
    check_product(m + k, [m], n, k, fmt, "silu", torch.float32, True, True, dtype, grouped=False)
    check_product(m + k, [m], n + 1, k, fmt, "none", torch.bfloat16, True, True, dtype, grouped=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,k", PAIRS)
@pytest.mark.parametrize("n", [200, 4200])
def test_experts(n, fmt, k, dtype):
    check_product(n + k, [300, 5, 0, 64, 259, 1], n, k, fmt, "swiglu", torch.float32, True, True, dtype)
    check_product(n + k, [1, 0, 131, 2, 30, 0, 0, 6], n, k, fmt, "relu", torch.bfloat16, True, False, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["44", "84", "88"])
@pytest.mark.parametrize("m", [17, 33, 64])
def test_few_rows_on_either_side_of_one_round(m, fmt, dtype):
    for n in (4096, 4130, 8300):
        check_product(m + n, [m], n, 256, fmt, "gelu", torch.float32, True, True, dtype, grouped=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,k", [(130, 328), (700, 4200), (2060, 4120)])
def test_weight_gradients(n, k, dtype):
    check_wgrad(n, [130, 33, 0, 257], n, k, dtype)
    check_wgrad(n, [1, 300, 47], n, k + 1, dtype, add=True, ld_extra=16)
