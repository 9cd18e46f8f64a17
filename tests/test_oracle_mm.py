"""The oracle of the matrix products against exact rational sums, torch's own
activations and their autograd."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp8, mm, mx
from oracle.formats import e2m1_value


def test_mxfp4_product_is_the_rational_sum():
    rng = np.random.default_rng(0)
    codes = [rng.integers(0, 256, (3, 32)).astype(np.uint8) for _ in range(2)]
    scales = [rng.integers(100, 150, (3, 2)).astype(np.uint8) for _ in range(2)]
    z, _ = mm.grouped_product(mm.operand_values(codes[0], scales[0]),
                              mm.operand_values(codes[1], scales[1])[None], [0, 3])
    for i in range(3):
        for j in range(3):
            s = Fraction(0)
            for t in range(64):
                v = [Fraction(e2m1_value((int(c[r, t // 2]) >> (4 * (t & 1))) & 15)) *
                     Fraction(2) ** (int(e[r, t // 32]) - 127) for c, e, r in
                     ((codes[0], scales[0], i), (codes[1], scales[1], j))]
                s += v[0] * v[1]
            assert abs(z[i, j] - float(s)) <= 64 * 2.0 ** -52 * abs(float(s)) + 2.0 ** -60


@pytest.mark.parametrize("name,f", [("relu", torch.relu), ("silu", torch.nn.functional.silu),
                                    ("gelu", lambda z: torch.nn.functional.gelu(z, approximate="tanh"))])
def test_activations_and_slopes_match_torch(name, f):
    z = torch.linspace(-9, 9, 4001, dtype=torch.float64, requires_grad=True)
    y = f(z)
    y.sum().backward()
    np.testing.assert_allclose(mm.act(z.detach().numpy(), name), y.detach().numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(mm.act_slope(z.detach().numpy(), name), z.grad.numpy(), rtol=1e-12, atol=1e-13)


def test_swiglu_gradient_matches_autograd():
    g = torch.Generator().manual_seed(0)
    z = torch.randn(5, 12, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(5, 6, generator=g, dtype=torch.float64)
    (torch.nn.functional.silu(z[:, 0::2]) * z[:, 1::2] * dy).sum().backward()
    np.testing.assert_allclose(mm.act_grad(dy.numpy(), z.detach().numpy(), "swiglu"), z.grad.numpy(), rtol=1e-12)


def test_column_values_undo_the_column_conversion():
    """FP8 columns of MXFP4 rows hold the rows' values where the conversion is exact."""
    rng = np.random.default_rng(1)
    offsets = np.array([0, 5, 5, 140, 300])
    codes = rng.integers(0, 256, (300, 32)).astype(np.uint8)
    e8 = rng.integers(126, 129, (300, 2)).astype(np.uint8)
    q8, s = fp8.mxfp4_rows_to_fp8_cols(codes, e8, offsets)
    np.testing.assert_array_equal(mm.column_values(q8, s, offsets), mx.mxfp4_dequantize_values(codes, e8).T)
