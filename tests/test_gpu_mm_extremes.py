"""FP8 operands whose scales lie at the ends of fp32's exponent range (zero and subnormal
scales, which count as 2^-127, and the largest) against operands that bring the products
back to ordinary numbers. Where both are widened to bf16 (fp32 results, few rows), an element below
2^-126 may be lost (2^-126 times the other operand's is in the bound), and one of 2^128 or more is
infinite, so its row or column is not finite; every other result is compared with the oracle."""
import numpy as np
import pytest
import torch

from mxfp4_microscaling_quantization_amd import mxq
from oracle import mm
from tests.gpu_helpers import require_gpu
from tests.mm_helpers import close, f64, fp8, gpu, mxfp4, out_bound, sum_bound

pytestmark = pytest.mark.gpu


def scaled(rng, rows, k, fields):
    """FP8 operand with the given exponent fields, and mantissa bits that do not count."""
    q, s = fp8(rng, rows, k)
    bits = (rng.choice(fields, s.shape).astype(np.uint32) << 23) | rng.integers(0, 1 << 23, s.shape).astype(np.uint32)
    bits[rng.random(s.shape) < 0.3] &= 0x7F800000
    return q, bits.view(np.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n", [(3, 72), (40, 72), (290, 72), (700, 4200), (4130, 4100)])
@pytest.mark.parametrize("a_fields,b_low,b_high", [((0, 1, 2), 245, 252), ((252, 253, 254), 0, 3), ((252, 254), 3, 6)])
@pytest.mark.parametrize("fmt", ["84", "88"])
def test_ends_of_the_range(fmt, a_fields, b_low, b_high, m, n, dtype):
    require_gpu()
    k = 384
    rng = np.random.default_rng(m + b_low)
    a = scaled(rng, m, k, a_fields)
    b = scaled(rng, n, k, range(b_low, b_high)) if fmt == "88" else mxfp4(rng, n, k, b_low, b_high)
    av, bv = mm.operand_values(*a), mm.operand_values(*b)
    z, mag = mm.grouped_product(av, bv[None], [0, m])
    lost = 2.0 ** -126 * (np.abs(av).sum(1)[:, None] + np.abs(bv).sum(1)[None])
    err = sum_bound(mag, k, dtype == torch.bfloat16) + lost
    bound = out_bound(z, err, dtype)
    d = mxq.mxq_gemm(gpu(*a), gpu(*b), out_dtype=dtype)
    widened = dtype == torch.float32 or m <= (64 if fmt == "84" else 16)
    beyond = (np.abs(av) >= 2.0 ** 128).any(1)[:, None] | (np.abs(bv) >= 2.0 ** 128).any(1)[None]
    if widened and beyond.any():
        assert np.array_equal(~np.isfinite(f64(d)), beyond)
        keep = ~beyond
        d, z, bound = d.cpu()[torch.from_numpy(keep)], z[keep], bound[keep]
    close(d, z, bound, f"{fmt} {m} {n} {dtype}")
