"""The activations' gradients far from zero, where the slopes are 0 and 1: no NaN from an
overflow up to the ends of both types' ranges and at infinity, NaN for NaN; in rows that
are whole vectors and in others, with the bias gradient's sums."""
import numpy as np
import pytest
import torch

from mxfp4_microscaling_quantization_amd import mxq
from tests.gpu_helpers import require_gpu
from tests.mm_helpers import f64

pytestmark = pytest.mark.gpu

FAR = [20.0, 100.0, 130.0, 1e4, 1e10, 1.8e19, 1.9e19, 1e20, 1e30, 3.3e38, float("inf")]


def values(dtype, n):
    z = torch.tensor([s * v for v in FAR for s in (1, -1)], dtype=dtype)
    return torch.cat([z, torch.full((n - z.numel(),), 1e20, dtype=dtype)])[None].repeat(5, 1).to("cuda:0")


@pytest.mark.parametrize("n", [24, 31])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_slopes(act, dtype, n):
    require_gpu()
    z = values(dtype, n)
    dy = torch.full_like(z, 3.0)
    dz, db = mxq.mxq_act_grad(dy, z, act, bias_grad=True)
    want = np.where(f64(z) > 0, 3.0, 0.0)
    # beyond 20 the slopes differ from 0 and 1 by less than 20 e^-20
    np.testing.assert_allclose(f64(dz), want, rtol=1e-6, atol=3 * 20 * np.exp(-20.0))
    np.testing.assert_allclose(f64(db), want.sum(0), rtol=1e-6, atol=15 * 20 * np.exp(-20.0))


@pytest.mark.parametrize("n", [48, 62])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_swiglu(dtype, n):
    """d gate = dy up silu'(gate), d up = dy silu(gate): the gate itself, or 0."""
    require_gpu()
    gate = values(dtype, n // 2)
    up = torch.full_like(gate, 2.0)
    dy = torch.full_like(gate, 0.5)
    dz = f64(mxq.mxq_act_grad(dy, torch.stack([gate, up], dim=-1).view(5, n).contiguous(), "swiglu"))
    g = f64(gate)
    np.testing.assert_allclose(dz[:, 0::2], np.where(g > 0, 1.0, 0.0), rtol=1e-6, atol=20 * np.exp(-20.0))
    ends = np.isneginf(g)  # (-inf times 0, as in the product's own silu: NaN)
    np.testing.assert_allclose(dz[:, 1::2][~ends], np.where(g > 0, 0.5 * g, 0.0)[~ends], rtol=1e-6,
                               atol=20 * np.exp(-20.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan(dtype):
    require_gpu()
    z = torch.zeros(3, 16, dtype=dtype, device="cuda:0")
    z[1, 4] = float("nan")
    dy = torch.ones_like(z)
    for act in ("gelu", "silu"):
        bad = torch.isnan(mxq.mxq_act_grad(dy, z, act))
        assert bad[1, 4] and int(bad.sum()) == 1
    bad = torch.isnan(mxq.mxq_act_grad(dy[:, ::2].contiguous(), z, "swiglu"))
    assert bad[1, 4:6].all() and int(bad.sum()) == 2
