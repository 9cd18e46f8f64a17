"""Every compiled form of the gradient from FP8 (type, with a gate, whole rows, with sums, with the
activation once more) against the float64 oracle. FORMS is also what
tests/test_fp8_act_grad_forms_cpu.py holds against the compiled kernels."""
import itertools

import numpy as np
import pytest
import torch

from mxfp4_microscaling_quantization_amd import mxq
from oracle import mm
from tests.gpu_helpers import require_gpu
from tests.mm_helpers import U, act_bound, close, f64, out_bound
from tests.test_gpu_act_grad import slope_bound
from tests.test_gpu_fp8_act_grad import make

pytestmark = pytest.mark.gpu

SIZES = [(65, 512), (130, 1026)]  # whole rows, and rows that start on no eight elements
FORMS = [(rows, n, act, bias, again) for (rows, n), act, bias, again in
         itertools.product(SIZES, ("gelu", "silu", "swiglu"), (False, True), (False, True))]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n,act,bias,again", FORMS)
def test_form(rows, n, act, bias, again, dtype):
    require_gpu()
    rng = np.random.default_rng(rows + n)
    z8, z, dy = make(rng, rows, n, act, dtype)
    got = mxq.mxq_fp8_act_grad(dy, z8, act, bias_grad=bias, recompute=again)
    got = list(got) if bias or again else [got]
    want, err = mm.act_grad(f64(dy), z, act), slope_bound(f64(dy), z, act)
    close(got.pop(0), want, out_bound(want, err, dtype), "dz")
    if bias:
        # (dz in fp32: its error and a rounding of each of the sum's additions)
        close(got.pop(0), want.sum(0), (2 * rows * U * np.abs(want) + err).sum(0) + 1e-300, "db")
    if again:
        h = mm.act(z, act)
        close(got.pop(0), h, out_bound(h, act_bound(z, np.zeros_like(z), act), dtype), "h")
    assert not got
