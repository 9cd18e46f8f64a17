"""The mixture-of-experts example: every product of one training step against float64
products of the very operands it was given, and the step as a whole against fp32 autograd."""
import numpy as np
import pytest
import torch

from examples import moe_ffn
from oracle import mm
from tests.gpu_helpers import require_gpu, u8
from tests.mm_helpers import close, f64, out_bound, sum_bound

pytestmark = pytest.mark.gpu


def test_step_against_its_operands():
    require_gpu()
    x, logits, w = moe_ffn.make(200, 128, 96, 5)
    out, s = moe_ffn.forward(x, logits, w, 2)
    z = f64(s.z)
    off = s.offsets.cpu().numpy()
    xv = mm.operand_values(u8(s.xq.codes_row), u8(s.xq.scales_row))
    w1 = np.stack([mm.operand_values(u8(c), u8(sc)) for c, sc in zip(*w.w1_rows)])
    zw, mag = mm.grouped_product(xv, w1, off, f64(w.b1))
    ez = sum_bound(mag, 129)
    close(s.z, zw, out_bound(zw, ez, torch.bfloat16), "z")
    grad = torch.randn(200, 128, device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(1))
    dx, dw1, db1, dw2, db2 = moe_ffn.backward(grad, s, w)
    # db2: the sums of the bf16 gradients that entered
    dy = f64((s.weight * grad[s.order]).bfloat16())
    want = np.stack([dy[a:b].sum(0) for a, b in zip(off[:-1], off[1:])])
    size = np.stack([np.abs(dy[a:b]).sum(0) for a, b in zip(off[:-1], off[1:])])
    close(db2, want, 2 * 400 * 2.0 ** -24 * size + 1e-30, "db2")
    assert dw1.shape == (5, 192, 128) and dw2.shape == (5, 128, 96) and dx.shape == (200, 128)
    assert not np.array_equal(f64(s.z), z)  # the gradient was written over z


@pytest.mark.parametrize("tokens,hidden,ffn,experts", [(300, 256, 128, 4), (2048, 512, 256, 8)])
def test_step_follows_fp32_autograd(tokens, hidden, ffn, experts):
    """MXFP4 keeps about 3 significant bits of each element (relative error up to 1/6 near the
    bottom of a binade, about 0.1 on average over both operands of a product): a step's
    outputs lie within 0.4 of fp32's in norm, and point the same way."""
    require_gpu()
    x, logits, w = moe_ffn.make(tokens, hidden, ffn, experts)
    grad = torch.randn(tokens, hidden, device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(2))
    out, s = moe_ffn.forward(x, logits, w, 2)
    got = (out, *moe_ffn.backward(grad, s, w))
    ref, ref_grads = moe_ffn.reference(x, logits, w, 2, grad)
    for name, a, b in zip(("output", "dx", "dW1", "db1", "dW2", "db2"), got, (ref, *ref_grads)):
        assert float((a - b).norm() / b.norm()) < 0.4, name
        assert float((a * b).sum() / (a.norm() * b.norm())) > 0.93, name
