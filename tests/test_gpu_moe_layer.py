"""The operators around the experts' products as a layer uses them: the example's step with z
kept in FP8 and the router's gradient, each piece against float64 on its own operands, the
whole against fp32 autograd, and captured in a graph."""
import numpy as np
import pytest
import torch

from examples import moe_ffn
from mxfp4_microscaling_quantization_amd import mxq
from oracle import mm, moe
from tests.gpu_helpers import bits32, require_gpu, u8
from tests.mm_helpers import U, close, f64, out_bound
from tests.moe_helpers import FLOOR, logit_depth, weight_bound
from tests.test_gpu_act_grad import slope_bound

pytestmark = pytest.mark.gpu
NAMES = ("output", "dx", "dW1", "db1", "dW2", "db2", "dlogits")


def gradient(tokens, hidden, seed=1):
    return torch.randn(tokens, hidden, device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(seed))


def test_pieces_against_their_operands():
    require_gpu()
    T, k, E = 150, 3, 7
    x, logits, w = moe_ffn.make(T, 128, 96, E)
    out, s = moe_ffn.forward(x, logits, w, k, keep="fp8")
    l = f64(logits)
    ww, we = moe.route(l, k, False)
    assert np.array_equal(s.experts.cpu().numpy(), we)
    close(s.weights, ww, weight_bound(ww, we, l), "weights")
    for got, want in zip(s.rows, moe.expert_sort(we, E)):
        assert np.array_equal(got.cpu().numpy(), want)
    pos, wf, y = s.rows.positions.cpu().numpy(), f64(s.weights), f64(s.y)
    q = mxq.mxq_quantize(x)
    for got, own in ((s.xq.codes_row, q.codes_row), (s.xq.scales_row, q.scales_row)):
        assert np.array_equal(u8(got), moe.dispatch(u8(own), pos, np.zeros(got.shape, np.uint8)))
    want, mag = moe.combine(y, pos, wf)
    close(out, want, out_bound(want, (k + 2) * U * mag, torch.float32), "output")
    # backward
    grad = gradient(T, 128)
    z = moe.fp8_row_values(u8(s.z[0]), bits32(s.z[1]))
    assert s.hq is None
    wdy, wdw, mag = moe.combine_grad(f64(grad), y, pos, wf)
    dy, dw = mxq.mxq_combine_grad(grad, s.y, s.rows.positions, s.weights)
    close(dy, wdy, out_bound(wdy, U * np.abs(wdy), torch.bfloat16), "dy")
    close(dw, wdw, 2 * 128 * U * mag + 1e-30, "dw")
    dh = mxq.mxq_grouped_gemm(moe_ffn.rows(mxq.mxq_quantize(dy)), w.w2_cols, s.offsets)
    dz, db1, h = mxq.mxq_fp8_act_grad(dh, s.z, "swiglu", s.offsets, bias_grad=True, recompute=True)
    wdz = mm.act_grad(f64(dh), z, "swiglu")
    close(dz, wdz, out_bound(wdz, slope_bound(f64(dh), z, "swiglu"), torch.bfloat16), "dz")
    got = moe_ffn.backward(grad, s, w, router=True)
    assert torch.equal(got[2], db1) and len(got) == 6
    wl, mag = moe.route_grad(f64(dw), wf, we, l, False)
    close(got[5], wl, out_bound(wl, (k + 8 + logit_depth(l) + 3 * E + 16) * U * mag + FLOOR, torch.float32), "dlogits")


@pytest.mark.parametrize("keep", ["bf16", "fp8"])
@pytest.mark.parametrize("tokens,hidden,ffn,experts,top_k", [(300, 256, 128, 4, 2), (2048, 512, 256, 8, 2), (700, 128, 64, 70, 6)])
def test_step_follows_fp32_autograd(tokens, hidden, ffn, experts, top_k, keep):
    """MXFP4 operands keep a step within 0.4 of fp32's in norm, pointing the same way (see
    test_gpu_moe_ffn.py); E4M3's half step of 2^-4 in z, 0.02 of its values on average, is small beside
    that. The router's gradient is made of sums of products of such outputs."""
    require_gpu()
    x, logits, w = moe_ffn.make(tokens, hidden, ffn, experts)
    grad = gradient(tokens, hidden, 2)
    out, s = moe_ffn.forward(x, logits, w, top_k, keep)
    got = (out, *moe_ffn.backward(grad, s, w, router=True))
    ref, ref_grads = moe_ffn.reference(x, logits, w, top_k, grad)
    for name, a, b in zip(NAMES, got, (ref, *ref_grads)):
        assert a.shape == b.shape, name
        assert float((a - b).norm() / b.norm()) < 0.4, name
        assert float((a * b).sum() / (a.norm() * b.norm())) > 0.93, name


@pytest.mark.parametrize("keep", ["bf16", "fp8"])
def test_step_in_a_graph(keep):
    """Forward and backward captured once, replayed with new tokens and logits between eager steps."""
    require_gpu()
    x, logits, w = moe_ffn.make(260, 128, 64, 6)
    grad = gradient(260, 128)

    def step():
        out, s = moe_ffn.forward(x, logits, w, 2, keep)
        return (out, *moe_ffn.backward(grad, s, w, router=True))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (0, 3, 4, 0):
        nx, nl, _ = moe_ffn.make(260, 128, 64, 6, seed=seed)
        x.copy_(nx)
        logits.copy_(nl)
        grad.copy_(gradient(260, 128, seed + 10))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for name, a, b in zip(NAMES, got, want):
            assert torch.equal(a, b), f"{name}, seed {seed}"


def test_padding_tokens():
    """Tokens whose logits are all -Inf have no rows: they come out as zeros, and get no gradients."""
    require_gpu()
    x, logits, w = moe_ffn.make(64, 128, 64, 4)
    logits[50:] = float("-inf")
    weights, experts = mxq.mxq_route(logits, 2)
    r = mxq.mxq_expert_sort(experts, 4)
    assert (experts[50:] == -1).all() and int(r.offsets[-1]) == 100
    xq = mxq.mxq_dispatch(x, r.positions, rows=100, fmt="mxfp4")
    y = mxq.mxq_grouped_gemm(xq, w.w1_rows, r.offsets, out_dtype=torch.float32)
    out = mxq.mxq_combine(y, r.positions, weights, out_dtype=torch.float32)
    assert (out[50:] == 0).all() and (out[:50] != 0).any(dim=1).all()
    dy, dw = mxq.mxq_combine_grad(torch.ones_like(out), y, r.positions, weights)
    assert (dw[50:] == 0).all() and torch.isfinite(dy).all()
    d = mxq.mxq_route_grad(dw, weights, experts, logits)
    assert (d[50:] == 0).all() and torch.isfinite(d).all() and (d[:50] != 0).any()
    assert (mxq.mxq_combine(dy, r.positions, out_dtype=torch.float32)[50:] == 0).all()
