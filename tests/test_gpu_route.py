"""The choice of experts and its gradient against the float64 oracle: every number of lanes
and of logits of a lane, both types, both softmaxes, strides, ties, masks and special values."""
import numpy as np
import pytest
import torch

from mxfp4_microscaling_quantization_amd import mxq
from oracle import moe
from tests.gpu_helpers import require_gpu
from tests.mm_helpers import U, close, f64, out_bound
from tests.moe_helpers import FLOOR, logit_depth, strided, to, weight_bound

pytestmark = pytest.mark.gpu

# (experts, k): 8, 16, 32 and 64 lanes of 8 logits, 64 lanes of 16, 32 and 64
SIZES = [(1, 1), (7, 7), (64, 1), (64, 64), (61, 33), (65, 6), (128, 64), (129, 8), (256, 8), (256, 64), (257, 5),
         (512, 8), (513, 9), (1000, 64), (1025, 3), (2048, 8), (2049, 10), (4096, 64)]


def check(logits, k, dtype, renorm, extra=0, first=0, seed=0):
    rng = np.random.default_rng(seed)
    t = to(logits, dtype)
    given = f64(t)
    if extra or first:
        t = strided(t, extra, first)
    w, e = mxq.mxq_route(t, k, renorm=renorm)
    ww, we = moe.route(given, k, renorm)
    assert np.array_equal(e.cpu().numpy(), we), "experts"
    close(w, ww, weight_bound(ww, we, given), "weights")
    # the gradient takes the weights that were computed
    dw = rng.normal(0, 1, w.shape).astype(np.float32)
    dw[we < 0] = np.nan  # (of choices that are none)
    d = mxq.mxq_route_grad(to(dw, torch.float32), w, e, t, renorm=renorm)
    wf = f64(w)
    want, mag = moe.route_grad(dw.astype(np.float64), wf, we, given, renorm)
    # k products and sums, the softmax's own error on the second term, a last subtraction
    err = (k + 8 + logit_depth(given) + 3 * given.shape[1] + 16) * U * mag + FLOOR
    close(d, want, out_bound(want, err, dtype), "gradient")
    assert d.dtype == dtype and d.is_contiguous()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,k", SIZES)
def test_sizes(E, k, dtype, renorm):
    require_gpu()
    rng = np.random.default_rng(E + k)
    for tokens in (1, 37):
        check(rng.normal(0, 2, (tokens, E)), k, dtype, renorm)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_alignments(dtype):
    require_gpu()
    rng = np.random.default_rng(0)
    for E, extra, first in ((64, 8, 0), (64, 8, 8), (64, 7, 1), (64, 1, 3), (61, 0, 2), (256, 5, 0), (256, 8, 4)):
        check(rng.normal(0, 2, (19, E)), 5, dtype, False, extra, first)


def test_no_tokens():
    require_gpu()
    w, e = mxq.mxq_route(torch.empty((0, 64), device="cuda:0"), 8)
    assert w.shape == e.shape == (0, 8)
    assert mxq.mxq_route_grad(w, w, e, torch.empty((0, 64), device="cuda:0")).shape == (0, 64)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E", [24, 200, 600])
def test_ties(E, dtype, renorm):
    """Few different values (zeros of both signs among them): equal logits by expert."""
    require_gpu()
    rng = np.random.default_rng(E)
    check(rng.choice([-1.0, -0.0, 0.0, 1.0, 1.0], (40, E)), 12, dtype, renorm)
    check(np.zeros((3, E)), 12, dtype, renorm)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_logits(dtype, renorm):
    """-Inf: rows with some, with fewer than k left, with one and with none left."""
    require_gpu()
    rng = np.random.default_rng(1)
    x = rng.normal(0, 2, (6, 96))
    x[0, rng.random(96) < 0.5] = -np.inf
    x[1, 3:] = -np.inf
    x[2, :95] = -np.inf
    x[3] = -np.inf
    x[4, ::2] = torch.finfo(dtype).min  # the type's lowest value is a value
    x[5] = torch.finfo(dtype).min
    check(x, 8, dtype, renorm)
    w, e = mxq.mxq_route(to(x, dtype), 8, renorm=renorm)
    assert (e[3] == -1).all() and (w[3] == 0).all()
    assert e[5].tolist() == list(range(8))


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_and_infinity(dtype, renorm):
    """NaN (either sign) before +Inf before the rest; the weights of such rows are NaN, other rows whole."""
    require_gpu()
    rng = np.random.default_rng(2)
    x = rng.normal(0, 2, (5, 70))
    x[0, 9] = np.nan
    x[1, 69] = np.inf
    x[2, 3], x[2, 5], x[2, 7] = np.inf, np.nan, -np.inf
    x[3, 1] = np.copysign(np.nan, -1.0)
    t = to(x, dtype)
    w, e = mxq.mxq_route(t, 4, renorm=renorm)
    _, we = moe.route(f64(t), 4, renorm)
    assert np.array_equal(e.cpu().numpy(), we)
    assert e[0, 0] == 9 and e[1, 0] == 69 and e[2, :2].tolist() == [5, 3] and e[3, 0] == 1
    assert torch.isnan(w[:4]).all() and torch.isfinite(w[4]).all()
    d = mxq.mxq_route_grad(torch.ones_like(w), w, e, t, renorm=renorm)
    assert torch.isnan(d[:4]).any(dim=1).all() and torch.isfinite(d[4]).all()


def test_far_logits():
    """Differences where the exponential vanishes, and large logits of one size."""
    require_gpu()
    x = np.array([[0.0, -80.0, -87.0, -100.0, -200.0, -1e30, 3.0, 2.0], [1e30, 1e30, -1e30, 0, 0, 0, 0, 0],
                  [3e38, -3e38, 3e38, 0, 0, 0, 0, 0]])
    for dtype in (torch.float32, torch.bfloat16):
        for renorm in (False, True):
            check(x, 8, dtype, renorm)


def test_choices_outside_are_left_out():
    """Experts that are none, whatever their weights and gradients, and the same expert twice."""
    require_gpu()
    rng = np.random.default_rng(3)
    x = rng.normal(0, 1, (4, 20))
    e = np.array([[3, -1, 3], [20, 2 ** 31 - 1, 7], [-2 ** 31, -1, 25], [0, 19, 0]], dtype=np.int32)
    w = rng.random((4, 3)).astype(np.float32)
    dw = rng.normal(0, 1, (4, 3)).astype(np.float32)
    w[1, 0] = dw[1, 1] = dw[2, 0] = np.nan
    for renorm in (False, True):
        d = mxq.mxq_route_grad(to(dw, torch.float32), to(w, torch.float32), to(e, torch.int32), to(x, torch.float32),
                               renorm=renorm)
        xs = f64(to(x, torch.float32))
        with np.errstate(invalid="ignore"):
            want, mag = moe.route_grad(dw.astype(np.float64), np.where((e >= 0) & (e < 20), w, 0).astype(np.float64), e, xs,
                                       renorm)
        close(d, want, out_bound(want, 100 * U * mag + FLOOR, torch.float32), "gradient")


def test_gradient_against_differences():
    """dlogits against the change of sum(w dw) over small steps, in the oracle's float64."""
    require_gpu()
    rng = np.random.default_rng(4)
    x = rng.normal(0, 1, (3, 12)).astype(np.float32)
    dw = rng.normal(0, 1, (3, 4)).astype(np.float32)
    for renorm in (False, True):
        w, e = mxq.mxq_route(to(x, torch.float32), 4, renorm=renorm)
        d = f64(mxq.mxq_route_grad(to(dw, torch.float32), w, e, to(x, torch.float32), renorm=renorm))
        h = 1e-4  # (h^2 times a third derivative of at most 6 |dw|; no two logits are as near as h)
        for i in range(12):
            up, down = x.astype(np.float64), x.astype(np.float64)
            up[:, i] += h
            down[:, i] -= h
            slope = ((moe.route(up, 4, renorm)[0] - moe.route(down, 4, renorm)[0]) * dw).sum(1) / (2 * h)
            assert np.abs(slope - d[:, i]).max() <= 6 * h * h * np.abs(dw).sum() + 400 * U * np.abs(dw).sum()
