"""The oracle of the operators around the experts' products against torch's own softmax, sort,
casts and autograd in float64, and against exact rationals."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp8, moe
from oracle.formats import e4m3_decode


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(1, 1), (5, 5), (40, 6)])
def test_route_and_its_gradient_match_autograd(E, k, renorm):
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(7, E, generator=g, dtype=torch.float64, requires_grad=True)
    dw = torch.randn(7, k, generator=g, dtype=torch.float64)
    top, at = torch.sort(logits, dim=1, descending=True, stable=True)
    w = torch.softmax(top[:, :k], 1) if renorm else torch.softmax(logits, 1).gather(1, at[:, :k])
    (w * dw).sum().backward()
    weights, experts = moe.route(logits.detach().numpy(), k, renorm)
    assert np.array_equal(experts, at[:, :k].numpy())
    np.testing.assert_allclose(weights, w.detach().numpy(), rtol=1e-12)
    d, mag = moe.route_grad(dw.numpy(), weights, experts, logits.detach().numpy(), renorm)
    np.testing.assert_allclose(d, logits.grad.numpy(), rtol=1e-10, atol=1e-13)
    assert (mag >= np.abs(d) - 1e-12).all()


def test_choice_of_special_values():
    inf, nan = np.inf, np.nan
    assert moe.choose(np.array([1.0, 3.0, 3.0, -inf, nan, inf, -0.0, 0.0]), 8) == [4, 5, 1, 2, 0, 6, 7, -1]
    w, e = moe.route(np.array([[-inf] * 4, [-inf, 2.0, -inf, -inf], [nan, 0.0, 1.0, 2.0]]), 2, False)
    assert e.tolist() == [[-1, -1], [1, -1], [0, 3]]
    assert w[0].tolist() == [0, 0] and w[1].tolist() == [1, 0] and np.isnan(w[2]).all()
    # a masked choice's gradient of the weight does not matter
    d, _ = moe.route_grad(np.array([[2.0, nan]]), np.array([[1.0, 0.0]]), np.array([[1, -1]]),
                          np.array([[-inf, 2.0, -inf]]), False)
    assert d.tolist() == [[0, 0, 0]]


@pytest.mark.parametrize("E", [1, 3, 64])
def test_expert_sort_is_a_stable_sort(E):
    rng = np.random.default_rng(E)
    e = rng.integers(-2, E + 2, (50, 3)).astype(np.int32)
    offsets, positions, order = moe.expert_sort(e, E)
    flat = e.reshape(-1)
    kept = np.flatnonzero((flat >= 0) & (flat < E))
    want = kept[np.argsort(flat[kept], kind="stable")]
    assert np.array_equal(order[:len(want)], want) and (order[len(want):] == -1).all()
    assert np.array_equal(np.diff(offsets), np.bincount(flat[kept], minlength=E))
    assert np.array_equal(positions.reshape(-1)[want], np.arange(len(want)))
    assert (positions.reshape(-1)[(flat < 0) | (flat >= E)] == -1).all()


def test_combine_and_its_gradient_match_autograd():
    g = torch.Generator().manual_seed(0)
    y = torch.randn(9, 6, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(4, 2, generator=g, dtype=torch.float64, requires_grad=True)
    res = torch.randn(4, 6, generator=g, dtype=torch.float64)
    grad = torch.randn(4, 6, generator=g, dtype=torch.float64)
    pos = np.array([[3, 0], [-1, 8], [5, 12], [1, 2]], dtype=np.int32)
    out = torch.stack([res[t] + sum(w[t, j] * y[r] for j, r in enumerate(pos[t]) if 0 <= r < 9) for t in range(4)])
    (out * grad).sum().backward()
    got, mag = moe.combine(y.detach().numpy(), pos, w.detach().numpy(), res.numpy())
    np.testing.assert_allclose(got, out.detach().numpy(), rtol=1e-12)
    assert (mag >= np.abs(got) - 1e-12).all()
    dy, dw, _ = moe.combine_grad(grad.numpy(), y.detach().numpy(), pos, w.detach().numpy())
    np.testing.assert_allclose(dw, w.grad.numpy(), rtol=1e-12, atol=1e-15)
    used = sorted(r for r in pos.reshape(-1) if 0 <= r < 9)
    np.testing.assert_allclose(dy[used], y.grad.numpy()[used], rtol=1e-12)
    assert np.isnan(np.delete(dy, used, axis=0)).all()
    # combine without weights is the gradient of dispatch
    x = torch.randn(4, 6, dtype=torch.float64, generator=g, requires_grad=True)
    rows = torch.stack([x[t] for t in range(4) for r in pos[t] if 0 <= r < 9])
    at = [r for row in pos for r in row if 0 <= r < 9]
    d = torch.randn(9, 6, generator=g, dtype=torch.float64)
    (rows * d[at]).sum().backward()
    np.testing.assert_allclose(moe.combine(d.numpy(), pos)[0], x.grad.numpy(), rtol=1e-12, atol=1e-15)
    assert np.array_equal(moe.dispatch(x.detach().numpy(), pos, np.full((9, 6), -7.0))[at], rows.detach().numpy())


def test_fp8_rows_are_the_casts_of_the_scaled_values():
    rng = np.random.default_rng(0)
    x = rng.normal(0, 1, (6, 300)) * np.ldexp(1.0, rng.integers(-30, 30, (6, 1)))
    x[2, :128] = 0.0
    x[3, 5], x[4, 200] = np.nan, -np.inf
    x = x.astype(np.float32).astype(np.float64)
    q, s = moe.fp8_rows(x)
    for r in range(6):
        for g in range(3):
            part = x[r, 128 * g:128 * g + 128]
            codes = q[r, 128 * g:128 * g + 128]
            if not np.isfinite(part).all():
                assert s[r, g] == 0x7FC00000 and (codes == 0x7F).all()
                continue
            scale = np.float64(s[r, g:g + 1].view(np.float32)[0])
            if (part == 0).all():
                assert scale == 1.0 and (codes == 0).all()
                continue
            assert np.abs(part).max() <= 448 * scale and np.abs(part).max() > 224 * scale
            cast = torch.from_numpy(part / scale).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            assert np.array_equal(codes, cast)
    assert np.isnan(moe.fp8_row_values(q, s)[3, :128]).all() and not np.isnan(moe.fp8_row_values(q, s)[3, 128:]).any()


def test_fp8_rows_round_to_the_nearest_value():
    """Against every finite E4M3 value, in rationals."""
    grid = [Fraction(float(e4m3_decode(np.array([c], dtype=np.uint8))[0])) for c in range(127)]
    rng = np.random.default_rng(1)
    x = rng.normal(0, 30, (1, 128))
    x[0, 0], x[0, 1] = 448.0, grid[3] / 2 + grid[4] / 2  # scale 1, a tie
    q, s = moe.fp8_rows(x)
    assert s[0, 0] == 0x3F800000
    for v, c in zip(x[0], q[0]):
        d = [abs(abs(Fraction(float(v))) - g) for g in grid]
        best = [i for i in range(127) if d[i] == min(d)]
        assert int(c) & 127 in best and (len(best) == 1 or int(c) % 2 == 0) and (int(c) >> 7) == int(v < 0)


def test_fp8_rows_are_what_the_products_read():
    rng = np.random.default_rng(2)
    x = rng.normal(0, 1, (3, 256))
    q, s = moe.fp8_rows(x)
    assert np.array_equal(moe.fp8_row_values(q, s), fp8.fp8_values(q, s))
    tiny = np.full((1, 130), 1e-44)
    q, s = moe.fp8_rows(tiny)
    assert (s == 1 << 23).all() and (q == 0).all()  # the least scale is 2^-126
