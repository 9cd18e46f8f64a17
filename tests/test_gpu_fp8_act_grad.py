"""The activation's gradient from values kept in FP8, against the float64 oracle on those values:
every activation and type, odd widths, groups, the activation's values once more, in place."""
import numpy as np
import pytest
import torch

from mxfp4_microscaling_quantization_amd import mxq
from oracle import mm, moe
from tests.gpu_helpers import bits32, require_gpu, u8
from tests.mm_helpers import U, act_bound, close, f64, out_bound
from tests.moe_helpers import to
from tests.test_gpu_act_grad import slope_bound
from tests.test_gpu_mm_malformed import PATTERNS, banded, offsets

pytestmark = pytest.mark.gpu


def make(rng, rows, n, act, dtype):
    z = rng.normal(0, 2, (rows, n))
    z8 = mxq.mxq_fp8_quantize(to(z, dtype))
    return z8, moe.fp8_row_values(u8(z8[0]), bits32(z8[1])), to(rng.normal(0, 1, (rows, n // 2 if act == "swiglu" else n)), dtype)


def check(seed, counts, n, act, dtype, grouped=True, over=False):
    require_gpu()
    rng = np.random.default_rng(seed)
    rows = sum(counts)
    offsets = np.concatenate([[0], np.cumsum(counts)]) if grouped else np.array([0, rows])
    z8, z, dy = make(rng, rows, n, act, dtype)
    dyv = f64(dy)
    off = torch.from_numpy(offsets).to("cuda:0") if grouped else None
    dz, db, h = mxq.mxq_fp8_act_grad(dy, z8, act, off, bias_grad=True, recompute=True, h=dy if over else None)
    want = mm.act_grad(dyv, z, act)
    err = slope_bound(dyv, z, act)
    what = f"{counts} {n} {act} {dtype}"
    close(dz, want, out_bound(want, err, dtype), f"dz {what}")
    sums = np.stack([want[a:b].sum(0) for a, b in zip(offsets[:-1], offsets[1:])])
    bound = np.stack([(2 * rows * U * np.abs(want[a:b]) + err[a:b]).sum(0) for a, b in zip(offsets[:-1], offsets[1:])])
    close(db if grouped else db[None], sums, bound + 1e-300, f"db {what}")
    wh = mm.act(z, act)
    close(h, wh, out_bound(wh, act_bound(z, np.zeros_like(z), act), dtype), f"h {what}")
    assert (h is dy) == over


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", mm.ACTS)
@pytest.mark.parametrize("rows,n", [(1, 2), (1, 512), (3, 70), (64, 520), (65, 1026), (200, 8), (130, 1336)])
def test_dense(rows, n, act, dtype):
    check(rows + n, [rows], n, act, dtype, grouped=False)


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("counts", [[1], [0, 2, 0], [64, 65, 63], [300, 0, 1, 129], [1] * 130, [0] * 80 + [70]],
                         ids=lambda c: f"{len(c)}x{sum(c)}")
def test_groups(counts, act):
    for n in (264, 34):
        check(n, counts, n, act, torch.bfloat16)
        check(n, counts, n, act, torch.float32, over=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["relu", "swiglu"])
def test_each_output_alone(act, dtype):
    require_gpu()
    rng = np.random.default_rng(0)
    for n in (264, 130):
        z8, z, dy = make(rng, 90, n, act, dtype)
        dz, db, h = mxq.mxq_fp8_act_grad(dy, z8, act, bias_grad=True, recompute=True)
        assert torch.equal(mxq.mxq_fp8_act_grad(dy, z8, act), dz)
        got = mxq.mxq_fp8_act_grad(dy, z8, act, bias_grad=True)
        assert torch.equal(got[0], dz) and torch.equal(got[1], db)
        got = mxq.mxq_fp8_act_grad(dy, z8, act, recompute=True)
        assert torch.equal(got[0], dz) and torch.equal(got[1], h)


def test_odd_width():
    require_gpu()
    rng = np.random.default_rng(1)
    for dtype in (torch.float32, torch.bfloat16):
        for n in (1, 131, 1025):
            z8, z, dy = make(rng, 37, n, "silu", dtype)
            want = mm.act_grad(f64(dy), z, "silu")
            close(mxq.mxq_fp8_act_grad(dy, z8, "silu"), want, out_bound(want, slope_bound(f64(dy), z, "silu"), dtype), "odd")


def test_same_bits_as_from_the_widened_values():
    """From z in fp32 with the values of z8, mxq_act_grad forms the same gradient (16 rows and more a block
    alike, so also the same sums)."""
    require_gpu()
    rng = np.random.default_rng(2)
    for act in mm.ACTS:
        z8, z, dy = make(rng, 300, 520, act, torch.float32)
        off = torch.tensor([0, 11, 11, 300], device="cuda:0")
        a = mxq.mxq_fp8_act_grad(dy, z8, act, off, bias_grad=True)
        b = mxq.mxq_act_grad(dy, to(z, torch.float32), act, off, bias_grad=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), act


def test_scales_of_every_exponent_and_nan():
    """A scale is read through its exponent field: 0 is 2^-127, 255 NaN, in its 128 columns only."""
    require_gpu()
    rows, n = 256, 200
    q = torch.from_numpy(np.random.default_rng(3).integers(0, 127, (rows, n)).astype(np.uint8)).to("cuda:0")
    bits = torch.arange(256, dtype=torch.int32)[:, None].repeat(1, 2) << 23
    bits[:, 0] |= 0x2AAAAA  # (the mantissa does not matter)
    bits[:, 1] = 127 << 23
    s = bits.view(torch.float32).to("cuda:0")
    z = moe.fp8_row_values(u8(q), bits.numpy().view(np.uint32))
    dy = torch.ones((rows, n), device="cuda:0")
    dz, h = mxq.mxq_fp8_act_grad(dy, (q, s), "none", recompute=True)
    assert torch.equal(dz, dy)
    with np.errstate(over="ignore", invalid="ignore"):
        want = z.astype(np.float32)  # rounded once where fp32 has fewer bits, infinite past its end
    assert np.array_equal(h.cpu().numpy(), want, equal_nan=True)
    assert torch.isnan(h[255, :128]).all() and torch.isfinite(h[255, 128:]).all()


def test_nan_codes_and_saturation():
    require_gpu()
    z = torch.zeros((4, 256), device="cuda:0")
    z[0], z[1], z[2, 5], z[3] = 1e4, -1e4, float("nan"), 0.0
    z8 = mxq.mxq_fp8_quantize(z)
    for act in ("silu", "gelu", "relu"):
        dz, h = mxq.mxq_fp8_act_grad(torch.full_like(z, 3.0), z8, act, recompute=True)
        zv = f64(moe_values(z8))
        assert (dz[0] == 3.0).all() and (dz[1] == 0.0).all() and (h[1] == 0).all()
        np.testing.assert_allclose(f64(h[0]), zv[0], rtol=1e-6)
        if act != "relu":
            assert torch.isnan(dz[2, :128]).all()
        assert torch.isfinite(dz[2, 128:]).all()


def moe_values(z8):
    return torch.from_numpy(moe.fp8_row_values(u8(z8[0]), bits32(z8[1])))


def test_no_rows():
    require_gpu()
    z8 = mxq.mxq_fp8_quantize(torch.empty((0, 24), device="cuda:0"))
    dy = torch.empty((0, 24), device="cuda:0")
    dz, db, h = mxq.mxq_fp8_act_grad(dy, z8, "relu", bias_grad=True, recompute=True)
    assert dz.shape == h.shape == (0, 24) and torch.equal(db, torch.zeros(24, device="cuda:0"))


@pytest.mark.parametrize("kind", PATTERNS)
@pytest.mark.parametrize("groups", [5, 130])
@pytest.mark.parametrize("m", [40, 700])
def test_malformed_offsets(m, groups, kind):
    """Results are unspecified, but nothing outside the buffers is read into a sum or written."""
    require_gpu()
    n = 136
    z8 = mxq.mxq_fp8_quantize(torch.ones(m, n, device="cuda:0"))
    (dz, dz_ok), (h, h_ok) = banded((m, n), torch.float32), banded((m, n), torch.float32)
    db, db_ok = banded((groups, n), torch.float32)
    need = mxq.lib().mxq_act_grad_workspace(m, n, groups)
    ws = torch.full((need // 4 + 2 * 65536,), float("nan"), device="cuda:0")
    inner = ws[65536:65536 + need // 4]
    inner.zero_()
    mxq.mxq_fp8_act_grad(torch.ones(m, n, device="cuda:0"), z8, "relu", offsets(kind, m, groups), bias_grad=True,
                         recompute=True, out=dz, db=db, h=h, workspace=inner.view(torch.uint8))
    assert dz_ok() and db_ok() and h_ok()
    assert torch.isnan(ws[:65536]).all() and torch.isnan(ws[65536 + need // 4:]).all()
    assert torch.isfinite(db).all() and db.min() >= 0 and db.max() <= m


def test_against_differences():
    """act'(z) against the change of act over a small step around the kept values."""
    require_gpu()
    rng = np.random.default_rng(5)
    for act in ("gelu", "silu", "swiglu"):
        z8, z, dy = make(rng, 8, 48, act, torch.float32)
        dz, dyv = f64(mxq.mxq_fp8_act_grad(dy, z8, act)), f64(dy)
        h = 1e-4  # central difference in 64 bits: error h^2 / 6 of a third derivative below 4 per unit
        for j in range(48):
            up, down = z.copy(), z.copy()
            up[:, j] += h
            down[:, j] -= h
            slope = ((mm.act(up, act) - mm.act(down, act)) * dyv).sum(1) / (2 * h)
            zmax = 1 + np.abs(z).max()
            assert np.abs(slope - dz[:, j]).max() <= 4 * h * h * zmax * np.abs(dyv).max() + 64 * U * np.abs(dyv).max() * zmax ** 2 + 1e-9
