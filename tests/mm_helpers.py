"""Inputs and error bounds shared by the tests of the matrix products.

Bounds, all derived from the arithmetic (u = 2^-24):
  sum      a sum of K products in fp32, in any order and grouping, errs by at most
           2 K u times the sum of the products' magnitudes (K roundings of partial sums,
           doubled for instructions that truncate), for exact products;
  fp8 core the matrix cores keep about 16 bits of an FP8 product and add several before
           rounding: 2^-12 of the magnitudes' sum;
  act      the slopes of the activations are below 1.13 (gelu) and the hardware's
           exponential and reciprocal err by a few units: 8 u |z| (1 + |z|);
  output   one rounding, half a unit of the last place: 2^-8 of the result in bf16 (8
           significant bits), u in fp32 (24), and the least subnormal.
"""
import numpy as np
import torch

from oracle import mm

U = 2.0 ** -24
DEV = "cuda:0"


def mxfp4(rng, rows, k, lo=120, hi=131, zeros=0.1):
    c = rng.integers(0, 256, (rows, k // 2)).astype(np.uint8)
    c[rng.random(c.shape) < zeros] = 0
    return c, rng.integers(lo, hi, (rows, k // 32)).astype(np.uint8)


def fp8(rng, rows, k, lo=-4, hi=5):
    q = torch.from_numpy(rng.normal(0, 60, (rows, k))).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return q, np.ldexp(1.0, rng.integers(lo, hi, (rows, k // 128))).astype(np.float32)


def small_integers(rng, rows, k, fmt="4"):
    """Operand of integers -3..3 with scale 1: any block scale holds them exactly, and fp32
    sums of their products are exact in any order."""
    v = rng.integers(-3, 4, (rows, k)).astype(np.float32)
    if fmt == "8":
        return (torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy(),
                np.ones((rows, k // 128), dtype=np.float32))
    code = np.array([0, 2, 4, 5])[np.abs(v).astype(int)] | ((v < 0) << 3)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), np.full((rows, k // 32), 127, dtype=np.uint8)


def operand(rng, rows, k, fmt, **kw):
    return (fp8 if fmt == "8" else mxfp4)(rng, rows, k, **kw)


def columns(rng, cols, counts, ld_extra=0, lo=-4, hi=5):
    """FP8 columns of random tokens with garbage past the last token and last group."""
    rows, slots = sum(counts), sum((c + 127) // 128 for c in counts)
    ld = (rows + 15) // 16 * 16 + ld_extra
    q = rng.integers(0, 256, (cols, max(ld, 16))).astype(np.uint8)  # NaN codes among them
    v = rng.normal(0, 60, (cols, rows))
    q[:, :rows] = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    s = np.full((cols, max(1, (rows + 127 * len(counts)) // 128)), np.nan, dtype=np.float32)
    s[:, :slots] = np.ldexp(1.0, rng.integers(lo, hi, (cols, slots)))
    return q, s


def gpu(*arrays):
    return tuple(torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for a in arrays)


def f64(t):
    return t.detach().cpu().double().numpy()


def sum_bound(mag, k, fp8_core=False):
    return (2 * k * U + (2.0 ** -12 if fp8_core else 0.0)) * mag


def act_bound(z, ez, name):
    """Error bound of act(z) for an error bound ez of z."""
    own = 8 * U * np.abs(z) * (1 + np.abs(z))
    if name == "none":
        return ez
    if name == "relu":
        return ez
    if name == "swiglu":
        g, u, eg, eu = z[..., 0::2], z[..., 1::2], ez[..., 0::2], ez[..., 1::2]
        s = np.abs(mm.act(g, "silu"))
        return (1.13 * eg + own[..., 0::2]) * (np.abs(u) + eu) + s * eu
    return 1.13 * ez + own


def out_bound(want, err, dtype):
    """Bound of the stored value: the computed one is off by err, then rounded once."""
    u = 2.0 ** -8 if dtype == torch.bfloat16 else U
    return err + u * (np.abs(want) + err) + 2.0 ** -126


def close(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, f"{what}: shape {got.shape} != {want.shape}"
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN places differ ({np.isnan(got).sum()} and {nan.sum()})"
    bad = (np.abs(got - want) > bound) & ~nan
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {i}: got {got[i]!r}, expected "
                             f"{want[i]!r} within {bound[i]!r}")
