"""Tokens' rows sent to their experts, against the oracle and the row quantisers, bit for bit:
every format, unit and type, strides, assignments without a row, rows left as they were."""
import numpy as np
import pytest
import torch

from mxfp4_microscaling_quantization_amd import mxq
from oracle import moe
from tests.gpu_helpers import require_gpu
from tests.mm_helpers import f64
from tests.moe_helpers import positions, strided, to

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def fill(t, byte=0x5A):
    t.view(torch.uint8).fill_(byte)
    return t


def check_copy(tokens, k, width, dtype, extra=0, first=0, missing=0.2, spare=5, seed=0):
    rng = np.random.default_rng(seed + tokens + width)
    x = to(rng.normal(0, 1, (tokens, width)), dtype)
    rows = tokens * k + spare
    pos = positions(rng, tokens, k, rows, missing)
    out = fill(torch.empty((rows, width), dtype=dtype, device="cuda:0"))
    before = bits(out).cpu().numpy()
    xs = strided(x, extra, first) if extra or first else x
    got = mxq.mxq_dispatch(xs, torch.from_numpy(pos).to("cuda:0"), out=out)
    assert got is out
    want = moe.dispatch(bits(x).cpu().numpy(), pos, before)
    assert np.array_equal(bits(got).cpu().numpy(), want)


COPIES = [(1, 1, 1), (1, 8, 8), (3, 2, 7), (5, 3, 130), (2, 64, 24), (7, 5, 2056), (4, 2, 4100), (2100, 2, 264),
          (2100, 3, 33)]
QUANTISED = [(1, 1, 128), (3, 2, 384), (6, 8, 2176), (5, 2, 4096), (2, 1, 16512), (1060, 2, 256), (1030, 1, 9216)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,width", COPIES)
def test_copy(tokens, k, width, dtype):
    require_gpu()
    check_copy(tokens, k, width, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_copy_strides(dtype):
    require_gpu()
    for width, extra, first in ((64, 8, 0), (64, 8, 8), (64, 2, 0), (64, 1, 1), (64, 3, 5), (63, 1, 0), (2, 0, 2)):
        check_copy(11, 3, width, dtype, extra, first)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("tokens,k,width", QUANTISED)
def test_quantised(tokens, k, width, fmt, dtype):
    """The bits of the row quantisers on the token's row, in the rows of its assignments only."""
    require_gpu()
    rng = np.random.default_rng(tokens + width)
    x = rng.normal(0, 1, (tokens, width)) * np.exp(rng.normal(0, 2, (tokens, width // 32))).repeat(32, axis=1)
    x[0, :32] = 0.0
    x[tokens // 2, 5] = np.nan
    x[-1, -1] = -np.inf
    x[-1, 0] = 1e-42
    x = to(x, dtype)
    rows = tokens * k + 3
    pos = positions(rng, tokens, k, rows, 0.2)
    q = mxq.mxq_quantize(x)
    own = (q.codes_row, q.scales_row) if fmt == "mxfp4" else mxq.mxq_fp8_quantize(x)
    out = tuple(fill(torch.empty((rows, t.shape[1]), dtype=t.dtype, device="cuda:0")) for t in own)
    before = [bits(t).cpu().numpy() for t in out]
    got = mxq.mxq_dispatch(strided(x, 16, 8), torch.from_numpy(pos).to("cuda:0"), fmt=fmt, out=out)
    for g, t, b in zip(got, own, before):
        assert np.array_equal(bits(g).cpu().numpy(), moe.dispatch(bits(t).cpu().numpy(), pos, b))
    fresh = mxq.mxq_dispatch(x, torch.from_numpy(pos).to("cuda:0"), fmt=fmt)
    assert fresh[0].shape == (tokens * k, own[0].shape[1])  # (rows past it are dropped)


def test_mxfp4_of_a_width_that_ends_inside_a_wave():
    require_gpu()
    rng = np.random.default_rng(9)
    for width in (32, 96, 2080):
        x = to(rng.normal(0, 1, (4, width)), torch.bfloat16)
        pos = torch.arange(8, dtype=torch.int32, device="cuda:0").view(4, 2)
        codes, scales = mxq.mxq_dispatch(x, pos, fmt="mxfp4")
        q = mxq.mxq_quantize(x)
        assert torch.equal(codes, q.codes_row.repeat_interleave(2, 0)) and torch.equal(scales, q.scales_row.repeat_interleave(2, 0))


def test_nothing_to_do():
    require_gpu()
    pos = torch.empty((0, 4), dtype=torch.int32, device="cuda:0")
    assert mxq.mxq_dispatch(torch.empty((0, 64), device="cuda:0"), pos).shape == (0, 64)
    pos = torch.full((3, 2), -1, dtype=torch.int32, device="cuda:0")
    assert mxq.mxq_dispatch(torch.ones((3, 64), device="cuda:0"), pos, rows=0, fmt="mxfp4")[0].shape == (0, 32)
    out = torch.full((6, 64), 7.0, device="cuda:0")
    assert (mxq.mxq_dispatch(torch.ones((3, 64), device="cuda:0"), pos, out=out) == 7.0).all()


def test_against_indexing_through_a_sort():
    """x[order // k] where every assignment has a row."""
    require_gpu()
    rng = np.random.default_rng(3)
    x = to(rng.normal(0, 1, (300, 96)), torch.bfloat16)
    e = to(rng.integers(0, 12, (300, 4)), torch.int32)
    r = mxq.mxq_expert_sort(e, 12)
    assert torch.equal(mxq.mxq_dispatch(x, r.positions), x[(r.order // 4).long()])
    assert f64(x).shape == (300, 96)
