"""The operators around the experts' products from a plain C program
(tests/c_caller/mxq_moe_caller.c: gcc, include/mxq_moe.h, hipMalloc; no PyTorch): one chain of
them, every output against the oracle on the outputs that went into it."""
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import mm, moe, mx
from tests import test_gpu_c_caller as caller
from tests.gpu_helpers import assert_equal_bits, require_gpu
from tests.mm_helpers import U, act_bound
from tests.moe_helpers import FLOOR, logit_depth, weight_bound
from tests.test_gpu_act_grad import slope_bound

pytestmark = pytest.mark.gpu


def near(got, want, bound, what):
    assert (np.abs(got.astype(np.float64) - want) <= bound).all(), what


@pytest.mark.parametrize("T,E,k,W", [(5, 4, 2, 96), (3000, 60, 4, 160)])
def test_chain(tmp_path, monkeypatch, T, E, k, W):
    require_gpu()
    monkeypatch.setattr(caller, "SRC", os.path.join(caller.ROOT, "tests", "c_caller", "mxq_moe_caller.c"))
    exe = caller.build(str(tmp_path))
    rng = np.random.default_rng(T)
    logits = rng.normal(0, 1, (T, E)).astype(np.float32)
    x = torch.from_numpy(rng.normal(0, 1, (T, W))).to(torch.bfloat16)
    lf, xf, prefix = (os.path.join(str(tmp_path), n) for n in ("l.bin", "x.bin", "out"))
    logits.tofile(lf)
    x.view(torch.int16).numpy().tofile(xf)
    r = subprocess.run([exe, *map(str, (T, E, k, W)), lf, xf, prefix], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr

    def out(name, dtype, *shape):
        return np.fromfile(f"{prefix}.{name}", dtype=dtype).reshape(shape)

    R, l = T * k, logits.astype(np.float64)
    weights, experts = out("weights", np.float32, T, k), out("experts", np.int32, T, k)
    ww, we = moe.route(l, k, True)
    assert np.array_equal(experts, we)
    near(weights, ww, weight_bound(ww, we, l), "weights")
    offsets, pos, order = moe.expert_sort(we, E)
    assert np.array_equal(out("offsets", np.int64, E + 1), offsets)
    assert np.array_equal(out("positions", np.int32, T, k), pos) and np.array_equal(out("order", np.int32, R), order)
    codes, scales = mx.mxfp4_quantize_rowwise(x.double().numpy())
    codes, scales = codes[order // k], scales[order // k]
    assert_equal_bits(out("codes", np.uint8, R, W // 2), codes, "codes")
    assert_equal_bits(out("scales", np.uint8, R, W // 32), scales, "scales")
    rows = out("rows", np.float32, R, W).astype(np.float64)
    assert np.array_equal(rows, mx.mxfp4_dequantize_values(codes, scales))
    wf = weights.astype(np.float64)
    want, mag = moe.combine(rows, pos, wf)
    res = out("out", np.float32, T, W).astype(np.float64)
    near(res, want, (k + 3) * U * mag + 2.0 ** -126, "out")
    dy, dw = out("dy", np.float32, R, W), out("dw", np.float32, T, k)
    wdy, wdw, mag = moe.combine_grad(res, rows, pos, wf)
    near(dy, wdy, 2 * U * np.abs(wdy) + 2.0 ** -126, "dy")
    near(dw, wdw, 2 * W * U * mag + 2.0 ** -126, "dw")
    want, mag = moe.route_grad(dw.astype(np.float64), wf, we, l, True)
    near(out("dlogits", np.float32, T, E), want, (k + 9 + logit_depth(l) + 3 * E + 16) * U * mag + FLOOR, "dlogits")
    q8, s8 = moe.fp8_rows(rows)
    assert_equal_bits(out("q8", np.uint8, R, W), q8, "FP8 codes")
    assert_equal_bits(out("s8", np.uint32, R, (W + 127) // 128), s8, "FP8 scales")
    z, g = moe.fp8_row_values(q8, s8), dy.astype(np.float64)
    want, err = mm.act_grad(g, z, "silu"), slope_bound(g, z, "silu")
    near(out("dz", np.float32, R, W), want, err + U * (np.abs(want) + err) + 2.0 ** -126, "dz")
    wh, eh = mm.act(z, "silu"), act_bound(z, np.zeros_like(z), "silu")
    near(out("h", np.float32, R, W), wh, eh + U * (np.abs(wh) + eh) + 2.0 ** -126, "h")
    db = out("db", np.float32, E, W)
    for e in range(E):
        part = slice(offsets[e], offsets[e + 1])
        near(db[e], want[part].sum(0), (2 * R * U * np.abs(want[part]) + err[part]).sum(0) + 1e-300, f"db {e}")
