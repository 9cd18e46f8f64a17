"""CPU-side checks of the C ABI and binding of the operators around the experts' products:
every declared entry point is exported, and invalid arguments are refused before the GPU is
touched. No kernel is launched here."""
import os
import re

import pytest
import torch

from mxfp4_microscaling_quantization_amd import mxq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # a 16-byte aligned, never dereferenced address
OK, EINVAL, ESHAPE, EALIGN = mxq.MXQ_OK, mxq.MXQ_EINVAL, mxq.MXQ_ESHAPE, mxq.MXQ_EALIGN


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "mxq_moe.h")).read()
    names = re.findall(r"^\s*(?:mxq_status|int64_t)\s+(mxq_\w+)\(", text, re.M)
    assert sorted(names) == ["mxq_combine", "mxq_combine_grad", "mxq_dispatch", "mxq_expert_sort",
                             "mxq_expert_sort_workspace", "mxq_fp8_act_grad", "mxq_fp8_quantize", "mxq_route",
                             "mxq_route_grad"]
    for n in names:
        assert hasattr(mxq.lib(), n), n


def call(name, defaults, kw):
    a = dict(defaults, **kw)
    assert len(a) == len(defaults)
    return getattr(mxq.lib(), name)(*a.values(), None)


ROUTE = dict(logits=FAKE, dt=0, tokens=4, experts=16, ld=16, k=2, renorm=0, weights=FAKE, chosen=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), EINVAL), (dict(weights=None), EINVAL), (dict(chosen=None), EINVAL), (dict(dt=2), EINVAL),
    (dict(tokens=-1), EINVAL), (dict(renorm=2), EINVAL), (dict(experts=0), EINVAL), (dict(experts=4097, ld=4097), EINVAL),
    (dict(k=0), EINVAL), (dict(k=17), EINVAL), (dict(experts=100, ld=100, k=65), EINVAL), (dict(ld=15), ESHAPE),
    (dict(tokens=2 ** 30), ESHAPE), (dict(tokens=2 ** 29, ld=2 ** 12), ESHAPE), (dict(logits=FAKE + 1), EALIGN),
    (dict(dt=1, logits=FAKE + 2), EALIGN), (dict(weights=FAKE + 2), EALIGN), (dict(chosen=FAKE + 1), EALIGN),
    (dict(tokens=0, logits=None, weights=None), OK),
])
def test_route_refusals(kw, status):
    assert call("mxq_route", ROUTE, kw) == status


ROUTE_GRAD = dict(dw=FAKE, weights=FAKE, chosen=FAKE, logits=FAKE, dt=0, tokens=4, experts=16, ld=16, k=2, renorm=0,
                  dlogits=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(dw=None), EINVAL), (dict(weights=None), EINVAL), (dict(chosen=None), EINVAL), (dict(dlogits=None), EINVAL),
    (dict(logits=None), EINVAL), (dict(dt=2), EINVAL), (dict(tokens=-1), EINVAL), (dict(renorm=-1), EINVAL),
    (dict(experts=0), EINVAL), (dict(experts=4097, ld=4097), EINVAL), (dict(k=0), EINVAL), (dict(k=17), EINVAL),
    (dict(ld=15), ESHAPE), (dict(tokens=2 ** 30), ESHAPE), (dict(tokens=2 ** 29, ld=2 ** 12), ESHAPE),
    (dict(logits=FAKE + 1), EALIGN), (dict(dlogits=FAKE + 1), EALIGN), (dict(dw=FAKE + 2), EALIGN),
    (dict(weights=FAKE + 2), EALIGN), (dict(chosen=FAKE + 2), EALIGN), (dict(tokens=0, dw=None), OK),
])
def test_route_grad_refusals(kw, status):
    assert call("mxq_route_grad", ROUTE_GRAD, kw) == status


SORT = dict(experts=FAKE, count=100, n=8, offsets=FAKE, positions=FAKE, order=FAKE, workspace=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(experts=None), EINVAL), (dict(offsets=None), EINVAL), (dict(positions=None), EINVAL), (dict(order=None), EINVAL),
    (dict(count=-1), EINVAL), (dict(n=0), EINVAL), (dict(n=4097), EINVAL), (dict(count=100000, workspace=None), EINVAL),
    (dict(count=2 ** 31), ESHAPE), (dict(experts=FAKE + 2), EALIGN), (dict(offsets=FAKE + 4), EALIGN),
    (dict(positions=FAKE + 1), EALIGN), (dict(order=FAKE + 2), EALIGN), (dict(workspace=FAKE + 8), EALIGN),
    (dict(count=0, offsets=None), EINVAL),
])
def test_sort_refusals(kw, status):
    assert call("mxq_expert_sort", SORT, kw) == status


def test_sort_workspace():
    ws = mxq.lib().mxq_expert_sort_workspace
    assert ws(0, 8) == 0 and ws(8192, 4096) == 0 and ws(10 ** 6, 0) == 0 and ws(10 ** 6, 4097) == 0 and ws(2 ** 31, 8) == 0
    for count, n in ((8193, 1), (524288, 256), (2 ** 21 + 1, 7), (2 ** 31 - 1, 4096)):
        chunk = 2048 if count <= 2 ** 21 else -(-count // 1024 // 256) * 256 or 256
        while chunk * 1024 < count:
            chunk += 256
        blocks = -(-count // chunk)
        assert blocks <= 1024 and ws(count, n) >= (blocks + 1) * n * 4 and ws(count, n) <= 1025 * n * 4


DISPATCH = dict(x=FAKE, dt=0, tokens=4, width=256, ldx=256, positions=FAKE, k=2, rows=8, fmt=1, out=FAKE, scales=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), EINVAL), (dict(positions=None), EINVAL), (dict(out=None), EINVAL), (dict(scales=None), EINVAL),
    (dict(dt=2), EINVAL), (dict(fmt=3), EINVAL), (dict(fmt=-1), EINVAL), (dict(tokens=-1), EINVAL), (dict(rows=-1), EINVAL),
    (dict(width=-32), EINVAL), (dict(k=0), EINVAL), (dict(k=65), EINVAL), (dict(width=0), ESHAPE),
    (dict(width=48), ESHAPE), (dict(fmt=2, width=96), ESHAPE), (dict(ldx=255), ESHAPE), (dict(rows=2 ** 31), ESHAPE),
    (dict(tokens=2 ** 30), ESHAPE), (dict(width=2 ** 22 + 32, ldx=2 ** 23), ESHAPE), (dict(tokens=2 ** 29, width=1024, ldx=2 ** 12), ESHAPE),
    (dict(x=FAKE + 8), EALIGN), (dict(ldx=260), EALIGN), (dict(out=FAKE + 8), EALIGN), (dict(positions=FAKE + 2), EALIGN),
    (dict(fmt=2, scales=FAKE + 2), EALIGN), (dict(fmt=0, x=FAKE + 1), EALIGN), (dict(fmt=0, dt=1, x=FAKE + 2), EALIGN),
    (dict(fmt=0, out=FAKE + 4), EALIGN), (dict(tokens=0, x=None), OK), (dict(rows=0, out=None, scales=None), OK),
])
def test_dispatch_refusals(kw, status):
    assert call("mxq_dispatch", DISPATCH, kw) == status


COMBINE = dict(y=FAKE, ydt=0, rows=8, width=33, positions=FAKE, weights=FAKE, tokens=4, k=2, residual=None, out=FAKE, odt=1)


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), EINVAL), (dict(positions=None), EINVAL), (dict(out=None), EINVAL), (dict(ydt=2), EINVAL),
    (dict(odt=-1), EINVAL), (dict(rows=-1), EINVAL), (dict(tokens=-1), EINVAL), (dict(width=-1), EINVAL), (dict(k=0), EINVAL),
    (dict(k=65), EINVAL), (dict(width=0), ESHAPE), (dict(width=2 ** 22 + 1), ESHAPE), (dict(rows=2 ** 31), ESHAPE),
    (dict(tokens=2 ** 30), ESHAPE), (dict(tokens=2 ** 28, width=4097), ESHAPE), (dict(y=FAKE + 8), EALIGN),
    (dict(positions=FAKE + 2), EALIGN), (dict(weights=FAKE + 2), EALIGN), (dict(residual=FAKE + 8), EALIGN),
    (dict(out=FAKE + 4), EALIGN), (dict(tokens=0, y=None, out=None), OK),
])
def test_combine_refusals(kw, status):
    assert call("mxq_combine", COMBINE, kw) == status


COMBINE_GRAD = dict(grad=FAKE, gdt=1, y=FAKE, ydt=0, rows=8, width=33, positions=FAKE, weights=FAKE, tokens=4, k=2, dy=FAKE,
                    dw=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(grad=None), EINVAL), (dict(y=None), EINVAL), (dict(positions=None), EINVAL), (dict(dy=None), EINVAL),
    (dict(gdt=2), EINVAL), (dict(ydt=2), EINVAL), (dict(rows=-1), EINVAL), (dict(tokens=-1), EINVAL), (dict(k=0), EINVAL),
    (dict(k=65), EINVAL), (dict(width=0), ESHAPE), (dict(width=2 ** 22 + 1), ESHAPE), (dict(rows=2 ** 31), ESHAPE),
    (dict(tokens=2 ** 30), ESHAPE), (dict(grad=FAKE + 8), EALIGN), (dict(y=FAKE + 4), EALIGN), (dict(dy=FAKE + 8), EALIGN),
    (dict(dw=FAKE + 2), EALIGN), (dict(positions=FAKE + 2), EALIGN), (dict(weights=FAKE + 2), EALIGN),
    (dict(tokens=0, grad=None), OK), (dict(rows=0, dw=None, y=None, dy=None), OK),
])
def test_combine_grad_refusals(kw, status):
    assert call("mxq_combine_grad", COMBINE_GRAD, kw) == status


FP8 = dict(x=FAKE, dt=0, rows=4, cols=200, ldx=200, q8=FAKE, scales=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), EINVAL), (dict(q8=None), EINVAL), (dict(scales=None), EINVAL), (dict(dt=2), EINVAL), (dict(rows=-1), EINVAL),
    (dict(cols=-1), EINVAL), (dict(cols=0), ESHAPE), (dict(ldx=199), ESHAPE), (dict(cols=2 ** 30, ldx=2 ** 30), ESHAPE),
    (dict(rows=2 ** 33), ESHAPE), (dict(x=FAKE + 1), EALIGN), (dict(dt=1, x=FAKE + 2), EALIGN), (dict(q8=FAKE + 8), EALIGN),
    (dict(scales=FAKE + 2), EALIGN), (dict(rows=0, x=None), OK),
])
def test_fp8_quantize_refusals(kw, status):
    assert call("mxq_fp8_quantize", FP8, kw) == status


FP8_GRAD = dict(dy=FAKE, dt=0, z8=FAKE, scales=FAKE, rows=4, n=8, act=1, off=None, E=1, dz=FAKE, db=None, h=None, ws=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), EINVAL), (dict(z8=None), EINVAL), (dict(scales=None), EINVAL), (dict(dz=None), EINVAL),
    (dict(db=FAKE), EINVAL), (dict(dt=2), EINVAL), (dict(act=5), EINVAL), (dict(act=-1), EINVAL), (dict(rows=-1), EINVAL),
    (dict(n=-1), EINVAL), (dict(E=2), EINVAL), (dict(off=FAKE, E=0), EINVAL), (dict(off=FAKE, E=4097), EINVAL),
    (dict(n=0), ESHAPE), (dict(act=4, n=7), ESHAPE), (dict(n=2 ** 31), ESHAPE), (dict(rows=2 ** 21, n=2 ** 20), ESHAPE),
    (dict(dt=1, rows=2 ** 30 + 2 ** 14, n=512), ESHAPE), (dict(rows=2 ** 30 + 2 ** 14, n=1024), ESHAPE),
    (dict(dy=FAKE + 8), EALIGN), (dict(z8=FAKE + 8), EALIGN), (dict(scales=FAKE + 2), EALIGN), (dict(dz=FAKE + 2), EALIGN),
    (dict(h=FAKE + 8), EALIGN), (dict(db=FAKE + 4, ws=FAKE), EALIGN), (dict(db=FAKE, ws=FAKE + 8), EALIGN),
    (dict(off=FAKE + 4), EALIGN), (dict(rows=0, dy=None, z8=None, dz=None), OK),
])
def test_fp8_act_grad_refusals(kw, status):
    assert call("mxq_fp8_act_grad", FP8_GRAD, kw) == status


U8, I32, F32, BF16, I64 = torch.uint8, torch.int32, torch.float32, torch.bfloat16, torch.int64


def cpu(shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


POS = cpu((4, 2), I32)


@pytest.mark.parametrize("make,error", [
    (lambda: mxq.mxq_route(cpu((4, 8), torch.float16), 2), TypeError),
    (lambda: mxq.mxq_route(cpu((8, 4)).t(), 2), ValueError),
    (lambda: mxq.mxq_route(cpu((4,)), 2), ValueError),
    (lambda: mxq.mxq_route(cpu((4, 8)), 2, out=(cpu((4, 3)), cpu((4, 2), I32))), ValueError),
    (lambda: mxq.mxq_route(cpu((4, 8)), 2, out=(cpu((4, 2)), cpu((4, 2), I64))), ValueError),
    (lambda: mxq.mxq_route_grad(cpu((3, 2)), cpu((4, 2)), cpu((4, 2), I32), cpu((4, 8))), ValueError),
    (lambda: mxq.mxq_route_grad(cpu((4, 2)), cpu((4, 3)), cpu((4, 2), I32), cpu((4, 8))), ValueError),
    (lambda: mxq.mxq_route_grad(cpu((4, 2)), cpu((4, 2)), cpu((4, 2), I64), cpu((4, 8))), ValueError),
    (lambda: mxq.mxq_route_grad(cpu((4, 2)), cpu((4, 2)), cpu((4, 2), I32), cpu((4, 8)), out=cpu((4, 8), BF16)), ValueError),
    (lambda: mxq.mxq_expert_sort(cpu((4, 2), I64), 8), ValueError),
    (lambda: mxq.mxq_expert_sort(cpu((2, 4), I32).t(), 8), ValueError),
    (lambda: mxq.mxq_expert_sort(cpu((4, 2), I32), 8, workspace=cpu((4, 4), U8)[:, ::2]), ValueError),
    (lambda: mxq.mxq_expert_sort(cpu((9000,), I32), 8, workspace=cpu((8,), U8)), ValueError),
    (lambda: mxq.mxq_expert_sort(cpu((4, 2), I32), 8, out=mxq.ExpertRows(cpu((8,), I64), POS, cpu((8,), I32))), ValueError),
    (lambda: mxq.mxq_dispatch(cpu((4, 32)), cpu((4, 2), I64)), ValueError),
    (lambda: mxq.mxq_dispatch(cpu((4, 32)), cpu((3, 2), I32)), ValueError),
    (lambda: mxq.mxq_dispatch(cpu((4, 32)), cpu((8,), I32)), ValueError),
    (lambda: mxq.mxq_dispatch(cpu((4, 32)), POS, fmt="int8"), KeyError),
    (lambda: mxq.mxq_dispatch(cpu((4, 32)), POS, rows=8, out=cpu((7, 32))), ValueError),
    (lambda: mxq.mxq_dispatch(cpu((4, 32)), POS, out=cpu((8, 32), BF16)), ValueError),
    (lambda: mxq.mxq_dispatch(cpu((4, 32)), POS, fmt="mxfp4", out=(cpu((8, 16), U8), cpu((8, 2), U8))), ValueError),
    (lambda: mxq.mxq_dispatch(cpu((4, 128)), POS, fmt="fp8", out=(cpu((8, 128), U8), cpu((8, 1), U8))), ValueError),
    (lambda: mxq.mxq_dispatch(cpu((4, 32), torch.float16), POS), TypeError),
    (lambda: mxq.mxq_combine(cpu((8, 32)), POS, cpu((4, 3))), ValueError),
    (lambda: mxq.mxq_combine(cpu((8, 32)), POS, cpu((4, 2), BF16)), ValueError),
    (lambda: mxq.mxq_combine(cpu((8, 32)), POS, residual=cpu((4, 32))), ValueError),          # result in bf16
    (lambda: mxq.mxq_combine(cpu((8, 32)), POS, residual=cpu((4, 31)), out_dtype=F32), ValueError),
    (lambda: mxq.mxq_combine(cpu((8, 32)), POS, out=cpu((3, 32))), ValueError),
    (lambda: mxq.mxq_combine(cpu((8, 64))[:, ::2], POS), ValueError),
    (lambda: mxq.mxq_combine_grad(cpu((4, 31)), cpu((8, 32)), POS), ValueError),
    (lambda: mxq.mxq_combine_grad(cpu((4, 32)), cpu((8, 32), torch.float16), POS), TypeError),
    (lambda: mxq.mxq_combine_grad(cpu((4, 32)), cpu((8, 32)), POS, cpu((2, 4))), ValueError),
    (lambda: mxq.mxq_combine_grad(cpu((4, 32)), cpu((8, 32)), POS, out=cpu((8, 32), BF16)), ValueError),
    (lambda: mxq.mxq_combine_grad(cpu((4, 32)), cpu((8, 32)), POS, dw=cpu((8,))), ValueError),
    (lambda: mxq.mxq_fp8_quantize(cpu((4, 32), torch.float16)), TypeError),
    (lambda: mxq.mxq_fp8_quantize(cpu((32, 4)).t()), ValueError),
    (lambda: mxq.mxq_fp8_quantize(cpu((4, 200)), out=(cpu((4, 200), U8), cpu((4, 1)))), ValueError),
    (lambda: mxq.mxq_fp8_act_grad(cpu((4, 8)), (cpu((4, 8), U8), cpu((4, 2)))), ValueError),
    (lambda: mxq.mxq_fp8_act_grad(cpu((4, 8)), (cpu((4, 8), U8), cpu((4, 1), BF16))), ValueError),
    (lambda: mxq.mxq_fp8_act_grad(cpu((4, 8)), (cpu((4, 8), U8), cpu((4, 1))), "swiglu"), ValueError),
    (lambda: mxq.mxq_fp8_act_grad(cpu((4, 8)), (cpu((4, 8), torch.int8), cpu((4, 1)))), ValueError),
    (lambda: mxq.mxq_fp8_act_grad(cpu((4, 8)), (cpu((4, 8), U8), cpu((4, 1))), offsets=cpu((3,), I32)), ValueError),
    (lambda: mxq.mxq_fp8_act_grad(cpu((4, 8)), (cpu((4, 8), U8), cpu((4, 1))), recompute=True, h=cpu((4, 4))), ValueError),
    (lambda: mxq.mxq_fp8_act_grad(cpu((4, 8)), (cpu((4, 8), U8), cpu((4, 1))), bias_grad=True, db=cpu((4,))), ValueError),
    (lambda: mxq.mxq_fp8_act_grad(cpu((4, 8)), (cpu((4, 8), U8), cpu((4, 1))), out=cpu((4, 8), BF16)), ValueError),
])
def test_binding_refusals(make, error):
    with pytest.raises(error):
        make()


def test_header_is_plain_c(tmp_path):
    """include/mxq_moe.h compiles as C and as C++ by itself."""
    import shutil
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "mxq_moe.h"\nint main(void) { return MXQ_ROWS_FP8 - 2 + MXQ_ROWS_COPY; }\n')
    for cc, std in (("gcc", "-std=c99"), ("g++", "-std=c++11")):
        if shutil.which(cc):
            subprocess.run([cc, std, "-Wall", "-Werror", "-x", "c" if cc == "gcc" else "c++", "-fsyntax-only", "-I",
                            os.path.join(ROOT, "include"), str(src)], check=True)
