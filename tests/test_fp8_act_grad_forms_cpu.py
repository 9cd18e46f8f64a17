"""Every compiled kernel of the gradient from FP8 is launched by the calls that
tests/test_gpu_fp8_act_grad_forms.py makes, without a GPU (tests/hip_recorder.py)."""
from mxfp4_microscaling_quantization_amd import mxq
from tests.hip_recorder import kernels, record
from tests.test_gpu_fp8_act_grad_forms import FORMS
from tests.test_moe_dispatch_cpu import BASE, name, of


def test_every_kernel_from_fp8_is_among_the_forms(tmp_path):
    compiled = {k for k in kernels(tmp_path) if name(k).startswith("fp8_act_grad")}
    calls = [of("mxq_fp8_act_grad", BASE, f32, BASE, BASE, rows, n, mxq._ACT[act], None, 1, BASE,
                BASE if bias else None, BASE if again else None, BASE)
             for f32 in (0, 1) for rows, n, act, bias, again in FORMS]
    reached = set()
    for status, launches, _ in record(calls, tmp_path):
        assert status == mxq.MXQ_OK
        reached |= {k for _, k, *_ in launches if name(k).startswith("fp8_act_grad")}
    assert len(compiled) == 32 and reached == compiled, compiled ^ reached
