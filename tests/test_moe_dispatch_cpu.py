"""Which kernels the operators around the experts' products launch, without a GPU
(tests/hip_recorder.py): every compiled one is reached by the sizes that the GPU tests run, and
grids and LDS stay within a launch's limits at the largest sizes that the ABI takes."""
import re

from mxfp4_microscaling_quantization_amd import mxq
from tests import test_gpu_combine as combine
from tests import test_gpu_dispatch as dispatch
from tests import test_gpu_expert_sort as sort
from tests import test_gpu_fp8_rows as fp8
from tests import test_gpu_route as route
from tests.hip_recorder import kernels, record

BASE = 0x10000  # a 16-byte aligned, never dereferenced address


def name(kernel):
    m = re.match(r"_ZN3mxq12_GLOBAL__N_1\d+(\w+_kernel)", kernel[0])
    return m.group(1) if m else kernel[0]


def is_mine(kernel):
    return bool(re.match(r"route|sort_|dispatch_|combine_|fp8_rows|fp8_act_grad", name(kernel)))


def of(entry, *args):
    return (0, 0, entry, [*args, None])


def calls():
    for f32 in (0, 1):
        for E, k in route.SIZES:
            yield of("mxq_route", BASE, f32, 37, E, E, k, 0, BASE, BASE)
            yield of("mxq_route_grad", BASE, BASE, BASE, BASE, f32, 37, E, E, k, 0, BASE)
        for tokens, k, width in dispatch.COPIES:
            yield of("mxq_dispatch", BASE, f32, tokens, width, width, BASE, k, tokens * k, 0, BASE, None)
        for fmt in (1, 2):
            for tokens, k, width in dispatch.QUANTISED:
                yield of("mxq_dispatch", BASE, f32, tokens, width, width, BASE, k, tokens * k, fmt, BASE, BASE)
        for rows, cols in fp8.SIZES:
            yield of("mxq_fp8_quantize", BASE, f32, rows, cols, cols, BASE, BASE)
        for out in (0, 1):
            for tokens, k, width in combine.SIZES:
                yield of("mxq_combine", BASE, f32, tokens * k, width, BASE, BASE, tokens, k, None, BASE, out)
                for dw in (None, BASE):
                    yield of("mxq_combine_grad", BASE, f32, BASE, out, tokens * k, width, BASE, BASE, tokens, k, BASE, dw)
        # (tests/test_gpu_fp8_act_grad.py: test_dense, test_each_output_alone and test_odd_width)
        for rows, n, acts in ((65, 512, (3, 4)), (130, 1026, (3, 4)), (37, 131, (3,))):
            for act in acts:
                for db in (None, BASE):
                    for h in (None, BASE):
                        yield of("mxq_fp8_act_grad", BASE, f32, BASE, BASE, rows, n, act, None, 1, BASE, db, h, BASE)
    for tokens, k, n in sort.ONE:
        yield of("mxq_expert_sort", BASE, tokens * min(k, n), n, BASE, BASE, BASE, BASE)
    for count, n in sort.MANY:
        yield of("mxq_expert_sort", BASE, count, n, BASE, BASE, BASE, BASE)


def test_every_compiled_kernel_is_among_the_tested_calls(tmp_path):
    compiled = {k for k in kernels(tmp_path) if is_mine(k)}
    reached = set()
    for status, launches, _ in record(list(calls()), tmp_path):
        assert status == mxq.MXQ_OK and launches
        for _, kernel, grid, threads, lds in launches:
            assert grid >= 1 and 64 <= threads <= 1024 and lds <= 65536
            reached |= {kernel} if is_mine(kernel) else set()
    assert len(compiled) > 60 and reached == compiled, compiled ^ reached


def test_largest_sizes_stay_within_a_launch(tmp_path):
    most = 2 ** 31 - 1
    big = [of("mxq_route", BASE, 0, most, 4, 4, 1, 0, BASE, BASE),
           of("mxq_route_grad", BASE, BASE, BASE, BASE, 0, most, 4, 4, 1, 0, BASE),
           of("mxq_route", BASE, 0, 2 ** 28 - 1, 4096, 4096, 8, 0, BASE, BASE),
           of("mxq_expert_sort", BASE, most, 4096, BASE, BASE, BASE, BASE),
           of("mxq_dispatch", BASE, 0, 2 ** 30, 256, 256, BASE, 1, most, 0, BASE, None),
           of("mxq_dispatch", BASE, 1, 2 ** 16, 2 ** 22, 2 ** 22, BASE, 2, 2 ** 17, 0, BASE, None),
           of("mxq_dispatch", BASE, 1, 2 ** 16, 2 ** 22, 2 ** 22, BASE, 2, 2 ** 17, 2, BASE, BASE),
           of("mxq_combine", BASE, 0, 2 ** 18, 2 ** 22 - 1, BASE, None, 2 ** 16, 64, None, BASE, 1),
           of("mxq_combine_grad", BASE, 0, BASE, 0, 2 ** 18, 2 ** 22, BASE, None, 2 ** 16, 64, BASE, BASE),
           of("mxq_fp8_act_grad", BASE, 1, BASE, BASE, 2 ** 30 - 2 ** 13, 512, 3, None, 1, BASE, BASE, BASE, BASE),
           of("mxq_fp8_act_grad", BASE, 0, BASE, BASE, 2 ** 31 - 2 ** 13, 512, 3, None, 1, BASE, None, BASE, BASE),
           of("mxq_fp8_quantize", BASE, 1, 2 ** 10, 2 ** 30 - 1, 2 ** 30 - 1, BASE, BASE)]
    for call, (status, launches, _) in zip(big, record(big, tmp_path)):
        assert status == mxq.MXQ_OK and launches, call
        for _, kernel, grid, threads, lds in launches:
            assert grid * threads < 2 ** 32 and lds <= 65536, (call, kernel, grid, threads)
