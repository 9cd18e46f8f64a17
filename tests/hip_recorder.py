"""What libmxq launches for a call, without a GPU: tests/host/hip_recorder.c stands in for
the HIP runtime in a process of its own.

record([(device, failures, entry point, arguments), ...]) returns, call by call, (status,
launches, attributes): launches [(device, kernel, workgroups, threads, dynamic LDS)], attributes [(device, kernel,
value)]; a kernel is (name, template arguments). kernels() lists every compiled one."""
import ctypes
import json
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp4_microscaling_quantization_amd", "libmxq.so")
SOURCE = os.path.join(ROOT, "tests", "host", "hip_recorder.c")


def _run(calls, tmp):
    cc = shutil.which("gcc")
    if not cc:
        pytest.skip("no C compiler")
    shim = os.path.join(str(tmp), "hip_recorder.so")
    if not os.path.exists(shim):
        subprocess.run([cc, "-std=c99", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", SOURCE, "-o", shim], check=True)
    r = subprocess.run([sys.executable, os.path.abspath(__file__), shim], input=json.dumps(calls), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout)


def parse(symbol):
    """(kernel, its template arguments: booleans and numbers, then the types "bf16" and "fp32")."""
    m = re.match(r"_ZN3mxq12_GLOBAL__N_1\d+(\w+?_kernel)(?:I((?:L[bi]\d+E|DF16b|f)*)E)?", symbol)
    if not m:
        return symbol, ()
    args = re.findall(r"L([bi])(\d+)E|(DF16b|f)", m.group(2) or "")
    return m.group(1), tuple({"DF16b": "bf16", "f": "fp32"}[t] if t else bool(int(v)) if k == "b" else int(v)
                             for k, v, t in args)


def record(calls, tmp):
    out = []
    for status, log in _run(calls, tmp)["calls"]:
        lines = [line.split() for line in log.splitlines()]
        out.append((status, [(int(x[1]), parse(x[2]), int(x[3]), int(x[4]), int(x[5])) for x in lines
                             if x[0] == "launch"],
                    [(int(x[1]), parse(x[2]), int(x[3])) for x in lines if x[0] == "attribute"]))
    return out


def kernels(tmp):
    return [parse(k) for k in _run([], tmp)["kernels"]]


def main():
    shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
    shim.rec_log.restype = shim.rec_kernel.restype = ctypes.c_char_p
    lib = ctypes.CDLL(LIB)
    out = []
    for device, failures, name, args in json.load(sys.stdin):
        shim.rec_start(device, failures)
        status = getattr(lib, name)(*(ctypes.c_int64(0 if a is None else a) for a in args))
        out.append((status, shim.rec_log().decode()))
    print(json.dumps({"calls": out, "kernels": [shim.rec_kernel(i).decode() for i in range(shim.rec_kernels())]}))


if __name__ == "__main__":
    main()
