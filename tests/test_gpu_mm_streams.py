"""The matrix products' stream contract: side streams, two host threads, and HIP graph capture
with new inputs between replays give the bits of eager calls on the default stream."""
import threading

import numpy as np
import pytest
import torch

from mxfp4_microscaling_quantization_amd import mxq
from tests.gpu_helpers import require_gpu
from tests.mm_helpers import columns, gpu, operand

pytestmark = pytest.mark.gpu


def calls(seed):
    """Every kernel family once: (name, inputs that may be overwritten, function of them)."""
    require_gpu()
    rng = np.random.default_rng(seed)
    out = []
    for name, fmt, m, n, k, dtype in (("one row", "44", 1, 264, 512, torch.bfloat16),
                                      ("rows", "84", 40, 264, 512, torch.float32),
                                      ("tiles", "44", 300, 520, 640, torch.bfloat16),
                                      ("block tails", "44", 300, 520, 672, torch.float32),
                                      ("exact tiles", "88", 300, 520, 640, torch.float32)):
        a, b = gpu(*operand(rng, m, k, fmt[0])), gpu(*operand(rng, n, k, fmt[1]))
        out.append((name, a, lambda a, b=b, dtype=dtype: mxq.mxq_gemm(a, b, act="gelu", out_dtype=dtype)))
    a, b = gpu(*operand(rng, 4200, 256, "4")), gpu(*operand(rng, 4096, 256, "4"))
    out.append(("large tiles", a, lambda a, b=b: mxq.mxq_gemm(a, b)))
    counts = [70, 0, 260, 33]
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), device="cuda:0")
    a, b = gpu(*operand(rng, 363, 384, "8")), tuple(t.view(4, 264, -1) for t in gpu(*operand(rng, 4 * 264, 384, "8")))
    out.append(("grouped", a, lambda a, b=b: mxq.mxq_grouped_gemm(a, b, off, act="swiglu", preact=True)))
    y, x = gpu(*columns(rng, 200, counts)), gpu(*columns(rng, 136, counts))
    out.append(("wgrad", y, lambda y, x=x: mxq.mxq_grouped_wgrad(y, x, off, 363)))
    z, dy = (torch.from_numpy(rng.normal(0, 1, (363, 264)).astype(np.float32)).to("cuda:0") for _ in range(2))
    out.append(("act_grad", (dy, z), lambda v: mxq.mxq_act_grad(v[0], v[1], "silu", off, bias_grad=True)))
    return out


def flat(v):
    return [v] if isinstance(v, torch.Tensor) else list(v)


def same(a, b, what):
    torch.cuda.synchronize()
    for x, y in zip(flat(a), flat(b)):
        kind = torch.int16 if x.dtype == torch.bfloat16 else torch.int32
        assert torch.equal(x.view(kind), y.view(kind)), what


def test_side_stream_and_threads():
    first, second = calls(0), calls(1)
    eager = [[f(v) for _, v, f in c] for c in (first, second)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]

    def work(i, c):
        with torch.cuda.stream(streams[i]):
            for _ in range(3):
                got[i] = [f(v) for _, v, f in c]
            streams[i].synchronize()

    threads = [threading.Thread(target=work, args=(i, c)) for i, c in enumerate((first, second))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i, c in enumerate((first, second)):
        for (name, _, _), a, b in zip(c, got[i], eager[i]):
            same(a, b, name)


def test_graph_replays_with_new_inputs():
    c = calls(2)
    other = {name: tuple(t.clone() for t in v) for name, v, _ in calls(3)}
    for name, v, f in c:
        f(v)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = f(v)
        mine = tuple(t.clone() for t in v)
        for turn in range(3):
            for src in (mine, other[name]):
                for t, s in zip(v, src):
                    t.copy_(s)
                want = [t.clone() for t in flat(f(v))]
                torch.cuda.synchronize()
                g.replay()
                same(got, want, f"{name} replay {turn}")
