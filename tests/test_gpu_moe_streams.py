"""The stream contract of the operators around the experts' products: side streams, two host
threads, and HIP graph capture with new inputs between replays give the bits of eager calls on
the default stream; and calls in flight together do not meet in a workspace."""
import threading

import numpy as np
import pytest
import torch

from mxfp4_microscaling_quantization_amd import mxq
from tests.gpu_helpers import require_gpu
from tests.moe_helpers import choices, positions, to
from tests.test_gpu_mm_streams import flat

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def calls(seed):
    """Every kernel family: (name, inputs that may be overwritten, function of them)."""
    require_gpu()
    rng = np.random.default_rng(seed)

    def normal(*shape, dtype=BF):
        return to(rng.normal(0, 1, shape), dtype)

    out = []
    for E, dtype, renorm in ((61, F32, True), (256, BF, False), (700, BF, True)):
        l = normal(301, E, dtype=dtype)
        w, e = mxq.mxq_route(l, 6, renorm=renorm)
        out.append((f"route {E}", (l,), lambda v, renorm=renorm: mxq.mxq_route(v[0], 6, renorm=renorm)))
        out.append((f"route gradient {E}", (normal(301, 6, dtype=F32), w, e, l),
                    lambda v, renorm=renorm: mxq.mxq_route_grad(*v, renorm=renorm)))
    for T in (40, 5000):
        out.append((f"sort {T}", (to(choices(rng, T, 64, 4, 0.1), I32),), lambda v: mxq.mxq_expert_sort(v[0], 64)))
    T, k, H = 130, 3, 1280
    pos = to(positions(rng, T, k, T * k), I32)
    w = normal(T, k, dtype=F32)
    for fmt in (None, "mxfp4", "fp8"):
        out.append((f"dispatch {fmt}", (normal(T, H), pos), lambda v, fmt=fmt: mxq.mxq_dispatch(*v, fmt=fmt)))
    for H in (1280, 333):
        y, g = normal(T * k, H), normal(T, H, dtype=F32)
        out.append((f"combine {H}", (y, pos, w, g), lambda v: mxq.mxq_combine(*v, out_dtype=F32)))
        out.append((f"combine gradient {H}", (g, y, pos, w), lambda v: mxq.mxq_combine_grad(*v)))
        z = normal(T * k, H)
        out.append((f"fp8 rows {H}", (z,), lambda v: mxq.mxq_fp8_quantize(v[0])))
        off = torch.tensor([0, 70, 70, T * k], device="cuda:0")
        out.append((f"fp8 gradient {H}", (normal(T * k, H), *mxq.mxq_fp8_quantize(z)),
                    lambda v, off=off: mxq.mxq_fp8_act_grad(v[0], (v[1], v[2]), "silu", off, bias_grad=True, recompute=True)))
    return out


def check(a, b, what):
    torch.cuda.synchronize()
    for x, y in zip(flat(a), flat(b)):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)), what


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
            check(a, b, name)


def test_graph_replays_with_new_inputs():
    other = {name: tuple(t.clone() for t in v) for name, v, _ in calls(3)}
    for name, v, f in calls(2):
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
                check(got, want, f"{name} replay {turn}")


def test_two_graphs_in_flight_together():
    """Sorts and gradients that each need a workspace, captured apart and replayed on two streams."""
    pairs = [[c for c in calls(s) if c[0] in ("sort 5000", "fp8 gradient 1280")] for s in (4, 5)]
    want = [[[t.clone() for t in flat(f(v))] for _, v, f in p] for p in pairs]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in pairs]
    torch.cuda.synchronize()
    for p in pairs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([f(v) for _, v, f in p])
        graphs.append(g)
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(5):
                    g.replay()
        torch.cuda.synchronize()
        for o, w, p in zip(outs, want, pairs):
            for got, ref, c in zip(o, w, p):
                check(got, ref, c[0])

