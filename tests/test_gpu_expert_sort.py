"""The rows of every expert against the oracle: one workgroup and many, every count of waves,
uneven experts, assignments without a row, and equal results from call to call."""
import numpy as np
import pytest
import torch

from mxfp4_microscaling_quantization_amd import mxq
from oracle import moe
from tests.gpu_helpers import require_gpu
from tests.moe_helpers import choices

pytestmark = pytest.mark.gpu


def want_of(flat: np.ndarray, n: int):
    """The oracle's answer by numpy's stable sort (pinned to the oracle by its own test and below)."""
    has = (flat >= 0) & (flat < n)
    kept = np.flatnonzero(has)
    rows = kept[np.argsort(flat[kept], kind="stable")]
    order = np.full(flat.size, -1, dtype=np.int32)
    order[:len(rows)] = rows
    positions = np.full(flat.size, -1, dtype=np.int32)
    positions[rows] = np.arange(len(rows))
    return np.concatenate([[0], np.cumsum(np.bincount(flat[kept], minlength=n))]), positions, order


def check(e: np.ndarray, n: int):
    r = mxq.mxq_expert_sort(torch.from_numpy(e).to("cuda:0"), n)
    offsets, positions, order = want_of(e.reshape(-1), n)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets), "offsets"
    assert np.array_equal(r.positions.cpu().numpy().reshape(-1), positions), "positions"
    assert np.array_equal(r.order.cpu().numpy(), order), "order"
    assert r.positions.shape == e.shape


ONE = [(tokens, k, n) for tokens, k in ((1, 1), (1, 8), (8, 8), (37, 3), (64, 1), (1365, 3), (4097, 1), (4096, 2))
       for n in (1, 2, 64, 512, 513, 4096)]
MANY = [(count, n) for count in (8193, 10007, 70001) for n in (1, 3, 65, 256, 512, 513, 1024, 1025, 4096)]
MANY += [(524288, 256), (524289, 256), (400000, 512), (360000, 512), (2 ** 21, 16), (2 ** 21 - 5, 17)]


@pytest.mark.parametrize("tokens,k,n", ONE)
def test_one_workgroup(tokens, k, n):
    require_gpu()
    rng = np.random.default_rng(n + tokens)
    check(choices(rng, tokens, n, min(k, n), 0.1), n)


@pytest.mark.parametrize("count,n", MANY)
def test_many_workgroups(count, n):
    require_gpu()
    rng = np.random.default_rng(n + count)
    p = rng.dirichlet(np.full(n, 0.3))
    e = rng.choice(n, count, p=p).astype(np.int32)
    e[rng.random(count) < 0.05] = -1
    check(e, n)


def test_more_than_a_thousand_blocks_worth():
    """Past 2^21 assignments a block takes more than 2048."""
    require_gpu()
    rng = np.random.default_rng(0)
    check(rng.integers(-1, 97, 2 ** 21 + 12345).astype(np.int32), 96)


@pytest.mark.parametrize("count", [100, 9000])
def test_extremes(count):
    require_gpu()
    check(np.zeros(count, dtype=np.int32), 7)                      # all of one expert
    check(np.full(count, 6, dtype=np.int32), 7)
    check(np.full(count, -1, dtype=np.int32), 7)                   # none has a row
    check((np.arange(count) % 7).astype(np.int32)[::-1].copy(), 7)
    e = np.full(count, 2 ** 31 - 1, dtype=np.int32)
    e[::3], e[1::3] = -2 ** 31, 3
    check(e, 7)
    check(np.full(count, 7, dtype=np.int32), 7)


def test_no_assignments():
    require_gpu()
    r = mxq.mxq_expert_sort(torch.empty((0, 4), dtype=torch.int32, device="cuda:0"), 9)
    assert torch.equal(r.offsets, torch.zeros(10, dtype=torch.int64, device="cuda:0"))
    assert r.positions.shape == (0, 4) and r.order.shape == (0,)


def test_the_oracle_on_the_same_choices():
    require_gpu()
    rng = np.random.default_rng(5)
    e = choices(rng, 700, 40, 7, 0.2)
    r = mxq.mxq_expert_sort(torch.from_numpy(e).to("cuda:0"), 40)
    for got, want in zip(r, moe.expert_sort(e, 40)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_workspace_contents_do_not_matter():
    require_gpu()
    rng = np.random.default_rng(6)
    e = torch.from_numpy(rng.integers(-1, 50, 20000).astype(np.int32)).to("cuda:0")
    need = mxq.lib().mxq_expert_sort_workspace(20000, 50)
    assert need > 0
    first = mxq.mxq_expert_sort(e, 50)
    for byte in (0, 255, 127):
        guard = torch.full((need + 64,), byte, dtype=torch.uint8, device="cuda:0")
        again = mxq.mxq_expert_sort(e, 50, workspace=guard[:need])
        for a, b in zip(first, again):
            assert torch.equal(a, b)
        assert (guard[need:] == byte).all()
