"""Inputs and error bounds shared by the tests of the operators around the experts' products
(u = 2^-24; bounds of sums, activations and outputs are those of tests/mm_helpers.py).

  exp      exp(x), x <= 0: the rounding of x (as l - max) moves the result by |x| u, the
           function itself by 8 u
  softmax  of E logits: the sum of E exponentials errs by 2 E u relative (its terms' |x| u
           weigh e^-|x| |x| <= 0.37), the quotient by u: (|x| + 3 E + 16) u in all
"""
import numpy as np
import torch

from tests.mm_helpers import DEV, U

FLOOR = 2.0 ** -120  # below it the exponentials of the hardware may be lost


def to(x: np.ndarray, dtype) -> torch.Tensor:
    """On the GPU, in this type."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).to(DEV)


def strided(t: torch.Tensor, extra: int, first: int = 0) -> torch.Tensor:
    """The same matrix inside wider rows, which start at column `first`; NaN around it."""
    wide = torch.full((t.shape[0], t.shape[1] + first + extra), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, first:first + t.shape[1]] = t
    return wide[:, first:first + t.shape[1]]


def logit_depth(logits: np.ndarray) -> np.ndarray:
    """|l - max| of every logit, 0 where that says nothing."""
    with np.errstate(invalid="ignore"):
        x = np.abs(logits - logits.max(axis=1, keepdims=True))
    return np.where(np.isfinite(x), x, 0.0)


def weight_bound(weights, experts, logits):
    x = np.take_along_axis(logit_depth(logits), np.maximum(experts, 0).astype(np.int64), axis=1)
    return np.nan_to_num(weights) * (x + 3 * logits.shape[1] + 16) * U + FLOOR


def choices(rng, tokens: int, experts: int, k: int, missing: float = 0.0) -> np.ndarray:
    """Distinct experts of every token, a share of them replaced by values that are none."""
    e = np.argsort(rng.random((tokens, experts)) * rng.random(experts), axis=1)[:, :k].astype(np.int32)
    gone = rng.random(e.shape) < missing
    return np.where(gone, rng.choice([-1, -2 ** 31, experts, 2 ** 31 - 1], e.shape), e).astype(np.int32)


def positions(rng, tokens: int, k: int, rows: int, missing: float = 0.0) -> np.ndarray:
    """Distinct rows [tokens, k] among `rows` (>= tokens k), some of them none."""
    p = rng.permutation(rows)[:tokens * k].reshape(tokens, k)
    gone = rng.random(p.shape) < missing
    return np.where(gone, rng.choice([-1, -2 ** 31, rows, 2 ** 31 - 1], p.shape), p).astype(np.int32)
