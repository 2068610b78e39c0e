"""Scores far past 2^24, where a product with log2(e) is no longer known to a unit: only differences between scores
count, and those of equal scores are zero.

A pattern's preference of -1e30 (a mask by a number, not by -infinity) makes all scores of the first rows equal:
their weights are 1 / n. Weights are then exact but for fp32's and, in the product, the type's rounding, and so is the
output: u for a weight, u for the output, and a step of the sums.
"""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from tests import _bounds, test_paged_gpu, test_quant_gpu
from tests.test_quant_gpu import _np, saf  # noqa: F401  (saf: the fixture)

pytestmark = pytest.mark.gpu

KINDS = ["8-bit", "paged"]


def _batch(kind, dtype, T, seed):
    make = test_quant_gpu.Batch if kind == "8-bit" else test_paged_gpu.Batch
    return make(dtype, 4, 2, T, 64, 16, (0, 200), (T, T), seed=seed)


def _values(x, n):
    """The first n values [n, Hkv, d] of sequence 0."""
    return x.rows(0, n)[1] if hasattr(x, "codes") else so.gather(_np(x.vc), x.table[0], n)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 40, 90])
@pytest.mark.parametrize("score", [-1e30, -3e8, 3e8, 1e30])
def test_patterns_of_large_equal_scores(saf, kind, dtype, T, score):  # noqa: F811
    x = _batch(kind, dtype, T, 61)
    x.a[1, :3], x.r[1] = score, 0.0
    o, lse = x.call(saf, [0, 1, 1, 0])
    v = _values(x, T)[:, 0]
    for t in range(min(T, 3)):   # rows that see keys of this score alone
        want, size = v[:t + 1].mean(0), np.abs(v[:t + 1]).mean(0)
        assert (np.abs(_np(o)[0, 1, t] - want) <= (2 * _bounds.HALF[dtype] + 2.0 ** -18) * size).all(), t
        assert abs(float(lse[0, 1, t]) - score) <= 2.0 ** -21 * abs(score) + np.log(3), t
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 40, 90])
@pytest.mark.parametrize("power", [5, 15, 40])
def test_large_products(saf, kind, dtype, T, power):  # noqa: F811
    # the first token sees one key, whatever its score
    x = _batch(kind, dtype, T, 62)
    x.q *= 2.0 ** power
    if kind == "8-bit":
        x.scales[0] *= 2.0 ** power
    else:
        x.kc *= 2.0 ** power
    o, lse = x.call(saf)
    for h in range(4):
        want = _values(x, 1)[0, h // 2]
        assert (np.abs(_np(o)[0, h, 0] - want) <= (2 * _bounds.HALF[dtype] + 2.0 ** -18) * np.abs(want)).all(), h
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
