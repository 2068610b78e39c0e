"""Patterns of the first and the last head, whose runs end with the array, at every place in a 16-byte line."""
import pytest
import torch

from tests.test_quant_gpu import Batch, saf  # noqa: F401  (saf: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("word", [0, 1, 2, 3])
@pytest.mark.parametrize("extra", [0, 1, 2, 3])
@pytest.mark.parametrize("ctx,T", [(0, 40), (77, 40), (300, 65)])
def test_runs_that_end_with_the_array(saf, word, extra, ctx, T):  # noqa: F811
    frozen = [1, 0, 0, 1]
    x = Batch("bf16", 4, 1, T, 64, 16, (ctx + extra, 0), (T, T), seed=92 + extra)
    L = x.a.shape[1]
    big = torch.full((2, 4 * L + 8), float("nan"), device="cuda")
    a, r = (y[word:word + 4 * L].view(4, L) for y in big)
    a.copy_(x.a)
    r.copy_(x.r)
    x.check(*x.call(saf, frozen, a=a, r=r), frozen)


def test_one_head_and_few_tokens(saf):  # noqa: F811
    # padded batches of one or two tokens: runs of a few entries at the array's first
    for T in (33, 34, 35, 36):
        for word in range(4):
            x = Batch("bf16", 1, 1, T, 64, 16, (0, 0), (1, 2), seed=T, max_len=T)
            big = torch.full((2, T + 8), float("nan"), device="cuda")
            a, r = (y[word:word + T].view(1, T) for y in big)
            a.copy_(x.a)
            r.copy_(x.r)
            x.check(*x.call(saf, [1], a=a, r=r), [1])
