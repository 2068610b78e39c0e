"""Attention over 8-bit caches where value scales lie many powers of two apart, against the fp64 reference.

What a key does not give to a row must not cost that row accuracy: the bounds of tests/test_quant_gpu.py, but
with the largest product of a weight and its value's scale over the keys that the row sees, in place of the
largest weight times the largest value of the whole sequence. For bf16, the weight of key j times its value's
scale s_j may be taken as terms that leave at most 2^-21 of the largest such product of the row, in each of n
keys with codes up to 448:
    |do| <= n 2^-21 448 max_j (W_j s_j)
"""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from tests import _bounds
from tests.test_quant_gpu import DT, E4M3, SOME, Batch, _np, saf  # noqa: F401  (saf: the fixture)

pytestmark = pytest.mark.gpu


def _bounds_of_rows(dtype, q, k, v, sv, W, o, lse, a, r, i, fz):
    """Bounds of one head's rows; sv [m]: the values' scales."""
    d = q.shape[1]
    s = _bounds.logit_error(q, k, a, r, i, fz)
    if not fz:
        s += 2 * _bounds.E * (np.abs(q) @ np.abs(k).T).max() / np.sqrt(d)
        if dtype == "bf16":
            s += 2.0 ** -17 * np.abs(q).max() * np.abs(k).sum(axis=1).max() / np.sqrt(d)
    o_tol, l_tol = _bounds.fwd(dtype, W, v, o, lse, s)
    o_tol = o_tol + 2 * _bounds.E * (W @ np.abs(v))
    if dtype == "bf16":
        o_tol = o_tol + len(v) * 2.0 ** -21 * 448 * (W * sv).max(axis=1, initial=0.0)[:, None]
    return o_tol, l_tol


def _value_scales(x, b, n):
    """Scales [.., Hkv] of the first n own values of sequence b, behind the prefix's."""
    s = x.scales[1].double().numpy()[..., None]
    return np.concatenate([so.gather(s, x.prefix_pages, x.prefix)[..., 0],
                           so.gather(s, x.table[b].clamp(min=0, max=len(s) - 1), n)[..., 0]])


def _check(x, o, lse, frozen, window=0, sinks=0):
    o, lse = _np(o), _np(lse)
    q, a, r = (_np(t) for t in (x.q, x.a, x.r))
    G = q.shape[1] // x.Hkv
    for b in range(len(q)):
        n = int(x.n_new[b])
        k, v = x.rows(b, int(x.ctx[b]) + n)
        sv = _value_scales(x, b, int(x.ctx[b]) + n)
        i = x.prefix + int(x.ctx[b]) + np.arange(n)
        for h in range(q.shape[1]):
            fz = bool(frozen[h])
            kk, vv, ss = k[:, h // G], v[:, h // G], sv[:, h // G]
            W, l_ref = so.row_weights(q[b, h, :n], kk, i, a[h], r[h], fz, window, sinks)
            ref = W @ vv
            o_tol, l_tol = _bounds_of_rows(x.dtype, q[b, h, :n], kk, vv, ss, W, ref, l_ref, a[h], r[h], i, fz)
            assert (np.abs(o[b, h, :n] - ref) <= o_tol).all(), (b, h)
            assert (np.abs(lse[b, h, :n] - l_ref) <= l_tol).all(), (b, h)


def _scale_value(x, b, at, factor):
    """Own value `at` of sequence b, of every head, times a power of two."""
    page = x.scales[1].shape[2]
    x.scales[1][int(x.table[b, at // page]), :, at % page] *= factor


@pytest.mark.parametrize("dtype,d", SOME)
@pytest.mark.parametrize("H,T", [(4, 2), (4, 5), (12, 3), (6, 9), (4, 40)])
@pytest.mark.parametrize("power", [12, 22, 40])
def test_a_later_token_with_a_large_value(saf, dtype, d, H, T, power):  # noqa: F811
    # rows before the last token do not see its value, however large it is
    frozen = [h % 4 == 2 for h in range(H)]
    x = Batch(dtype, H, 2, T, d, 16, (300, 40), (T, T), seed=31 + T)
    for b in range(2):
        _scale_value(x, b, int(x.ctx[b]) + T - 1, 2.0 ** power)
    _check(x, *x.call(saf, frozen), frozen)


@pytest.mark.parametrize("dtype,d", SOME)
@pytest.mark.parametrize("T", [1, 5, 40])
@pytest.mark.parametrize("power", [12, 22, 40])
def test_a_large_value_behind_the_window(saf, dtype, d, T, power):  # noqa: F811
    # the frozen heads of a group see it, the ordinary ones do not
    frozen = [0, 1, 0, 0]
    x = Batch(dtype, 4, 1, T, d, 16, (300, 160), (T, T), seed=33)
    for b in range(2):
        _scale_value(x, b, 101, 2.0 ** power)
    _check(x, *x.call(saf, frozen, 30, 2), frozen, 30, 2)


@pytest.mark.parametrize("dtype,d", SOME)
@pytest.mark.parametrize("T", [1, 5, 40])
@pytest.mark.parametrize("at", [0, 150, 290])
@pytest.mark.parametrize("prefix", [0, 90])
def test_a_large_value_without_weight(saf, dtype, d, T, at, prefix):  # noqa: F811
    # a weight of e^-60 times 2^40: 2^-46 of the others' part
    frozen = [1, 1, 1, 1]
    x = Batch(dtype, 4, 1, T, d, 16, (300, 295), (T, T), prefix=prefix, seed=34)
    x.a[:, prefix + at] = -60.0 - x.r.abs().max()
    for b in range(2):
        _scale_value(x, b, at, 2.0 ** 40)
    _check(x, *x.call(saf, frozen), frozen)


@pytest.mark.parametrize("dtype,d", SOME)
@pytest.mark.parametrize("T", [1, 5, 40])
@pytest.mark.parametrize("masked", [-float("inf"), torch.finfo(torch.float32).min])
def test_a_large_value_that_a_pattern_hides(saf, dtype, d, T, masked):  # noqa: F811
    # some heads' patterns leave it no weight at all, however large it is; the others do not hide it
    frozen = [1, 1, 0, 1]
    x = Batch(dtype, 4, 1, T, d, 16, (300, 120), (T, T), seed=36)
    for b in range(2):
        _scale_value(x, b, 70, 2.0 ** 90)
    x.a[:2, 70] = masked
    o, lse = x.call(saf, frozen)
    x.a[:2, 70] = -200.0   # e^-200 2^90: nothing in the outputs' bits
    _check(x, o, lse, frozen)


@pytest.mark.parametrize("dtype,d", SOME)
@pytest.mark.parametrize("T", [1, 5, 40])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_value_scales_over_many_powers_of_two(saf, dtype, d, T, order):  # noqa: F811
    # scales from 2^-60 to 2^60 along the sequence
    frozen = [0, 1, 0, 0]
    x = Batch(dtype, 4, 2, T, d, 16, (700, 300), (T, T), seed=35)
    for b in range(2):
        n = int(x.ctx[b]) + T
        for at in range(n):
            p = 120 * at // n - 60
            _scale_value(x, b, at, 2.0 ** (p if order == "rising" else -p if order == "falling" else at * 37 % 121 - 60))
    _check(x, *x.call(saf, frozen), frozen)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 5, 40])
def test_an_infinity_that_was_appended(saf, dtype, T):  # noqa: F811
    # its row of values stands for NaN, and so does every output that sees it
    H, Hkv, d, page = 4, 2, 64, 16
    g = torch.Generator().manual_seed(51)
    dt = DT[dtype]
    n = 100 + T
    k, v = (torch.randn(1, Hkv, n, d, generator=g).to(dt).cuda() for _ in range(2))
    v[0, 1, 60, 7] = float("inf")
    per = -(-n // page)
    cache = [torch.zeros(per, Hkv, page, d, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    cache += [torch.zeros(per, Hkv, page, device="cuda") for _ in range(2)]
    table = torch.arange(per, dtype=torch.int32, device="cuda")[None]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    saf.saf_kv_append_quant(k, v, *cache, table, zero)
    q = torch.randn(1, H, T, d, generator=g).to(dt).cuda()
    o, lse = saf.saf_attn_paged_quant(q, *cache, table, zero + 100, n)
    assert o[:, 2:].isnan().all()
    assert torch.isfinite(o[:, :2].float()).all() and torch.isfinite(lse).all()
