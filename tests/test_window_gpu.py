"""GPU parity of the layer with a sliding window and sinks (saf_attn_fwd_window,
saf_attn_bwd_window) against the fp64 reference, with bounds from tests/_bounds.py.

Sizes where it can go wrong: windows of one key, around a tile's edge and longer than
several tiles, sinks inside and across the first tile and behind the window, lengths of one
token, a full tile and odd ones, groups with and without frozen heads.
"""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from softmax_attention_hybrid_gb300.inputs import custom_workload, make_gqa_inputs
from tests import _bounds

pytestmark = pytest.mark.gpu

# (T, window, sinks)
SPANS = [(1, 1, 0), (1, 5, 3), (2, 1, 0), (64, 7, 0), (127, 1, 1), (129, 128, 0), (130, 127, 4), (257, 1, 0),
         (300, 64, 4), (385, 129, 130), (513, 100, 300), (640, 256, 0), (700, 333, 1), (701, 2, 700)]


@pytest.fixture(scope="module")
def saf():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from softmax_attention_hybrid_gb300 import saf as mod
    return mod


def _inputs(dtype, B, H, Hkv, T, d, frozen, seed):
    w = custom_workload(B, H, T, d=d, dtype=dtype, frozen=frozen, scale=1.0, slope=0.03)
    x = make_gqa_inputs(w, Hkv, seed=seed)
    g = {n: x[n].cuda() for n in ("q", "k", "v", "do", "a", "r")}
    return x, g


def _np(t):
    return t.double().cpu().numpy()


def _run(saf, g, frozen, window, sinks, **kw):
    o, lse = saf.saf_attn_fwd_window(g["q"], g["k"], g["v"], g["a"], g["r"], frozen, window, sinks, **kw)
    dq = torch.full_like(g["q"], 7.0)
    dq, dk, dv = saf.saf_attn_bwd_window(g["q"], g["k"], g["v"], o, g["do"], lse, g["a"], g["r"], frozen, window,
                                         sinks, dq=dq, **kw)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _check(dtype, x, out, frozen, window, sinks):
    """Ordinary heads and the groups without a frozen head, against the reference."""
    q, k, v, do, a, r = (_np(x[n]) for n in ("q", "k", "v", "do", "a", "r"))
    B, H, T, d = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    got = {n: _np(t) for n, t in out.items()}
    assert all(np.isfinite(t).all() for t in got.values())
    u = _bounds.HALF[dtype]
    i = np.arange(T)
    for b in range(B):
        for hk in range(Hkv):
            tk, tv = np.zeros((T, d)), np.zeros((T, d))
            dk, dv = np.zeros((T, d)), np.zeros((T, d))
            for h in range(hk * G, hk * G + G):
                if frozen[h]:
                    assert not got["dq"][b, h].any()
                    continue
                W, lse = so.row_weights(q[b, h], k[b, hk], i, a[h], r[h], False, window, sinks)
                o = W @ v[b, hk]
                s = _bounds.logit_error(q[b, h], k[b, hk], a[h], r[h], i, False)
                o_tol, l_tol = _bounds.fwd(dtype, W, v[b, hk], o, lse, s)
                assert (np.abs(got["o"][b, h] - o) <= o_tol).all()
                assert (np.abs(got["lse"][b, h] - lse) <= l_tol).all()
                dW = do[b, h] @ v[b, hk].T
                dS = W * (dW - (W * dW).sum(axis=1, keepdims=True)) / np.sqrt(d)
                tq, tk1, tv1 = _bounds.bwd(dtype, W, q[b, h], k[b, hk], v[b, hk], do[b, h], o, o_tol, s)
                dq = dS @ k[b, hk]
                assert (np.abs(got["dq"][b, h] - dq) <= tq + u * np.abs(dq) + 1e-30).all()
                tk, tv = tk + tk1, tv + tv1
                dk += dS.T @ q[b, h]
                dv += W.T @ do[b, h]
            if not any(frozen[hk * G:hk * G + G]):
                assert (np.abs(got["dk"][b, hk] - dk) <= tk + u * np.abs(dk) + 1e-30).all()
                assert (np.abs(got["dv"][b, hk] - dv) <= tv + u * np.abs(dv) + 1e-30).all()
            elif not all(frozen[hk * G:hk * G + G]):   # frozen heads add nothing to dk
                assert (np.abs(got["dk"][b, hk] - dk) <= tk + u * np.abs(dk) + 1e-30).all()
            else:
                assert not got["dk"][b, hk].any()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 96), ("bf16", 128), ("fp32", 64), ("fp32", 96),
                                     ("fp32", 128)])
@pytest.mark.parametrize("T,window,sinks", SPANS)
def test_multi_head(saf, dtype, d, T, window, sinks):
    frozen = [0, 1, 0]
    x, g = _inputs(dtype, 1, 3, 3, T, d, (1,), seed=T + d)
    out = _run(saf, g, frozen, window, sinks)
    _check(dtype, x, out, frozen, window, sinks)
    # a frozen head keeps the layer's bits
    o, lse = saf.saf_attn_fwd_gqa(g["q"], g["k"], g["v"], g["a"], g["r"], frozen)
    assert torch.equal(out["o"][:, 1], o[:, 1]) and torch.equal(out["lse"][:, 1], lse[:, 1])
    _, _, dv = saf.saf_attn_bwd_gqa(g["q"], g["k"], g["v"], o, g["do"], lse, g["a"], g["r"], frozen)
    assert torch.equal(out["dv"][:, 1], dv[:, 1])


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("frozen", [(), (1, 3, 6), (4, 5, 6, 7)])
@pytest.mark.parametrize("T,window,sinks", [(300, 64, 4), (513, 200, 0), (389, 1, 140)])
def test_grouped(saf, dtype, d, frozen, T, window, sinks):
    flags = [1 if h in frozen else 0 for h in range(8)]
    x, g = _inputs(dtype, 2, 8, 2, T, d, frozen, seed=T)
    out = _run(saf, g, flags, window, sinks)
    _check(dtype, x, out, flags, window, sinks)
    # dv of a group with frozen heads: the whole group against the reference, to bf16's rounding of
    # weights and result (u each, the factorised weights one more) and the fp32 terms of the bounds
    dv = so.window_bwd(*(_np(x[n]) for n in ("q", "k", "v", "do", "a", "r")), flags, window, sinks)[2]
    u = _bounds.HALF[dtype]
    for hk in range(2):
        A = np.zeros((2, T, d))
        for h in range(4 * hk, 4 * hk + 4):
            for b in range(2):
                W, _ = so.row_weights(_np(x["q"])[b, h], _np(x["k"])[b, hk], np.arange(T), _np(x["a"])[h],
                                      _np(x["r"])[h], flags[h], window, sinks)
                A[b] += W.T @ np.abs(_np(x["do"])[b, h])
        slack = 2e-5 + (1e-4 if any(flags[4 * hk:4 * hk + 4]) else 0)   # logits of frozen heads reach 60: 6 e |logit|
        assert (np.abs(_np(out["dv"])[:, hk] - dv[:, hk]) <= (2 * u + slack) * A + u * np.abs(dv[:, hk])).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 96), ("bf16", 128), ("fp32", 64), ("fp32", 96)])
@pytest.mark.parametrize("H,Hkv,frozen", [(8, 1, ()), (8, 1, (1, 3, 6)), (8, 2, (4, 5, 6, 7)), (8, 4, (1,)), (3, 3, (2,))])
@pytest.mark.parametrize("T,window,sinks", [(1100, 100, 200), (1409, 200, 16)])
def test_blocks_of_sinks_in_parts(saf, dtype, d, H, Hkv, frozen, T, window, sinks):
    # every query sees the blocks of sinks: their gradients are summed in parts where heads share them
    flags = [1 if h in frozen else 0 for h in range(H)]
    x, g = _inputs(dtype, 2 if Hkv == 2 else 1, H, Hkv, T, d, frozen, seed=T + d)
    out = _run(saf, g, flags, window, sinks)
    _check(dtype, x, out, flags, window, sinks)
    again = _run(saf, g, flags, window, sinks)
    assert torch.equal(out["dk"], again["dk"]) and torch.equal(out["dv"], again["dv"])


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 96), ("fp32", 64)])
def test_window_that_reaches_every_key_has_the_layers_bits(saf, dtype, d):
    frozen = [0, 1, 0, 0]
    x, g = _inputs(dtype, 2, 4, 2, 200, d, (1,), seed=3)
    o, lse = saf.saf_attn_fwd_gqa(g["q"], g["k"], g["v"], g["a"], g["r"], frozen)
    for window in (0, 200, 2 ** 31 - 1):
        for sinks in (0, 7, 2 ** 31 - 1):
            o2, lse2 = saf.saf_attn_fwd_window(g["q"], g["k"], g["v"], g["a"], g["r"], frozen, window, sinks)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # sinks that cover every key, with a window that does not: the masked kernels, the same weights
    o2, lse2 = saf.saf_attn_fwd_window(g["q"], g["k"], g["v"], g["a"], g["r"], frozen, 5, 2 ** 31 - 1)
    torch.testing.assert_close(lse, lse2, atol=1e-5, rtol=1e-5)


def test_prepared_state(saf):
    for dtype, d in (("bf16", 64), ("bf16", 128), ("fp32", 64)):
        frozen = [0, 1, 0, 1]
        x, g = _inputs(dtype, 1, 4, 4, 333, d, (1, 3), seed=9)
        state = saf.saf_frozen_prepare(g["a"], g["r"], frozen, 333, g["v"].dtype)
        a, b = _run(saf, g, frozen, 50, 3), _run(saf, g, frozen, 50, 3, state=state)
        assert torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"])
        assert torch.equal(a["dk"][:, ::2], b["dk"][:, ::2])
        _check(dtype, x, b, frozen, 50, 3)


def test_a_state_of_fewer_tokens_is_refused(saf):
    # the kernels read it by the call's sizes
    for dtype, d in (("bf16", 64), ("bf16", 128), ("fp32", 64)):
        frozen = [0, 1, 0, 1]
        _, g = _inputs(dtype, 1, 4, 4, 333, d, (1, 3), seed=9)
        state = saf.saf_frozen_prepare(g["a"], g["r"], frozen, 200, g["v"].dtype)
        lse = torch.zeros(1, 4, 333, device="cuda")
        fwd, bwd = [g["q"], g["k"], g["v"]], [g["q"], g["k"], g["v"], g["q"], g["do"], lse]
        tail = (g["a"], g["r"], frozen)
        for call in (lambda: saf.saf_attn_fwd_window(*fwd, *tail, 50, 3, state=state),
                     lambda: saf.saf_attn_bwd_window(*bwd, *tail, 50, 3, state=state),
                     lambda: saf.saf_attn_fwd_prepared(*fwd, *tail, state),
                     lambda: saf.saf_attn_bwd_prepared(*bwd, *tail, state)):
            before = saf.saf_launch_count()
            with pytest.raises(ValueError, match="state"):
                call()
            assert saf.saf_launch_count() == before


def test_every_head_frozen_without_q_and_k(saf):
    for dtype, d in (("bf16", 64), ("bf16", 128), ("fp32", 96)):
        x, g = _inputs(dtype, 1, 4, 2, 300, d, (0, 1, 2, 3), seed=40)
        frozen = bytes([1] * 4)
        o, lse = saf.saf_attn_fwd_window(None, None, g["v"], g["a"], g["r"], frozen, 20, 2)
        want, want_lse = saf.saf_attn_fwd_gqa(None, None, g["v"], g["a"], g["r"], frozen)
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
        dq, dk, dv = saf.saf_attn_bwd_window(None, None, g["v"], o, g["do"], lse, g["a"], g["r"], frozen, 20, 2)
        _, _, want_dv = saf.saf_attn_bwd_gqa(None, None, g["v"], o, g["do"], lse, g["a"], g["r"], frozen)
        assert not dq.any() and not dk.any() and torch.equal(dv, want_dv)


@pytest.mark.parametrize("B,T", [(0, 64), (2, 0)])
def test_empty(saf, B, T):
    q = torch.empty(B, 4, T, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(B, 2, T, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = saf.saf_attn_fwd_window(q, k, k, None, None, None, 8, 1)
    dq, dk, dv = saf.saf_attn_bwd_window(q, k, k, o, q, lse, None, None, None, 8, 1)
    assert o.shape == q.shape and dq.shape == q.shape and dk.shape == dv.shape == k.shape


def test_largest_head_count(saf):
    x, g = _inputs("bf16", 1, 256, 64, 140, 64, tuple(h for h in range(256) if h % 4 == 3), seed=41)
    flags = [h % 4 == 3 for h in range(256)]
    _check("bf16", x, _run(saf, g, flags, 9, 2), flags, 9, 2)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("frozen", [(), (255,)])
@pytest.mark.parametrize("window,sinks", [(9, 2), (0, 0)])
def test_one_group_of_the_largest_head_count(saf, dtype, d, frozen, window, sinks):
    # 256 query heads over one key/value head: a count of ordinary heads that takes more than 8 bits
    flags = [h in frozen for h in range(256)]
    x, g = _inputs(dtype, 1, 256, 1, 140, d, frozen, seed=43)
    if not frozen:
        g["a"] = g["r"] = None
    _check(dtype, x, _run(saf, g, flags, window, sinks), flags, window, sinks)
    if not window:
        o, lse = saf.saf_attn_fwd_gqa(g["q"], g["k"], g["v"], g["a"], g["r"], flags)
        dq, dk, dv = saf.saf_attn_bwd_gqa(g["q"], g["k"], g["v"], o, g["do"], lse, g["a"], g["r"], flags)
        _check(dtype, x, {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, flags, 0, 0)


@pytest.mark.parametrize("B,H,Hkv,frozen,T,window,sinks", [
    (8, 12, 12, (11,), 1590, 16, 1), (8, 16, 4, (15,), 2687, 96, 1), (3, 32, 32, tuple(range(3, 32, 4)), 1367, 2, 16),
    (8, 6, 2, (1, 3, 5), 3635, 8, 16), (8, 16, 16, (15,), 870, 62, 4), (8, 16, 16, (0, 5, 15), 870, 0, 0),
    (16, 12, 12, (0, 3, 6, 9, 11), 385, 0, 0)])
def test_frozen_heads_after_items_of_one_tile(saf, B, H, Hkv, frozen, T, window, sinks):
    # an odd number of query blocks: one of each pair's two row groups has nothing to do in a slice's
    # first item, and may come to a frozen item while that one's keys are still on their way
    flags = [h in frozen for h in range(H)]
    _, g = _inputs("bf16", B, H, Hkv, T, 64, frozen, seed=T)
    call = lambda: saf.saf_attn_fwd_window(g["q"], g["k"], g["v"], g["a"], g["r"], flags, window, sinks)   # noqa: E731
    o, lse = call()
    i = torch.arange(T, device="cuda")
    gap = i[:, None] - i[None, :]
    # weights and results rounded to bf16, and 1e-4 of the terms for logits of up to 60 in fp32
    u = _bounds.HALF["bf16"]
    for h in frozen:
        logits = (g["a"][h, :T].double()[None, :] + g["r"][h].double()[gap.clamp(min=0)]).masked_fill(gap < 0, -np.inf)
        W = torch.softmax(logits, -1)
        v = g["v"][:, h // (H // Hkv)].double()
        want = W @ v
        assert ((o[:, h].double() - want).abs() <= (u + 1e-4) * (W @ v.abs()) + u * want.abs()).all(), h
    for _ in range(60):
        o2, lse2 = call()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [96, 128])
@pytest.mark.parametrize("frozen", [(1, 2), (1, 2, 3, 4, 6), (0, 1, 2, 4, 5)])
@pytest.mark.parametrize("T,window,sinks", [(100, 9, 2), (100, 0, 0), (300, 40, 0), (520, 130, 3)])
def test_adjacent_frozen_heads_between_ordinary_ones(saf, d, frozen, T, window, sinks):
    # short runs of a head's tiles: a stage's Q goes unused once or more before an ordinary head's is loaded
    flags = [h in frozen for h in range(8)]
    x, g = _inputs("bf16", 2, 8, 1, T, d, frozen, seed=T + d)
    out = _run(saf, g, flags, window, sinks)
    _check("bf16", x, out, flags, window, sinks)
    for _ in range(8):
        again = _run(saf, g, flags, window, sinks)
        assert all(torch.equal(out[n], again[n]) for n in out)


def test_nan_keys_outside_every_window(saf):
    # whole key blocks that no row of a query block sees are not visited: a NaN there stays there.
    # 640 tokens, window 100, no sinks: rows from 384 on see keys from 285 on, in blocks from 256 on
    for dtype, d in (("bf16", 64), ("bf16", 128), ("fp32", 64)):
        x, g = _inputs(dtype, 1, 2, 2, 640, d, (), seed=12)
        clean, _ = saf.saf_attn_fwd_window(g["q"], g["k"], g["v"], None, None, None, 100, 0)
        g["k"][:, :, :128], g["v"][:, :, :128] = float("nan"), float("nan")
        o, _ = saf.saf_attn_fwd_window(g["q"], g["k"], g["v"], None, None, None, 100, 0)
        assert torch.equal(o[:, :, 384:], clean[:, :, 384:])


def _visits(T, window, sinks, rows, keys, key_blocks):
    """Boolean [T]: rows whose block (of `rows`) visits one of the key blocks (of `keys`)."""
    out = np.zeros(T, dtype=bool)
    for r0 in range(0, T, rows):
        first = max(0, r0 - window + 1) // keys
        last = (min(T, r0 + rows) - 1) // keys
        seen = set(range(first, last + 1)) | set(range(min(-(-sinks // keys), last + 1)))
        out[r0:r0 + rows] = bool(seen & key_blocks)
    return out


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 96), ("bf16", 128), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("T,window,sinks,p0,p1", [(256, 128, 0, 0, 1), (640, 100, 0, 128, 256), (640, 100, 0, 0, 128),
                                                  (900, 130, 5, 200, 201), (1100, 60, 3, 500, 640)])
def test_nan_reaches_the_rows_that_visit_its_block_only(saf, dtype, d, T, window, sinks, p0, p1):
    # as the header states it: what a block of rows (256 in the d 64 forward) does not visit may be anything
    x, g = _inputs(dtype, 1, 4, 2, T, d, (), seed=T + d)
    clean = _run(saf, g, None, window, sinks)
    keys, fwd = (128, 256 if d == 64 else 128) if dtype == "bf16" else (64, 64)
    blocks = set(range(p0 // keys, (p1 - 1) // keys + 1))
    for what in ("k", "v"):
        y = dict(g)
        y[what] = g[what].clone()
        y[what][:, :, p0:p1] = float("nan")
        o, lse = saf.saf_attn_fwd_window(y["q"], y["k"], y["v"], None, None, None, window, sinks)
        free = torch.from_numpy(~_visits(T, window, sinks, fwd, keys, blocks)).cuda()
        assert torch.equal(o[:, :, free], clean["o"][:, :, free])
        assert torch.equal(lse[:, :, free], clean["lse"][:, :, free])
        dq, dk, dv = saf.saf_attn_bwd_window(y["q"], y["k"], y["v"], clean["o"], y["do"], clean["lse"], None, None,
                                             None, window, sinks)
        free = torch.from_numpy(~_visits(T, window, sinks, keys, keys, blocks)).cuda()
        if dtype == "bf16" and d == 64:   # key blocks' shares in any order, then one rounding
            torch.testing.assert_close(dq[:, :, free], clean["dq"][:, :, free], rtol=2.0 ** -7, atol=1e-5)
        else:
            assert torch.equal(dq[:, :, free], clean["dq"][:, :, free])
        other = torch.ones(T, dtype=torch.bool, device="cuda")
        other[p0:p1] = False
        for got, want in ((dk, clean["dk"]), (dv, clean["dv"])):
            assert torch.equal(got[:, :, other], want[:, :, other])
    for what in ("q", "do", "o", "lse"):   # of rows: the keys of the blocks that theirs visit
        y = dict(g, o=clean["o"], lse=clean["lse"])
        y[what] = y[what].clone()
        y[what][:, :, p0:p1] = float("nan")
        _, dk, dv = saf.saf_attn_bwd_window(y["q"], y["k"], y["v"], y["o"], y["do"], y["lse"], None, None, None, window,
                                            sinks)
        free = torch.ones(T, dtype=torch.bool, device="cuda")
        for kb in range(-(-T // keys)):
            visited = _visits(T, window, sinks, keys, keys, {kb})[p0:p1].any()
            free[kb * keys:(kb + 1) * keys] = not visited
        assert torch.equal(dk[:, :, free], clean["dk"][:, :, free])
        assert torch.equal(dv[:, :, free], clean["dv"][:, :, free])


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("T,window,sinks", [(600, 2, 0), (601, 3, 0), (555, 3, 1), (4, 9, 0), (700, 15, 1), (32, 40, 0)])
def test_rows_of_few_keys_lose_nothing_to_the_rounded_output(saf, d, T, window, sinks):
    # dq, dk: dS and the result are rounded, each off by a step of 2^-7 / sqrt(12) over a mantissa m in
    # [1, 2), root mean square 2^-7 / sqrt(12) sqrt(mean 1 / m^2) = 2^-7 / sqrt(24): together 0.00226 of
    # the norm, and 15% for the scatter of m. (D from the rounded o adds up to 0.003 at two keys.)
    B = 3 if T > 16 else 64
    x, g = _inputs("bf16", B, 4, 2, T, d, (1,), seed=T + d)
    out = _run(saf, g, [0, 1, 0, 0], window, sinks)
    ref = so.window_bwd(*(_np(x[n]) for n in ("q", "k", "v", "do", "a", "r")), [0, 1, 0, 0], window, sinks)
    for n, want in zip(("dq", "dk"), ref):
        err = np.linalg.norm(_np(out[n]) - want) / np.linalg.norm(want)
        assert err <= 0.0026, (n, err)


def test_gradients_against_differences(saf):
    # fp32: <o, do> along a direction; central differences at h = 0.02 are off by h^2 f''' / 6
    # (about 1e-4 of |f'| for scores of size 1) and 2^-24 sqrt(n) |f| / h of rounding
    x, g = _inputs("fp32", 1, 2, 1, 150, 64, (), seed=21)
    for n in ("q", "k"):
        g[n] *= 0.3
    out = _run(saf, g, None, 40, 3)
    gen = torch.Generator().manual_seed(5)
    for n, grad in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        dirn = torch.randn(g[n].shape, generator=gen).cuda()
        dirn /= dirn.norm()
        f = []
        for h in (0.02, -0.02):
            y = dict(g)
            y[n] = g[n] + h * dirn
            o, _ = saf.saf_attn_fwd_window(y["q"], y["k"], y["v"], None, None, None, 40, 3)
            f.append((o.double() * g["do"].double()).sum().item())
        diff, want = (f[0] - f[1]) / 0.04, (out[grad].double() * dirn.double()).sum().item()
        scale = out[grad].double().norm().item()
        assert abs(diff - want) <= 2e-3 * scale, (n, diff, want)


@pytest.mark.parametrize("dtype,d,T", [("bf16", 64, 20011), ("bf16", 128, 20011), ("fp32", 64, 6007)])
def test_a_long_sequence(saf, dtype, d, T):
    """Every element against 64-bit sums over the visible keys alone (window + sinks of them a row).

    Off by at most: the weights' rounding (u), the results' (u), D from the rounded o, dS' rounding (u),
    and 1e-4 of the terms for fp32: a score of d products is off by d 2^-24 sum |q k| / sqrt(d), below
    8e-5 here, which its weight takes over as a factor."""
    window, sinks, H = 200, 7, 4
    x, g = _inputs(dtype, 1, H, 1, T, d, (), seed=77)
    out = _run(saf, g, [0] * H, window, sinks)
    u = _bounds.HALF[dtype]
    eps = 1e-4
    i = torch.arange(T, device="cuda")[:, None]
    recent = i - torch.arange(window, device="cuda")          # the window's keys
    first = torch.arange(sinks, device="cuda").expand(T, -1)   # the sinks before it
    idx = torch.cat([recent, first], 1)
    seen = torch.cat([recent >= 0, first <= i - window], 1)
    idx = idx.clamp(min=0)
    f = {n: g[n].double()[0] for n in ("q", "k", "v", "do")}
    k, v = f["k"][0], f["v"][0]
    K, V = k[idx], v[idx]
    dk, dv, tk, tv = (torch.zeros_like(k) for _ in range(4))
    for h in range(H):
        q, do = f["q"][h], f["do"][h]
        S = torch.einsum("td,tjd->tj", q, K) / d ** 0.5
        S = S.masked_fill(~seen, -float("inf"))
        P = torch.softmax(S, 1)
        o = torch.einsum("tj,tjd->td", P, V)
        to = (u + eps) * torch.einsum("tj,tjd->td", P, V.abs()) + u * o.abs()
        assert ((out["o"][0, h].double() - o).abs() <= to).all()
        assert ((out["lse"][0, h].double() - torch.logsumexp(S, 1)).abs() <= 2e-4).all()
        dP = torch.einsum("td,tjd->tj", do, V)
        D = (do * o).sum(1, keepdim=True)
        dS = P * (dP - D)
        err = P * (u * (dP - D).abs() + (do.abs() * to).sum(1, keepdim=True) + eps * (dP.abs() + D.abs()))
        dq = torch.einsum("tj,tjd->td", dS, K) / d ** 0.5
        tq = torch.einsum("tj,tjd->td", err, K.abs()) / d ** 0.5 + u * dq.abs()
        assert ((out["dq"][0, h].double() - dq).abs() <= tq).all()
        flat = idx.flatten()
        for total, w, y in ((dk, dS / d ** 0.5, q), (tk, err / d ** 0.5, q.abs()), (dv, P, do),
                            (tv, (u + eps) * P, do.abs())):
            total.index_add_(0, flat, (w[:, :, None] * y[:, None, :]).reshape(-1, d))
    assert ((out["dk"][0, 0].double() - dk).abs() <= tk + u * dk.abs()).all()
    assert ((out["dv"][0, 0].double() - dv).abs() <= tv + u * dv.abs()).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
def test_parts_captured_and_beside_another_call(saf, dtype, d):
    # a captured backward with blocks of sinks in parts, replayed while an eager call with its own
    # workspace runs on another stream
    frozen = [0, 0, 1, 0, 0, 0, 0, 0]
    x, g = _inputs(dtype, 1, 8, 1, 1100, d, (2,), seed=31)
    first = _run(saf, g, frozen, 100, 16)
    ws = saf.alloc_workspace(1, 8, 1100, d, g["v"].dtype, True)
    grads = [torch.empty_like(first[n]) for n in ("dq", "dk", "dv")]

    def step():
        saf.saf_attn_bwd_window(g["q"], g["k"], g["v"], first["o"], g["do"], first["lse"], g["a"], g["r"], frozen,
                                100, 16, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    side = torch.cuda.Stream()
    for _ in range(3):
        for t in grads:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        other = saf.saf_attn_bwd_window(g["q"], g["k"], g["v"], first["o"], g["do"], first["lse"], g["a"], g["r"],
                                        frozen, 100, 16, stream=side)
        torch.cuda.synchronize()
        for dq, dk, dv in (grads, other):
            assert torch.equal(dk, first["dk"]) and torch.equal(dv, first["dv"])
            torch.testing.assert_close(dq, first["dq"], rtol=2.0 ** -7, atol=1e-5)


def test_captured_and_replayed(saf):
    x, g = _inputs("bf16", 2, 4, 2, 260, 64, (1,), seed=30)
    frozen = [0, 1, 0, 0]
    first = _run(saf, g, frozen, 70, 2)
    ws = [saf.alloc_workspace(2, 4, 260, 64, torch.bfloat16, b) for b in (False, True)]
    o, lse = torch.empty_like(first["o"]), torch.empty_like(first["lse"])
    grads = [torch.empty_like(first[n]) for n in ("dq", "dk", "dv")]

    def step():
        saf.saf_attn_fwd_window(g["q"], g["k"], g["v"], g["a"], g["r"], frozen, 70, 2, o=o, lse=lse, workspace=ws[0])
        saf.saf_attn_bwd_window(g["q"], g["k"], g["v"], o, g["do"], lse, g["a"], g["r"], frozen, 70, 2, dq=grads[0],
                                dk=grads[1], dv=grads[2], workspace=ws[1])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for t in (o, lse, *grads):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, first["o"]) and torch.equal(lse, first["lse"])
        assert torch.equal(grads[1], first["dk"]) and torch.equal(grads[2], first["dv"])
        # dq adds key blocks' shares in fp32 in any order, then rounds to bf16: one step apart
        torch.testing.assert_close(grads[0], first["dq"], rtol=2.0 ** -7, atol=1e-5)
