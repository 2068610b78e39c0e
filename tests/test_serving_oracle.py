"""The fp64 reference of the windowed layer and the paged calls, pinned on the CPU."""
import numpy as np
import pytest

import oracle
from oracle import serving_oracle as so

RNG = np.random.default_rng


def _layer(seed, B=1, H=4, Hkv=2, T=23, d=8):
    g = RNG(seed)
    x = {n: g.standard_normal((B, H if n in ("q", "do") else Hkv, T, d)) for n in ("q", "k", "v", "do")}
    x["a"], x["r"] = g.standard_normal((H, T)), g.standard_normal((H, T)) - 0.1 * np.arange(T)
    return x


def test_visible_by_hand():
    # window 2, one sink: query 4 sees keys 0, 3, 4; query 0 sees key 0 only
    assert so.visible([4], range(6), 2, 1).tolist() == [[True, False, False, True, True, False]]
    assert so.visible([0, 1], range(3), 1, 0).tolist() == [[True, False, False], [False, True, False]]
    assert so.visible([2], range(4), 0, 0).tolist() == [[True, True, True, False]]


def test_no_window_is_the_layer():
    x = _layer(1)
    frozen = [0, 1, 0, 0]
    o, lse = so.window_fwd(x["q"], x["k"], x["v"], x["a"], x["r"], frozen, 0, 0)
    o2, lse2 = oracle.gqa_fwd(x["q"], x["k"], x["v"], x["a"], x["r"], frozen)
    np.testing.assert_allclose(o, o2, atol=1e-12)
    np.testing.assert_allclose(lse, lse2, atol=1e-12)
    g = so.window_bwd(x["q"], x["k"], x["v"], x["do"], x["a"], x["r"], frozen, 99, 3)
    for got, want in zip(g, oracle.gqa_bwd(x["q"], x["k"], x["v"], x["do"], x["a"], x["r"], frozen)):
        np.testing.assert_allclose(got, want, atol=1e-12)


def test_window_of_one_returns_the_values():
    x = _layer(2)
    o, _ = so.window_fwd(x["q"], x["k"], x["v"], x["a"], x["r"], [0] * 4, 1, 0)
    np.testing.assert_allclose(o, np.repeat(x["v"], 2, axis=1), atol=1e-14)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 2), (9, 0), (3, 30)])
def test_window_gradients_against_differences(window, sinks):
    x = _layer(3, T=13, d=4)
    frozen = [0, 1, 0, 0]

    def loss(q, k, v):
        return (so.window_fwd(q, k, v, x["a"], x["r"], frozen, window, sinks)[0] * x["do"]).sum()

    grads = so.window_bwd(x["q"], x["k"], x["v"], x["do"], x["a"], x["r"], frozen, window, sinks)
    g = RNG(4)
    for n, grad in zip(("q", "k", "v"), grads):
        dirn = g.standard_normal(x[n].shape)
        args = [{m: x[m] + (s * 1e-5 * dirn if m == n else 0) for m in ("q", "k", "v")} for s in (1, -1)]
        diff = (loss(**args[0]) - loss(**args[1])) / 2e-5
        assert abs(diff - (grad * dirn).sum()) <= 1e-7 * (1 + abs(diff))


def test_rotation_turns_pairs_and_keeps_products_of_distances():
    g = RNG(5)
    f = 100.0 ** (-np.arange(4) / 4)
    x, y = g.standard_normal((1, 8)), g.standard_normal((1, 8))
    for inter in (False, True):
        dots = [(so.rotate(x, [p + 7], f, inter) @ so.rotate(y, [p], f, inter).T)[0, 0] for p in (0, 3, 1000)]
        np.testing.assert_allclose(dots, dots[0], atol=1e-11)
        np.testing.assert_allclose(so.rotate(x, [0], f, inter), x)
    # one quarter turn of pair 0: (x0, x1) -> (-x1, x0)
    z = so.rotate(np.arange(4.0)[None], [1], [np.pi / 2], True)
    np.testing.assert_allclose(z, [[-1, 0, 2, 3]], atol=1e-15)
    z = so.rotate(np.arange(4.0)[None], [1], [np.pi / 2, 0.0], False)
    np.testing.assert_allclose(z, [[-2, 1, 0, 3]], atol=1e-15)


def test_paged_is_the_layer_on_gathered_keys():
    g = RNG(6)
    x = _layer(7, B=1, H=4, Hkv=2, T=20, d=8)
    page, perm = 8, np.array([2, 0, 3])
    kc, vc = np.full((4, 2, page, 8), np.nan), np.full((4, 2, page, 8), np.nan)
    for j in range(20):
        kc[perm[j // page], :, j % page] = x["k"][0, :, j]
        vc[perm[j // page], :, j % page] = x["v"][0, :, j]
    frozen = [1, 0, 0, 0]
    want, lse = so.window_fwd(x["q"], x["k"], x["v"], x["a"], x["r"], frozen, 6, 2)
    o, l = so.paged_fwd(x["q"][:, :, 17:], kc, vc, perm[None], [17], [3], x["a"], x["r"], frozen, 6, 2)
    np.testing.assert_allclose(o, want[:, :, 17:], atol=1e-13)
    np.testing.assert_allclose(l, lse[:, :, 17:], atol=1e-13)
    # the first page as a shared prefix
    o, l = so.paged_fwd(x["q"][:, :, 17:], kc, vc, perm[None, 1:], [9], [3], x["a"], x["r"], frozen, 6, 2, perm[:1], 8)
    np.testing.assert_allclose(o, want[:, :, 17:], atol=1e-13)
    o, l = so.paged_fwd(x["q"][:, :, 17:], kc, vc, perm[None], [17], [0], x["a"], x["r"], frozen)
    assert not o.any() and np.isneginf(l).all()
