"""GPU parity of the calls on 8-bit caches against the fp64 reference, over what the codes stand for.

Whatever no token owns is poisoned: free pages and the slots behind a sequence's last token hold codes
of NaN and of the largest value with scales that are NaN, infinite or negative, and the page table's
entries behind it hold numbers that are no page.

Bounds. Those of tests/_bounds.py, for the values code * scale, with u, e as there, and
  - logits: the scale is applied to the sum (or to each product) in fp32: a relative e (2 e with
    the product's own rounding) of sum |q k|. For bf16, q may be taken as two terms of e4m3 of the row
    scaled by a power of two so that its largest element lies in (224, 448]: what the terms leave
    is half a step of their smallest, 2^-10, at most 2^-17 of the largest |q|, in each of d products:
        ds <= 2^-17 max |q| sum_c |k_c| / sqrt(d)
  - outputs: the scale is applied to the weight or to the value, a relative e (2 e). For bf16 the weight
    times the value's scale may be taken as terms of e4m3 (off by at most u of itself, as in bf16, or, near
    zero, by 2^-20 of the largest weight times the largest scale of the row's keys):
        |do| <= n 2^-20 max_j W_j max_j |v_j|
"""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from tests import _bounds

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
ALL = [("bf16", 64), ("bf16", 96), ("bf16", 128), ("fp32", 64), ("fp32", 96), ("fp32", 128)]
SOME = [("bf16", 64), ("bf16", 128), ("fp32", 96)]


@pytest.fixture(scope="module")
def saf():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from softmax_attention_hybrid_gb300 import saf as mod
    return mod


def _np(t):
    return t.double().cpu().numpy()


def _quantise(y):
    scale = (y.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    return (y / scale[..., None]).to(E4M3).view(torch.uint8), scale


class Batch:
    """Sequences of ctx + n_new tokens in shuffled pages, with poison in every free place."""

    def __init__(self, dtype, H, Hkv, T, d, page, ctx, n_new, prefix=0, seed=0, max_len=None, scale=1.0,
                 first_seen=0, spread=0.3):
        g = torch.Generator().manual_seed(seed)
        B = len(ctx)
        total = [c + n for c, n in zip(ctx, n_new)]
        self.max_len = max_len or max(1, max(total, default=1))
        per = -(-self.max_len // page)
        npp = -(-prefix // page)
        count = sum(-(-t // page) for t in total) + npp + 2
        order = torch.randperm(count, generator=g).tolist()
        odd = torch.tensor([float("nan"), float("inf"), -1.0, 0.0, 1e30])
        shape = (count, Hkv, page)
        self.codes = [torch.tensor([127, 255, 126, 254])[torch.randint(0, 4, (*shape, d), generator=g)].to(torch.uint8)
                      for _ in range(2)]
        self.scales = [odd[torch.randint(0, 5, shape, generator=g)] for _ in range(2)]

        def fill(pg, n):
            for c, s in zip(self.codes, self.scales):
                size = torch.exp(spread * torch.randn(Hkv, n, 1, generator=g))
                c[pg, :, :n], s[pg, :, :n] = _quantise(torch.randn(Hkv, n, d, generator=g) * scale * size)

        self.table = torch.full((B, per), -7, dtype=torch.int32)
        self.table[:, 1::2] = 2 ** 30
        self.prefix_pages = torch.tensor([order.pop() for _ in range(npp)], dtype=torch.int32)
        for at in range(npp):
            fill(int(self.prefix_pages[at]), min(page, prefix - at * page))
        for b in range(B):
            for at in range(-(-total[b] // page)):
                pg = order.pop()
                fill(pg, min(page, total[b] - at * page))
                # a page that lies before everything that is seen may be gone
                self.table[b, at] = pg if (at + 1) * page > first_seen else -3
        self.q = (torch.randn(B, H, T, d, generator=g) * scale).to(DT[dtype])
        L = prefix + self.max_len
        self.a = torch.randn(H, L, generator=g)
        self.r = 0.5 * torch.randn(H, L, generator=g) - 0.03 * torch.arange(L)
        self.ctx, self.n_new = (torch.tensor(x, dtype=torch.int32) for x in (ctx, n_new))
        self.dtype, self.prefix, self.Hkv = dtype, prefix, Hkv

    def cache(self):
        return [c.cuda().view(E4M3) for c in self.codes] + [s.cuda() for s in self.scales]

    def call(self, saf, frozen=None, window=0, sinks=0, **kw):
        c = lambda t: t.cuda()   # noqa: E731
        args = dict(n_new=c(self.n_new), a=c(self.a), r=c(self.r), frozen=frozen, window=window, sinks=sinks)
        args.update(kw)
        tail = (c(self.table), c(self.ctx), self.max_len)
        if self.prefix:
            return saf.saf_attn_paged_shared_quant(c(self.q), *self.cache(), c(self.prefix_pages), self.prefix, *tail,
                                                   **args)
        return saf.saf_attn_paged_quant(c(self.q), *self.cache(), *tail, **args)

    def rows(self, b, n):
        """What the first n own keys of sequence b, behind the prefix, stand for: k, v [.., Hkv, d]."""
        table = self.table[b].clamp(min=0, max=self.codes[0].shape[0] - 1)
        out = []
        for c, s in zip(self.codes, self.scales):
            c, s = c.numpy(), s.double().numpy()
            parts = [so.dequantise(so.gather(c, pages, m), so.gather(s[..., None], pages, m)[..., 0])
                     for pages, m in ((self.prefix_pages, self.prefix), (table, n))]
            out.append(np.concatenate(parts))
        return out

    def check(self, o, lse, frozen=None, window=0, sinks=0, rows=slice(None)):
        o, lse = _np(o), _np(lse)
        q, a, r = (_np(t) for t in (self.q, self.a, self.r))
        B, H, T, d = q.shape
        G = H // self.Hkv
        for b in range(B):
            n = int(self.n_new[b])
            k, v = self.rows(b, int(self.ctx[b]) + n)
            i = self.prefix + int(self.ctx[b]) + np.arange(n)
            assert not o[b, :, n:].any() and np.isneginf(lse[b, :, n:]).all()
            if n == 0:
                continue
            if window and not any(frozen or [0]):
                # keys behind every window may be gone: they carry no weight
                hidden = ~so.visible(i, np.arange(len(k)), window, sinks).any(axis=0)
                k[hidden], v[hidden] = 0, 0
            for h in range(H):
                fz = bool(frozen and frozen[h])
                kk, vv = np.nan_to_num(k[:, h // G]), v[:, h // G]
                W, l_ref = so.row_weights(q[b, h, :n], kk, i, a[h], r[h], fz, window, sinks)
                ref = W @ vv
                o_tol, l_tol = bounds(self.dtype, q[b, h, :n], kk, vv, W, ref, l_ref, a[h], r[h], i, fz)
                assert (np.abs(o[b, h, :n] - ref) <= o_tol).all(), (b, h)
                assert (np.abs(lse[b, h, :n] - l_ref) <= l_tol).all(), (b, h)


def bounds(dtype, q, k, v, W, o, lse, a, r, i, fz):
    """The module's bounds for one head's rows."""
    d = q.shape[1]
    s = _bounds.logit_error(q, k, a, r, i, fz)
    if not fz and len(k):
        s += 2 * _bounds.E * (np.abs(q) @ np.abs(k).T).max() / np.sqrt(d)
        if dtype == "bf16":
            s += 2.0 ** -17 * np.abs(q).max() * np.abs(k).sum(axis=1).max() / np.sqrt(d)
    o_tol, l_tol = _bounds.fwd(dtype, W, v, o, lse, s)
    o_tol = o_tol + 2 * _bounds.E * (W @ np.abs(v))
    if dtype == "bf16":
        o_tol = o_tol + len(v) * 2.0 ** -20 * W.max(axis=1, initial=0.0)[:, None] * np.abs(v).max(initial=0.0)
    return o_tol, l_tol


LENS = [(0,), (63, 0, 64), (127, 128, 129), (200, 7, 391), (1030, 515)]


@pytest.mark.parametrize("dtype,d", ALL)
@pytest.mark.parametrize("page", [8, 64, 256])
@pytest.mark.parametrize("ctx", LENS)
def test_one_new_token(saf, dtype, d, page, ctx):
    frozen = [0, 1, 0, 0, 1, 1]
    x = Batch(dtype, 6, 2, 1, d, page, ctx, [1] * len(ctx), seed=page + d)
    x.check(*x.call(saf, frozen), frozen)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 1), (12, 4), (40, 1)])
@pytest.mark.parametrize("T,n_new", [(1, (1, 1)), (4, (4, 2)), (5, (0, 3)), (9, (1, 9)), (33, (33, 32)),
                                     (150, (150, 0))])
def test_new_tokens_and_groups(saf, dtype, H, Hkv, T, n_new):
    frozen = [h % 3 == 1 for h in range(H)]
    x = Batch(dtype, H, Hkv, T, 64, 16, (90, 37), n_new, seed=H + T)
    x.check(*x.call(saf, frozen), frozen)


@pytest.mark.parametrize("dtype,d", SOME)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 0), (100, 130), (129, 4), (700, 2), (5000, 9)])
@pytest.mark.parametrize("T", [1, 6, 40])
@pytest.mark.parametrize("fz", [False, True])
def test_window(saf, dtype, d, window, sinks, T, fz):
    frozen = [0, 0, 1, 0] if fz else None
    # pages before the window and past the sinks are gone when no head sees them
    ctx = (600, 333, 12)
    first = 0 if fz or sinks else max(0, 12 - window + 1)
    x = Batch(dtype, 4, 2, T, d, 16, ctx, [T, T, min(T, 2)], seed=window, first_seen=first)
    x.check(*x.call(saf, frozen, window, sinks), frozen, window, sinks)


def test_pages_before_the_window_may_be_gone(saf):
    for dtype in ("bf16", "fp32"):
        for T in (3, 50):
            x = Batch(dtype, 4, 2, T, 64, 16, (600, 640), (T, 2), seed=4, first_seen=600 - 100 + 1)
            ws = saf.alloc_paged_quant_workspace(2, 4, 2, T, 64, x.max_len, DT[dtype])
            x.check(*x.call(saf, None, 100, 0, workspace=ws), None, 100, 0)
            assert saf.saf_device_status(ws) == saf.SAF_OK


@pytest.mark.parametrize("dtype,d", SOME)
@pytest.mark.parametrize("prefix,page", [(1, 8), (100, 32), (129, 64), (700, 256)])
@pytest.mark.parametrize("H,Hkv,T", [(3, 3, 1), (8, 2, 1), (8, 2, 3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 4), (40, 200)])
def test_shared_prefix(saf, dtype, d, prefix, page, H, Hkv, T, window, sinks):
    for fz in ([h % 4 == 3 for h in range(H)], None):
        x = Batch(dtype, H, Hkv, T, d, page, (0, 5, 77, 31, 200), [T, T, 1, 0, T], prefix=prefix, seed=prefix)
        x.check(*x.call(saf, fz, window, sinks), fz, window, sinks)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("prefix", [0, 100])
@pytest.mark.parametrize("frozen", [(), (0,), tuple(range(256))])
def test_one_group_of_the_largest_head_count(saf, dtype, d, prefix, frozen):
    flags = [h in frozen for h in range(256)]
    x = Batch(dtype, 256, 1, 2, d, 16, (90, 37), (2, 1), prefix=prefix, seed=44)
    none = {} if frozen else dict(a=None, r=None)
    x.check(*x.call(saf, flags, **none), flags)
    if not frozen:
        x.check(*x.call(saf, flags, 20, 3, **none), flags, 20, 3)


def test_many_sequences_share_a_prefix(saf):
    for dtype in ("bf16", "fp32"):
        B = 70
        ctx, n_new = [(7 * b) % 40 for b in range(B)], [1 + (b % 2) for b in range(B)]
        frozen = [0, 1, 0, 0]
        x = Batch(dtype, 4, 2, 2, 64, 16, ctx, n_new, prefix=300, seed=1)
        x.check(*x.call(saf, frozen), frozen)


@pytest.mark.parametrize("dtype,d", SOME)
@pytest.mark.parametrize("masked", [-float("inf"), torch.finfo(torch.float32).min])
@pytest.mark.parametrize("prefix,T", [(0, 2), (40, 2), (0, 40)])
def test_keys_that_a_pattern_masks(saf, dtype, d, masked, prefix, T):
    # a head whose pattern leaves nothing: zeros and -infinity; one that masks some keys: no weight there
    frozen = [0, 1, 1, 0]
    x = Batch(dtype, 4, 2, T, d, 16, (0, 100, 300), (2, T, 1), prefix=prefix, seed=3)
    x.a[1], x.a[2, 3:7] = masked, masked
    o, lse = x.call(saf, frozen)
    assert not o[:, 1].any() and torch.isneginf(lse[:, 1]).all()
    x.a[1], x.a[2, 3:7] = 0.0, -200.0   # e^-200: nothing in the outputs' bits
    o[:, 1], lse[:, 1] = (t[:, 1] for t in x.call(saf, frozen))
    x.check(o, lse, frozen)


@pytest.mark.parametrize("T", [2, 40])
def test_every_head_frozen_reads_no_keys(saf, T):
    for dtype in ("bf16", "fp32"):
        x = Batch(dtype, 4, 2, T, 64, 16, (30, 50), (T, 1), seed=2)
        _, vc, _, vs = x.cache()
        o, lse = saf.saf_attn_paged_quant(torch.full_like(x.q, float("nan")).cuda(), None, vc, None, vs, x.table.cuda(),
                                          x.ctx.cuda(), x.max_len, x.n_new.cuda(), x.a.cuda(), x.r.cuda(), [1] * 4)
        x.check(o, lse, [1] * 4)


def test_bound_above_the_lengths(saf):
    for dtype in ("bf16", "fp32"):
        for T in (1, 50):
            x = Batch(dtype, 4, 2, T, 64, 16, (3, 300, 0), (1, T, 1), seed=8, max_len=9000)
            x.check(*x.call(saf, [0, 0, 0, 1]), [0, 0, 0, 1])


@pytest.mark.parametrize("T", [1, 2, 50])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_scores(saf, dtype, T):
    # scores in the hundreds: one key takes nearly all the weight, others vanish
    x = Batch(dtype, 2, 1, T, 64, 16, (500, 130), (T, T), seed=11, scale=6.0)
    x.check(*x.call(saf))


@pytest.mark.parametrize("dtype,d", SOME)
@pytest.mark.parametrize("T", [1, 12, 50])
def test_scales_of_very_different_size(saf, dtype, d, T):
    # rows a thousand times larger and smaller than others, empty ones and ones at the smallest scale
    x = Batch(dtype, 4, 2, T, d, 16, (700, 300), (T, T), seed=21, scale=0.3, spread=2.5)
    pg = int(x.table[0, 3])
    for c, s in zip(x.codes, x.scales):
        c[pg, :, 2:5], s[pg, :, 2:5] = 0, 2.0 ** -126
        s[pg, :, 7] = 2.0 ** -126
        s[pg, :, 8] = 0.0
    x.check(*x.call(saf, [0, 1, 0, 0]), [0, 1, 0, 0])


@pytest.mark.parametrize("T", [1, 50])
def test_values_that_grow_along_the_sequence(saf, T):
    # the largest scale so far rises from tile to tile, and falls behind the middle
    for dtype in ("bf16", "fp32"):
        x = Batch(dtype, 4, 2, T, 64, 64, (1500, 900), (T, T), seed=22)
        for b in range(2):
            for at in range(int(x.ctx[b] + x.n_new[b] + 63) // 64):
                x.scales[1][int(x.table[b, at])] *= 2.0 ** (at if at < 12 else 24 - 2 * at)
        x.check(*x.call(saf))


@pytest.mark.parametrize("T", [1, 50])
def test_queries_of_any_size(saf, T):
    # rows of q scaled by powers of two from 2^-100 to 2^100, against keys scaled the other way, and zero rows
    for p in (-100, -20, 20, 100):
        x = Batch("bf16", 4, 2, T, 128, 16, (200, 100), (T, T), seed=23)
        x.q *= 2.0 ** p
        x.scales[0] *= 2.0 ** -p
        x.q[0, 1] = 0
        x.check(*x.call(saf))


@pytest.mark.parametrize("dtype,d", SOME)
@pytest.mark.parametrize("ctx", [3, 40, 5000])
@pytest.mark.parametrize("bad", ["q", "inf"])
@pytest.mark.parametrize("T", [2, 40])
def test_a_row_of_nan_stays_one_and_alone(saf, dtype, d, ctx, bad, T):
    x = Batch(dtype, 4, 2, T, d, 64, (ctx, 7), (T, 2), seed=71)
    want, want_lse = x.call(saf)
    x.q[0, 1, 0] = float("nan") if bad == "q" else float("inf")
    o, lse = x.call(saf)
    assert o[0, 1, 0].isnan().all() and lse[0, 1, 0].isnan()
    o[0, 1, 0], lse[0, 1, 0] = want[0, 1, 0], want_lse[0, 1, 0]
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_a_nan_in_the_cache_reaches_the_rows_that_see_it(saf):
    for dtype in ("bf16", "fp32"):
        for what in (0, 1):   # k, v
            for T in (1, 50):
                x = Batch(dtype, 4, 2, T, 64, 16, (100, 60), (T, T), seed=72)
                want = x.call(saf)
                x.codes[what][int(x.table[0, 2]), 1, 5, 7] = 127
                o, lse = x.call(saf)
                assert torch.equal(o[1], want[0][1]) and torch.equal(o[0, :2], want[0][0, :2])
                if what == 0:
                    assert o[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
                else:
                    assert o[0, 2:, :, 7].isnan().all() and torch.equal(lse, want[1])


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("G,T", [(1, 1), (4, 1), (5, 1), (8, 1), (3, 3), (4, 4), (17, 1), (6, 4), (5, 5), (8, 4), (11, 3),
                                 (2, 63), (43, 3), (4, 64), (1, 257), (6, 100)])
@pytest.mark.parametrize("kind", ["ordinary", "frozen", "mixed", "window"])
def test_every_number_of_rows_to_a_block(saf, d, G, T, kind):
    # (1 to 600 rows to a key/value head: every size of block, full and with one row more)
    H = 2 * G
    frozen = [kind == "frozen" or (kind == "mixed" and h % 2 == 1) for h in range(H)]
    window, sinks = (70, 3) if kind == "window" else (0, 0)
    x = Batch("bf16", H, 2, T, d, 32, (300, 0, 161), (T, max(1, T // 3), T), seed=G + T)
    x.check(*x.call(saf, frozen, window, sinks), frozen, window, sinks)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("G,T", [(1, 1), (2, 1), (3, 1), (1, 4), (5, 1), (3, 2), (1, 7), (4, 2), (3, 3), (5, 5), (1, 40)])
@pytest.mark.parametrize("kind", ["ordinary", "frozen", "mixed", "window", "prefix"])
def test_every_number_of_rows_to_a_block_fp32(saf, d, G, T, kind):
    H = 2 * G
    frozen = [kind == "frozen" or (kind in ("mixed", "prefix") and h % 2 == 1) for h in range(H)]
    window, sinks = (70, 3) if kind == "window" else (0, 0)
    ctx, n_new = ((300, 0, 161), (T, max(1, T // 3), T)) if (G + T) % 2 else ((257,), (T,))
    x = Batch("fp32", H, 2, T, d, 32, ctx, n_new, prefix=150 if kind == "prefix" else 0, seed=G + T)
    x.check(*x.call(saf, frozen, window, sinks), frozen, window, sinks)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_magnitudes_of_q_and_of_the_scales(saf, dt):
    # sums over codes of q of every size: scores, not what leads to them, decide
    for q, k in ((2.0 ** 100, 2.0 ** -100), (2.0 ** -100, 2.0 ** 100), (2.0 ** -110, 2.0 ** -10), (2.0 ** 60, 2.0 ** -60)):
        x = Batch(dt, 4, 2, 2, 64, 16, (90, 33), (2, 2), seed=95)
        x.q = x.q * q
        x.scales[0] = x.scales[0] * k
        x.check(*x.call(saf))


@pytest.mark.parametrize("H,T,d,page,window,sinks", [
    (32, 1, 128, 128, 1000, 4), (32, 1, 128, 128, 0, 0), (32, 1, 64, 128, 1000, 4), (32, 1, 128, 16, 1000, 4),
    (64, 1, 128, 128, 1000, 4), (160, 1, 128, 128, 1000, 4), (32, 4, 128, 128, 1000, 4), (32, 64, 128, 128, 300, 4)])
def test_the_same_bits_every_time(saf, H, T, d, page, window, sinks):
    # several blocks to an SM, all of them with masked tiles: what one block holds up, another must wait for
    B, Hkv, max_len = 48, 8, 1500
    g = torch.Generator(device="cuda").manual_seed(96)
    per = -(-max_len // page)
    shape = (B * per, Hkv, page, d)
    cache = [torch.randn(*shape, generator=g, device="cuda").to(E4M3) for _ in range(2)]
    scales = [0.5 + torch.rand(shape[:3], generator=g, device="cuda") for _ in range(2)]
    table = torch.randperm(B * per, generator=g, device="cuda").int().view(B, per)
    ctx = torch.randint(T, max_len - T, (B,), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(B, H, T, d, generator=g, device="cuda").to(torch.bfloat16)
    first = None
    for _ in range(12):
        o, lse = saf.saf_attn_paged_quant(q, *cache, *scales, table, ctx, max_len, window=window, sinks=sinks)
        torch.cuda.synchronize()
        if first is None:
            first = o.clone(), lse.clone()
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_many_sequences(saf):
    # more sequences than a block of many rows puts in order, of very unequal lengths
    for B, H, T in ((300, 40, 1), (300, 2, 1), (257, 2, 20), (256, 40, 1)):
        ctx = [(37 * b) % 200 if b % 7 else 0 for b in range(B)]
        frozen = [h % 5 == 4 for h in range(H)]
        x = Batch("bf16", H, 1, T, 64, 16, ctx, [T if b % 3 else T // 2 for b in range(B)], seed=B + H)
        x.check(*x.call(saf, frozen), frozen)


def test_positions_far_apart_in_blocks_of_many_rows(saf):
    # the frozen heads' patterns of a block do not fit into shared memory, or just do
    for spread in (1500, 2300, 4000):
        ctx = [0, spread] + [(spread * b) // 20 for b in range(18)]
        frozen = [0, 0, 1, 1]
        x = Batch("bf16", 4, 1, 1, 64, 64, ctx, [1] * 20, prefix=150, seed=spread)
        x.check(*x.call(saf, frozen), frozen)


def test_priors_of_any_alignment(saf):
    # rows of a and r that begin anywhere in a 16-byte line, ending with the last position
    for extra in range(4):
        for T in (1, 40):
            x = Batch("bf16", 4, 1, T, 64, 16, (77 + extra, 3), (T, T), seed=91)
            big = torch.full((2, 4 * x.a.shape[1] + 1), float("nan"))
            a, r = (y[1:].view(4, x.a.shape[1]) for y in big.cuda())   # 4 bytes into a line
            a.copy_(x.a)
            r.copy_(x.r)
            o, lse = x.call(saf, [0, 1, 1, 0], a=a, r=r)
            x.check(o, lse, [0, 1, 1, 0])


def test_sequences_that_share_pages(saf):
    # the same pages in two sequences' tables, and twice in one
    x = Batch("bf16", 4, 2, 2, 64, 16, (100, 100, 40), (2, 2, 2), seed=92)
    x.table[1] = x.table[0]
    x.table[0, 1] = x.table[0, 0]
    x.q[1] = x.q[0]
    o, lse = x.call(saf, [0, 1, 0, 0])
    x.check(o, lse, [0, 1, 0, 0])
    x.table[1] = x.table[0]
    o, lse = x.call(saf, [0, 1, 0, 0])
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])


def test_empty_calls(saf):
    x = Batch("bf16", 4, 2, 1, 64, 16, (10,), (1,), seed=93)
    none = torch.zeros(0, x.table.shape[1], dtype=torch.int32, device="cuda")
    count = torch.zeros(0, dtype=torch.int32, device="cuda")
    o, lse = saf.saf_attn_paged_quant(x.q[:0].cuda(), *x.cache(), none, count, 16)
    assert o.shape == (0, 4, 1, 64) and lse.shape == (0, 4, 1)
    k, v = saf.saf_kv_read_quant(*x.cache(), x.table.cuda(), T=0, dtype=torch.bfloat16)
    assert k.shape == v.shape == (1, 2, 0, 64)
    k, v = saf.saf_kv_read_quant(*x.cache(), none, T=5, dtype=torch.float32)
    assert k.shape == v.shape == (0, 2, 5, 64)
    rows = torch.zeros(1, 2, 0, 64, dtype=torch.bfloat16, device="cuda")
    before = x.cache()
    assert saf.saf_kv_append_quant(rows, rows, *before, x.table.cuda(), x.ctx.cuda()) is None


def test_refused_tensors(saf):
    x = Batch("bf16", 4, 2, 1, 64, 16, (10,), (1,), seed=94)
    kc, vc, ks, vs = x.cache()
    q, table, ctx = x.q.cuda(), x.table.cuda(), x.ctx.cuda()
    call = saf.saf_attn_paged_quant
    for args, err in (((q, kc.view(torch.uint8), vc, ks, vs), TypeError), ((q, kc, vc.view(torch.uint8), ks, vs), TypeError),
                      ((q, kc, vc, ks.double(), vs), TypeError), ((q, kc, vc, ks, vs.half()), TypeError),
                      ((q, kc, vc, ks, vs[:, :, :8]), ValueError), ((q, kc, vc, ks[1:], vs), ValueError),
                      ((q, kc, vc, ks.transpose(0, 1).contiguous().transpose(0, 1), vs), ValueError),
                      ((q, kc, vc, ks, vs.cpu()), ValueError), ((q.half(), kc, vc, ks, vs), TypeError),
                      ((q[..., :32].contiguous(), kc, vc, ks, vs), ValueError)):
        with pytest.raises(err):
            call(*args, table, ctx, 11)
    for kw in (dict(), dict(T=3), dict(dtype=torch.bfloat16), dict(T=3, dtype=torch.float16),
               dict(k_out=torch.zeros(1, 2, 4, 64, device="cuda"), v_out=torch.zeros(1, 2, 3, 64, device="cuda")),
               dict(v_out=torch.zeros(1, 2, 3, 64, device="cuda"), T=4),
               dict(T=3, dtype=torch.float32, status=torch.zeros(1, dtype=torch.int32, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            saf.saf_kv_read_quant(kc, vc, ks, vs, table, **kw)
    with pytest.raises(ValueError):
        saf.saf_kv_read_quant(None, vc, ks, vs, table, T=3, dtype=torch.float32)
    with pytest.raises(TypeError):
        saf.saf_kv_append_quant(q[:, :2], q[:, :2], kc.view(torch.uint8), vc, ks, vs, table, ctx)


def test_positions_far_apart(saf):
    for dtype, d in SOME:
        frozen = [0, 1, 0, 0]
        x = Batch(dtype, 4, 2, 1, d, 64, (0, 2500, 1200), (1, 1, 1), prefix=200, seed=13)
        x.check(*x.call(saf, frozen), frozen)
        x = Batch(dtype, 4, 2, 1, d, 64, (0, 2500, 1200), (1, 1, 1), prefix=200, seed=14)
        x.check(*x.call(saf, frozen, 300, 5), frozen, 300, 5)


def test_a_long_chunk_of_a_prompt(saf):
    for dtype, d in (("bf16", 64), ("bf16", 96), ("bf16", 128), ("fp32", 64)):
        frozen = [0, 0, 0, 1]
        x = Batch(dtype, 4, 1, 400, d, 32, (700, 0), (400, 399), seed=15)
        x.check(*x.call(saf, frozen, 260, 3), frozen, 260, 3)
        x.check(*x.call(saf, frozen), frozen)


def test_large_pages_and_no_prefix(saf):
    for dtype in ("bf16", "fp32"):
        for page in (512, 1024):
            x = Batch(dtype, 4, 4, 2, 64, page, (1500, 3), (2, 2), seed=page)
            o, lse = x.call(saf, [0, 1, 0, 0])
            x.check(o, lse, [0, 1, 0, 0])
            o2, lse2 = saf.saf_attn_paged_shared_quant(x.q.cuda(), *x.cache(), None, 0, x.table.cuda(), x.ctx.cuda(),
                                                       x.max_len, x.n_new.cuda(), x.a.cuda(), x.r.cuda(),
                                                       [0, 1, 0, 0])
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 64)])
def test_offsets_past_32_bits(saf, dtype, d):
    # caches of more than 2^32 codes, of which the last pages are used (the rest is never touched)
    Hkv, page, used = 8, 64, 12
    num = 2 ** 32 // (Hkv * page * d) + 1 + used
    dt = DT[dtype]
    g = torch.Generator().manual_seed(1)
    cache = [torch.empty(num, Hkv, page, d, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    cache += [torch.empty(num, Hkv, page, device="cuda") for _ in range(2)]
    x = Batch(dtype, 8, Hkv, 1, d, page, (300, 290), (1, 1), seed=3)
    perm = num - used + torch.randperm(used, generator=g)[:10].reshape(2, 5)
    table = perm.int().cuda()
    k, v = (torch.randn(2, Hkv, 300, d, generator=g).to(dt).cuda() for _ in range(2))
    ctx0, n0 = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor([300, 290], dtype=torch.int32).cuda()
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    saf.saf_kv_append_quant(k, v, *cache, table, ctx0, n0, status=status)
    k1, v1 = (torch.randn(2, Hkv, 1, d, generator=g).to(dt).cuda() for _ in range(2))
    saf.saf_kv_append_quant(k1, v1, *cache, table, n0, status=status)
    o, lse = saf.saf_attn_paged_quant(x.q.cuda(), *cache, table, n0, 301)
    small = [(c.view(torch.uint8) if c.dtype == E4M3 else c)[num - used:].clone() for c in cache]
    small = [c.view(E4M3) if c.dtype == torch.uint8 else c for c in small]
    near = (table - (num - used)).int()
    o2, lse2 = saf.saf_attn_paged_quant(x.q.cuda(), *small, near, n0, 301)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    back = saf.saf_kv_read_quant(*cache, table, None, n0, T=300, dtype=dt, status=status)
    again = saf.saf_kv_read_quant(*small, near, None, n0, T=300, dtype=dt)
    assert saf.saf_device_status(status) == saf.SAF_OK
    for got, ref, y in zip(back, again, (k, v)):
        assert torch.equal(got, ref)
        off = (got.double() - y.double()).abs()
        step = 2.0 ** -4 * y.double().abs() + 2.0 ** -10 / 448 * y.double().abs().amax(-1, keepdim=True)
        assert (off <= step * 1.01 + 2.0 ** -8 * y.double().abs())[0].all()


def test_on_a_given_stream_beside_a_busy_one(saf):
    # what a call allocates and clears belongs to the stream it is given, not to the current one
    for T in (3, 40):
        x = Batch("bf16", 4, 2, T, 64, 16, (900, 60), (T, 2), seed=6)
        head = [x.q.cuda(), *x.cache(), x.table.cuda(), x.ctx.cuda()]
        kw = dict(n_new=x.n_new.cuda(), a=x.a.cuda(), r=x.r.cuda(), frozen=[0, 1, 0, 0])
        k, v = (torch.randn(2, 2, T, 64, device="cuda").bfloat16() for _ in range(2))
        freq = [1.0, 0.1, 0.01, 0.5, 0.2, 0.3, 0.4, 0.6]
        pages = torch.arange(6, dtype=torch.int32, device="cuda").reshape(2, 3)
        none = torch.zeros_like(head[6])

        def step(**on):
            c = [torch.zeros(head[1].shape, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
            c += [torch.zeros_like(head[3]) for _ in range(2)]
            torch.cuda.synchronize()
            if on:
                torch.cuda._sleep(100_000_000)   # about 50 ms on the current stream
            q = saf.saf_kv_append_quant(k, v, *c, pages, none, kw["n_new"], q=head[0], inv_freq=freq, **on)
            rows = saf.saf_kv_read_quant(*c, pages, none, kw["n_new"], T=T, dtype=torch.bfloat16, **on)
            out = saf.saf_attn_paged_quant(*head, x.max_len, **kw, **on)
            torch.cuda.synchronize()
            return [q, *rows, *out, c[0].view(torch.uint8), c[3]]

        want = step()
        for got, ref in zip(step(stream=torch.cuda.Stream()), want):
            assert torch.equal(got, ref)


@pytest.mark.parametrize("T", [2, 40])
def test_counts_and_pages_out_of_bounds_are_reported(saf, T):
    # a bad entry reaches no memory: the keys of such a page are not seen, the counts are cut
    for dtype in ("bf16", "fp32"):
        for what in ("page", "ctx", "n_new", "past"):
            x = Batch(dtype, 2, 2, T, 64, 16, (100, 60), (T, 2), seed=5)
            ws = saf.alloc_paged_quant_workspace(2, 2, 2, T, 64, x.max_len, DT[dtype])
            good = x.call(saf, workspace=ws)
            assert saf.saf_device_status(ws) == saf.SAF_OK
            if what == "page":
                x.table[0, 1] = x.codes[0].shape[0]
            elif what == "ctx":
                x.ctx[0] = -1
            elif what == "n_new":
                x.n_new[0] = T + 1
            else:
                x.ctx[0] = x.max_len
            o, lse = x.call(saf, workspace=ws)
            assert saf.saf_device_status(ws) == saf.SAF_EPAGE
            assert torch.equal(o[1], good[0][1]) and torch.equal(lse[1], good[1][1])
            assert torch.isfinite(o[0].float()).all()
            if what in ("ctx", "past"):
                assert not o[0].any() and torch.isneginf(lse[0]).all()
            elif what == "page":
                k, v = x.rows(0, 100 + T)
                k, v = (np.delete(y, np.arange(16, 32), axis=0) for y in (k, v))
                i = np.array([len(k) - 1])   # the last token sees every key that is left
                for h in range(2):
                    qh = _np(x.q)[0, h, -1:]
                    W, l_ref = so.row_weights(qh, k[:, h], i, None, None, False)
                    ref = W @ v[:, h]
                    tol, _ = bounds(dtype, qh, k[:, h], v[:, h], W, ref, l_ref, None, None, i, False)
                    assert (np.abs(_np(o)[0, h, -1:] - ref) <= tol).all()


# ---------------------------------------------------------------------------
# Append and read
# ---------------------------------------------------------------------------
def _append_case(dtype, H, Hkv, T, d, page, ctx, n_new, seed, strided):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    B = len(ctx)
    per = -(-(max(c + n for c, n in zip(ctx, n_new)) + 1) // page)
    table = torch.randperm(B * per + 3, generator=g)[:B * per].reshape(B, per).int()
    shape = (B * per + 3, Hkv, page)
    codes = [torch.randint(0, 256, (*shape, d), generator=g).to(torch.uint8) for _ in range(2)]
    scales = [torch.randn(shape, generator=g) for _ in range(2)]
    if strided:   # one projection's output, token by token
        qkv = torch.randn(B, T, H + 2 * Hkv, d, generator=g).to(dt).cuda().transpose(1, 2)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    else:
        q, k, v = (torch.randn(B, n, T, d, generator=g).to(dt).cuda() for n in (H, Hkv, Hkv))
    return table, codes, scales, q, k, v


def _device(codes, scales):
    return [c.cuda().view(E4M3) for c in codes] + [s.cuda() for s in scales]


def _check_rows(codes, scales, want, err):
    """Rows [..., d] as codes and scales against the values: half a step of e4m3 (2^-4 of the value, or
    2^-10 scale near zero), the arithmetic before it (err, absolute), and 2^-21 for the scale and its inverse."""
    top = np.abs(want).max(axis=-1) / 448
    assert (np.abs(scales - top) <= 2.0 ** -22 * top + err.max(axis=-1) / 448 + 2.0 ** -126).all()
    got = so.dequantise(codes, scales)
    tol = np.maximum(2.0 ** -4 * (np.abs(want) + err), 2.0 ** -10 * scales[..., None]) * (1 + 2.0 ** -20)
    assert (np.abs(got - want) <= tol + err + 2.0 ** -21 * np.abs(want)).all()


@pytest.mark.parametrize("dtype,d", ALL)
@pytest.mark.parametrize("page", [8, 32, 1024])
@pytest.mark.parametrize("rope", [0, 16, 48, -1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(saf, dtype, d, page, rope, interleaved):
    rope = d if rope < 0 else rope
    H, Hkv = 6, 3
    frozen = [0, 1, 1, 1, 0, 0]   # the second key/value head serves frozen query heads only
    ctx, n_new, T = (0, 31, 77), (5, 0, 3), 5
    freq = 10000.0 ** (-np.arange(0, rope, 2) / max(rope, 1))
    for strided in (False, True):
        table, codes, scales, q, k, v = _append_case(dtype, H, Hkv, T, d, page, ctx, n_new, rope + page, strided)
        cache = _device(codes, scales)
        q_out = torch.full((3, H, T, d), 9.0, dtype=DT[dtype], device="cuda")
        args = (table.cuda(), torch.tensor(ctx).int().cuda(), torch.tensor(n_new).int().cuda())
        kw = dict(q=q, inv_freq=torch.from_numpy(freq) if rope else None, interleaved=interleaved, pos_base=11,
                  frozen=frozen)
        saf.saf_kv_append_quant(k, v, *cache, *args, q_out=q_out, **kw)
        # q is the plain append's, to the bit
        plain = [torch.zeros(*codes[0].shape, dtype=DT[dtype], device="cuda") for _ in range(2)]
        q_plain = torch.full_like(q_out, 9.0)
        saf.saf_kv_append(k, v, *plain, *args, q_out=q_plain, **kw)
        assert torch.equal(q_out, q_plain)
        got = [c.view(torch.uint8).cpu().numpy() for c in cache[:2]] + [s.cpu().double().numpy() for s in cache[2:]]
        touched = np.zeros((2, *scales[0].shape), bool)
        for b in range(3):
            for t in range(n_new[b]):
                x = ctx[b] + t
                pg, at = int(table[b, x // page]), x % page
                touched[1, pg, :, at] = True
                vr = _np(v)[b, :, t]
                _check_rows(got[1][pg, :, at], got[3][pg, :, at], vr, np.zeros_like(vr))
                for hk in (0, 2):
                    touched[0, pg, hk, at] = True
                    kr = so.rotate(_np(k)[b, hk, t][None], [11 + x], freq, interleaved)[0]
                    err = np.full_like(kr, (6 * _bounds.E + 2.0 ** -21) * 2 * np.abs(_np(k)[b, hk, t]).max())
                    _check_rows(got[0][pg, hk, at], got[2][pg, hk, at], kr, err if rope else 0 * err)
        for i in range(2):
            assert np.array_equal(got[i][~touched[i]], codes[i].numpy()[~touched[i]])
            assert np.array_equal(got[2 + i][~touched[i]], scales[i].double().numpy()[~touched[i]])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_rows_that_are_not_ordinary(saf, dtype):
    # zeros, one element, the smallest and the largest numbers, NaN, infinity: in one call, beside ordinary rows
    d, T = 96, 8
    table, codes, scales, _, k, v = _append_case(dtype, 2, 2, T, d, 8, (3,), (T,), 9, False)
    big = torch.finfo(DT[dtype]).max
    for y in (k, v):
        y[0, :, 0] = 0
        y[0, :, 1] = 0
        y[0, :, 1, 95] = -3.0
        y[0, :, 2] *= 2.0 ** -125
        y[0, :, 3] = y[0, :, 3].sign() * big
        y[0, :, 4, 5] = float("nan")
        y[0, :, 5, 7] = -float("inf")
    cache = _device(codes, scales)
    saf.saf_kv_append_quant(k, v, *cache, table.cuda(), torch.tensor([3]).int().cuda())
    at = 3 + np.arange(T)
    pg = table[0].numpy()[at // 8]
    for y, c, s in zip((k, v), cache[:2], cache[2:]):
        c, s = c.view(torch.uint8).cpu().numpy()[pg, :, at % 8], s.double().cpu().numpy()[pg, :, at % 8]
        y, got = _np(y)[0].transpose(1, 0, 2), so.dequantise(c, s)
        assert (s[0] == 2.0 ** -126).all() and not got[0].any()
        assert not got[1, :, :95].any() and np.allclose(got[1, :, 95], -3.0, rtol=2.0 ** -22, atol=0)
        for t in (2, 3, 6, 7):
            _check_rows(c[t], s[t], y[t], np.zeros_like(y[t]))
        assert np.isnan(got[4, :, 5]).all() and np.isnan(got[4]).sum() == 2
        rest = np.delete(np.arange(d), 5)
        _check_rows(c[4][:, rest], s[4], y[4][:, rest], np.zeros_like(y[4][:, rest]))
        assert np.isinf(s[5]).all() and np.isnan(got[5]).all()


def test_append_out_of_bounds_is_reported_and_writes_nothing(saf):
    for what in ("page", "negative page", "ctx", "past"):
        table, codes, scales, q, k, v = _append_case("bf16", 2, 2, 2, 64, 16, (20, 40), (2, 2), 3, False)
        ctx = torch.tensor([20, 40]).int()
        if what == "page":
            table[0, 1] = codes[0].shape[0]
        elif what == "negative page":
            table[0, 1] = -1
        elif what == "ctx":
            ctx[0] = -2
        else:
            ctx[0] = table.shape[1] * 16
        cache = _device(codes, scales)
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        saf.saf_kv_append_quant(k, v, *cache, table.cuda(), ctx.cuda(), q=q, inv_freq=[1.0] * 32, status=status)
        assert saf.saf_device_status(status) == saf.SAF_EPAGE
        for s, before in zip(cache[2:], scales):
            pages, slots = np.nonzero((_np(s) != _np(before)).any(axis=1))
            assert sorted(zip(pages, slots)) == sorted([(int(table[1, 2]), 8), (int(table[1, 2]), 9)])
        changed = (cache[1].view(torch.uint8).cpu() != codes[1]).any(dim=-1).any(dim=1)
        assert changed.sum() == 2


@pytest.mark.parametrize("dtype,d", ALL)
@pytest.mark.parametrize("page", [8, 64, 1024])
def test_read(saf, dtype, d, page):
    g = torch.Generator().manual_seed(page + d)
    B, Hkv, T, num = 4, 3, 70, 40
    per = -(-200 // page)
    codes = [torch.randint(0, 256, (num, Hkv, page, d), generator=g).to(torch.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 127) == 127] = 0
    scales = [torch.exp(3 * torch.randn(num, Hkv, page, generator=g)) for _ in range(2)]
    table = torch.randint(0, num, (B, per), generator=g).int()
    first, count = torch.tensor([0, 5, 130, 199]).int(), torch.tensor([70, 0, 33, 1]).int()
    cache = _device(codes, scales)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    outs = [torch.full((B, Hkv, T, d), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2)]
    got = saf.saf_kv_read_quant(*cache, table.cuda(), first.cuda(), count.cuda(), k_out=outs[0], v_out=outs[1],
                                status=status)
    assert got[0] is outs[0] and got[1] is outs[1] and saf.saf_device_status(status) == saf.SAF_OK
    for y, c, s in zip(got, codes, scales):
        want = torch.zeros(B, Hkv, T, d)
        for b in range(B):
            at = int(first[b]) + torch.arange(int(count[b]))
            pg, x = table[b][at // page].long(), at % page
            val = c.view(E4M3).float()[pg, :, x] * s[pg, :, x][..., None]
            want[b, :, :int(count[b])] = val.transpose(0, 1)
        assert torch.equal(y.cpu(), want.to(DT[dtype]))   # a product in fp32, rounded once
    # values only, everything from slot 0, sizes given
    none, v = saf.saf_kv_read_quant(None, cache[1], None, cache[3], table.cuda(), T=9, dtype=DT[dtype])
    assert none is None and v.shape == (B, Hkv, 9, d)
    k0, v0 = saf.saf_kv_read_quant(*cache, table.cuda(), T=9, dtype=DT[dtype])
    assert torch.equal(v, v0) and torch.equal(v0[0], got[1][0, :, :9]) and torch.equal(k0[0], got[0][0, :, :9])


def test_read_out_of_bounds_is_reported_and_zero(saf):
    for what in ("page", "first", "count", "past"):
        table, codes, scales, *_ = _append_case("bf16", 2, 2, 2, 64, 16, (20, 40), (2, 2), 3, False)
        first, count = torch.tensor([10, 20]).int(), torch.tensor([12, 3]).int()
        cache = _device(codes, scales)
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        good = saf.saf_kv_read_quant(*cache, table.cuda(), first.cuda(), count.cuda(), T=12, dtype=torch.float32)
        zero, room = slice(6, 12), table.shape[1] * 16
        if what == "page":
            table[0, 1] = -1
        elif what == "first":
            first[0], zero = -1, slice(0, 12)
        elif what == "count":
            count[0], zero = 13, slice(12, 12)
        else:
            first[0], zero = room - 4, slice(4, 12)
        got = saf.saf_kv_read_quant(*cache, table.cuda(), first.cuda(), count.cuda(), T=12, dtype=torch.float32,
                                    status=status)
        assert saf.saf_device_status(status) == saf.SAF_EPAGE
        for y, ref in zip(got, good):
            assert torch.equal(y[1].nan_to_num(), ref[1].nan_to_num())
            assert not y[0, :, zero].any()
            if what in ("page", "count"):
                assert torch.equal(y[0, :, :zero.start].nan_to_num(), ref[0, :, :zero.start].nan_to_num())


# ---------------------------------------------------------------------------
# The calls together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4)])
def test_prompt_then_steps(saf, dtype, d, window, sinks):
    """A padded batch of prompts into the cache, then single tokens and drafted ones: every output against
    fp64 over what the cache stands for, which lies within half a step of the keys and values; and the
    prompt through the windowed layer on the rows read back."""
    H, Hkv, page, frozen = 4, 2, 16, [0, 1, 0, 0]
    prompts, steps = [130, 75], [1, 1, 3, 1]
    Tp, B = max(prompts), 2
    total = Tp + sum(steps)
    g = torch.Generator().manual_seed(77)
    dt = DT[dtype]
    q, k, v = (torch.randn(B, n, total, d, generator=g).to(dt) for n in (H, Hkv, Hkv))
    a = torch.randn(H, total, generator=g)
    r = 0.5 * torch.randn(H, total, generator=g) - 0.03 * torch.arange(total)
    freq = 10000.0 ** (-np.arange(0, d, 2) / d)
    per = -(-total // page)
    table = torch.randperm(B * per, generator=g).reshape(B, per).int().cuda()
    cache = [torch.full((B * per, Hkv, page, d), 127, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    cache += [torch.full((B * per, Hkv, page), float("nan"), device="cuda") for _ in range(2)]
    rope = torch.from_numpy(freq)
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    n_new = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    ac, rc = a.cuda(), r.cuda()
    outs, qs, layer = [[] for _ in range(B)], [[] for _ in range(B)], None

    def piece(x, starts, n):   # tokens starts[b] .. + n of each sequence
        return torch.stack([x[b, :, s:s + n] for b, s in enumerate(starts)]).contiguous().cuda()

    at = [0, 0]
    for t, new in [(Tp, prompts)] + [(t, [t, t]) for t in steps]:
        n_new.copy_(torch.tensor(new, dtype=torch.int32))
        qr = saf.saf_kv_append_quant(piece(k, at, t), piece(v, at, t), *cache, table, ctx, n_new, q=piece(q, at, t),
                                     inv_freq=rope, frozen=frozen)
        o, lse = saf.saf_attn_paged_quant(qr, *cache, table, ctx, total, n_new, a=ac, r=rc, frozen=frozen,
                                          window=window, sinks=sinks)
        if t == Tp:
            rows = saf.saf_kv_read_quant(*cache, table, None, n_new, T=t, dtype=dt)
            layer = saf.saf_attn_fwd_window(qr, *rows, ac, rc, frozen, window, sinks)[0]
        for b in range(B):
            outs[b].append(_np(o[b, :, :new[b]]))
            qs[b].append(_np(qr[b, :, :new[b]]))
        ctx += n_new
        at = [x + n for x, n in zip(at, new)]
    codes = [c.view(torch.uint8).cpu().numpy() for c in cache[:2]]
    scales = [s.double().cpu().numpy() for s in cache[2:]]
    for b in range(B):
        n = at[b]
        i = np.arange(n)
        pages = table[b].cpu()
        kc, vc = ((so.gather(c, pages, n), so.gather(s[..., None], pages, n)[..., 0]) for c, s in zip(codes, scales))
        _check_rows(*vc, _np(v)[b, :, :n].transpose(1, 0, 2), np.zeros((n, Hkv, d)))
        rot = so.rotate(_np(k)[b, :, :n], i, freq, False).transpose(1, 0, 2)
        _check_rows(*kc, rot, np.full(rot.shape, (6 * _bounds.E + 2.0 ** -21) * 2 * np.abs(_np(k)).max()))
        kk, vv = so.dequantise(*kc), so.dequantise(*vc)
        got, qq = np.concatenate(outs[b], axis=1), np.concatenate(qs[b], axis=1)
        m = prompts[b]
        for h in range(H):
            W, l = so.row_weights(qq[h], kk[:, h // 2], i, _np(a)[h], _np(r)[h], frozen[h], window, sinks)
            ref = W @ vv[:, h // 2]
            tol, _ = bounds(dtype, qq[h], kk[:, h // 2], vv[:, h // 2], W, ref, l, _np(a)[h], _np(r)[h], i, frozen[h])
            assert (np.abs(got[h] - ref) <= tol).all(), (b, h)
            # the layer takes the rows rounded to dt: u of each key in the logits, u of each value
            u = _bounds.HALF[dtype]
            near = u * (np.abs(qq[h]) @ np.abs(kk[:, h // 2]).T).max() / np.sqrt(d)
            mag = W @ np.abs(vv[:, h // 2])
            extra = (2 * np.expm1(near) + u + (1e-4 if frozen[h] else 0)) * mag
            assert (np.abs(_np(layer)[b, h, :m] - ref[:m]) <= (tol + extra)[:m]).all(), (b, h)


@pytest.mark.parametrize("T", [1, 40])
def test_captured_steps(saf, T):
    """Two captured graphs (append, then attention) serve every step, each with a workspace of its own, beside
    an eager step on another stream: the counts live on the device."""
    H, Hkv, d, page, B, total = 4, 2, 64, 16, 3, 64 + 12 * T
    per = -(-total // page)
    g = torch.Generator().manual_seed(3)
    table = torch.randperm(B * per, generator=g).reshape(B, per).int().cuda()
    ctx = torch.tensor([0, 20, 45], dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros(B, n, T, d, dtype=torch.bfloat16, device="cuda") for n in (H, Hkv, Hkv))
    freq = torch.ones(32, dtype=torch.float64)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")

    def new_cache():   # the slots before ctx hold zeros
        return [torch.zeros(B * per, Hkv, page, d, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)] + \
               [torch.ones(B * per, Hkv, page, device="cuda") for _ in range(2)]

    def step(cache, qo, **kw):
        saf.saf_kv_append_quant(k, v, *cache, table, ctx, q=q, q_out=qo, inv_freq=freq, status=status)
        return saf.saf_attn_paged_quant(qo, *cache, table, ctx, total, **kw)

    kept = []
    for _ in range(2):
        own = dict(o=torch.empty_like(q), lse=torch.empty(B, H, T, device="cuda"),
                   workspace=saf.alloc_paged_quant_workspace(B, H, Hkv, T, d, total, torch.bfloat16))
        cache, qo = new_cache(), torch.empty_like(q)
        step(cache, qo, **own)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(cache, qo, **own)
        kept.append((graph, own, cache, qo))
    eager, side = new_cache(), [torch.cuda.Stream() for _ in range(2)]
    for n in range(12):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))
        for s, (graph, *_) in zip(side, kept):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                graph.replay()
        o, lse = step(eager, torch.empty_like(q))
        for s, (_, own, *_) in zip(side, kept):
            torch.cuda.current_stream().wait_stream(s)
            assert torch.equal(o, own["o"]) and torch.equal(lse, own["lse"]), n
        ctx += T
    assert saf.saf_device_status(status) == saf.SAF_OK
    for _, own, *_ in kept:
        assert saf.saf_device_status(own["workspace"]) == saf.SAF_OK


def test_same_bits_on_every_run(saf):
    for dtype in ("bf16", "fp32"):
        for T in (2, 40):
            x = Batch(dtype, 8, 2, T, 64, 16, (1000, 333, 700), (2, 1, T), prefix=500, seed=6)
            frozen = [0, 0, 1, 0, 0, 0, 0, 1]
            first = x.call(saf, frozen)
            for _ in range(3):
                again = x.call(saf, frozen)
                assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
