"""GPU parity of the paged calls (saf_kv_append, saf_attn_paged, saf_attn_paged_shared) against
the fp64 reference, with bounds from tests/_bounds.py.

Whatever no token owns is poisoned: free pages, the slots behind a sequence's last token and the
page table's entries behind it hold NaN, infinities or numbers that are no page.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from tests import _bounds

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def saf():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from softmax_attention_hybrid_gb300 import saf as mod
    return mod


def _np(t):
    return t.double().cpu().numpy()


class Batch:
    """Sequences of ctx + n_new tokens in shuffled pages, with poison in every free place."""

    def __init__(self, dtype, H, Hkv, T, d, page, ctx, n_new, prefix=0, seed=0, max_len=None, scale=1.0,
                 first_seen=0):
        g = torch.Generator().manual_seed(seed)
        dt = DT[dtype]
        B = len(ctx)
        total = [c + n for c, n in zip(ctx, n_new)]
        self.max_len = max_len or max(1, max(total, default=1))
        per = -(-self.max_len // page)
        npp = -(-prefix // page)
        count = sum(-(-t // page) for t in total) + npp + 2
        order = torch.randperm(count, generator=g).tolist()
        rand = lambda *s: (torch.randn(*s, generator=g) * scale).to(dt)   # noqa: E731
        poison = torch.tensor([float("nan"), float("inf"), -float("inf")])
        self.kc = poison[torch.randint(0, 3, (count, Hkv, page, d), generator=g)].to(dt)
        self.vc = poison[torch.randint(0, 3, (count, Hkv, page, d), generator=g)].to(dt)
        self.table = torch.full((B, per), -7, dtype=torch.int32)
        self.table[:, 1::2] = 2 ** 30
        self.prefix_pages = torch.tensor([order.pop() for _ in range(npp)], dtype=torch.int32)
        for cache in (self.kc, self.vc):
            for x in range(prefix):
                cache[self.prefix_pages[x // page], :, x % page] = rand(Hkv, d)
        for b in range(B):
            for at in range(-(-total[b] // page)):
                pg = order.pop()
                n = min(page, total[b] - at * page)
                for cache in (self.kc, self.vc):
                    cache[pg, :, :n] = rand(Hkv, n, d)
                # a page that lies before everything that is seen may be gone
                self.table[b, at] = pg if (at + 1) * page > first_seen else -3
        self.q = rand(B, H, T, d)
        L = prefix + self.max_len
        self.a = torch.randn(H, L, generator=g)
        self.r = 0.5 * torch.randn(H, L, generator=g) - 0.03 * torch.arange(L)
        self.ctx, self.n_new = (torch.tensor(x, dtype=torch.int32) for x in (ctx, n_new))
        self.dtype, self.prefix, self.Hkv = dtype, prefix, Hkv

    def call(self, saf, frozen=None, window=0, sinks=0, **kw):
        c = lambda t: t.cuda()   # noqa: E731
        args = dict(n_new=c(self.n_new), a=c(self.a), r=c(self.r), frozen=frozen, window=window, sinks=sinks)
        args.update(kw)
        head = (c(self.q), c(self.kc), c(self.vc))
        tail = (c(self.table), c(self.ctx), self.max_len)
        if self.prefix:
            return saf.saf_attn_paged_shared(*head, c(self.prefix_pages), self.prefix, *tail, **args)
        return saf.saf_attn_paged(*head, *tail, **args)

    def check(self, o, lse, frozen=None, window=0, sinks=0):
        o, lse = _np(o), _np(lse)
        q, kc, vc, a, r = (_np(t) for t in (self.q, self.kc, self.vc, self.a, self.r))
        B, H, T, d = q.shape
        G = H // self.Hkv
        P = self.prefix
        kp, vp = so.gather(kc, self.prefix_pages, P), so.gather(vc, self.prefix_pages, P)
        for b in range(B):
            n = int(self.n_new[b])
            L = int(self.ctx[b]) + n
            table = self.table[b].clamp(min=0, max=kc.shape[0] - 1)
            k = np.concatenate([kp, so.gather(kc, table, L)])
            v = np.concatenate([vp, so.gather(vc, table, L)])
            i = P + int(self.ctx[b]) + np.arange(n)
            assert not o[b, :, n:].any() and np.isneginf(lse[b, :, n:]).all()
            if n == 0:
                continue
            if not all(frozen or [0]) and (window and not any(frozen or [0])):
                # keys behind every window may be gone: they carry no weight
                hidden = ~so.visible(i, np.arange(len(k)), window, sinks).any(axis=0)
                k[hidden], v[hidden] = 0, 0
            for h in range(H):
                fz = bool(frozen and frozen[h])
                kk, vv = np.nan_to_num(k[:, h // G]), v[:, h // G]
                W, l_ref = so.row_weights(q[b, h, :n], kk, i, a[h], r[h], fz, window, sinks)
                ref = W @ vv
                s = _bounds.logit_error(q[b, h, :n], kk, a[h], r[h], i, fz)
                o_tol, l_tol = _bounds.fwd(self.dtype, W, vv, ref, l_ref, s)
                assert (np.abs(o[b, h, :n] - ref) <= o_tol).all(), (b, h)
                assert (np.abs(lse[b, h, :n] - l_ref) <= l_tol).all(), (b, h)


LENS = [(0,), (1,), (63, 0, 64), (127, 128, 129), (200, 7, 391), (1030, 515)]


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 96), ("bf16", 128), ("fp32", 64), ("fp32", 96),
                                     ("fp32", 128)])
@pytest.mark.parametrize("page", [8, 16, 64, 256])
@pytest.mark.parametrize("ctx", LENS)
def test_one_new_token(saf, dtype, d, page, ctx):
    frozen = [0, 1, 0, 0, 1, 1]
    x = Batch(dtype, 6, 2, 1, d, page, ctx, [1] * len(ctx), seed=page + d)
    x.check(*x.call(saf, frozen), frozen)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 1), (12, 4), (5, 5), (40, 1)])
@pytest.mark.parametrize("T,n_new", [(1, (1, 1)), (4, (4, 2)), (5, (0, 3)), (9, (1, 9)), (70, (70, 33)),
                                     (150, (150, 0))])
def test_new_tokens_and_groups(saf, dtype, H, Hkv, T, n_new):
    frozen = [h % 3 == 1 for h in range(H)]
    x = Batch(dtype, H, Hkv, T, 64, 16, (90, 37), n_new, seed=H + T)
    x.check(*x.call(saf, frozen), frozen)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 96)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 0), (100, 130), (129, 4), (700, 2), (5000, 9)])
@pytest.mark.parametrize("T", [1, 6])
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
        x = Batch(dtype, 4, 2, 3, 64, 16, (600, 640), (3, 2), seed=4, first_seen=600 - 100 + 1)
        status = saf.alloc_paged_workspace(2, 4, 2, 3, 64, x.max_len, DT[dtype])
        x.check(*x.call(saf, None, 100, 0, workspace=status), None, 100, 0)
        assert saf.saf_device_status(status) == saf.SAF_OK


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 96), ("bf16", 128), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("prefix,page", [(1, 8), (16, 16), (100, 32), (129, 64), (700, 256)])
@pytest.mark.parametrize("H,Hkv,T", [(3, 3, 1), (8, 2, 1), (8, 2, 3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 4), (40, 200)])
def test_shared_prefix(saf, dtype, d, prefix, page, H, Hkv, T, window, sinks):
    for fz in ([h % 4 == 3 for h in range(H)], None):
        ctx = (0, 5, 77, 31, 200)
        n_new = [T, T, 1, 0, T]
        x = Batch(dtype, H, Hkv, T, d, page, ctx, n_new, prefix=prefix, seed=prefix)
        x.check(*x.call(saf, fz, window, sinks), fz, window, sinks)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("prefix", [0, 100])
@pytest.mark.parametrize("frozen", [(), (0,), tuple(range(256))])
def test_one_group_of_the_largest_head_count(saf, dtype, d, prefix, frozen):
    # 256 query heads over one key/value head: a count of ordinary heads that takes more than 8 bits
    flags = [h in frozen for h in range(256)]
    x = Batch(dtype, 256, 1, 2, d, 16, (90, 37), (2, 1), prefix=prefix, seed=44)
    none = {} if frozen else dict(a=None, r=None)
    x.check(*x.call(saf, flags, **none), flags)
    if not frozen:
        x.check(*x.call(saf, flags, 20, 3, **none), flags, 20, 3)


def test_many_sequences_share_a_prefix(saf):
    # more rows than one tile holds, in both kinds of head
    for dtype in ("bf16", "fp32"):
        B = 70
        ctx, n_new = [(7 * b) % 40 for b in range(B)], [1 + (b % 2) for b in range(B)]
        frozen = [0, 1, 0, 0]
        x = Batch(dtype, 4, 2, 2, 64, 16, ctx, n_new, prefix=300, seed=1)
        x.check(*x.call(saf, frozen), frozen)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("masked", [-float("inf"), torch.finfo(torch.float32).min])
@pytest.mark.parametrize("prefix", [0, 40])
def test_keys_that_a_pattern_masks(saf, dtype, d, masked, prefix):
    # a head whose pattern leaves nothing: zeros and -infinity; one that masks some keys: no weight there
    frozen = [0, 1, 1, 0]
    x = Batch(dtype, 4, 2, 2, d, 16, (0, 100, 300), (2, 2, 1), prefix=prefix, seed=3)
    x.a[1], x.a[2, 3:7] = masked, masked
    o, lse = x.call(saf, frozen)
    assert not o[:, 1].any() and torch.isneginf(lse[:, 1]).all()
    # (the first row sees key 0 alone and the next ones 1, 2, ...: never only masked keys)
    x.a[1], x.a[2, 3:7] = 0.0, -200.0   # e^-200: nothing in the outputs' bits
    o[:, 1], lse[:, 1] = (t[:, 1] for t in x.call(saf, frozen))
    x.check(o, lse, frozen)


def test_every_head_frozen_reads_no_keys(saf):
    for dtype in ("bf16", "fp32"):
        x = Batch(dtype, 4, 2, 2, 64, 16, (30, 50), (2, 1), seed=2)
        x.kc.fill_(float("nan"))
        x.q.fill_(float("nan"))
        o, lse = x.call(saf, [1] * 4)
        x.q.fill_(0)
        x.check(o, lse, [1] * 4)


def test_bound_above_the_lengths(saf):
    # max_len far above what the sequences hold: empty work items on every side
    for dtype in ("bf16", "fp32"):
        x = Batch(dtype, 4, 2, 1, 64, 16, (3, 300, 0), (1, 1, 1), seed=8, max_len=9000)
        x.check(*x.call(saf, [0, 0, 0, 1]), [0, 0, 0, 1])


def test_large_scores(saf):
    # scores in the hundreds: one key takes nearly all the weight, others vanish
    for dtype in ("bf16", "fp32"):
        x = Batch(dtype, 2, 1, 2, 64, 16, (500, 130), (2, 2), seed=11, scale=6.0)
        x.check(*x.call(saf))


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("ctx", [3, 40, 5000])
@pytest.mark.parametrize("bad", ["q", "inf"])
def test_a_row_of_nan_stays_one_and_alone(saf, dtype, d, ctx, bad):
    # a NaN query has NaN for its output, in one item or joined from several; so has one whose scores
    # are infinite. The other rows of its block keep their bits.
    x = Batch(dtype, 4, 2, 2, d, 64, (ctx, 7), (2, 2), seed=71)
    want, want_lse = x.call(saf)
    x.q[0, 1, 0] = float("nan") if bad == "q" else float("inf")
    o, lse = x.call(saf)
    assert o[0, 1, 0].isnan().all() and lse[0, 1, 0].isnan()
    o[0, 1, 0], lse[0, 1, 0] = want[0, 1, 0], want_lse[0, 1, 0]
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_positions_far_apart(saf):
    # rows of one block 2500 positions apart: the frozen heads' patterns do not fit beside the tiles
    for dtype, d in (("bf16", 64), ("bf16", 128), ("fp32", 64)):
        frozen = [0, 1, 0, 0]
        x = Batch(dtype, 4, 2, 1, d, 64, (0, 2500, 1200), (1, 1, 1), prefix=200, seed=13)
        x.check(*x.call(saf, frozen), frozen)
        x = Batch(dtype, 4, 2, 1, d, 64, (0, 2500, 1200), (1, 1, 1), prefix=200, seed=14)
        x.check(*x.call(saf, frozen, 300, 5), frozen, 300, 5)


def test_a_long_chunk_of_a_prompt(saf):
    for dtype in ("bf16", "fp32"):
        frozen = [0, 0, 0, 1]
        x = Batch(dtype, 4, 1, 400, 64, 32, (700, 0), (400, 399), seed=15)
        x.check(*x.call(saf, frozen, 260, 3), frozen, 260, 3)


def test_large_pages_and_no_prefix(saf):
    for dtype in ("bf16", "fp32"):
        for page in (512, 1024):
            x = Batch(dtype, 4, 4, 2, 64, page, (1500, 3), (2, 2), seed=page)
            o, lse = x.call(saf, [0, 1, 0, 0])
            x.check(o, lse, [0, 1, 0, 0])
            o2, lse2 = saf.saf_attn_paged_shared(x.q.cuda(), x.kc.cuda(), x.vc.cuda(), None, 0, x.table.cuda(),
                                                 x.ctx.cuda(), x.max_len, x.n_new.cuda(), x.a.cuda(), x.r.cuda(),
                                                 [0, 1, 0, 0])
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 64)])
def test_offsets_past_32_bits(saf, dtype, d):
    # caches of more than 2^32 elements, of which the last pages are used (the rest is never touched)
    Hkv, page, used = 8, 64, 12
    num = 2 ** 32 // (Hkv * page * d) + 1 + used
    dt = DT[dtype]
    g = torch.Generator().manual_seed(1)
    kc, vc = (torch.empty(num, Hkv, page, d, dtype=dt, device="cuda") for _ in range(2))
    assert kc[num - used:].storage_offset() > 2 ** 32
    x = Batch(dtype, 8, Hkv, 1, d, page, (300, 290), (1, 1), seed=3)
    perm = num - used + torch.randperm(used, generator=g)[:10].reshape(2, 5)
    table = perm.int().cuda()
    k, v = (torch.randn(2, Hkv, 300, d, generator=g).to(dt).cuda() for _ in range(2))
    ctx0, n0 = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor([300, 290], dtype=torch.int32).cuda()
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    saf.saf_kv_append(k, v, kc, vc, table, ctx0, n0, status=status)
    k1, v1 = (torch.randn(2, Hkv, 1, d, generator=g).to(dt).cuda() for _ in range(2))
    saf.saf_kv_append(k1, v1, kc, vc, table, n0, status=status)
    o, lse = saf.saf_attn_paged(x.q.cuda(), kc, vc, table, n0, 301)
    small = kc[num - used:].clone(), vc[num - used:].clone()
    o2, lse2 = saf.saf_attn_paged(x.q.cuda(), *small, (table - (num - used)).int(), n0, 301)
    assert saf.saf_device_status(status) == saf.SAF_OK
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for b, n in ((0, 300), (1, 290)):
        at = torch.arange(n + 1)
        got = small[1][(perm[b] - (num - used))[at // page].cuda(), :, (at % page).cuda()]
        assert torch.equal(got[:n].transpose(0, 1), v[b, :, :n]) and torch.equal(got[n], v1[b, :, 0])


def test_on_a_given_stream(saf):
    x = Batch("bf16", 4, 2, 1, 64, 16, (100, 60), (1, 1), seed=5)
    want = x.call(saf)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ws = saf.alloc_paged_workspace(2, 4, 2, 1, 64, x.max_len, torch.bfloat16)
    torch.cuda.synchronize()
    got = x.call(saf, stream=side, workspace=ws)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_on_a_stream_beside_a_busy_one(saf):
    # what a call allocates and clears belongs to the stream it is given, not to the current one
    x = Batch("bf16", 4, 2, 3, 64, 16, (900, 60), (3, 2), seed=6)
    head = [t.cuda() for t in (x.q, x.kc, x.vc, x.table, x.ctx)]
    n_new, a, r = (t.cuda() for t in (x.n_new, x.a, x.r))
    k, v = (torch.randn(2, 2, 3, 64, device="cuda").bfloat16() for _ in range(2))
    side = torch.cuda.Stream()
    kw = dict(n_new=n_new, a=a, r=r, frozen=[0, 1, 0, 0])
    freq = [1.0, 0.1, 0.01, 0.5, 0.2, 0.3, 0.4, 0.6]
    # the new tokens go to the first slots of pages of their own: a sequence has its page alone
    pages = torch.arange(2, dtype=torch.int32, device="cuda")[:, None].contiguous()
    kc, vc, none = torch.zeros_like(head[1]), torch.zeros_like(head[2]), torch.zeros_like(head[4])
    want = saf.saf_kv_append(k, v, kc, vc, pages, none, n_new, q=head[0], inv_freq=freq), \
        *saf.saf_attn_paged(*head, x.max_len, **kw)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)   # about 50 ms on the current stream
    q = saf.saf_kv_append(k, v, kc, vc, pages, none, n_new, q=head[0], inv_freq=freq, stream=side)
    o, lse = saf.saf_attn_paged(*head, x.max_len, **kw, stream=side)
    torch.cuda.synchronize()
    for got, ref in zip((q, o, lse), want):
        assert torch.equal(got, ref)


def test_counts_and_pages_out_of_bounds_are_reported(saf):
    # a bad entry reaches no memory: the keys of such a page are not seen, the counts are cut
    for dtype in ("bf16", "fp32"):
        for what in ("page", "ctx", "n_new", "past"):
            x = Batch(dtype, 2, 2, 2, 64, 16, (100, 60), (2, 2), seed=5)
            ws = saf.alloc_paged_workspace(2, 2, 2, 2, 64, x.max_len, DT[dtype])
            good = x.call(saf, workspace=ws)
            assert saf.saf_device_status(ws) == saf.SAF_OK
            if what == "page":
                x.table[0, 1] = x.kc.shape[0]
            elif what == "ctx":
                x.ctx[0] = -1
            elif what == "n_new":
                x.n_new[0] = 3
            else:
                x.ctx[0] = x.max_len
            o, lse = x.call(saf, workspace=ws)
            assert saf.saf_device_status(ws) == saf.SAF_EPAGE
            assert torch.equal(o[1], good[0][1]) and torch.equal(lse[1], good[1][1])
            assert torch.isfinite(o[0].float()).all()
            if what in ("ctx", "past"):
                assert not o[0].any() and torch.isneginf(lse[0]).all()
            elif what == "page":
                keep = [j for j in range(102) if j // 16 != 1]
                table = x.table[0].clone()
                table[1] = table[0]
                k, v = (so.gather(_np(c), table, 102)[keep] for c in (x.kc, x.vc))
                for h in range(2):
                    W, l_ref = so.row_weights(_np(x.q)[0, h, 1:], k[:, h], np.array([len(keep) - 1]), None, None, False)
                    ref = W @ v[:, h]
                    s = _bounds.logit_error(_np(x.q)[0, h, 1:], k[:, h], None, None, np.array([0]), False)
                    tol, _ = _bounds.fwd(dtype, W, v[:, h], ref, l_ref, s)
                    assert (np.abs(_np(o)[0, h, 1:] - ref) <= tol).all()


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------
def _append_case(dtype, H, Hkv, T, d, page, ctx, n_new, seed, strided):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    B = len(ctx)
    per = -(-(max(c + n for c, n in zip(ctx, n_new)) + 1) // page)
    table = torch.randperm(B * per + 3, generator=g)[:B * per].reshape(B, per).int()
    shape = (B * per + 3, Hkv, page, d)
    kc, vc = torch.randn(shape, generator=g).to(dt), torch.randn(shape, generator=g).to(dt)
    if strided:   # one projection's output, token by token
        qkv = torch.randn(B, T, H + 2 * Hkv, d, generator=g).to(dt).cuda().transpose(1, 2)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    else:
        q, k, v = (torch.randn(B, n, T, d, generator=g).to(dt).cuda() for n in (H, Hkv, Hkv))
    return table, kc, vc, q, k, v


def _append_check(dtype, got, want, rows, angle_err):
    """Rotated rows: fp32 products and one rounding: u |y| + (4 e + angle_err) (|x0| + |x1|), which
    the pair's norm, at most sqrt(2) |row|_max, bounds."""
    u = _bounds.HALF[dtype]
    tol = u * np.abs(want) + (6 * _bounds.E + angle_err) * 2 * rows
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 96), ("bf16", 128), ("fp32", 64), ("fp32", 96),
                                     ("fp32", 128)])
@pytest.mark.parametrize("page", [8, 32, 1024])
@pytest.mark.parametrize("rope", [0, 16, 48, -1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(saf, dtype, d, page, rope, interleaved):
    rope = d if rope < 0 else rope
    H, Hkv = 6, 3
    frozen = [0, 1, 1, 1, 0, 0]   # the second key/value head serves frozen query heads only
    ctx, n_new, T = (0, 31, 77), (5, 0, 3), 5
    for strided in (False, True):
        table, kc, vc, q, k, v = _append_case(dtype, H, Hkv, T, d, page, ctx, n_new, rope + page, strided)
        kc2, vc2 = kc.cuda(), vc.cuda()
        q_out = torch.full((3, H, T, d), 9.0, dtype=DT[dtype], device="cuda")
        freq = 10000.0 ** (-np.arange(0, rope, 2) / max(rope, 1))
        saf.saf_kv_append(k, v, kc2, vc2, table.cuda(), torch.tensor(ctx).int().cuda(),
                          torch.tensor(n_new).int().cuda(), q=q, q_out=q_out,
                          inv_freq=torch.from_numpy(freq) if rope else None, interleaved=interleaved, pos_base=11,
                          frozen=frozen)
        kr, vr, qr = _np(kc), _np(vc), np.full(q_out.shape, 9.0)
        rows_k, rows_q = np.zeros(kr.shape[:3] + (1,)), np.zeros(qr.shape[:3] + (1,))
        for b in range(3):
            for t in range(n_new[b]):
                x = ctx[b] + t
                pg, at = int(table[b, x // page]), x % page
                vr[pg, :, at] = _np(v)[b, :, t]
                for hk in (0, 2):
                    kr[pg, hk, at] = so.rotate(_np(k)[b, hk, t][None], [11 + x], freq, interleaved)[0]
                    rows_k[pg, hk, at] = np.abs(_np(k)[b, hk, t]).max()
                for h in (0, 4, 5):
                    qr[b, h, t] = so.rotate(_np(q)[b, h, t][None], [11 + x], freq, interleaved)[0]
                    rows_q[b, h, t] = np.abs(_np(q)[b, h, t]).max()
        assert np.array_equal(_np(vc2), vr)
        _append_check(dtype, _np(kc2), kr, rows_k, 2.0 ** -21)
        _append_check(dtype, _np(q_out), qr, rows_q, 2.0 ** -21)
        untouched = rows_k[..., 0] == 0
        assert np.array_equal(_np(kc2)[untouched], _np(kc)[untouched])


def test_append_at_far_positions(saf):
    # the angle of position 10^9 keeps its digits: (y0, y1) against 64-bit integers modulo a turn
    d, far = 64, 10 ** 9
    table, kc, vc, q, k, v = _append_case("fp32", 1, 1, 1, d, 16, (3,), (1,), 4, False)
    kc2, vc2 = kc.cuda(), vc.cuda()
    freq = 10000.0 ** (-np.arange(0, d, 2) / d)
    saf.saf_kv_append(k, v, kc2, vc2, table.cuda(), torch.tensor([3]).int().cuda(), inv_freq=freq, pos_base=far)
    turns = np.array([(far + 3) * int(f / (2 * np.pi) * 2 ** 64) % 2 ** 64 / 2 ** 64 for f in freq])
    want = so.rotate(_np(k)[0, 0], [1], 2 * np.pi * turns, False)[0]
    got = _np(kc2)[int(table[0, 0]), 0, 3]
    # the frequencies are doubles: pos * 2^-53 * freq radians of them, and a few steps of fp32
    assert np.abs(got - want).max() <= (2.0 ** -20 + far * 2.0 ** -53) * 2 * np.abs(_np(k)).max()


def _turns(f, pos):
    """pos * f / (2 pi) modulo 1 as a float, pi from Machin's formula in integers of 400 bits."""
    one = 1 << 400

    def arctan(n):   # of 1 / n
        term = total = one // n
        k = 1
        while term:
            term = -term // (n * n)
            k += 2
            total += term // k
        return total

    two_pi = Fraction(8 * (4 * arctan(5) - arctan(239)), one)
    return float(pos * Fraction(f) / two_pi % 1)


@pytest.mark.parametrize("pos", [0, 1, 12345, 10 ** 9, 2 ** 36 + 7, 2 ** 40])
@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_of_far_positions_are_exact(saf, pos, interleaved):
    # a frequency is taken to 2^-64 of a turn; from the reduced angle on, x half turns in fp32 (2^-25 of a
    # half turn) and its sine and cosine
    d = 64
    table, kc, vc, q, k, v = _append_case("fp32", 1, 1, 1, d, 16, (3,), (1,), 4, False)
    freq = 10000.0 ** (-np.arange(0, d, 2) / d)
    freq[1:6] = (-0.3, 3.7, 1e5, -1e-30, 2.0 ** -60)
    kc2, vc2 = kc.cuda(), vc.cuda()
    ctx = torch.tensor([3 if pos >= 3 else pos]).int().cuda()
    saf.saf_kv_append(k, v, kc2, vc2, table.cuda(), ctx, inv_freq=freq, interleaved=interleaved,
                      pos_base=pos - int(ctx))
    angles = 2 * np.pi * np.array([_turns(f, pos) for f in freq])
    want = so.rotate(_np(k)[0, 0], [1], angles, interleaved)[0]
    got = _np(kc2)[int(table[0, 0]), 0, int(ctx)]
    _append_check("fp32", got, want, np.abs(_np(k)).max(), 2 * np.pi * pos * 2.0 ** -64 + np.pi * 2.0 ** -25)


def test_append_in_place_and_without_q(saf):
    table, kc, vc, q, k, v = _append_case("bf16", 4, 2, 3, 64, 16, (5, 9), (3, 2), 8, False)
    freq = 100.0 ** (-np.arange(0, 64, 2) / 64)
    ctx, n_new = torch.tensor([5, 9]).int().cuda(), torch.tensor([3, 2]).int().cuda()
    a, b = [(kc.cuda(), vc.cuda()) for _ in range(2)]
    out = saf.saf_kv_append(k, v, *a, table.cuda(), ctx, n_new, q=q, inv_freq=freq)
    assert not out[1, :, 2].any()
    qq = q.clone()
    assert saf.saf_kv_append(k, v, *b, table.cuda(), ctx, n_new, q=qq, q_out=qq, inv_freq=freq) is qq
    assert torch.equal(qq[0], out[0]) and torch.equal(qq[1, :, :2], out[1, :, :2])
    assert torch.equal(qq[1, :, 2], q[1, :, 2])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = (kc.cuda(), vc.cuda())
    assert saf.saf_kv_append(k, v, *c, table.cuda(), ctx, n_new, inv_freq=freq) is None
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_append_out_of_bounds_is_reported_and_writes_nothing(saf):
    for what in ("page", "negative page", "ctx", "past"):
        table, kc, vc, q, k, v = _append_case("bf16", 2, 2, 2, 64, 16, (20, 40), (2, 2), 3, False)
        ctx = torch.tensor([20, 40]).int()
        if what == "page":
            table[0, 1] = kc.shape[0]
        elif what == "negative page":
            table[0, 1] = -1
        elif what == "ctx":
            ctx[0] = -2
        else:
            ctx[0] = table.shape[1] * 16
        kc2, vc2 = kc.cuda(), vc.cuda()
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        saf.saf_kv_append(k, v, kc2, vc2, table.cuda(), ctx.cuda(), q=q, inv_freq=[1.0] * 32, status=status)
        assert saf.saf_device_status(status) == saf.SAF_EPAGE
        changed = (_np(vc2) != _np(vc)).any(axis=(1, 3))
        pages, slots = np.nonzero(changed)
        assert sorted(zip(pages, slots)) == sorted([(int(table[1, 2]), 8), (int(table[1, 2]), 9)])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_cuts_counts_for_q_too(saf, dtype):
    # tokens past the pages' room are none: their q rows stay as they were, like those behind n_new
    table, kc, vc, q, k, v = _append_case(dtype, 2, 2, 3, 64, 16, (20, 40), (3, 3), 6, False)
    room = table.shape[1] * 16
    ctx = torch.tensor([room - 1, 40]).int().cuda()
    q_out = torch.full(q.shape, 9.0, dtype=DT[dtype], device="cuda")
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    kc2, vc2 = kc.cuda(), vc.cuda()
    saf.saf_kv_append(k, v, kc2, vc2, table.cuda(), ctx, torch.tensor([3, 7]).int().cuda(), q=q, q_out=q_out,
                      inv_freq=[1.0] * 32, status=status)
    assert saf.saf_device_status(status) == saf.SAF_EPAGE
    assert (q_out[0, :, 1:] == 9.0).all() and (q_out[0, :, 0] != 9.0).any()
    assert (q_out[1] != 9.0).any(dim=-1).all()   # 7 of 3 tokens: all three
    pages, slots = np.nonzero((_np(vc2) != _np(vc)).any(axis=(1, 3)))
    want = [(int(table[0, -1]), 15)] + [(int(table[1, 2]), x) for x in (8, 9, 10)]
    assert sorted(zip(pages, slots)) == sorted(want)


# ---------------------------------------------------------------------------
# The calls together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4)])
def test_prompt_then_steps(saf, dtype, d, window, sinks):
    """A padded batch of prompts through the windowed layer and into the cache, then single tokens
    and drafted ones: every output against the layer on the whole sequence."""
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
    kc = torch.full((B * per, Hkv, page, d), float("nan"), dtype=dt, device="cuda")
    vc = kc.clone()
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
        qr = saf.saf_kv_append(piece(k, at, t), piece(v, at, t), kc, vc, table, ctx, n_new, q=piece(q, at, t),
                               inv_freq=rope, frozen=frozen)
        o, lse = saf.saf_attn_paged(qr, kc, vc, table, ctx, total, n_new, a=ac, r=rc, frozen=frozen, window=window,
                                    sinks=sinks)
        if t == Tp:   # the prompt through the layer itself, on the keys that the cache holds
            keys = torch.zeros(B, Hkv, t, d, dtype=dt, device="cuda")
            for b in range(B):
                keys[b, :, :new[b]] = torch.from_numpy(so.gather(_np(kc), table[b].cpu(), new[b])).transpose(0, 1).to(dt)
            layer = _np(saf.saf_attn_fwd_window(qr, keys, piece(v, at, t), ac, rc, frozen, window, sinks)[0])
        for b in range(B):
            outs[b].append(_np(o[b, :, :new[b]]))
            qs[b].append(_np(qr[b, :, :new[b]]))
        ctx += n_new
        at = [x + n for x, n in zip(at, new)]
    for b in range(B):
        n = at[b]
        i = np.arange(n)
        kk, vv = so.gather(_np(kc), table[b].cpu(), n), so.gather(_np(vc), table[b].cpu(), n)
        assert np.array_equal(vv, _np(v)[b, :, :n].transpose(1, 0, 2))
        rot = so.rotate(_np(k)[b, :, :n], i, freq, False).transpose(1, 0, 2)
        assert (np.abs(kk - rot) <= _bounds.HALF[dtype] * np.abs(rot) + 2.0 ** -18 * np.abs(_np(k)).max()).all()
        got, qq = np.concatenate(outs[b], axis=1), np.concatenate(qs[b], axis=1)
        for h in range(H):
            W, l = so.row_weights(qq[h], kk[:, h // 2], i, _np(a)[h], _np(r)[h], frozen[h], window, sinks)
            ref = W @ vv[:, h // 2]
            s = _bounds.logit_error(qq[h], kk[:, h // 2], _np(a)[h], _np(r)[h], i, frozen[h])
            tol, _ = _bounds.fwd(dtype, W, vv[:, h // 2], ref, l, s)
            assert (np.abs(got[h] - ref) <= tol).all(), (b, h)
            m = prompts[b]
            # (the layer's factorised form of a frozen head rounds its weights' factors: 2^-22 each,
            # and its normaliser's inverse)
            extra = 1e-4 * (W @ np.abs(vv[:, h // 2])) if frozen[h] else 0.0
            assert (np.abs(layer[b, h, :m] - ref[:m]) <= (tol + extra)[:m] if frozen[h]
                    else np.abs(layer[b, h, :m] - ref[:m]) <= tol[:m]).all(), (b, h)


def test_captured_steps(saf):
    """One captured graph (append, then attention) serves every step: the counts live on the device."""
    H, Hkv, d, page, B, total = 4, 2, 64, 16, 3, 64
    g = torch.Generator().manual_seed(3)
    table = torch.randperm(B * 4, generator=g).reshape(B, 4).int().cuda()
    caches = [torch.zeros(B * 4, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    q, k, v = (torch.zeros(B, n, 1, d, dtype=torch.bfloat16, device="cuda") for n in (H, Hkv, Hkv))
    ctx = torch.tensor([0, 20, 45], dtype=torch.int32, device="cuda")
    freq = torch.ones(32, dtype=torch.float64)
    q_out = torch.empty_like(q)
    ws = saf.alloc_paged_workspace(B, H, Hkv, 1, d, total, torch.bfloat16)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")

    def step(kc, vc, qo, **kw):
        saf.saf_kv_append(k, v, kc, vc, table, ctx, q=q, q_out=qo, inv_freq=freq, status=status)
        return saf.saf_attn_paged(qo, kc, vc, table, ctx, total, **kw)

    o, lse = torch.empty_like(q), torch.empty(B, H, 1, device="cuda")
    step(caches[0], caches[1], q_out, o=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0], caches[1], q_out, o=o, lse=lse, workspace=ws)
    side = torch.cuda.Stream()
    for n in range(12):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):   # an eager step on another stream, its own caches
            o2, lse2 = step(caches[2], caches[3], torch.empty_like(q))
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, o2) and torch.equal(lse, lse2), n
        ctx += 1
    assert saf.saf_device_status(status) == saf.SAF_OK and saf.saf_device_status(ws) == saf.SAF_OK


def test_same_bits_on_every_run(saf):
    for dtype in ("bf16", "fp32"):
        x = Batch(dtype, 8, 2, 2, 64, 16, (1000, 333, 700), (2, 1, 2), prefix=500, seed=6)
        frozen = [0, 0, 1, 0, 0, 0, 0, 1]
        first = x.call(saf, frozen)
        for _ in range(3):
            again = x.call(saf, frozen)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
