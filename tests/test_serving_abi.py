"""Refusals of the windowed and paged calls, before any device work, on the CPU."""
import ctypes
import os

import pytest
import torch

F = 0x10000   # a fake device address: the calls below must fail before any access


@pytest.fixture(scope="module")
def saf():
    from softmax_attention_hybrid_gb300 import build_lib
    if not os.path.exists(build_lib.LIB):
        build_lib.build()
    from softmax_attention_hybrid_gb300 import saf as mod
    return mod


def _fwd_window(lib, **kw):
    x = dict(q=F, k=F, v=F, a=F, r=F, ld=256, frozen=None, state=None, window=8, sinks=0, B=1, H=4, Hkv=2, T=256, d=64,
             dt=0, o=F, lse=F, ws=F, wsb=1 << 30)
    x.update(kw)
    return lib.saf_attn_fwd_window(x["q"], x["k"], x["v"], x["a"], x["r"], x["ld"], x["frozen"], x["state"],
                                   x["window"], x["sinks"], x["B"], x["H"], x["Hkv"], x["T"], x["d"], x["dt"], x["o"],
                                   x["lse"], x["ws"], x["wsb"], None)


def _bwd_window(lib, **kw):
    x = dict(do=F, lse=F, state=None, window=8, sinks=0, H=4, Hkv=2, T=256, d=64, dq=F, dk=F, dv=F, wsb=1 << 30)
    x.update(kw)
    return lib.saf_attn_bwd_window(F, F, F, F, x["do"], x["lse"], None, None, 0, None, x["state"], x["window"],
                                   x["sinks"], 1, x["H"], x["Hkv"], x["T"], x["d"], 0, x["dq"], x["dk"], x["dv"], F,
                                   x["wsb"], None)


def test_window_refusals(saf):
    lib = saf.library()
    fz = bytes([0, 1, 0, 0])
    for call in (_fwd_window, _bwd_window):
        assert call(lib, window=-1) == saf.SAF_EINVAL
        assert call(lib, sinks=-1) == saf.SAF_EINVAL
        assert call(lib, Hkv=3) == saf.SAF_EINVAL
        assert call(lib, d=80) == saf.SAF_EUNSUPPORTED
        assert call(lib, state=F + 16) == saf.SAF_EALIGN
        assert call(lib, wsb=64) == saf.SAF_EWORKSPACE
        assert call(lib, T=0) == saf.SAF_OK
        assert call(lib, H=512, Hkv=512) == saf.SAF_EINVAL
    assert _fwd_window(lib, frozen=fz, ld=255) == saf.SAF_EINVAL
    assert _fwd_window(lib, frozen=fz, a=None) == saf.SAF_EINVAL
    assert _fwd_window(lib, o=None) == saf.SAF_EINVAL
    assert _fwd_window(lib, q=F + 2) == saf.SAF_EALIGN
    assert _bwd_window(lib, dq=None) == saf.SAF_EINVAL
    assert _bwd_window(lib, dv=F + 8) == saf.SAF_EALIGN


def _paged(lib, shared=False, **kw):
    x = dict(q=F, k=F, v=F, pp=F, P=100, table=F, mp=8, ctx=F, new=None, a=F, r=F, ld=1000, frozen=None, window=0,
             sinks=0, B=2, H=4, Hkv=2, T=1, d=64, ml=512, np=64, ps=64, dt=0, o=F, lse=F, ws=F, wsb=1 << 30)
    x.update(kw)
    fn = lib.saf_attn_paged_shared if shared else lib.saf_attn_paged
    mid = (x["pp"], x["P"]) if shared else ()
    return fn(x["q"], x["k"], x["v"], *mid, x["table"], x["mp"], x["ctx"], x["new"], x["a"], x["r"], x["ld"],
              x["frozen"], x["window"], x["sinks"], x["B"], x["H"], x["Hkv"], x["T"], x["d"], x["ml"], x["np"], x["ps"],
              x["dt"], x["o"], x["lse"], x["ws"], x["wsb"], None)


@pytest.mark.parametrize("shared", [False, True])
def test_paged_refusals(saf, shared):
    lib = saf.library()
    bad = lambda **kw: _paged(lib, shared, **kw)   # noqa: E731
    for kw in (dict(B=-1), dict(H=0), dict(Hkv=3), dict(H=300, Hkv=300), dict(T=-1), dict(dt=3), dict(ml=0),
               dict(ml=513), dict(window=-1), dict(sinks=-2), dict(np=0), dict(mp=0), dict(ps=4), dict(ps=24),
               dict(ps=2048), dict(v=None), dict(q=None), dict(k=None), dict(table=None), dict(ctx=None), dict(o=None),
               dict(lse=None), dict(np=2 ** 30, Hkv=4), dict(B=2 ** 20, T=2 ** 10)):
        assert bad(**kw) == saf.SAF_EINVAL, kw
    assert bad(d=80) == saf.SAF_EUNSUPPORTED
    fz = bytes([0, 0, 1, 0])
    assert bad(frozen=fz, a=None) == saf.SAF_EINVAL
    assert bad(frozen=fz, ld=511) == saf.SAF_EINVAL
    if shared:
        assert bad(frozen=fz, ld=611) == saf.SAF_EINVAL
        assert bad(pp=None) == saf.SAF_EINVAL
        assert bad(P=-1) == saf.SAF_EINVAL
        assert bad(P=2 ** 30) == saf.SAF_EINVAL
    for kw in (dict(q=F + 8), dict(k=F + 4), dict(v=F + 2), dict(o=F + 8), dict(lse=F + 2), dict(table=F + 1),
               dict(ctx=F + 2), dict(new=F + 3), dict(ws=F + 64)):
        assert bad(**kw) == saf.SAF_EALIGN, kw
    assert bad(ws=None) == saf.SAF_EWORKSPACE
    need = lib.saf_attn_paged_workspace_bytes(2, 4, 2, 1, 64, 512, 100 if shared else 0, 0)
    assert need > 256 and bad(wsb=need - 1) == saf.SAF_EWORKSPACE
    assert bad(T=0, q=None, v=None, ws=None) == saf.SAF_OK
    assert bad(B=0, q=None, v=None, ws=None) == saf.SAF_OK


def test_paged_workspace_bytes(saf):
    f = saf.saf_attn_paged_workspace_bytes
    assert f(2, 4, 2, 1, 64, 128, "bf16") % 256 == 0
    assert f(1, 4, 2, 1, 64, 16, "bf16") == 256            # one item per row: nothing to join
    assert f(0, 4, 2, 1, 64, 16, "bf16") == 256
    for wrong in ((2, 4, 3, 1, 64, 128), (2, 4, 2, 1, 80, 128), (2, 4, 2, 1, 64, 0), (2, 0, 1, 1, 64, 128)):
        assert f(*wrong, "bf16") == 0, wrong
    # a long cache of one sequence is split; more sequences share the same number of items
    assert f(1, 8, 8, 1, 128, 1 << 20, "bf16") > f(1, 8, 8, 1, 128, 1 << 10, "bf16")


def _append(lib, **kw):
    x = dict(q=F, k=F, v=F, st=None, ctx=F, new=None, table=F, mp=8, freq=(ctypes.c_double * 32)(*[1.0] * 32), rope=64,
             inter=0, base=0, frozen=None, B=2, H=4, Hkv=2, T=1, d=64, np=64, ps=16, dt=0, qo=F + 0x1000, kc=F, vc=F,
             status=F)
    x.update(kw)
    return lib.saf_kv_append(x["q"], x["k"], x["v"], x["st"], x["ctx"], x["new"], x["table"], x["mp"], x["freq"],
                             x["rope"], x["inter"], x["base"], x["frozen"], x["B"], x["H"], x["Hkv"], x["T"], x["d"],
                             x["np"], x["ps"], x["dt"], x["qo"], x["kc"], x["vc"], x["status"], None)


def test_append_refusals(saf):
    lib = saf.library()
    inf = (ctypes.c_double * 32)(*[float("inf")] * 32)
    nan = (ctypes.c_double * 32)(*[float("nan")] * 32)
    for kw in (dict(B=-1), dict(Hkv=3), dict(H=300, Hkv=300), dict(dt=9), dict(rope=8), dict(rope=80), dict(rope=-16),
               dict(freq=None), dict(freq=inf), dict(freq=nan), dict(inter=2), dict(base=-1), dict(ps=12), dict(ps=4),
               dict(np=0), dict(mp=0), dict(v=None), dict(vc=None), dict(k=None), dict(kc=None), dict(qo=None),
               dict(ctx=None), dict(table=None), dict(B=2 ** 20, T=2 ** 11),
               dict(T=2 ** 21 + 1)):
        assert _append(lib, **kw) == saf.SAF_EINVAL, kw
    assert _append(lib, d=72) == saf.SAF_EUNSUPPORTED
    odd = (ctypes.c_int64 * 9)(512, 128, 64, 256, 68, 64, 256, 128, 64)
    for kw in (dict(q=F + 4), dict(k=F + 8), dict(v=F + 2), dict(qo=F + 8), dict(kc=F + 8), dict(vc=F + 8),
               dict(ctx=F + 2), dict(new=F + 2), dict(table=F + 2), dict(status=F + 2), dict(st=odd)):
        assert _append(lib, **kw) == saf.SAF_EALIGN, kw
    # q_out = q needs q laid out as q_out
    turned = (ctypes.c_int64 * 9)(256, 64, 256, 128, 64, 128, 128, 64, 128)
    assert _append(lib, qo=F, T=2, st=turned) == saf.SAF_EINVAL
    assert _append(lib, B=0, q=None, k=None, v=None) == saf.SAF_OK


def test_append_takes_positions_whose_angles_keep_their_digits(saf):
    lib = saf.library()
    assert _append(lib, base=2 ** 40, B=0) == saf.SAF_OK
    assert _append(lib, base=2 ** 40 + 1, B=0) == saf.SAF_EINVAL


def test_binding_refusals_without_a_device(saf):
    x = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        saf.saf_attn_paged(x, x, x, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 1)
    with pytest.raises(ValueError):
        saf.saf_attn_fwd_window(x, x, x, None, None, None, 1)
    with pytest.raises(ValueError):
        saf.saf_kv_append(x, x, x, x, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_binding_refuses_numbers_past_a_c_integer(saf):
    # cut to 32 bits, a window of 2^32 + 5 would be one of 5
    x = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    table, ctx = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    big = 2 ** 32 + 5
    for n in ("window", "sinks"):
        kw = {"window": 1, n: big}
        with pytest.raises(ValueError, match=n):
            saf.saf_attn_fwd_window(x, x, x, None, None, None, **kw)
        with pytest.raises(ValueError, match=n):
            saf.saf_attn_bwd_window(x, x, x, x, x, x, None, None, None, **kw)
        with pytest.raises(ValueError, match=n):
            saf.saf_attn_paged(x, x, x, table, ctx, 1, **kw)
    with pytest.raises(ValueError, match="max_len"):
        saf.saf_attn_paged(x, x, x, table, ctx, big)
    with pytest.raises(ValueError, match="prefix_len"):
        saf.saf_attn_paged_shared(x, x, x, None, big, table, ctx, 1)
    with pytest.raises(ValueError, match="pos_base"):
        saf.saf_kv_append(x, x, x, x, table, ctx, pos_base=2 ** 64 + 1)
    assert saf.saf_attn_paged_workspace_bytes(2, 4, 2, 1, 64, big, "bf16") == 0
    assert saf.saf_attn_paged_workspace_bytes(2, 4, 2, 1, 64, 128, "bf16", prefix_len=big) == 0
