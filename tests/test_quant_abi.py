"""Refusals of the calls on 8-bit caches, before any device work, on the CPU."""
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


def _paged(lib, shared=False, **kw):
    x = dict(q=F, k=F, v=F, ks=F, vs=F, pp=F, P=100, table=F, mp=8, ctx=F, new=None, a=F, r=F, ld=1000, frozen=None,
             window=0, sinks=0, B=2, H=4, Hkv=2, T=1, d=64, ml=512, np=64, ps=64, dt=0, o=F, lse=F, ws=F, wsb=1 << 30)
    x.update(kw)
    fn = lib.saf_attn_paged_shared_quant if shared else lib.saf_attn_paged_quant
    mid = (x["pp"], x["P"]) if shared else ()
    return fn(x["q"], x["k"], x["v"], x["ks"], x["vs"], *mid, x["table"], x["mp"], x["ctx"], x["new"], x["a"], x["r"],
              x["ld"], x["frozen"], x["window"], x["sinks"], x["B"], x["H"], x["Hkv"], x["T"], x["d"], x["ml"],
              x["np"], x["ps"], x["dt"], x["o"], x["lse"], x["ws"], x["wsb"], None)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("dt", [0, 1])
def test_paged_refusals(saf, shared, dt):
    lib = saf.library()
    bad = lambda **kw: _paged(lib, shared, **{"dt": dt, **kw})   # noqa: E731
    for kw in (dict(B=-1), dict(H=0), dict(Hkv=3), dict(H=300, Hkv=300), dict(T=-1), dict(dt=3), dict(ml=0),
               dict(ml=513), dict(window=-1), dict(sinks=-2), dict(np=0), dict(mp=0), dict(ps=4), dict(ps=24),
               dict(ps=2048), dict(v=None), dict(q=None), dict(k=None), dict(ks=None), dict(vs=None),
               dict(table=None), dict(ctx=None), dict(o=None), dict(lse=None), dict(np=2 ** 30, Hkv=4),
               dict(B=2 ** 20, T=2 ** 10)):
        assert bad(**kw) == saf.SAF_EINVAL, kw
    assert bad(d=80) == saf.SAF_EUNSUPPORTED
    fz = bytes([0, 0, 1, 0])
    assert bad(frozen=fz, a=None) == saf.SAF_EINVAL
    assert bad(frozen=fz, ld=511) == saf.SAF_EINVAL
    assert bad(frozen=bytes([1] * 4), k=None, ks=None, wsb=16) == saf.SAF_EWORKSPACE   # no keys are needed
    assert bad(frozen=bytes([1] * 4), k=None, ks=None, vs=None) == saf.SAF_EINVAL
    for kw in (dict(q=F + 8), dict(k=F + 4), dict(v=F + 8), dict(ks=F + 4), dict(vs=F + 8), dict(o=F + 2),
               dict(lse=F + 2), dict(ctx=F + 1), dict(new=F + 2), dict(table=F + 2), dict(ws=F + 16)):
        assert bad(**kw) == saf.SAF_EALIGN, kw
    for kw in (dict(ws=None), dict(wsb=0), dict(wsb=255)):
        assert bad(**kw) == saf.SAF_EWORKSPACE, kw
    assert bad(B=0, q=None, v=None, vs=None) == saf.SAF_OK
    assert bad(T=0, ws=None) == saf.SAF_OK
    if shared:
        assert bad(pp=None) == saf.SAF_EINVAL
        assert bad(P=-1) == saf.SAF_EINVAL


def test_workspace_queries(saf):
    size = saf.saf_attn_paged_quant_workspace_bytes
    for dtype in ("bf16", "fp32"):
        for kw in (dict(B=-1), dict(H=0), dict(Hkv=3), dict(d=80), dict(max_len=0), dict(prefix_len=-1),
                   dict(max_len=2 ** 32 + 5), dict(T=-1)):
            x = {**dict(B=2, H=4, Hkv=2, T=1, d=64, max_len=128), **kw}
            assert size(**x, dtype=dtype) == 0, kw
        assert size(0, 4, 2, 1, 64, 128, dtype) == 256
        n = size(2, 4, 2, 1, 64, 10000, dtype)
        assert n > 256
        assert _paged(saf.library(), ml=10000, mp=200, dt=0 if dtype == "bf16" else 1, wsb=n - 1) == saf.SAF_EWORKSPACE


def _append(lib, **kw):
    x = dict(q=F, k=F, v=F, st=None, ctx=F, new=None, table=F, mp=4, freq=None, rope=0, inter=0, base=0, frozen=None,
             B=2, H=4, Hkv=2, T=2, d=64, np=16, ps=16, dt=0, qo=F + 0x1000, kc=F, vc=F, ks=F, vs=F, status=None)
    x.update(kw)
    return lib.saf_kv_append_quant(x["q"], x["k"], x["v"], x["st"], x["ctx"], x["new"], x["table"], x["mp"], x["freq"],
                                   x["rope"], x["inter"], x["base"], x["frozen"], x["B"], x["H"], x["Hkv"], x["T"],
                                   x["d"], x["np"], x["ps"], x["dt"], x["qo"], x["kc"], x["vc"], x["ks"], x["vs"],
                                   x["status"], None)


def test_append_refusals(saf):
    lib = saf.library()
    inf = (ctypes.c_double * 32)(*[float("inf")] * 32)
    for kw in (dict(B=-1), dict(Hkv=3), dict(H=300, Hkv=300), dict(dt=9), dict(rope=8), dict(rope=80),
               dict(rope=32), dict(rope=32, freq=inf), dict(inter=2), dict(base=-1), dict(ps=12), dict(ps=4),
               dict(np=0), dict(mp=0), dict(v=None), dict(vc=None), dict(k=None), dict(kc=None), dict(ks=None),
               dict(vs=None), dict(qo=None), dict(ctx=None), dict(table=None), dict(B=2 ** 20, T=2 ** 11)):
        assert _append(lib, **kw) == saf.SAF_EINVAL, kw
    assert _append(lib, d=72) == saf.SAF_EUNSUPPORTED
    for kw in (dict(q=F + 4), dict(k=F + 8), dict(v=F + 2), dict(qo=F + 8), dict(kc=F + 8), dict(vc=F + 8),
               dict(ks=F + 4), dict(vs=F + 8), dict(ctx=F + 2), dict(new=F + 2), dict(table=F + 2),
               dict(status=F + 2)):
        assert _append(lib, **kw) == saf.SAF_EALIGN, kw
    assert _append(lib, B=0, q=None, k=None, v=None, vs=None) == saf.SAF_OK


def _read(lib, **kw):
    x = dict(kc=F, vc=F, ks=F, vs=F, table=F, mp=4, first=None, count=None, B=2, Hkv=2, T=5, d=64, np=16, ps=16, dt=0,
             ko=F, vo=F, status=None)
    x.update(kw)
    return lib.saf_kv_read_quant(x["kc"], x["vc"], x["ks"], x["vs"], x["table"], x["mp"], x["first"], x["count"], x["B"],
                                 x["Hkv"], x["T"], x["d"], x["np"], x["ps"], x["dt"], x["ko"], x["vo"], x["status"],
                                 None)


def test_read_refusals(saf):
    lib = saf.library()
    for kw in (dict(B=-1), dict(Hkv=0), dict(Hkv=257), dict(T=-1), dict(dt=2), dict(ps=12), dict(ps=2048), dict(np=0),
               dict(mp=0), dict(vc=None), dict(vs=None), dict(vo=None), dict(table=None), dict(ks=None), dict(ko=None),
               dict(kc=None), dict(T=2 ** 21 + 1), dict(B=2 ** 10, T=2 ** 21)):
        assert _read(lib, **kw) == saf.SAF_EINVAL, kw
    assert _read(lib, d=80) == saf.SAF_EUNSUPPORTED
    for kw in (dict(kc=F + 8), dict(vc=F + 4), dict(ks=F + 4), dict(vs=F + 8), dict(ko=F + 8), dict(vo=F + 2),
               dict(table=F + 2), dict(first=F + 2), dict(count=F + 1), dict(status=F + 2)):
        assert _read(lib, **kw) == saf.SAF_EALIGN, kw
    assert _read(lib, B=0, vc=None) == saf.SAF_OK and _read(lib, T=0, vo=None) == saf.SAF_OK


def test_binding_refusals_without_a_device(saf):
    x = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    c = torch.zeros(1, 4, 8, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(1, 4, 8)
    table, ctx = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: saf.saf_attn_paged_quant(x, c, c, s, s, table, ctx, 1),
                 lambda: saf.saf_attn_paged_shared_quant(x, c, c, s, s, None, 0, table, ctx, 1),
                 lambda: saf.saf_kv_append_quant(x, x, c, c, s, s, table, ctx),
                 lambda: saf.saf_kv_read_quant(c, c, s, s, table, T=1, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    big = 2 ** 32 + 5
    with pytest.raises(ValueError, match="window"):
        saf.saf_attn_paged_quant(x, c, c, s, s, table, ctx, 1, window=big)
    with pytest.raises(ValueError, match="prefix_len"):
        saf.saf_attn_paged_shared_quant(x, c, c, s, s, None, big, table, ctx, 1)
    with pytest.raises(ValueError, match="pos_base"):
        saf.saf_kv_append_quant(x, x, c, c, s, s, table, ctx, pos_base=2 ** 64 + 1)
