"""GPU: the backward calls with dq in the buffer of q or of dO, against the same calls with buffers
of their own.

dk and dv are sums in a fixed order: the same bits. dq at d = 96, 128 and in fp32 too; at d = 64 in
bf16 it adds key blocks' shares in fp32 in any order and rounds to bf16, one step apart. A windowed
call that may not use dq as scratch adds its blocks of sinks up in another order: it is compared
with the fp64 reference.
"""
import pytest
import torch

from tests.test_window_gpu import _check, _inputs

pytestmark = pytest.mark.gpu

KINDS = [("bf16", 64), ("bf16", 96), ("bf16", 128), ("fp32", 64), ("fp32", 96), ("fp32", 128)]


@pytest.fixture(scope="module")
def saf():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from softmax_attention_hybrid_gb300 import saf as mod
    return mod


def _same(got, want, dtype, d):
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    if dtype == "bf16" and d == 64:
        torch.testing.assert_close(got[0], want[0], rtol=2.0 ** -7, atol=1e-5)
    else:
        assert torch.equal(got[0], want[0])


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("over", ["q", "do"])
@pytest.mark.parametrize("B,H,Hkv,T,frozen", [(1, 2, 2, 65, ()), (1, 4, 4, 250, (1,)), (2, 4, 2, 300, (0, 2, 3)),
                                              (1, 4, 2, 200, (0, 1, 2, 3)), (2, 16, 4, 2000, (3, 7, 8, 9, 10, 11))])
def test_layer(saf, dtype, d, over, B, H, Hkv, T, frozen):
    flags = [h in frozen for h in range(H)]
    _, g = _inputs(dtype, B, H, Hkv, T, d, frozen, seed=T + d)
    o, lse = saf.saf_attn_fwd_gqa(g["q"], g["k"], g["v"], g["a"], g["r"], flags)
    state = saf.saf_frozen_prepare(g["a"], g["r"], flags, T, g["v"].dtype)
    calls = [lambda y, dq: saf.saf_attn_bwd_gqa(y["q"], y["k"], y["v"], o, y["do"], lse, y["a"], y["r"], flags, dq=dq),
             lambda y, dq: saf.saf_attn_bwd_prepared(y["q"], y["k"], y["v"], o, y["do"], lse, y["a"], y["r"], flags,
                                                     state, dq=dq)]
    if H == Hkv:
        calls.append(lambda y, dq: saf.saf_attn_bwd(y["q"], y["k"], y["v"], o, y["do"], lse, y["a"], y["r"], flags,
                                                    dq=dq))
    for call in calls:
        want = call(g, None)
        for _ in range(3):
            y = dict(g)
            y[over] = g[over].clone()
            got = call(y, y[over])
            assert got[0].data_ptr() == y[over].data_ptr()
            _same(got, want, dtype, d)


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("over", ["q", "do"])
@pytest.mark.parametrize("H,Hkv,T,window,sinks,frozen", [(4, 4, 250, 100, 3, (1,)), (8, 1, 1100, 100, 200, (2,)),
                                                         (4, 2, 700, 5, 0, ()), (4, 2, 300, 0, 0, (3,))])
def test_windowed(saf, dtype, d, over, H, Hkv, T, window, sinks, frozen):
    flags = [h in frozen for h in range(H)]
    x, g = _inputs(dtype, 1, H, Hkv, T, d, frozen, seed=T + d)
    o, lse = saf.saf_attn_fwd_window(g["q"], g["k"], g["v"], g["a"], g["r"], flags, window, sinks)
    y = dict(g)
    y[over] = g[over].clone()
    dq, dk, dv = saf.saf_attn_bwd_window(y["q"], y["k"], y["v"], o, y["do"], lse, y["a"], y["r"], flags, window, sinks,
                                         dq=y[over])
    _check(dtype, x, {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, flags, window, sinks)
