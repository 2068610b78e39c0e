"""The README's serving examples, run as they stand."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _examples():
    text = open(os.path.join(ROOT, "README.md")).read()
    text = text[text.index("## Serving in short"):]
    return re.findall(r"```python\n(.*?)```", text[:text.index("\n## ", 5)], re.S)


@pytest.mark.parametrize("T", [1, 3])
def test_serving_examples(T):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from softmax_attention_hybrid_gb300 import saf
    plain, quant = _examples()
    B, H, Hkv, d, page, max_len = 2, 4, 2, 64, 16, 96
    g = torch.Generator().manual_seed(5)
    pages = B * max_len // page
    frozen = [0, 0, 0, 1]
    for code, eight in ((plain, False), (quant, True)):
        q, k, v = (torch.randn(B, n, T, d, generator=g).bfloat16().cuda() for n in (H, Hkv, Hkv))
        shape = (pages, Hkv, page, d)
        k_cache, v_cache = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) if eight
                            else torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k_scale, v_scale = (torch.ones(shape[:3], device="cuda") for _ in range(2))
        alloc = saf.alloc_paged_quant_workspace if eight else saf.alloc_paged_workspace
        ns = dict(saf=saf, q=q, k=k, v=v, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                  page_table=torch.randperm(pages, generator=g).int().reshape(B, -1).cuda(),
                  ctx=torch.tensor([20, 7], dtype=torch.int32, device="cuda"),
                  n_new=torch.full((B,), T, dtype=torch.int32, device="cuda"),
                  inv_freq=10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d), frozen=frozen,
                  a=torch.zeros(H, max_len, device="cuda"), r=torch.zeros(H, max_len, device="cuda"), max_len=max_len, T=T,
                  ws=alloc(B, H, Hkv, T, d, max_len, torch.bfloat16))
        exec(code, ns)
        assert ns["o"].shape == q.shape and torch.isfinite(ns["o"].float()).all()
        assert saf.saf_device_status(ns["ws"]) == saf.SAF_OK
        assert ns["ctx"].tolist() == [20 + T, 7 + T]
        if eight:   # every token up to the newest is read back
            for b, n in enumerate(ns["ctx"].tolist()):
                got = ns["vb"][b, :, n - T:n].double()
                want = v[b].double()
                step = 2.0 ** -4 * want.abs() + 2.0 ** -10 / 448 * want.abs().amax(-1, keepdim=True)
                assert ((got - want).abs() <= 1.01 * step + 2.0 ** -8 * want.abs()).all()
                assert not ns["vb"][b, :, n:].any()
