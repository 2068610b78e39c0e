"""The cases by which the serving and windowed-attention operators are measured.

Four operators of the hybrid attention layer (ordinary and frozen heads):

  window   sliding-window attention with sinks, forward and backward. Query i of an
           ordinary head sees the keys j <= i with i - j < window or j < sinks
           (window 0: every j <= i); frozen heads keep their whole pattern.
  append   keys and values of new tokens written into a paged cache, with the rotary
           position rotation applied to k (and to q) on the way.
  paged    attention of the newest tokens of each sequence over its paged cache, with
           the window, the sinks and the frozen heads' patterns.
  shared   the same for a batch whose sequences share one long prefix.

`run` computes a case in its plain form (torch, 32 bits) or, with `own` set, through
the library's entry points; `exact` gives the outputs in 64 bits from the definition.
Layouts: q, o [B, H, T, d]; k, v [B, Hkv, T, d]; caches [pages, Hkv, page, d].
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
ROPE_BASE = 10000.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _window(name, B, H, Hkv, F, T, d, dtype, window, sinks, backward):
    return {"name": name, "op": "window", "B": B, "H": H, "Hkv": Hkv, "F": F, "T": T, "d": d, "dtype": dtype,
            "window": window, "sinks": sinks, "backward": backward}


def _append(name, B, H, Hkv, F, T, d, dtype, page, max_len, rope, interleaved):
    return {"name": name, "op": "append", "B": B, "H": H, "Hkv": Hkv, "F": F, "T": T, "d": d, "dtype": dtype,
            "page": page, "max_len": max_len, "rope": rope, "interleaved": interleaved}


def _paged(name, B, H, Hkv, F, T, d, dtype, page, max_len, window, sinks, prefix=0):
    return {"name": name, "op": "shared" if prefix else "paged", "B": B, "H": H, "Hkv": Hkv, "F": F, "T": T, "d": d,
            "dtype": dtype, "page": page, "max_len": max_len, "window": window, "sinks": sinks, "prefix": prefix}


def listed():
    return [
        # a training step of a 124M layer whose nine ordinary heads see 1024 tokens
        _window("window_train_gpt2", 8, 12, 12, 3, 4096, 64, "bf16", 1024, 4, True),
        # a training step of a grouped-query layer, 32 query heads over 8, head dimension 128
        _window("window_train_gqa_d128", 2, 32, 8, 8, 4096, 128, "bf16", 512, 16, True),
        # the prompt of one long sequence: forward only
        _window("window_prefill_16k", 1, 12, 12, 3, 16384, 64, "bf16", 2048, 4, False),
        # the smallest training step, in 32 bits, at a ragged length
        _window("window_train_tiny_fp32", 1, 4, 4, 1, 250, 64, "fp32", 100, 3, True),
        # one decoding step of 32 sequences: one new token each
        _append("append_step", 32, 32, 8, 8, 1, 128, "bf16", 64, 8192, 128, False),
        # the prompts of eight sequences, padded to the longest
        _append("append_prompts", 8, 12, 12, 3, 4096, 64, "bf16", 128, 4096, 64, True),
        # one token of one sequence: latency counts
        _paged("decode_one", 1, 12, 12, 3, 1, 64, "bf16", 64, 4096, 0, 0),
        # a batch of 32 sequences of 4K to 16K tokens
        _paged("decode_batch", 32, 32, 8, 8, 1, 128, "bf16", 64, 16384, 0, 0),
        # a batch of 64 sequences whose heads see the last 1024 tokens and four sinks
        _paged("decode_window", 64, 32, 8, 0, 1, 128, "bf16", 128, 16384, 1024, 4),
        # five drafted tokens of each of four sequences, in 32 bits
        _paged("draft_fp32_d96", 4, 16, 16, 4, 5, 96, "fp32", 16, 2000, 0, 0),
        # eight sequences after a 4K system prompt
        _paged("shared_small", 8, 12, 12, 3, 1, 64, "bf16", 64, 256, 0, 0, 4096),
        # 64 sequences after a 32K document
        _paged("shared_large", 64, 32, 8, 8, 1, 128, "bf16", 128, 1024, 0, 0, 32768),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    H, Hkv = rng.choice([(1, 1), (4, 4), (6, 2), (8, 1), (12, 12), (16, 4), (16, 16), (32, 8), (32, 32)])
    return H, Hkv, rng.choice([0, 1, H // 4, H // 2, H]) if H > 1 else rng.choice([0, 1])


def _cost(c):
    w = work(c)
    return w["flops"] / 1e15 + w["bytes"] / 6e12


def _draw_one(rng, op):
    H, Hkv, F = _heads(rng)
    d = rng.choice([64, 64, 96, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "window":
        T = _log_int(rng, 1, 1024 if dtype == "fp32" else 8192)
        window = rng.choice([_log_int(rng, 1, 2 * T), _log_int(rng, 1, 512)])
        return _window("", rng.choice([1, 2, 3, 8]), H, Hkv, F, T, d, dtype, window,
                       rng.choice([0, 1, 4, 16, 130]), rng.random() < 0.6)
    page = rng.choice([16, 32, 64, 128, 256])
    B = _log_int(rng, 1, 64)
    if op == "append":
        T = _log_int(rng, 1, 4096)
        return _append("", B, H, Hkv, F, T, d, dtype, page, T + _log_int(rng, 1, 8192), rng.choice([d, d // 2, 16]),
                       rng.random() < 0.5)
    T = rng.choice([1, 1, 1, rng.randint(2, 8), _log_int(rng, 1, 64)])
    window, sinks = rng.choice([(0, 0), (0, 0), (_log_int(rng, 1, 4096), rng.choice([0, 1, 4, 64]))])
    if op == "paged":
        return _paged("", B, H, Hkv, F, T, d, dtype, page, T + _log_int(rng, 1, 16384), window, sinks)
    return _paged("", B, H, Hkv, F, T, d, dtype, page, T + _log_int(rng, 1, 1024), window, sinks,
                  _log_int(rng, 1, 32768))


def draw(rng):
    op = rng.choice(["window", "append", "paged", "shared"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        c = _draw_one(rng, op)
        # fp32 runs on the CUDA cores: those cases stay a fifth as large
        if _cost(c) <= most * (0.2 if c["dtype"] == "fp32" else 1.0) and _elements(c) < 3e9:
            del c["name"]
            return c


def _elements(c):
    """Elements of the largest tensor of the plain form."""
    if c["op"] == "window":
        return c["B"] * c["H"] * c["T"] ** 2
    if c["op"] == "append":
        return c["B"] * c["H"] * c["T"] * c["d"]
    return max(c["B"] * c["Hkv"] * c["max_len"] * c["d"], c["Hkv"] * c["prefix"] * c["d"],
               c["B"] * c["H"] * c["T"] * (c["prefix"] + c["max_len"]))


def _frozen(c):
    """F of the H heads are frozen, evenly spaced, the last one among them."""
    return [(h + 1) * c["F"] // c["H"] > h * c["F"] // c["H"] for h in range(c["H"])]


def _live_kv(c):
    """Key/value heads that an ordinary query head reads: the others need no keys."""
    G, fz = c["H"] // c["Hkv"], _frozen(c)
    return [not all(fz[hk * G:(hk + 1) * G]) for hk in range(c["Hkv"])]


def _tokens(c):
    """(tokens before, new tokens) of each sequence: between a quarter and all of max_len
    together, one of the batch at max_len; of several new tokens some sequences bring
    fewer, one in ten none."""
    ctx, new = [], []
    for b in range(c["B"]):
        total = max(1, c["max_len"] * (c["B"] + 3 * (b + 1)) // (4 * c["B"]))
        n = min(c["T"], total)
        if c["T"] > 1 and b + 1 < c["B"]:
            n = min(n, c["T"] * (b % 10) // 9)
        ctx.append(total - n)
        new.append(n)
    return ctx, new


def _seen(i0, n, window, sinks):
    """Visible (query, key) pairs of the queries at i0 .. i0 + n - 1, and the keys that one of them sees."""
    if n == 0:
        return 0, 0
    if window == 0:
        return sum(range(i0 + 1, i0 + n + 1)), i0 + n
    pairs = sum(min(i + 1, window + min(sinks, max(0, i + 1 - window))) for i in range(i0, i0 + n))
    lo = max(0, i0 - window + 1)
    return pairs, i0 + n - lo + min(sinks, lo)


def work(case):
    c = case
    B, H, Hkv, T, d = (c[n] for n in ("B", "H", "Hkv", "T", "d"))
    e = 2 if c["dtype"] == "bf16" else 4
    G, fz, live = H // Hkv, _frozen(c), _live_kv(c)
    F = sum(fz)
    if c["op"] == "window":
        ordinary = _seen(0, T, c["window"], c["sinks"])[0]
        causal = T * (T + 1) // 2
        contractions = (7, 2) if c["backward"] else (2, 1)
        flops = 2 * d * B * ((H - F) * contractions[0] * ordinary + F * contractions[1] * causal)
        row = B * T * d * e
        moved = row * (H - F + sum(live) + Hkv + H) + B * H * T * 4 + F * T * 8    # q, k, v, o; lse; a, r
        if c["backward"]:
            moved += row * (H + H + 2 * Hkv)                                      # dO; dq, dk, dv
        return {"bytes": moved, "flops": flops}
    ctx, new = _tokens(c)
    if c["op"] == "append":
        tokens = sum(new)
        rotated = H - F + sum(live)
        return {"bytes": tokens * 2 * d * e * (rotated + Hkv) + B * 8 + 4 * sum(-(-n // c["page"]) for n in new),
                "flops": tokens * rotated * c["rope"] * 3}
    # frozen heads see every earlier key, ordinary ones those of the window
    P = c["prefix"]
    flops = keys_k = keys_v = 0
    first_k, first_v = P, P
    for x, n in zip(ctx, new):
        pairs, k = _seen(P + x, n, c["window"], c["sinks"])
        causal = _seen(P + x, n, 0, 0)[0]
        flops += 2 * d * ((H - F) * 2 * pairs + F * causal)
        if P:   # own keys; the prefix is counted once, below
            lo = 0 if c["window"] == 0 else max(0, x - c["window"] + 1)
            k = (x + n - lo if n else 0) + min(lo, max(0, c["sinks"] - P))
            if n:
                lo = max(0, P + x - c["window"] + 1) if c["window"] else 0
                first_k = min(first_k, max(0, lo - min(lo, c["sinks"])))
                first_v = 0
        keys_k += k
        keys_v += x + n if n else 0
    if P:
        keys_k += P - first_k
        keys_v += P - first_v
    v_all = sum(any(fz[hk * G:(hk + 1) * G]) for hk in range(Hkv))   # groups that read every value
    moved = d * e * (sum(live) * keys_k + v_all * keys_v + (Hkv - v_all) * keys_k)
    moved += sum(new) * d * e * (H - F) + B * T * H * (d * e + 4)
    return {"bytes": moved + F * 8 * (P + c["max_len"]), "flops": flops}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    dt = DTYPES[c["dtype"]]
    B, H, Hkv, T, d = (c[n] for n in ("B", "H", "Hkv", "T", "d"))

    def normal(*shape, scale=0.5):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

    def prior(L):   # per head: key preference ~ N(0, 1), distance preference with a recency slope
        a = torch.randn(H, L, generator=g, device="cuda")
        r = 0.5 * torch.randn(H, L, generator=g, device="cuda")
        return a, r - min(0.05, 80.0 / L) * torch.arange(L, device="cuda")

    s = {"case": c, "frozen": bytes(_frozen(c)), "frz": torch.tensor(_frozen(c), device="cuda")}
    if c["op"] == "window":
        s.update(q=normal(B, H, T, d), k=normal(B, Hkv, T, d), v=normal(B, Hkv, T, d), do=normal(B, H, T, d))
        s["a"], s["r"] = prior(T)
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, H, T, device="cuda")
        s["dq"], s["dk"], s["dv"] = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
        s["workspace"] = {}
        return s

    ps = c["page"]
    ctx, new = _tokens(c)
    order = torch.randperm(B, generator=g, device="cuda")
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")[order].contiguous()
    s["n_new"] = torch.tensor(new, dtype=torch.int32, device="cuda")[order].contiguous()
    per_seq = -(-c["max_len"] // ps)
    own_pages = B * per_seq
    prefix_pages = -(-c.get("prefix", 0) // ps)
    total = own_pages + prefix_pages
    pages = torch.randperm(total, generator=g, device="cuda").int()
    table = pages[:own_pages].reshape(B, per_seq)
    # a sequence holds pages for its own tokens only
    used = -(-(s["ctx"] + s["n_new"]) // ps)
    s["table"] = torch.where(torch.arange(per_seq, device="cuda")[None, :] < used[:, None], table, -1).int()
    s["k_cache"], s["v_cache"] = normal(total, Hkv, ps, d), normal(total, Hkv, ps, d)
    if c["op"] == "append":
        # one projection's output, token by token: the query heads, then the key and the value heads
        qkv = normal(B, T, H + 2 * Hkv, d).transpose(1, 2)
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        s["q_out"] = torch.zeros(B, H, T, d, dtype=dt, device="cuda")
        s["inv_freq"] = ROPE_BASE ** (-torch.arange(0, c["rope"], 2, dtype=torch.float64) / c["rope"])
        s["live"] = torch.tensor(_live_kv(c), device="cuda")
        return s
    s["q"] = normal(B, H, T, d)
    s["prefix_pages"] = pages[own_pages:].contiguous()
    s["a"], s["r"] = prior(c["prefix"] + c["max_len"])
    s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, H, T, device="cuda")
    s["workspace"] = {}
    return s


# ---------------------------------------------------------------------------
# Plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _plain_scores(s, q, k, i, j):
    """Logits [B, H, T, L] of queries at positions i [B or 1, T] and keys at positions j [L]
    (scaled products, or the pattern of frozen heads; -inf where a query does not see a key).
    q: [B, H, T, d] fp32; k: [B or 1, H, L, d] fp32."""
    c = s["case"]
    S = (q @ k.transpose(-1, -2)) / math.sqrt(c["d"])
    gap = i[:, None, :, None] - j
    if c["F"]:
        a, r = s["a"][s["frz"]], s["r"][s["frz"]]
        pattern = a[None, :, None, j] + r[:, gap[:, 0].clamp(min=0)].transpose(0, 1)
        S[:, s["frz"]] = pattern.expand(S.shape[0], -1, -1, -1)
    seen = gap >= 0
    if c["window"]:
        near = seen & ((gap < c["window"]) | (j < c["sinks"]))
        seen = torch.where(s["frz"][None, :, None, None], seen, near)
    return S.masked_fill_(~seen, -math.inf)


def _softmax(S):
    """Row softmax and log-sum-exp; a row that sees nothing has weights 0 and log-sum-exp -inf."""
    m = S.amax(-1, keepdim=True)
    e = torch.exp(S - m.clamp(min=-1e30))
    z = e.sum(-1, keepdim=True)
    return e / z.clamp(min=1e-37), (m + torch.log(z)).squeeze(-1)


def _plain_window(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    G = c["H"] // c["Hkv"]
    q = s["q"].float()
    k, v = (s[n].float().repeat_interleave(G, 1) for n in ("k", "v"))
    j = torch.arange(c["T"], device="cuda")
    P, lse = _softmax(_plain_scores(s, q, k, j[None], j))
    o = P @ v
    if not c["backward"]:
        return [o.to(dt), lse]
    do = s["do"].float()
    dv = P.transpose(-1, -2) @ do
    dS = P * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
    dS[:, s["frz"]] = 0
    dS /= math.sqrt(c["d"])
    dq, dk = dS @ k, dS.transpose(-1, -2) @ q
    dk, dv = (x.unflatten(1, (c["Hkv"], G)).sum(2) for x in (dk, dv))
    return [o.to(dt), lse, dq.to(dt), dk.to(dt), dv.to(dt)]


def _rotate(x, cos, sin, interleaved):
    """x [B, heads, T, d]: the first 2 * cos.shape[-1] elements of each row rotated by the angles [B, T, .]."""
    n = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    x = x.float()
    if interleaved:
        x0, x1 = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2)
    else:
        x0, x1 = x[..., :n], x[..., n:2 * n]
        y = torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _plain_append(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    t = torch.arange(c["T"], device="cuda")
    pos = s["ctx"].long()[:, None] + t
    valid = t < s["n_new"][:, None]
    angle = pos.double()[..., None] * s["inv_freq"].cuda()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotate(s["q"], cos, sin, c["interleaved"]).to(dt)
    k = _rotate(s["k"], cos, sin, c["interleaved"]).to(dt)
    q_keep = valid[:, None, :, None] & ~s["frz"][None, :, None, None]
    s["q_out"].copy_(torch.where(q_keep, q, s["q_out"]))
    slot = pos.clamp(max=s["table"].shape[1] * c["page"] - 1)
    page = s["table"].gather(1, slot // c["page"])[valid].long()
    slot = (slot % c["page"])[valid]
    s["v_cache"][page, :, slot] = s["v"].transpose(1, 2)[valid]
    kept = s["k_cache"][page, :, slot]
    s["k_cache"][page, :, slot] = torch.where(s["live"][None, :, None], k.transpose(1, 2)[valid], kept)
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _gather(cache, table, L, G):
    """[B, H, L, d] fp32 from a paged cache and a page table [B, pages]."""
    x = cache[table.clamp(min=0).long()].transpose(1, 2).flatten(2, 3)[:, :, :L]
    return x.float().repeat_interleave(G, 1)


def _plain_paged(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    G, P, L = c["H"] // c["Hkv"], c["prefix"], c["max_len"]
    q = s["q"].float()
    t = torch.arange(c["T"], device="cuda")
    i = P + s["ctx"].long()[:, None] + t
    i = torch.where(t < s["n_new"][:, None], i, -1)     # rows past the new tokens see nothing
    j = torch.arange(P + L, device="cuda")
    S = _plain_scores(s, q, _gather(s["k_cache"], s["table"], L, G), i, j[P:])
    v = _gather(s["v_cache"], s["table"], L, G)
    if not P:
        W, lse = _softmax(S)
        return [(W @ v).to(dt), lse]
    kp, vp = (_gather(s[n], s["prefix_pages"][None], P, G) for n in ("k_cache", "v_cache"))
    W, lse = _softmax(torch.cat([_plain_scores(s, q, kp, i, j[:P]), S], -1))
    # one product per head with the shared values for all sequences
    op = (W[..., :P].permute(1, 0, 2, 3).flatten(1, 2) @ vp[0]).unflatten(1, (c["B"], c["T"])).transpose(0, 1)
    return [(op + W[..., P:] @ v).to(dt), lse]


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    s = state
    c = s["case"]
    if not own:
        if c["op"] == "window":
            return _plain_window(s)
        return _plain_append(s) if c["op"] == "append" else _plain_paged(s)
    return _own(s)


def _own(s):
    from softmax_attention_hybrid_gb300 import saf

    c = s["case"]
    fz = s["frozen"] if c["F"] else None
    if c["op"] == "append":
        saf.saf_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["n_new"], q=s["q"],
                          q_out=s["q_out"], inv_freq=s["inv_freq"], interleaved=c["interleaved"], frozen=fz)
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    ws = s["workspace"]
    B, H, Hkv, T, d = (c[n] for n in ("B", "H", "Hkv", "T", "d"))
    if c["op"] == "window":
        if not ws:
            ws["fwd"] = saf.alloc_workspace(B, H, T, d, s["q"].dtype, False)
            ws["bwd"] = saf.alloc_workspace(B, H, T, d, s["q"].dtype, True) if c["backward"] else None
        o, lse = saf.saf_attn_fwd_window(s["q"], s["k"], s["v"], s["a"], s["r"], fz, c["window"], c["sinks"],
                                         o=s["o"], lse=s["lse"], workspace=ws["fwd"])
        if not c["backward"]:
            return [o, lse]
        dq, dk, dv = saf.saf_attn_bwd_window(s["q"], s["k"], s["v"], o, s["do"], lse, s["a"], s["r"], fz, c["window"],
                                             c["sinks"], dq=s["dq"], dk=s["dk"], dv=s["dv"], workspace=ws["bwd"])
        return [o, lse, dq, dk, dv]
    if not ws:
        ws["w"] = saf.alloc_paged_workspace(B, H, Hkv, T, d, c["max_len"], s["q"].dtype, prefix_len=c["prefix"])
    if c["op"] == "paged":
        o, lse = saf.saf_attn_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], c["max_len"],
                                    n_new=s["n_new"], a=s["a"], r=s["r"], frozen=fz, window=c["window"],
                                    sinks=c["sinks"], o=s["o"], lse=s["lse"], workspace=ws["w"])
    else:
        o, lse = saf.saf_attn_paged_shared(s["q"], s["k_cache"], s["v_cache"], s["prefix_pages"], c["prefix"],
                                           s["table"], s["ctx"], c["max_len"], n_new=s["n_new"], a=s["a"], r=s["r"],
                                           frozen=fz, window=c["window"], sinks=c["sinks"], o=s["o"], lse=s["lse"],
                                           workspace=ws["w"])
    return [o, lse]


# ---------------------------------------------------------------------------
# From the definition, in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(c, fz, h, q, keys, i, a, r):
    """Weights and log-sum-exp of head h: queries q [n, d] at positions i [n], keys [m, d] at 0 .. m - 1."""
    gap = i[:, None] - torch.arange(keys.shape[0], device="cuda")[None, :]
    hidden = gap < 0
    if fz[h]:
        logits = a[h, :keys.shape[0]].double()[None, :] + r[h].double()[gap.clamp(min=0)]
    else:
        logits = q.double() @ keys.double().t() * c["d"] ** -0.5
        if c["window"]:
            far = gap >= c["window"]
            far[:, :c["sinks"]] = False
            hidden = hidden | far
    logits = torch.where(hidden, -math.inf, logits)
    lse = torch.logsumexp(logits, -1)
    return torch.exp(logits - lse[:, None]).nan_to_num(0.0), lse


def exact(case, seed):
    c, s = case, prepare(case, seed)
    fz, G = _frozen(c), c["H"] // c["Hkv"]
    if c["op"] == "append":
        return _exact_append(c, s, fz)
    o = torch.zeros(c["B"], c["H"], c["T"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["H"], c["T"]), -math.inf, dtype=torch.float64, device="cuda")
    if c["op"] == "window":
        dq = torch.zeros_like(o)
        dk, dv = (torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
        i = torch.arange(c["T"], device="cuda")
        for b in range(c["B"]):
            for h in range(c["H"]):
                k, v, do = s["k"][b, h // G].double(), s["v"][b, h // G].double(), s["do"][b, h].double()
                W, lse[b, h] = _exact_rows(c, fz, h, s["q"][b, h], k, i, s["a"], s["r"])
                o[b, h] = W @ v
                if c["backward"]:
                    dv[b, h // G] += W.t() @ do
                    if not fz[h]:
                        dS = W * (do @ v.t() - (do * o[b, h]).sum(-1, keepdim=True)) * c["d"] ** -0.5
                        dq[b, h] = dS @ k
                        dk[b, h // G] += dS.t() @ s["q"][b, h].double()
        return [o, lse, dq, dk, dv] if c["backward"] else [o, lse]
    P, ps = c["prefix"], c["page"]
    ctx, new = s["ctx"].tolist(), s["n_new"].tolist()
    for b in range(c["B"]):
        n, L = new[b], ctx[b] + new[b]
        if n == 0:
            continue
        at = torch.arange(L, device="cuda")
        page, slot = s["table"][b][at // ps].long(), at % ps
        if P:
            head = torch.arange(P, device="cuda")
            page = torch.cat([s["prefix_pages"][head // ps].long(), page])
            slot = torch.cat([head % ps, slot])
        i = P + ctx[b] + torch.arange(n, device="cuda")
        for hk in range(c["Hkv"]):
            k, v = s["k_cache"][page, hk, slot].double(), s["v_cache"][page, hk, slot].double()
            for h in range(hk * G, hk * G + G):
                W, lse[b, h, :n] = _exact_rows(c, fz, h, s["q"][b, h, :n], k, i, s["a"], s["r"])
                o[b, h, :n] = W @ v
    return [o, lse]


def _exact_append(c, s, fz):
    """The caches and the rotated queries as complex rotations in 64 bits."""
    q_out, kc, vc = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
    ctx, new, n = s["ctx"].tolist(), s["n_new"].tolist(), c["rope"] // 2
    freq = ROPE_BASE ** (-2 * torch.arange(n, dtype=torch.float64, device="cuda") / c["rope"])
    live = _live_kv(c)
    heads = [h for h in range(c["H"]) if not fz[h]]
    kv_heads = [hk for hk in range(c["Hkv"]) if live[hk]]

    def turn(x, pos):   # x [heads, tokens, d]
        z = x[..., :2 * n].reshape(*x.shape[:-1], *((n, 2) if c["interleaved"] else (2, n)))
        z = z if c["interleaved"] else z.transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(freq), pos * freq))
        y = y if c["interleaved"] else y.transpose(-1, -2)
        return torch.cat([y.flatten(-2), x[..., 2 * n:]], -1)

    for b in range(c["B"]):
        m = new[b]
        if m == 0:
            continue
        at = ctx[b] + torch.arange(m, device="cuda")
        page, slot = s["table"][b][at // c["page"]].long(), at % c["page"]
        pos = at.double()[:, None]
        vc[page, :, slot] = s["v"][b, :, :m].double().transpose(0, 1)
        if heads:
            q_out[b, heads, :m] = turn(s["q"][b, heads, :m].double(), pos)
        for hk in kv_heads:
            kc[page, hk, slot] = turn(s["k"][b, hk:hk + 1, :m].double(), pos)[0]
    return [q_out, kc, vc]
