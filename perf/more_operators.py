"""The cases by which the operators of the 8-bit paged cache are measured.

A row (one token of one key/value head) of the cache is d values of float8 e4m3 and one
fp32 scale: y is held as  scale = max(max |y| / 448, 2^-126),  code = e4m3(y / scale).
Four operators:

  append   keys and values of new tokens quantised into the paged cache, with the rotary
           position rotation applied to k (and to q) before it.
  read     a range of each sequence's slots read back as rows of bf16 or fp32.
  paged    attention of the newest tokens of each sequence over its paged cache, with
           windows, sinks and the fixed patterns of frozen heads.
  shared   the same for a batch whose sequences share one long prefix.

`run` computes a case in its plain form (torch, 32 bits) or, with `own` set, through
the library's entry points; `exact` gives the outputs in 64 bits from the definition.
Layouts: q, o [B, H, T, d]; k, v [B, Hkv, T, d]; caches [pages, Hkv, page, d] with
scales [pages, Hkv, page].
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
ROPE_BASE = 10000.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _append(name, B, H, Hkv, F, T, d, dtype, page, max_len, rope, interleaved):
    return {"name": name, "op": "append", "B": B, "H": H, "Hkv": Hkv, "F": F, "T": T, "d": d, "dtype": dtype,
            "page": page, "max_len": max_len, "rope": rope, "interleaved": interleaved}


def _read(name, B, Hkv, T, d, dtype, page, max_len):
    return {"name": name, "op": "read", "B": B, "H": Hkv, "Hkv": Hkv, "F": 0, "T": T, "d": d, "dtype": dtype,
            "page": page, "max_len": max_len}


def _paged(name, B, H, Hkv, F, T, d, dtype, page, max_len, window, sinks, prefix=0):
    return {"name": name, "op": "shared" if prefix else "paged", "B": B, "H": H, "Hkv": Hkv, "F": F, "T": T, "d": d,
            "dtype": dtype, "page": page, "max_len": max_len, "window": window, "sinks": sinks, "prefix": prefix}


def listed():
    return [
        # one decoding step of 32 sequences: one new token each
        _append("append8_step", 32, 32, 8, 8, 1, 128, "bf16", 64, 8192, 128, False),
        # the prompts of eight sequences, padded to the longest
        _append("append8_prompts", 8, 12, 12, 3, 4096, 64, "bf16", 128, 4096, 64, True),
        # the last tokens of a few short sequences, in 32 bits
        _read("read8_tail_fp32", 3, 4, 250, 96, "fp32", 16, 1000),
        # whole contexts back as bf16, for the dense layer
        _read("read8_contexts", 4, 8, 16384, 128, "bf16", 64, 16384),
        # one token of one sequence: latency counts
        _paged("decode8_one", 1, 12, 12, 3, 1, 64, "bf16", 64, 4096, 0, 0),
        # a batch of 32 sequences of 4K to 16K tokens
        _paged("decode8_batch", 32, 32, 8, 8, 1, 128, "bf16", 64, 16384, 0, 0),
        # a batch of 64 sequences whose heads see the last 1024 tokens and four sinks
        _paged("decode8_window", 64, 32, 8, 0, 1, 128, "bf16", 128, 16384, 1024, 4),
        # five drafted tokens of each of four sequences, in 32 bits
        _paged("draft8_fp32_d96", 4, 16, 16, 4, 5, 96, "fp32", 16, 2000, 0, 0),
        # up to five drafted tokens of each of 16 sequences
        _paged("draft8_batch", 16, 32, 8, 8, 5, 128, "bf16", 64, 8192, 0, 0),
        # 512 more tokens of the prompts of four sequences
        _paged("chunk8_512", 4, 32, 8, 8, 512, 128, "bf16", 64, 8192, 0, 0),
        # eight sequences after a 4K system prompt
        _paged("shared8_small", 8, 12, 12, 3, 1, 64, "bf16", 64, 256, 0, 0, 4096),
        # 64 sequences after a 32K document
        _paged("shared8_large", 64, 32, 8, 8, 1, 128, "bf16", 128, 1024, 0, 0, 32768),
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
    page = rng.choice([16, 32, 64, 128, 256])
    B = _log_int(rng, 1, 64)
    if op == "append":
        T = _log_int(rng, 1, 4096)
        return _append("", B, H, Hkv, F, T, d, dtype, page, T + _log_int(rng, 1, 8192), rng.choice([d, d // 2, 16]),
                       rng.random() < 0.5)
    if op == "read":
        T = _log_int(rng, 1, 16384)
        return _read("", B, Hkv, T, d, dtype, page, T + _log_int(rng, 1, 4096))
    T = rng.choice([1, 1, 1, rng.randint(2, 8), _log_int(rng, 1, 600)])
    window, sinks = rng.choice([(0, 0), (0, 0), (_log_int(rng, 1, 4096), rng.choice([0, 1, 4, 64]))])
    if op == "paged":
        return _paged("", B, H, Hkv, F, T, d, dtype, page, T + _log_int(rng, 1, 16384), window, sinks)
    return _paged("", B, H, Hkv, F, T, d, dtype, page, T + _log_int(rng, 1, 1024), window, sinks,
                  _log_int(rng, 1, 32768))


def draw(rng):
    op = rng.choice(["append", "read", "paged", "paged", "shared"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        c = _draw_one(rng, op)
        # fp32 attention runs on the CUDA cores: those cases stay a fifth as large
        slow = c["dtype"] == "fp32" and op in ("paged", "shared")
        if _cost(c) <= most * (0.2 if slow else 1.0) and _elements(c) < 3e9:
            del c["name"]
            return c


def _elements(c):
    """Elements of the largest tensor of the plain form."""
    if c["op"] in ("append", "read"):
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
    together, one of the batch at max_len; of several new tokens sequences bring between
    half and all, one in ten none."""
    ctx, new = [], []
    for b in range(c["B"]):
        total = max(1, c["max_len"] * (c["B"] + 3 * (b + 1)) // (4 * c["B"]))
        n = min(c["T"], total)
        if c["T"] > 1 and b + 1 < c["B"]:
            n = 0 if b % 10 == 9 else n - n * (b % 5 + 1) // 10
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
    row = d + 4   # a row of the cache and its scale
    G, fz, live = H // Hkv, _frozen(c), _live_kv(c)
    F = sum(fz)
    ctx, new = _tokens(c)
    if c["op"] == "append":
        tokens = sum(new)
        moved = 2 * (H - F) * d * e + (sum(live) + Hkv) * (d * e + row)
        pages = sum(-(-n // c["page"]) for n in new)
        return {"bytes": tokens * moved + B * 8 + 4 * pages,
                "flops": tokens * ((H - F + sum(live)) * c["rope"] * 3 + (sum(live) + Hkv) * 2 * d)}
    if c["op"] == "read":
        tokens = sum(new)
        return {"bytes": 2 * Hkv * (tokens * row + B * T * d * e) + B * 8, "flops": 2 * Hkv * tokens * d}
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
    moved = row * (sum(live) * keys_k + v_all * keys_v + (Hkv - v_all) * keys_k)
    moved += sum(new) * d * e * (H - F) + B * T * H * (d * e + 4)
    return {"bytes": moved + F * 8 * (P + c["max_len"]), "flops": flops}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _quantise(y):
    """Codes and scales of the rows of y (fp32)."""
    scale = (y.abs().amax(-1) / 448.0).clamp(min=2.0 ** -126)
    return (y / scale[..., None]).to(E4M3), scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    dt = DTYPES[c["dtype"]]
    B, H, Hkv, T, d = (c[n] for n in ("B", "H", "Hkv", "T", "d"))

    def normal(*shape, scale=0.5):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

    ps = c["page"]
    s = {"case": c, "frozen": bytes(_frozen(c)), "frz": torch.tensor(_frozen(c), device="cuda")}
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
    # keys with a few channels larger than the others, values of rows of different size
    wide = 1.0 + 3.0 * (torch.arange(d, device="cuda") % 16 == 5)
    y = torch.randn(total, Hkv, ps, d, generator=g, device="cuda") * (0.4 * wide)
    s["k_cache"], s["k_scale"] = _quantise(y)
    y = torch.randn(total, Hkv, ps, d, generator=g, device="cuda", out=y)
    y *= 0.5 * torch.exp(0.3 * torch.randn(total, Hkv, ps, 1, generator=g, device="cuda"))
    s["v_cache"], s["v_scale"] = _quantise(y)
    if c["op"] == "append":
        # one projection's output, token by token: the query heads, then the key and the value heads
        qkv = normal(B, T, H + 2 * Hkv, d).transpose(1, 2)
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        s["q_out"] = torch.zeros(B, H, T, d, dtype=dt, device="cuda")
        s["inv_freq"] = ROPE_BASE ** (-torch.arange(0, c["rope"], 2, dtype=torch.float64) / c["rope"])
        s["live"] = torch.tensor(_live_kv(c), device="cuda")
        return s
    if c["op"] == "read":
        s["k_out"], s["v_out"] = (torch.empty(B, Hkv, T, d, dtype=dt, device="cuda") for _ in range(2))
        return s
    s["q"] = normal(B, H, T, d)
    s["prefix_pages"] = pages[own_pages:].contiguous()
    L = c["prefix"] + c["max_len"]   # per head: key preference ~ N(0, 1), distance preference with a recency slope
    s["a"] = torch.randn(H, L, generator=g, device="cuda")
    s["r"] = 0.5 * torch.randn(H, L, generator=g, device="cuda")
    s["r"] -= min(0.05, 80.0 / L) * torch.arange(L, device="cuda")
    s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, H, T, device="cuda")
    s["workspace"] = {}
    return s


# ---------------------------------------------------------------------------
# Plain forms, in 32 bits
# ---------------------------------------------------------------------------
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
    q_keep = valid[:, None, :, None] & ~s["frz"][None, :, None, None]
    s["q_out"].copy_(torch.where(q_keep, q, s["q_out"]))
    k, k_scale = _quantise(_rotate(s["k"], cos, sin, c["interleaved"]))
    v, v_scale = _quantise(s["v"].float())
    slot = pos.clamp(max=s["table"].shape[1] * c["page"] - 1)
    page = s["table"].gather(1, slot // c["page"])[valid].long()
    slot = (slot % c["page"])[valid]
    live = s["live"][None, :]
    for new, to, keep in ((v.view(torch.uint8), s["v_cache"].view(torch.uint8), None), (v_scale, s["v_scale"], None),
                          (k.view(torch.uint8), s["k_cache"].view(torch.uint8), live[..., None]),
                          (k_scale, s["k_scale"], live)):
        rows = new.transpose(1, 2)[valid]
        to[page, :, slot] = rows if keep is None else torch.where(keep, rows, to[page, :, slot])
    return [s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _plain_read(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    t = torch.arange(c["T"], device="cuda")
    slot = s["ctx"].long()[:, None] + t
    valid = t < s["n_new"][:, None]
    slot = slot.clamp(max=s["table"].shape[1] * c["page"] - 1)
    page = s["table"].gather(1, slot // c["page"]).clamp(min=0).long()
    slot = slot % c["page"]
    out = []
    for n in ("k", "v"):
        x = s[n + "_cache"].view(torch.uint8)[page, :, slot].view(E4M3).float() * s[n + "_scale"][page, :, slot][..., None]
        out.append(torch.where(valid[..., None, None], x, 0.0).transpose(1, 2).to(dt))
    return out


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


def _gather(s, name, table, L, G):
    """[B, H, L, d] fp32 from a cache, its scales and a page table [B, pages]."""
    at = table.clamp(min=0).long()
    x = s[name + "_cache"].view(torch.uint8)[at].view(E4M3).float() * s[name + "_scale"][at][..., None]
    return x.transpose(1, 2).flatten(2, 3)[:, :, :L].repeat_interleave(G, 1)


def _plain_paged(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    G, P, L = c["H"] // c["Hkv"], c["prefix"], c["max_len"]
    q = s["q"].float()
    t = torch.arange(c["T"], device="cuda")
    i = P + s["ctx"].long()[:, None] + t
    i = torch.where(t < s["n_new"][:, None], i, -1)     # rows past the new tokens see nothing
    j = torch.arange(P + L, device="cuda")
    S = _plain_scores(s, q, _gather(s, "k", s["table"], L, G), i, j[P:])
    v = _gather(s, "v", s["table"], L, G)
    if not P:
        W, lse = _softmax(S)
        return [(W @ v).to(dt), lse]
    kp, vp = (_gather(s, n, s["prefix_pages"][None], P, G) for n in ("k", "v"))
    W, lse = _softmax(torch.cat([_plain_scores(s, q, kp, i, j[:P]), S], -1))
    # one product per head with the shared values for all sequences
    op = (W[..., :P].permute(1, 0, 2, 3).flatten(1, 2) @ vp[0]).unflatten(1, (c["B"], c["T"])).transpose(0, 1)
    return [(op + W[..., P:] @ v).to(dt), lse]


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return _plain_append(s) if op == "append" else _plain_read(s) if op == "read" else _plain_paged(s)
    return _own(s)


def _own(s):
    from softmax_attention_hybrid_gb300 import saf

    c = s["case"]
    fz = s["frozen"] if c["F"] else None
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if c["op"] == "append":
        saf.saf_kv_append_quant(s["k"], s["v"], *cache, s["table"], s["ctx"], s["n_new"], q=s["q"], q_out=s["q_out"],
                               inv_freq=s["inv_freq"], interleaved=c["interleaved"], frozen=fz)
        return [s["q_out"], *cache]
    if c["op"] == "read":
        return list(saf.saf_kv_read_quant(*cache, s["table"], s["ctx"], s["n_new"], k_out=s["k_out"],
                                         v_out=s["v_out"]))
    ws = s["workspace"]
    B, H, Hkv, T, d = (c[n] for n in ("B", "H", "Hkv", "T", "d"))
    if not ws:
        ws["w"] = saf.alloc_paged_quant_workspace(B, H, Hkv, T, d, c["max_len"], s["q"].dtype, prefix_len=c["prefix"])
    if c["op"] == "paged":
        o, lse = saf.saf_attn_paged_quant(s["q"], *cache, s["table"], s["ctx"], c["max_len"], n_new=s["n_new"],
                                         a=s["a"], r=s["r"], frozen=fz, window=c["window"], sinks=c["sinks"],
                                         o=s["o"], lse=s["lse"], workspace=ws["w"])
    else:
        o, lse = saf.saf_attn_paged_shared_quant(s["q"], *cache, s["prefix_pages"], c["prefix"], s["table"], s["ctx"],
                                                c["max_len"], n_new=s["n_new"], a=s["a"], r=s["r"], frozen=fz,
                                                window=c["window"], sinks=c["sinks"], o=s["o"], lse=s["lse"],
                                                workspace=ws["w"])
    return [o, lse]


# ---------------------------------------------------------------------------
# From the definition, in 64 bits
# ---------------------------------------------------------------------------
def _exact_row(c, frozen, q, keys, i, a, r):
    """Weights and log-sum-exp of one head: queries q [n, d] at positions i [n], keys [m, d] at 0 .. m - 1."""
    gap = i[:, None] - torch.arange(keys.shape[0], device="cuda")[None, :]
    hidden = gap < 0
    if frozen:
        logits = a[:keys.shape[0]].double()[None, :] + r.double()[gap.clamp(min=0)]
    else:
        logits = q.double() @ keys.t() * c["d"] ** -0.5
        if c["window"]:
            far = gap >= c["window"]
            far[:, :c["sinks"]] = False
            hidden = hidden | far
    logits = torch.where(hidden, -math.inf, logits)
    lse = torch.logsumexp(logits, -1)
    return torch.exp(logits - lse[:, None]).nan_to_num(0.0), lse


def _slots(c, s, b, first, n):
    """(page, slot in the page) of n slots of sequence b."""
    at = first + torch.arange(n, device="cuda")
    return s["table"][b][at // c["page"]].long(), at % c["page"]


def _exact_rows(s, name, page, hk, slot):
    """What the cache's rows stand for."""
    code = s[name + "_cache"].view(torch.uint8)[page, hk, slot].view(E4M3).double()
    return code * s[name + "_scale"][page, hk, slot].double()[..., None]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    fz, G = _frozen(c), c["H"] // c["Hkv"]
    if c["op"] == "append":
        return _exact_append(c, s, fz)
    if c["op"] == "read":
        return _exact_read(c, s)
    o = torch.zeros(c["B"], c["H"], c["T"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["H"], c["T"]), -math.inf, dtype=torch.float64, device="cuda")
    P, ps = c["prefix"], c["page"]
    ctx, new = s["ctx"].tolist(), s["n_new"].tolist()
    for b in range(c["B"]):
        n = new[b]
        if n == 0:
            continue
        page, slot = _slots(c, s, b, 0, ctx[b] + n)
        if P:
            head = torch.arange(P, device="cuda")
            page = torch.cat([s["prefix_pages"][head // ps].long(), page])
            slot = torch.cat([head % ps, slot])
        i = P + ctx[b] + torch.arange(n, device="cuda")
        for hk in range(c["Hkv"]):
            k, v = (_exact_rows(s, name, page, hk, slot) for name in ("k", "v"))
            for h in range(hk * G, hk * G + G):
                W, lse[b, h, :n] = _exact_row(c, fz[h], s["q"][b, h, :n], k, i, s["a"][h], s["r"][h])
                o[b, h, :n] = W @ v
    return [o, lse]


def _exact_read(c, s):
    out = [torch.zeros(c["B"], c["Hkv"], c["T"], c["d"], dtype=torch.float64, device="cuda") for _ in range(2)]
    ctx, new = s["ctx"].tolist(), s["n_new"].tolist()
    for b in range(c["B"]):
        page, slot = _slots(c, s, b, ctx[b], new[b])
        for hk in range(c["Hkv"]):
            for x, name in zip(out, ("k", "v")):
                x[b, hk, :new[b]] = _exact_rows(s, name, page, hk, slot)
    return out


def _exact_append(c, s, fz):
    """The rotated queries, and the caches as y / scale before it is rounded to e4m3, with the scales; the
    rotation as a complex product."""
    q_out, kc, vc, ks, vs = (s[n].double() for n in ("q_out", "k_cache", "v_cache", "k_scale", "v_scale"))
    ctx, new, n = s["ctx"].tolist(), s["n_new"].tolist(), c["rope"] // 2
    freq = ROPE_BASE ** (-2 * torch.arange(n, dtype=torch.float64, device="cuda") / c["rope"])
    live = _live_kv(c)
    heads = [h for h in range(c["H"]) if not fz[h]]

    def turn(x, pos):   # x [heads, tokens, d]
        z = x[..., :2 * n].reshape(*x.shape[:-1], *((n, 2) if c["interleaved"] else (2, n)))
        z = z if c["interleaved"] else z.transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(freq), pos * freq))
        y = y if c["interleaved"] else y.transpose(-1, -2)
        return torch.cat([y.flatten(-2), x[..., 2 * n:]], -1)

    def put(codes, scales, page, hk, slot, y):
        top = torch.maximum(y.amax(-1), -y.amin(-1)) / 448
        scales[page, hk, slot] = top
        codes[page, hk, slot] = y / top[:, None]

    for b in range(c["B"]):
        m = new[b]
        if m == 0:
            continue
        page, slot = _slots(c, s, b, ctx[b], m)
        pos = (ctx[b] + torch.arange(m, device="cuda")).double()[:, None]
        if heads:
            q_out[b, heads, :m] = turn(s["q"][b, heads, :m].double(), pos)
        for hk in range(c["Hkv"]):
            put(vc, vs, page, hk, slot, s["v"][b, hk, :m].double())
            if live[hk]:
                put(kc, ks, page, hk, slot, turn(s["k"][b, hk:hk + 1, :m].double(), pos)[0])
    return [q_out, kc, vc, ks, vs]
