"""Measured cases of the operators round the paged KV cache.

Four operators: attention of a request's newest tokens over the paged cache
(``qsa.paged_attn``), writing new keys and values into the pages with rotary
positions and E4M3 quantisation (``qsa.kv_append``), reading the cache back
(``qsa.kv_gather``) and rotary positions alone (``qsa.rope``).

``run`` computes a case in plain torch operations, or, with ``own`` true, with
the library's kernels. ``exact`` gives the result from the definition in 64
bits.
"""

import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attn(name, batch, n_q, ctx_lo, ctx_hi, kv, n_q_heads=16, n_kv_heads=2, head_dim=128, page_size=64, window=0,
          pad=0):
    return {"name": name, "op": "paged_attn", "batch": batch, "n_q": n_q, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "kv": kv,
            "n_q_heads": n_q_heads, "n_kv_heads": n_kv_heads, "head_dim": head_dim, "page_size": page_size,
            "window": window, "pad": pad}


def _append(name, batch, n_tok, start, kv, scaling, layout="half", rot_dim=128, n_q_heads=16, n_kv_heads=2,
            head_dim=128, page_size=64, ragged=0):
    return {"name": name, "op": "kv_append", "batch": batch, "n_tok": n_tok, "start": start, "kv": kv,
            "scaling": scaling, "layout": layout, "rot_dim": rot_dim, "n_q_heads": n_q_heads,
            "n_kv_heads": n_kv_heads, "head_dim": head_dim, "page_size": page_size, "ragged": ragged}


def _gather(name, batch, n_tok, kv, n_kv_heads=2, head_dim=128, page_size=64, ragged=0):
    return {"name": name, "op": "kv_gather", "batch": batch, "n_tok": n_tok, "kv": kv, "n_kv_heads": n_kv_heads,
            "head_dim": head_dim, "page_size": page_size, "ragged": ragged}


def _rope(name, batch, n_tok, start, scaling, layout, rot_dim, n_heads, head_dim=128, inverse=False):
    return {"name": name, "op": "rope", "batch": batch, "n_tok": n_tok, "start": start, "scaling": scaling,
            "layout": layout, "rot_dim": rot_dim, "n_heads": n_heads, "head_dim": head_dim, "inverse": inverse}


def listed():
    return [
        # one short chat turn, one new token: the latency of a call
        _attn("attn b1 decode 1k bf16", 1, 1, 1000, 1000, "bf16"),
        # one request verifying 4 draft tokens at the context of the 50K workload
        _attn("attn b1 verify 50k bf16", 1, 4, 50004, 50004, "bf16"),
        # a serving batch over agent turns (50,000 + 800 t tokens), one token each
        _attn("attn b32 decode 50k bf16", 32, 1, 50001, 61201, "bf16"),
        # the same batch verifying 4 draft tokens on an E4M3 cache
        _attn("attn b32 verify 50k fp8", 32, 4, 50004, 61204, "fp8"),
        # a mixed batch of short and long requests, small heads, small pages, a sliding window, two padding rows
        _attn("attn b13 window d64 p16", 13, 2, 1, 9001, "bf16", 12, 4, 64, 16, 1000, 2),
        # a decode step's new token of every request: rotate q and k, write k and v
        _append("append b32 decode bf16", 32, 1, 1500, "bf16", "none"),
        # a verify step on an E4M3 cache, positions scaled for long contexts, a quarter of the head rotated
        _append("append b24 verify fp8", 24, 4, 2045, "fp8", "yarn", "half", 32, 16, 2, 128, 64, 1),
        # a ragged prefill chunk of two requests on an E4M3 cache
        _append("append b2 prefill 16385 fp8", 2, 16385, 7, "fp8", "linear", "half", 128, 16, 2, 128, 64, 1001),
        # index queries of a verify step
        _rope("rope b32 index queries", 32, 4, 50000, "none", "half", 128, 4),
        # a prefill chunk's queries, interleaved pairs on half of the head (rotated back: the gradient's direction)
        _rope("rope b1 chunk 32768 back", 1, 32768, 100000, "ntk", "interleaved", 64, 16, 128, True),
        # a cached prefix read back for a dense layer's prefill
        _gather("gather b1 prefix 50k bf16", 1, 50001, "bf16"),
        # short prefixes of a batch from an E4M3 cache
        _gather("gather b4 prefix 777 fp8", 4, 777, "fp8", 2, 128, 16, 100),
    ]


_MAX_KV_BYTES = 32 * 55000 * 2 * 2 * 128 * 2  # about the largest listed case's cache
_MAX_TOK_VALUES = 32768 * 16 * 128


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["paged_attn", "paged_attn", "kv_append", "kv_append", "rope", "kv_gather"])
    kv = rng.choice(["bf16", "fp8"])
    page_size = rng.choice([16, 32, 64, 64, 128, 256])
    head_dim = rng.choice([64, 128, 128, 256])
    n_kv = rng.choice([1, 2, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8, 8, 16])
    if op == "paged_attn":
        batch = _log_int(rng, 1, 32)
        n_q = rng.randint(1, 4)
        esz = 2 if kv == "bf16" else 1
        cap = int(_MAX_KV_BYTES / (batch * n_kv * 2 * head_dim * esz * max(1, n_q * group // 32)))
        hi = _log_int(rng, 2, max(3, min(61204, cap // 2)))
        lo = rng.randint(1, hi)
        window = rng.choice([0, 0, 0, _log_int(rng, 1, 4096)])
        pad = rng.randint(0, batch - 1) if rng.random() < 0.2 else 0
        c = _attn("", batch, n_q, lo, hi, kv, n_kv * group, n_kv, head_dim, page_size, window, pad)
    elif op == "kv_gather":
        batch = _log_int(rng, 1, 16)
        n_tok = _log_int(rng, 1, max(1, min(50001, _MAX_TOK_VALUES // (2 * batch * n_kv * head_dim))))
        c = _gather("", batch, n_tok, kv, n_kv, head_dim, page_size, rng.randint(0, n_tok - 1))
    else:
        batch = _log_int(rng, 1, 32)
        heads = n_kv * group
        rows = _MAX_TOK_VALUES // (2 * batch * (heads + 2 * n_kv) * head_dim)
        n_tok = _log_int(rng, 1, max(1, min(16385, rows)))
        rot = rng.choice([head_dim, head_dim // 2, head_dim // 4, 2 * rng.randint(2, head_dim // 2)])
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        layout = rng.choice(["half", "interleaved"])
        if op == "rope":
            c = _rope("", batch, n_tok, _log_int(rng, 1, 1000000), scaling, layout, rot, heads, head_dim,
                      rng.random() < 0.5)
        else:
            c = _append("", batch, n_tok, _log_int(rng, 1, 4096), kv, scaling, layout, rot, heads, n_kv, head_dim,
                        page_size, rng.randint(0, n_tok - 1))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# sizes that follow from a case alone
# ---------------------------------------------------------------------------
def _spread(r):
    """A fixed sequence in [0, 1), well spread over its prefixes."""
    return (0.6180339887498949 * (r + 1)) % 1.0


def _contexts(c):
    span = c["ctx_hi"] - c["ctx_lo"]
    return [c["ctx_lo"] + int(span * _spread(r)) for r in range(c["batch"])]


def _query_positions(c):
    """The n_q newest tokens of each request; -1 where there is none, and for the padding requests at the end."""
    out = []
    for r, ctx in enumerate(_contexts(c)):
        live = r < c["batch"] - c["pad"]
        out.append([max(-1, ctx - c["n_q"] + j) if live else -1 for j in range(c["n_q"])])
    return out


def _lengths(c):
    """New (or read) tokens of each request: n_tok less a share of `ragged`."""
    return [c["n_tok"] - int(c.get("ragged", 0) * _spread(r)) for r in range(c["batch"])]


def _token_positions(c):
    start = c.get("start", 0)
    out = np.full((c["batch"], c["n_tok"]), -1, dtype=np.int32)
    for r, n in enumerate(_lengths(c)):
        first = start + 3 * r
        out[r, :n] = np.arange(first, first + n)
    return out


def _inv_freq(c):
    """Angular frequency of each rotated pair (radians per position) in 64 bits, and the amplitude."""
    R = c["rot_dim"]
    base, amp, factor, orig = 10000.0, 1.0, 4.0, 32768.0
    if c["scaling"] == "ntk":
        base *= factor ** (R / (R - 2))
    w = base ** (-2.0 * np.arange(R // 2, dtype=np.float64) / R)
    if c["scaling"] == "linear":
        w = w / factor
    elif c["scaling"] == "yarn":
        g = np.clip((orig * w / (2 * math.pi) - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        w = w * ((1 - g) / factor + g)
        amp = 0.1 * math.log(factor) + 1.0
    return w, amp


def work(case):
    c, D = case, case["head_dim"]
    if c["op"] == "paged_attn":
        esz = 2 if c["kv"] == "bf16" else 1
        seen, pairs, pages = 0, 0, 0
        for row in _query_positions(c):
            row = [p for p in row if p >= 0]
            if not row:
                continue
            w = c["window"] or (1 << 40)
            lo = max(0, min(row) - w + 1)
            seen += max(row) + 1 - lo
            pages += max(row) // c["page_size"] + 1 - lo // c["page_size"]
            pairs += sum(min(p + 1, w) for p in row)
        rows = c["batch"] * c["n_q"] * c["n_q_heads"]
        return {"bytes": 2 * seen * c["n_kv_heads"] * D * esz + rows * (4 * D + 4) + 4 * (pages + c["batch"] * c["n_q"]),
                "flops": 4 * D * c["n_q_heads"] * pairs}
    tokens = c["batch"] * c["n_tok"] if c["op"] == "rope" else sum(_lengths(c))
    idx = 4 * c["batch"] * c["n_tok"]
    if c["op"] == "rope":
        return {"bytes": idx + tokens * c["n_heads"] * D * 4, "flops": tokens * c["n_heads"] * 3 * c["rot_dim"]}
    esz = 2 if c["kv"] == "bf16" else 1
    kvals = tokens * c["n_kv_heads"] * D
    if c["op"] == "kv_gather":
        return {"bytes": idx + 2 * kvals * (esz + 2), "flops": 2 * kvals}
    qvals = tokens * c["n_q_heads"] * D
    return {"bytes": idx + 2 * kvals * (2 + esz) + 4 * qvals,
            "flops": 3 * c["rot_dim"] * tokens * (c["n_q_heads"] + c["n_kv_heads"]) + 2 * kvals}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _cache(c, num_pages, gen):
    """K and V pages of N(0, 1) values (BF16, or E4M3 codes as bytes) and the scale of each KV head."""
    shape = (num_pages, c["n_kv_heads"], c["page_size"], c["head_dim"])
    scales = [(0.010 + 0.002 * torch.rand(c["n_kv_heads"], generator=gen, device="cuda")) for _ in range(2)]
    if c["kv"] == "bf16":
        return _normal(shape, gen), _normal(shape, gen), scales[0], scales[1]
    caches = []
    for s in scales:
        x = torch.randn(shape, generator=gen, device="cuda") / s.view(1, -1, 1, 1)
        caches.append(x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8))
    return caches[0], caches[1], scales[0], scales[1]


def _page_table(tokens, page_size, gen):
    """Randomly placed pages for each request's tokens (-1 behind them), and their number with one page to spare."""
    need = [-(-t // page_size) for t in tokens]
    total = max(1, sum(need))
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(tokens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return table.cuda(), total + 1


def _rope_state(c):
    w, amp = _inv_freq(c)
    return torch.from_numpy(w).cuda(), amp


def _own_rope(c, qsa):
    factor = 1.0 if c["scaling"] == "none" else 4.0
    return qsa.make_rope(c["rot_dim"], base=10000.0, layout=c["layout"], scaling=c["scaling"], factor=factor,
                         orig_len=32768.0)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": c}
    D = c["head_dim"]
    if c["op"] == "rope":
        # the heads to rotate are a slice of a packed projection's output
        H = c["n_heads"]
        st["x"] = _normal((c["batch"], c["n_tok"], H + 2, D), gen)[:, :, :H]
        st["y"] = torch.zeros((c["batch"], c["n_tok"], H, D), dtype=torch.bfloat16, device="cuda")
        first = c["start"] + 3 * np.arange(c["batch"])[:, None]
        st["pos"] = torch.from_numpy((first + np.arange(c["n_tok"])[None]).astype(np.int32)).cuda()
        st["freq"], st["amp"] = _rope_state(c)
        if own:
            from block_sparse_attention_qsa_gb300 import qsa
            st["rope"] = _own_rope(c, qsa)
        return st
    if c["op"] == "paged_attn":
        tokens = _contexts(c)
        st["q_pos"] = torch.tensor(_query_positions(c), dtype=torch.int32).cuda()
        st["q"] = _normal((c["batch"], c["n_q"], c["n_q_heads"], D), gen)
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((c["batch"], c["n_q"], c["n_q_heads"]), device="cuda")
        n_q = c["n_q"]
    else:
        pos = _token_positions(c)
        tokens = [int(row.max()) + 1 for row in pos]
        st["pos"] = torch.from_numpy(pos).cuda()
        n_q = 1
    st["page_table"], num_pages = _page_table(tokens, c["page_size"], gen)
    st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"] = _cache(c, num_pages, gen)
    B, Hk = c["batch"], c["n_kv_heads"]
    if c["op"] == "kv_append":
        # queries, keys and values side by side, as one projection writes them
        H = c["n_q_heads"]
        qkv = _normal((B, c["n_tok"], H + 2 * Hk, D), gen)
        st["q"], st["k"], st["v"] = qkv[:, :, :H], qkv[:, :, H:H + Hk], qkv[:, :, H + Hk:]
        st["q_out"] = torch.zeros((B, c["n_tok"], H, D), dtype=torch.bfloat16, device="cuda")
        st["freq"], st["amp"] = _rope_state(c)
    elif c["op"] == "kv_gather":
        st["k_out"] = torch.zeros((B, c["n_tok"], Hk, D), dtype=torch.bfloat16, device="cuda")
        st["v_out"] = torch.zeros_like(st["k_out"])
    if own:
        from block_sparse_attention_qsa_gb300 import qsa
        max_pages = st["page_table"].shape[1]
        st["d"] = qsa.make_dims(B, n_q, max(1, max_pages * c["page_size"] // 4), max_pages, num_pages, 1, c["kv"],
                                c["page_size"], c.get("n_q_heads", Hk), Hk, D)
        st["ws"] = qsa.make_kv_workspace(st["d"])
        if c["op"] == "kv_append":
            st["rope"] = _own_rope(c, qsa)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _values(cache, kv):
    """A cache as the values that it holds (E4M3 codes without their head's scale)."""
    return cache if kv == "bf16" else cache.view(torch.float8_e4m3fn)


def _rotate(x, pos, freq, amp, layout, sign):
    """Rotary positions of x [B][n][H][D] in 32 bits; the angles in 64."""
    half = freq.numel()
    a = pos.to(torch.float64).unsqueeze(-1) * freq
    cos = (amp * torch.cos(a)).float().unsqueeze(2)
    sin = (sign * amp * torch.sin(a)).float().unsqueeze(2)
    x = x.float()
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if layout == "half":
        x1, x2 = r[..., :half], r[..., half:]
        y = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    else:
        x1, x2 = r[..., 0::2], r[..., 1::2]
        y = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
    return torch.cat([y, rest], -1)


def _store(cache, scale, page, slot, live, x, kv):
    """Writes x [B][n][H_kv][D] to the slots of the live tokens; the others rewrite what the spare page holds."""
    if kv == "bf16":
        new = x.to(torch.bfloat16)
    else:
        new = (x.float() / scale.view(1, 1, -1, 1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    cache[page, :, slot] = torch.where(live, new, cache[page, :, slot])


def _plain_append(st):
    c, pos = st["case"], st["pos"]
    live = (pos >= 0).unsqueeze(-1).unsqueeze(-1)
    p = pos.long().clamp(min=0)
    page = torch.gather(st["page_table"].long(), 1, p // c["page_size"])
    page = torch.where(pos >= 0, page, st["k_cache"].shape[0] - 1)
    slot = p % c["page_size"]
    q = _rotate(st["q"], pos, st["freq"], st["amp"], c["layout"], 1.0).to(torch.bfloat16)
    k = _rotate(st["k"], pos, st["freq"], st["amp"], c["layout"], 1.0)
    _store(st["k_cache"], st["k_scale"], page, slot, live, k, c["kv"])
    _store(st["v_cache"], st["v_scale"], page, slot, live, st["v"], c["kv"])
    return torch.where(live, q, st["q_out"]), _values(st["k_cache"], c["kv"]), _values(st["v_cache"], c["kv"])


def _plain_gather(st):
    c, pos = st["case"], st["pos"]
    live = (pos >= 0).unsqueeze(-1).unsqueeze(-1)
    p = pos.long().clamp(min=0)
    page = torch.gather(st["page_table"].long(), 1, p // c["page_size"]).clamp(min=0)
    slot = p % c["page_size"]
    k, v = (_values(st[n], c["kv"])[page, :, slot].float() for n in ("k_cache", "v_cache"))
    if c["kv"] == "fp8":
        k, v = k * st["k_scale"].view(1, 1, -1, 1), v * st["v_scale"].view(1, 1, -1, 1)
    return (torch.where(live, k.to(torch.bfloat16), st["k_out"]),
            torch.where(live, v.to(torch.bfloat16), st["v_out"]))


def _plain_attn(st):
    c = st["case"]
    B, n_q, Hk, D = c["batch"], c["n_q"], c["n_kv_heads"], c["head_dim"]
    G = c["n_q_heads"] // Hk
    pages = st["page_table"].long().clamp(min=0)
    k, v = (_values(st[n], c["kv"])[pages].transpose(1, 2).flatten(2, 3).float() for n in ("k_cache", "v_cache"))
    if c["kv"] == "fp8":
        k, v = k * st["k_scale"].view(1, -1, 1, 1), v * st["v_scale"].view(1, -1, 1, 1)
    q = st["q"].float().view(B, n_q, Hk, G, D).transpose(1, 2).reshape(B, Hk, n_q * G, D)
    s = (q @ k.transpose(2, 3)) / math.sqrt(D)
    t = torch.arange(k.shape[2], device="cuda").view(1, 1, -1)
    p = st["q_pos"].long().unsqueeze(-1)
    seen = t <= p
    if c["window"]:
        seen = seen & (t > p - c["window"])
    seen = seen.repeat_interleave(G, 1).unsqueeze(1)
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    o = (e @ v) / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, -math.inf, m + torch.log(total)).squeeze(-1)
    o = o.view(B, Hk, n_q, G, D).transpose(1, 2).reshape(B, n_q, Hk * G, D)
    lse = lse.view(B, Hk, n_q, G).transpose(1, 2).reshape(B, n_q, Hk * G)
    return o.to(torch.bfloat16), lse


def run(state):
    st, c = state, state["case"]
    if own:
        from block_sparse_attention_qsa_gb300 import qsa
        if c["op"] == "rope":
            qsa.rope(st["rope"], st["x"], st["pos"], st["y"], inverse=c["inverse"])
            return st["y"]
        cache = (st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["page_table"])
        if c["op"] == "paged_attn":
            qsa.paged_attn(st["d"], st["q"], *cache, st["q_pos"], st["out"], st["ws"], lse=st["lse"],
                           window=c["window"])
            return st["out"], st["lse"]
        if c["op"] == "kv_gather":
            qsa.kv_gather(st["d"], *cache, st["pos"], st["k_out"], st["v_out"], st["ws"])
            return st["k_out"], st["v_out"]
        qsa.kv_append(st["d"], st["k"], st["v"], *cache, st["pos"], st["ws"], rope=st["rope"], q=st["q"],
                      q_out=st["q_out"])
        return st["q_out"], _values(st["k_cache"], c["kv"]), _values(st["v_cache"], c["kv"])
    if c["op"] == "rope":
        return _rotate(st["x"], st["pos"], st["freq"], st["amp"], c["layout"],
                       -1.0 if c["inverse"] else 1.0).to(torch.bfloat16)
    if c["op"] == "paged_attn":
        return _plain_attn(st)
    return _plain_gather(st) if c["op"] == "kv_gather" else _plain_append(st)


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------
def _exact_rotation(x, positions, c, sign):
    """x [n][H][D] (64 bits): every pair as a complex number times amp * exp(i sign angle)."""
    w, amp = _inv_freq(c)
    angle = torch.from_numpy(np.outer(positions.astype(np.float64), w)).cuda()
    turn = torch.polar(torch.full_like(angle, amp), sign * angle).unsqueeze(1)
    R = c["rot_dim"]
    first = torch.arange(R // 2, device="cuda") if c["layout"] == "half" else torch.arange(0, R, 2, device="cuda")
    second = first + (R // 2 if c["layout"] == "half" else 1)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _cache_rows(st, r, positions):
    """(page, slot) of request r's positions."""
    ps = st["case"]["page_size"]
    table = st["page_table"][r].cpu().numpy()
    return torch.from_numpy(table[positions // ps].astype(np.int64)).cuda(), torch.from_numpy(positions % ps).cuda()


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    D = c["head_dim"]
    if c["op"] == "rope":
        pos = st["pos"].cpu().numpy()
        sign = -1.0 if c["inverse"] else 1.0
        return torch.stack([_exact_rotation(st["x"][r].double(), pos[r], c, sign) for r in range(c["batch"])])
    fp8 = c["kv"] == "fp8"
    kc, vc = (_values(st[n], c["kv"]).double() if c["op"] == "kv_append" else _values(st[n], c["kv"])
              for n in ("k_cache", "v_cache"))
    Hk = c["n_kv_heads"]
    ks, vs = (st[n].double().view(1, Hk, 1) if fp8 else 1.0 for n in ("k_scale", "v_scale"))
    if c["op"] == "kv_append":
        q_out = st["q_out"].double()
        for r, row in enumerate(st["pos"].cpu().numpy().astype(np.int64)):
            n = int((row >= 0).sum())
            page, slot = _cache_rows(st, r, row[:n])
            q_out[r, :n] = _exact_rotation(st["q"][r, :n].double(), row[:n], c, 1.0)
            k = _exact_rotation(st["k"][r, :n].double(), row[:n], c, 1.0) / ks
            v = st["v"][r, :n].double() / vs
            kc[page, :, slot] = k.clamp(-E4M3_MAX, E4M3_MAX) if fp8 else k
            vc[page, :, slot] = v.clamp(-E4M3_MAX, E4M3_MAX) if fp8 else v
        return q_out, kc, vc
    if c["op"] == "kv_gather":
        k_out, v_out = st["k_out"].double(), st["v_out"].double()
        for r, row in enumerate(st["pos"].cpu().numpy().astype(np.int64)):
            n = int((row >= 0).sum())
            page, slot = _cache_rows(st, r, row[:n])
            k_out[r, :n] = kc[page, :, slot].double() * ks
            v_out[r, :n] = vc[page, :, slot].double() * vs
        return k_out, v_out
    G = c["n_q_heads"] // Hk
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for r, row in enumerate(_query_positions(c)):
        for j, p in enumerate(row):
            if p < 0:
                continue
            lo = max(0, p + 1 - c["window"]) if c["window"] else 0
            page, slot = _cache_rows(st, r, np.arange(lo, p + 1))
            k = (kc[page, :, slot].double() * ks).transpose(0, 1)  # [H_kv][t][D]
            v = (vc[page, :, slot].double() * vs).transpose(0, 1)
            s = st["q"][r, j].double().view(Hk, G, D) @ k.transpose(1, 2) / math.sqrt(D)
            lse[r, j] = torch.logsumexp(s, -1).view(-1)
            out[r, j] = (torch.softmax(s, -1) @ v).reshape(-1, D)
    return out, lse
