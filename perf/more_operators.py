"""Measured cases of the operators for serving a batch in a bounded cache.

Four operators: attention of a batch whose requests share a long prefix
(``qsa.prefix_attn``), the attention weight that each cached position gets
(``qsa.kv_weight``), eviction of the positions with the least of it
(``qsa.kv_evict``), and verification of drafted tokens against the target's
probabilities (``qsa.verify_drafts``).

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
def _prefix(name, batch, n_q, prefix, own_lo, own_hi, kv, n_q_heads=16, n_kv_heads=2, head_dim=128, page_size=64,
            pad=0):
    """`prefix` pages are shared; each request has own_lo .. own_hi tokens behind them."""
    return {"name": name, "op": "prefix_attn", "batch": batch, "n_q": n_q, "prefix": prefix, "own_lo": own_lo,
            "own_hi": own_hi, "kv": kv, "n_q_heads": n_q_heads, "n_kv_heads": n_kv_heads, "head_dim": head_dim,
            "page_size": page_size, "pad": pad}


def _weight(name, batch, n_q, ctx_lo, ctx_hi, kv, decay, n_q_heads=16, n_kv_heads=2, head_dim=128, page_size=64,
            pad=0):
    return {"name": name, "op": "kv_weight", "batch": batch, "n_q": n_q, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "kv": kv,
            "decay": decay, "n_q_heads": n_q_heads, "n_kv_heads": n_kv_heads, "head_dim": head_dim,
            "page_size": page_size, "pad": pad}


def _evict(name, batch, ctx_lo, ctx_hi, keep, sinks, recent, kv, n_kv_heads=2, head_dim=128, page_size=64):
    return {"name": name, "op": "kv_evict", "batch": batch, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "keep": keep,
            "sinks": sinks, "recent": recent, "kv": kv, "n_kv_heads": n_kv_heads, "head_dim": head_dim,
            "page_size": page_size}


def _verify(name, batch, n_draft, vocab, probs, drafts, accept):
    """`drafts`: "sampled" (the draft's probabilities are given) or "greedy" (they are not)."""
    return {"name": name, "op": "verify_drafts", "batch": batch, "n_draft": n_draft, "vocab": vocab, "probs": probs,
            "drafts": drafts, "accept": accept}


def listed():
    return [
        # a few chats over one short system prompt, small heads, small pages, a padding row: the latency of a call
        _prefix("prefix b5 1k d64 p16 bf16", 5, 2, 63, 1, 300, "bf16", 12, 4, 64, 16, 1),
        # one new token of 64 requests over a common document on an E4M3 cache
        _prefix("prefix b64 decode 16k fp8", 64, 1, 257, 1, 2001, "fp8"),
        # agents branched from one 50,000-token history (own turns of 800 t tokens), 4 verify queries each
        _prefix("prefix b32 verify 50k bf16", 32, 4, 782, 4, 6401, "bf16"),
        # the same on an E4M3 cache
        _prefix("prefix b32 verify 50k fp8", 32, 4, 782, 4, 6401, "fp8"),
        # one short chat turn's weights: the latency of a call
        _weight("weight b1 decode 1k fp8", 1, 1, 1000, 1000, "fp8", 0.0),
        # a serving batch over agent turns, 4 verify queries, older weights fading
        _weight("weight b32 verify 50k bf16", 32, 4, 50004, 61204, "bf16", 0.95),
        # one request over its bound by a few tokens: the latency of a call
        _evict("evict b1 4200 to 4097 fp8", 1, 4200, 4200, 4097, 4, 128, "fp8"),
        # a serving batch brought down to a third of its contexts
        _evict("evict b32 50k to 16k bf16", 32, 50001, 61201, 16385, 4, 1000, "bf16"),
        # one request, three greedily drafted tokens, a vocabulary of odd size: the latency of a call
        _verify("drafts b1 greedy 32001 fp32", 1, 3, 32001, "fp32", "greedy", 0.8),
        # a small batch with long sampled drafts, probabilities in 16 bits
        _verify("drafts b8 sampled 100k bf16", 8, 7, 100352, "bf16", "sampled", 0.8),
        # a large batch, three sampled drafts each
        _verify("drafts b256 sampled 150k fp32", 256, 3, 150001, "fp32", "sampled", 0.7),
    ]


_MAX_KV_BYTES = 32 * 55000 * 2 * 2 * 128 * 2  # about the largest listed case's cache
_MAX_PAIRS = 32 * 4 * 16 * 56000 * 128        # its products: query rows x positions x head dim
_MAX_PROBS = 256 * 7 * 150001 * 4             # bytes of the largest listed case's probabilities


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefix_attn", "prefix_attn", "kv_weight", "kv_evict", "verify_drafts"])
    if op == "verify_drafts":
        probs, drafts = rng.choice(["fp32", "fp32", "bf16"]), rng.choice(["sampled", "sampled", "greedy"])
        n_draft = rng.randint(1, 8)
        batch = _log_int(rng, 1, 256)
        rows = batch * (n_draft + 1 + (n_draft if drafts == "sampled" else 0))
        vocab = _log_int(rng, 1000, min(160000, _MAX_PROBS // (rows * 4)))
        c = _verify("", batch, n_draft, vocab, probs, drafts, rng.choice([0.3, 0.7, 0.9]))
        del c["name"]
        return c
    kv = rng.choice(["bf16", "fp8"])
    page_size = rng.choice([16, 32, 64, 64, 128, 256])
    head_dim = rng.choice([64, 128, 128, 256])
    n_kv = rng.choice([1, 2, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8, 8, 16])
    esz = 2 if kv == "bf16" else 1
    row = 2 * n_kv * head_dim * esz
    if op == "kv_evict":
        batch = _log_int(rng, 1, 32)
        hi = _log_int(rng, 64, min(61201, _MAX_KV_BYTES // (2 * batch * row)))
        lo = rng.randint(hi // 2, hi)
        keep = rng.randint(hi // 8 + 1, hi)
        sinks = rng.randint(0, min(keep // 4, 64))
        c = _evict("", batch, lo, hi, keep, sinks, rng.randint(0, (keep - sinks) // 2), kv, n_kv, head_dim, page_size)
    else:
        n_q = rng.randint(1, 4)
        batch = _log_int(rng, 1, 64 if op == "prefix_attn" else 32)
        pairs = _MAX_PAIRS // (batch * n_q * n_kv * group * head_dim)
        if op == "prefix_attn":
            prefix = _log_int(rng, 64, max(65, min(61000, pairs // 2, _MAX_KV_BYTES // (2 * row))))
            hi = _log_int(rng, 1, max(2, min(8000, pairs // 4, _MAX_KV_BYTES // (4 * batch * row))))
            pad = rng.randint(0, batch - 1) if rng.random() < 0.2 else 0
            c = _prefix("", batch, n_q, max(1, prefix // page_size), rng.randint(1, hi), hi, kv, n_kv * group, n_kv,
                        head_dim, page_size, pad)
        else:
            hi = _log_int(rng, 2, max(3, min(61204, pairs // 2, _MAX_KV_BYTES // (2 * batch * row))))
            pad = rng.randint(0, batch - 1) if rng.random() < 0.2 else 0
            c = _weight("", batch, n_q, rng.randint(1, hi), hi, kv, rng.choice([0.0, 0.95, 1.0]), n_kv * group, n_kv,
                        head_dim, page_size, pad)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# sizes that follow from a case alone
# ---------------------------------------------------------------------------
def _spread(r):
    """A fixed sequence in [0, 1), well spread over its prefixes."""
    return (0.6180339887498949 * (r + 1)) % 1.0


def _between(c, lo, hi):
    return [c[lo] + int((c[hi] - c[lo]) * _spread(r)) for r in range(c["batch"])]


def _contexts(c):
    """Cached tokens of each request, the prefix's among them."""
    if c["op"] == "prefix_attn":
        return [c["prefix"] * c["page_size"] + n for n in _between(c, "own_lo", "own_hi")]
    return _between(c, "ctx_lo", "ctx_hi")


def _query_positions(c):
    """The n_q newest tokens of each request; -1 where there is none, and for the padding requests at the end."""
    out = []
    for r, ctx in enumerate(_contexts(c)):
        live = r < c["batch"] - c["pad"]
        out.append([max(-1, ctx - c["n_q"] + j) if live else -1 for j in range(c["n_q"])])
    return out


def work(case):
    c = case
    if c["op"] == "verify_drafts":
        esz = 4 if c["probs"] == "fp32" else 2
        # the target's row that is sampled from, and the draft's where a token was rejected
        rejected = 1.0 - c["accept"] ** c["n_draft"] if c["drafts"] == "sampled" else 0.0
        n = c["batch"] * c["vocab"]
        small = c["batch"] * (c["n_draft"] * (2 * esz + 4) + (c["n_draft"] + 1) * 8 + 4)
        return {"bytes": int(n * esz * (1.0 + rejected)) + small, "flops": int(n * (1.0 + 2 * rejected))}
    D, Hk = c["head_dim"], c["n_kv_heads"]
    esz = 2 if c["kv"] == "bf16" else 1
    if c["op"] == "kv_evict":
        n = _contexts(c)
        kept = sum(min(x, c["keep"]) for x in n)
        out = c["batch"] * -(-c["keep"] // c["page_size"]) * c["page_size"]
        idx = 4 * (sum(n) + out + c["batch"] * (c["keep"] + 2)) + 8 * kept // c["page_size"]
        return {"bytes": 4 * kept * Hk * D * esz + idx, "flops": sum(n)}
    shared = c["prefix"] * c["page_size"] if c["op"] == "prefix_attn" else 0
    seen, pairs = shared, 0
    for row in _query_positions(c):
        row = [p for p in row if p >= 0]
        if row:
            seen += max(0, max(row) + 1 - shared)
            pairs += sum(p + 1 for p in row)
    rows = c["batch"] * c["n_q"] * c["n_q_heads"]
    idx = 4 * (seen // c["page_size"] + c["batch"] * c["n_q"])
    if c["op"] == "prefix_attn":
        return {"bytes": 2 * seen * Hk * D * esz + rows * (4 * D + 4) + idx, "flops": 4 * D * c["n_q_heads"] * pairs}
    weights = seen * (4 if c["decay"] == 0.0 else 8)
    return {"bytes": seen * Hk * D * esz + weights + rows * (2 * D + 4) + idx, "flops": 2 * D * c["n_q_heads"] * pairs}


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


def _page_tables(need_lists, gen):
    """Tables of randomly placed pages, one of len(need) rows for each list `need` of page numbers (-1 behind a row's
    last); and the number of pages with one to spare."""
    total = sum(sum(need) for need in need_lists)
    order = torch.randperm(max(1, total), generator=gen, device="cuda").to(torch.int32).cpu()
    tables, at = [], 0
    for need in need_lists:
        table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32)
        for r, n in enumerate(need):
            table[r, :n] = order[at:at + n]
            at += n
        tables.append(table)
    return tables, total + 1


def _prepare_verify(c, gen):
    B, n, V = c["batch"], c["n_draft"], c["vocab"]
    dt = torch.float32 if c["probs"] == "fp32" else torch.bfloat16
    target = torch.softmax(3.0 * torch.randn((B, n + 1, V), generator=gen, device="cuda"), -1)
    st = {"case": c, "draft": None}
    uniform = torch.rand((B, n + 1), generator=gen, device="cuda")
    if c["drafts"] == "sampled":
        # `accept` of the draft's probability lies where the target's is, the rest elsewhere
        draft = c["accept"] * target[:, :n] + (1.0 - c["accept"]) * target[:, :n].roll(V // 2, -1)
        flat = draft.reshape(B * n, V)
        x = torch.rand((B * n, 1), generator=gen, device="cuda", dtype=torch.float64)
        tokens = torch.searchsorted(torch.cumsum(flat.double(), -1), x).clamp_(max=V - 1).view(B, n)
        st["draft"] = draft.to(dt)
    else:
        # the target's likeliest token, made as likely as `accept`
        tokens = target[:, :n].argmax(-1)
        at = tokens.unsqueeze(-1)
        rest = 1.0 - torch.gather(target[:, :n], 2, at)
        target[:, :n] *= (1.0 - c["accept"]) / rest
        target[:, :n].scatter_(2, at, c["accept"])
    st["target"], st["uniform"], st["tokens"] = target.to(dt), uniform, tokens.to(torch.int32)
    st["accepted"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    st["out_tokens"] = torch.zeros((B, n + 1), dtype=torch.int32, device="cuda")
    if own:
        from block_sparse_attention_qsa_gb300 import qsa
        st["ws"] = qsa.make_kv_workspace(qsa.make_dims(B, 1, 1, 1, 1))
    return st


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "verify_drafts":
        return _prepare_verify(c, gen)
    st = {"case": c}
    B, D, Hk, ps = c["batch"], c["head_dim"], c["n_kv_heads"], c["page_size"]
    tokens = _contexts(c)
    n_q = c.get("n_q", 1)
    if c["op"] == "prefix_attn":
        need = [-(-t // ps) - c["prefix"] for t in tokens]
        (shared, table), num_pages = _page_tables([[c["prefix"]], need], gen)
        st["prefix_table"] = shared[0].cuda()
        st["page_table"] = torch.cat([shared.expand(B, -1), table], 1).cuda()
    elif c["op"] == "kv_evict":
        need = [-(-t // ps) for t in tokens]
        (table, table_out), num_pages = _page_tables([need, [-(-c["keep"] // ps)] * B], gen)
        st["page_table"], st["page_table_out"] = table.cuda(), table_out.cuda()
    else:
        (table,), num_pages = _page_tables([[-(-t // ps) for t in tokens]], gen)
        st["page_table"] = table.cuda()
    st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"] = _cache(c, num_pages, gen)
    max_pages = st["page_table"].shape[1]
    if c["op"] == "kv_evict":
        st["length"] = torch.tensor(tokens, dtype=torch.int32).cuda()
        # accumulated weights: a few positions with most of it, and many that never got any (equal: the lower stays)
        w = torch.exp(2.0 * torch.randn((B, max_pages * ps), generator=gen, device="cuda"))
        dead = torch.rand(w.shape, generator=gen, device="cuda") < 0.3
        st["weight"] = torch.where(dead, 0.0, w)
        st["weight_out"] = torch.zeros((B, st["page_table_out"].shape[1] * ps), device="cuda")
        st["kept"] = torch.zeros((B, c["keep"]), dtype=torch.int32, device="cuda")
        st["new_length"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    else:
        st["q_pos"] = torch.tensor(_query_positions(c), dtype=torch.int32).cuda()
        st["q"] = _normal((B, n_q, c["n_q_heads"], D), gen)
        if c["op"] == "prefix_attn":
            st["out"] = torch.zeros_like(st["q"])
            st["lse"] = torch.zeros((B, n_q, c["n_q_heads"]), device="cuda")
        else:
            # scores of such keys are about N(0, 1): the log of their softmax's sum over n positions is about ln n + 1/2
            noise = 0.1 * torch.randn((B, n_q, c["n_q_heads"]), generator=gen, device="cuda")
            st["lse"] = torch.log(st["q_pos"].clamp(min=0) + 1.0).unsqueeze(-1) + 0.5 + noise
            st["weight"] = torch.rand((B, max_pages * ps), generator=gen, device="cuda") / 64.0
    if own:
        from block_sparse_attention_qsa_gb300 import qsa
        st["d"] = qsa.make_dims(B, n_q, max(1, max_pages * ps // 4), max_pages, num_pages, 1, c["kv"], ps,
                                c.get("n_q_heads", Hk), Hk, D)
        st["ws"] = (qsa.make_prefix_workspace(st["d"], c["prefix"]) if c["op"] == "prefix_attn"
                    else qsa.make_kv_workspace(st["d"]))
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _values(cache, kv):
    """A cache as the values that it holds (E4M3 codes without their head's scale)."""
    return cache if kv == "bf16" else cache.view(torch.float8_e4m3fn)


def _paged(st, name, pages):
    """K or V of the pages [..., n] in 32 bits, as [..., H_kv][positions][D]."""
    x = _values(st[name + "_cache"], st["case"]["kv"])[pages.long().clamp(min=0)]
    x = x.transpose(-4, -3).flatten(-3, -2).float()
    return x if st["case"]["kv"] == "bf16" else x * st[name + "_scale"].view(-1, 1, 1)


def _rows(st):
    """The queries in 32 bits as [B][H_kv][n_q x group][D]."""
    c = st["case"]
    B, n_q, Hk, D = c["batch"], c["n_q"], c["n_kv_heads"], c["head_dim"]
    return st["q"].float().view(B, n_q, Hk, -1, D).transpose(1, 2).reshape(B, Hk, -1, D)


def _seen(st, first, n):
    """Whether position first + t is a query's, as [B][1][n_q x group][n]."""
    c = st["case"]
    t = first + torch.arange(n, device="cuda").view(1, 1, -1)
    s = t <= st["q_pos"].long().unsqueeze(-1)
    return s.repeat_interleave(c["n_q_heads"] // c["n_kv_heads"], 1).unsqueeze(1)


def _by_query(x, c):
    """[B][H_kv][n_q x group][...] as [B][n_q][H_q][...]."""
    B, n_q, Hk = c["batch"], c["n_q"], c["n_kv_heads"]
    x = x.view(B, Hk, n_q, -1, *x.shape[3:]).transpose(1, 2)
    return x.reshape(B, n_q, c["n_q_heads"], *x.shape[4:])


def _plain_prefix(st):
    c = st["case"]
    B, Hk, D, n = c["batch"], c["n_kv_heads"], c["head_dim"], c["prefix"] * c["page_size"]
    q = _rows(st)
    flat = q.transpose(0, 1).reshape(Hk, -1, D)  # the rows of all requests, for the keys that they share
    k, v = _paged(st, "k", st["prefix_table"]), _paged(st, "v", st["prefix_table"])
    mine = st["page_table"][:, c["prefix"]:]
    k1, v1 = _paged(st, "k", mine), _paged(st, "v", mine)
    s = (flat @ k.transpose(1, 2)).view(Hk, B, -1, n).transpose(0, 1) / math.sqrt(D)
    s = torch.where(_seen(st, 0, n), s, -math.inf)
    s1 = torch.where(_seen(st, n, k1.shape[2]), (q @ k1.transpose(2, 3)) / math.sqrt(D), -math.inf)
    m = torch.maximum(s.amax(-1, keepdim=True), s1.amax(-1, keepdim=True))
    base = torch.where(m == -math.inf, 0.0, m)
    e, e1 = torch.exp(s - base), torch.exp(s1 - base)
    total = e.sum(-1, keepdim=True) + e1.sum(-1, keepdim=True)
    o = (e.transpose(0, 1).reshape(Hk, -1, n) @ v).view(Hk, B, -1, D).transpose(0, 1) + e1 @ v1
    o = o / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, -math.inf, m + torch.log(total)).squeeze(-1)
    return _by_query(o, c).to(torch.bfloat16), _by_query(lse, c)


def _plain_weight(st):
    c = st["case"]
    k = _paged(st, "k", st["page_table"])
    s = (_rows(st) @ k.transpose(2, 3)) / math.sqrt(c["head_dim"])
    B, n_q, Hk = c["batch"], c["n_q"], c["n_kv_heads"]
    lse = st["lse"].view(B, n_q, Hk, -1).transpose(1, 2).reshape(B, Hk, -1, 1)
    new = torch.where(_seen(st, 0, k.shape[2]), torch.exp(s - lse), 0.0).sum((1, 2))
    touched = torch.arange(k.shape[2], device="cuda") <= st["q_pos"].amax(1, keepdim=True)
    st["weight"] = torch.where(touched, c["decay"] * st["weight"] + new, st["weight"])
    return st["weight"]


def _plain_evict(st):
    c = st["case"]
    B, keep, ps = c["batch"], c["keep"], c["page_size"]
    n = st["length"].long().unsqueeze(1)
    t = torch.arange(st["weight"].shape[1], device="cuda").expand(B, -1)
    always = (t < c["sinks"]) | (t >= n - c["recent"]) | (n <= keep)
    key = torch.where(t >= n, -math.inf, torch.where(always, math.inf, st["weight"]))
    best = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :keep]
    kept = torch.sort(torch.where(best < n, best, t.shape[1]), dim=1).values
    live = kept < n
    kept = torch.where(live, kept, 0)
    # (a case may keep more than the longest request has)
    kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[1]))
    live = torch.nn.functional.pad(live, (0, keep - live.shape[1]))
    to = torch.arange(keep, device="cuda").expand(B, -1)
    src = torch.gather(st["page_table"].long(), 1, kept // ps).clamp(min=0)
    dst = torch.where(live, torch.gather(st["page_table_out"].long(), 1, to // ps), st["k_cache"].shape[0] - 1)
    mask = live.unsqueeze(-1).unsqueeze(-1)
    st["k_cache"][dst, :, to % ps] = torch.where(mask, st["k_cache"][src, :, kept % ps], st["k_cache"][dst, :, to % ps])
    st["v_cache"][dst, :, to % ps] = torch.where(mask, st["v_cache"][src, :, kept % ps], st["v_cache"][dst, :, to % ps])
    w = torch.where(live, torch.gather(st["weight"], 1, kept), 0.0)
    weight_out = torch.nn.functional.pad(w, (0, st["weight_out"].shape[1] - keep))
    return (_values(st["k_cache"], c["kv"]), _values(st["v_cache"], c["kv"]), weight_out,
            torch.where(live, kept, -1).to(torch.int32), st["length"].clamp(max=keep))


def _plain_verify(st):
    c = st["case"]
    B, n, V = c["batch"], c["n_draft"], c["vocab"]
    at = st["tokens"].long().unsqueeze(-1)
    p = torch.gather(st["target"][:, :n], 2, at).squeeze(-1).double()
    q = torch.gather(st["draft"], 2, at).squeeze(-1).double() if st["draft"] is not None else torch.ones_like(p)
    ok = st["uniform"][:, :n].double() * q < p
    m = torch.cumprod(ok.int(), 1).sum(1)
    r = torch.arange(B, device="cuda")
    row = st["target"][r, m].double()
    cut = (m < n).unsqueeze(-1)
    last = m.clamp(max=n - 1)
    if st["draft"] is not None:
        minus = st["draft"][r, last].double()
    else:
        minus = torch.nn.functional.one_hot(st["tokens"][r, last].long(), V).double()
    rest = torch.where(cut, (row - minus).clamp(min=0.0), row)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, row)
    total = torch.cumsum(rest, -1)
    pick = (total <= st["uniform"][:, n:].double() * total[:, -1:]).sum(-1).clamp(max=V - 1)
    j = torch.arange(n + 1, device="cuda")
    drafted = torch.nn.functional.pad(st["tokens"].long(), (0, 1))
    mm = m.unsqueeze(-1)
    out = torch.where(j < mm, drafted, torch.where(j == mm, pick.unsqueeze(-1), -1))
    return m.to(torch.int32), out.to(torch.int32)


def run(state):
    st, c = state, state["case"]
    if own:
        from block_sparse_attention_qsa_gb300 import qsa
        if c["op"] == "verify_drafts":
            qsa.verify_drafts(st["target"], st["draft"], st["tokens"], st["uniform"], st["accepted"],
                              st["out_tokens"], st["ws"])
            return st["accepted"], st["out_tokens"]
        if c["op"] == "prefix_attn":
            qsa.prefix_attn(st["d"], st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"],
                            st["prefix_table"], st["page_table"], st["q_pos"], st["out"], st["ws"], lse=st["lse"])
            return st["out"], st["lse"]
        if c["op"] == "kv_weight":
            qsa.kv_weight(st["d"], st["q"], st["k_cache"], st["k_scale"], st["page_table"], st["q_pos"], st["lse"],
                          st["weight"], st["ws"], decay=c["decay"])
            return st["weight"]
        qsa.kv_evict(st["d"], st["k_cache"], st["v_cache"], st["page_table"], st["page_table_out"], st["length"],
                     st["weight"], st["weight_out"], st["kept"], st["new_length"], st["ws"], sinks=c["sinks"],
                     recent=c["recent"])
        return (_values(st["k_cache"], c["kv"]), _values(st["v_cache"], c["kv"]), st["weight_out"], st["kept"],
                st["new_length"])
    if c["op"] == "verify_drafts":
        return _plain_verify(st)
    if c["op"] == "prefix_attn":
        return _plain_prefix(st)
    return _plain_weight(st) if c["op"] == "kv_weight" else _plain_evict(st)


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------
def _cache_rows(st, r, positions, which="page_table"):
    """(page, slot) of request r's positions."""
    ps = st["case"]["page_size"]
    table = st[which][r].cpu().numpy()
    return torch.from_numpy(table[positions // ps].astype(np.int64)).cuda(), torch.from_numpy(positions % ps).cuda()


def _exact_verify(st):
    c = st["case"]
    accepted, out = np.zeros(c["batch"], np.int32), np.full((c["batch"], c["n_draft"] + 1), -1, np.int32)
    tokens, u = st["tokens"].cpu().numpy(), st["uniform"].double().cpu().numpy()
    for r in range(c["batch"]):
        m = 0
        for x in tokens[r]:
            chance = float(st["draft"][r, m, x]) if st["draft"] is not None else 1.0
            if not u[r, m] * chance < float(st["target"][r, m, x]):
                break
            out[r, m] = x
            m += 1
        p = st["target"][r, m].double().cpu().numpy()
        rest = p
        if m < c["n_draft"]:
            rest = p.copy()
            if st["draft"] is not None:
                rest = np.maximum(rest - st["draft"][r, m].double().cpu().numpy(), 0.0)
            else:
                rest[tokens[r, m]] = 0.0
            if not rest.any():
                rest = p
        total = np.cumsum(rest)
        out[r, m] = min(c["vocab"] - 1, int(np.searchsorted(total, u[r, c["n_draft"]] * total[-1], side="right")))
        accepted[r] = m
    return torch.from_numpy(accepted), torch.from_numpy(out)


def _exact_evict(st):
    c = st["case"]
    kc, vc = (_values(st[n], c["kv"]).double() for n in ("k_cache", "v_cache"))
    kept_all = np.full((c["batch"], c["keep"]), -1, np.int32)
    weight_out = torch.zeros(st["weight_out"].shape, dtype=torch.float64, device="cuda")
    lengths = _contexts(c)
    for r, n in enumerate(lengths):
        kept = np.arange(n)
        if n > c["keep"]:
            middle = np.arange(c["sinks"], n - c["recent"])
            w = st["weight"][r].cpu().numpy()[middle]
            best = middle[np.lexsort((middle, -w))][:c["keep"] - c["sinks"] - c["recent"]]
            kept = np.sort(np.concatenate([kept[:c["sinks"]], best, kept[n - c["recent"]:]]))
        src = _cache_rows(st, r, kept)
        dst = _cache_rows(st, r, np.arange(len(kept)), "page_table_out")
        for x in (kc, vc):
            x[dst[0], :, dst[1]] = x[src[0], :, src[1]]
        kept_all[r, :len(kept)] = kept
        weight_out[r, :len(kept)] = st["weight"][r, torch.from_numpy(kept).cuda()].double()
    return kc, vc, weight_out, torch.from_numpy(kept_all), torch.tensor([min(n, c["keep"]) for n in lengths],
                                                                        dtype=torch.int32)


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] == "verify_drafts":
        return _exact_verify(st)
    if c["op"] == "kv_evict":
        return _exact_evict(st)
    D, Hk = c["head_dim"], c["n_kv_heads"]
    G = c["n_q_heads"] // Hk
    fp8 = c["kv"] == "fp8"
    ks, vs = (st[n].double().view(1, Hk, 1) if fp8 else 1.0 for n in ("k_scale", "v_scale"))
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    weight = st["weight"].double() if c["op"] == "kv_weight" else None
    for r, row in enumerate(_query_positions(c)):
        n = max(row) + 1
        if n == 0:
            continue
        page, slot = _cache_rows(st, r, np.arange(n))
        k = (_values(st["k_cache"], c["kv"])[page, :, slot].double() * ks).transpose(0, 1)  # [H_kv][t][D]
        q = st["q"][r].double().view(c["n_q"], Hk, G, D)
        if c["op"] == "kv_weight":
            weight[r, :n] *= c["decay"]
            for j, p in enumerate(row):
                s = q[j] @ k[:, :p + 1].transpose(1, 2) / math.sqrt(D)
                weight[r, :p + 1] += torch.exp(s - st["lse"][r, j].double().view(Hk, G, 1)).sum((0, 1))
            continue
        v = (_values(st["v_cache"], c["kv"])[page, :, slot].double() * vs).transpose(0, 1)
        for j, p in enumerate(row):
            if p >= 0:
                s = q[j] @ k[:, :p + 1].transpose(1, 2) / math.sqrt(D)
                lse[r, j] = torch.logsumexp(s, -1).view(-1)
                out[r, j] = (torch.softmax(s, -1) @ v[:, :p + 1]).reshape(-1, D)
    return weight if c["op"] == "kv_weight" else (out, lse)
