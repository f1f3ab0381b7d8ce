"""64-bit references of the operators round the paged cache (numpy, CPU), and
the pages and tables their tests use. Written from the definitions in
include/qsa_kv.h; nothing here is shared with the library."""

import math

import numpy as np
import torch

E4M3_MAX = 448.0


def frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, alpha=1.0, beta=32.0):
    """(radians per position of each pair, amplitude)."""
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    w = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    amp = 1.0
    if scaling == "linear":
        w = [x / factor for x in w]
    if scaling == "yarn":
        g = [min(1.0, max(0.0, (orig_len * x / (2 * math.pi) - alpha) / (beta - alpha))) for x in w]
        w = [gi * x + (1 - gi) * x / factor for gi, x in zip(g, w)]
        amp = 0.1 * math.log(factor) + 1.0
    return np.array(w), amp


def pairs(rot_dim, layout):
    i = np.arange(rot_dim // 2)
    return (i, i + rot_dim // 2) if layout == "half" else (2 * i, 2 * i + 1)


def rotate(x, pos, w, amp, layout, inverse=False):
    """x [..., H, D] float64, pos [...]: every head rotated to its position."""
    x = np.asarray(x, dtype=np.float64)
    a, b = pairs(2 * len(w), layout)
    ang = np.asarray(pos, dtype=np.float64)[..., None, None] * w * (-1.0 if inverse else 1.0)
    y = x.copy()
    y[..., a] = amp * (x[..., a] * np.cos(ang) - x[..., b] * np.sin(ang))
    y[..., b] = amp * (x[..., b] * np.cos(ang) + x[..., a] * np.sin(ang))
    return y


def pair_size(x, w, layout):
    """|x_a| + |x_b| at both components of every pair, 0 at the others."""
    a, b = pairs(2 * len(w), layout)
    s = np.zeros_like(np.asarray(x, dtype=np.float64))
    s[..., a] = s[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return s


def f64(t):
    """A tensor's values (E4M3 codes held in uint8 included) as float64 numpy."""
    t = t.detach().cpu()
    if t.dtype == torch.uint8:
        t = t.view(torch.float8_e4m3fn)
    return t.float().numpy().astype(np.float64)


def attention(q, k, v, scale, lo, hi):
    """q [H][D], k, v [T][H_kv][D] float64; positions lo .. hi - 1. Returns
    (out [H][D], lse [H], sum of weight * |v| [H][D], largest sum of |q k| [H],
    largest weight * sum of |v| [H][D])."""
    H = q.shape[0]
    out, mag, small = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    lse, qk = np.full(H, -np.inf), np.zeros(H)
    if hi <= lo:
        return out, lse, mag, qk, small
    G = H // k.shape[1]
    for h in range(H):
        kk, vv = k[lo:hi, h // G], v[lo:hi, h // G]
        s = kk @ q[h] * scale
        m = s.max()
        e = np.exp(s - m)
        p = e / e.sum()
        out[h], mag[h] = p @ vv, p @ np.abs(vv)
        small[h] = p.max() * np.abs(vv).sum(0)
        lse[h] = m + math.log(e.sum())
        qk[h] = (np.abs(kk) @ np.abs(q[h])).max() * scale
    return out, lse, mag, qk, small


def page_table(tokens, page_size, seed, spare=1):
    """Randomly placed pages, -1 behind a request's last; (table, num_pages)."""
    need = [-(-t // page_size) for t in tokens]
    rng = np.random.RandomState(seed)
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(tokens), max(1, max(need))), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table), sum(need) + spare


def rows(cache, table_row, n):
    """Positions 0 .. n - 1 of a request as [n][H_kv][D] (numpy cache)."""
    ps = cache.shape[2]
    t = np.arange(n)
    return cache[table_row[t // ps], :, t % ps]


def make_cache(num_pages, n_kv, page_size, D, kv, seed, device="cuda"):
    """(k_cache, v_cache, k_scale, v_scale) of N(0, 1) values."""
    g = torch.Generator(device=device).manual_seed(seed)
    out, scales = [], []
    for i in range(2):
        x = torch.randn((num_pages, n_kv, page_size, D), generator=g, device=device)
        s = 0.01 + 0.003 * torch.rand(n_kv, generator=g, device=device)
        scales.append(s)
        if kv == "fp8":
            x = (x / s.view(1, -1, 1, 1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            x = x.to(torch.bfloat16)
        out.append(x)
    return out[0], out[1], scales[0], scales[1]
