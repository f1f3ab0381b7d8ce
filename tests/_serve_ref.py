"""64-bit references of the operators for serving a batch in a bounded cache
(numpy, CPU). Written from the definitions in include/qsa_serve.h; nothing here
is shared with the library."""

import math

import numpy as np

from tests import _kv_ref as R


def attn_tol(ref, mag, lse, qk, D, kv, small):
    """Output: half a BF16 step of the result; every weight is off by its own
    rounding (2^-8 at most), by the score's error as an exponent, and by the
    exponential and the sums (2^-18 covers a few thousand FP32 steps taken in
    trees); the score's error is that of an FP32 sum of D products, at most
    2^-23 of the sum of their magnitudes for each of about D / 8 + 8 partial
    sums. lse: the score's error and a few FP32 steps. With an E4M3 cache a
    position of a request's own may add 2^-21 of the largest weight (two E4M3
    codes a weight), one of the prefix 2^-31."""
    eps_s = (D / 8 + 8) * 2.0 ** -23 * qk
    w = 2.0 ** -8 + 2.0 ** -18
    tiny = 2.0 ** -21 * small if kv == "fp8" else 0.0
    fin = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return 2.0 ** -8 * np.abs(ref) + (w + 2 * eps_s)[..., None] * mag + tiny, eps_s + 2.0 ** -18 * (1 + fin)


def weights(q, k, scale, lse, pos, old, decay, fp8):
    """q [n_q][H][D], k [T][H_kv][D], lse [n_q][H], old [T] float64, pos [n_q]:
    (weights [T], their tolerance [T]). A score is off by the error of an FP32
    sum of D products (as in attn_tol), with an E4M3 cache by 2^-22 of the
    head's largest |q| in each component, and the exponent's product and
    difference by 2^-22 of their sizes; the exponentials and sums by 2^-18."""
    T, H = k.shape[0], q.shape[1]
    G, D = H // k.shape[1], q.shape[2]
    new, err = np.zeros(T), np.zeros(T)
    for j, p in enumerate(pos):
        for h in range(H):
            if p < 0 or lse[j, h] == -np.inf:
                continue
            kk = k[:p + 1, h // G]
            s = kk @ q[j, h] * scale
            size = np.abs(kk) @ np.abs(q[j, h]) * scale
            e = (D / 8 + 8) * 2.0 ** -23 * size + 2.0 ** -22 * (np.abs(s) + abs(lse[j, h]) + 1)
            if fp8:
                e = e + 2.0 ** -22 * np.abs(q[j, h]).max() * np.abs(kk).sum(1) * scale
            w = np.exp(s - lse[j, h])
            new[:p + 1] += w
            err[:p + 1] += w * np.expm1(2 * e)
    total = new + (decay * old if decay else 0.0)
    return total, err + 2.0 ** -18 * new + 2.0 ** -22 * np.abs(total)


def evict(w, n, keep, sinks, recent):
    """Old positions that stay, ascending. w [>= n] float32."""
    if n <= keep:
        return np.arange(n)
    mid = np.arange(sinks, n - recent)
    x = w[mid].astype(np.float64)
    nan = np.isnan(x)
    # heaviest first; NaN behind everything, equal ones by position
    order = sorted(range(len(mid)), key=lambda i: (bool(nan[i]), 0.0 if nan[i] else -x[i], i))
    best = mid[np.array(order[:keep - sinks - recent], dtype=int)]
    return np.sort(np.concatenate([np.arange(sinks), best, np.arange(n - recent, n)])).astype(int)


def clean(p):
    p = np.asarray(p, dtype=np.float64)
    return np.where(np.isnan(p), 0.0, np.clip(p, 0.0, 1.0))


def fixed54(p):
    return np.rint(clean(p) * 2.0 ** 54).astype(np.int64)  # (24 significant bits: the product is exact)


def uniform(u):
    u = float(u)
    if math.isnan(u):
        return 0.0
    return min(max(u, 0.0), 1.0 - 2.0 ** -24)


def verify(target, draft, tokens, u):
    """One request: target [n + 1][V], draft [n][V] or None (float64), tokens
    [n], u [n + 1]. Returns (accepted, out [n + 1])."""
    n, V = target.shape[0] - 1, target.shape[1]
    out = [-1] * (n + 1)
    if tokens[0] == -2:
        return 0, out
    m, rejected = 0, False
    while m < n and 0 <= tokens[m] < V:
        q = float(clean(draft[m, tokens[m]])) if draft is not None else 1.0
        if not uniform(u[m]) * q < float(clean(target[m, tokens[m]])):
            rejected = True
            break
        out[m] = int(tokens[m])
        m += 1
    p = fixed54(target[m])
    w = p
    if rejected:
        if draft is not None:
            w = np.where(clean(target[m]) > clean(draft[m]), p - fixed54(draft[m]), 0)
        else:
            w = p.copy()
            w[tokens[m]] = 0
        if not w.any():
            w = p
    cum = np.cumsum(w, dtype=np.int64)
    total = int(cum[-1])
    if total:
        t = total * int(uniform(u[n]) * 2.0 ** 64) >> 64
        out[m] = int(np.searchsorted(cum, t, side="right"))
    return m, out


def rows_of(cache, table_row, n):
    return R.rows(cache, table_row, n)
