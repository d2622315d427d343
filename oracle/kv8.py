"""The 8-bit key/value cache in float64 (test infrastructure only).

A cache here is a dict of numpy arrays: ``k8``, ``v8`` [B, Hk, cap, d] the E4M3 *values* of the
codes (NaN for the NaN code), ``ks``, ``vs`` [B, Hk, cap / block] the scales, ``w`` [B, Hk, cap]
the accumulated weights and ``lengths`` [B].  One token, one row, one block at a time.
"""
from __future__ import annotations

import math

import numpy as np

from .fp8 import round_e4m3


def block_scale(values):
    """Least power of two s in 2^-100 .. 2^120 with |x| <= 448 s for every finite value x."""
    x = np.abs(np.asarray(values, dtype=np.float64))
    x = x[np.isfinite(x)]
    a = float(x.max()) if x.size else 0.0
    e = -100
    while e < 120 and a > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def codes(x, scale):
    """E4M3 values of x / scale; what is not finite becomes NaN."""
    x = np.asarray(x, dtype=np.float64)
    fin = np.isfinite(x)
    return np.where(fin, round_e4m3(np.where(fin, x, 0.0) / scale), np.nan)


def positions(length, count, n):
    """Positions of the ``count`` new tokens: token i at length - count + i."""
    return [length - count + i for i in range(min(count, n))]


def append(cache, k_new, v_new, counts=None):
    """Writes k_new, v_new [B, Hk, n, d] into the cache (a new dict)."""
    out = {key: np.array(val, copy=True) for key, val in cache.items()}
    B, Hk, cap, _ = out["k8"].shape
    n, block = k_new.shape[2], cap // out["ks"].shape[2]
    for b in range(B):
        length = int(out["lengths"][b])
        cnt = n if counts is None else int(counts[b])
        pos = positions(length, cnt, n)
        first = max(0, length - cnt)
        for h in range(Hk):
            for x, c, s in ((k_new, out["k8"], out["ks"]), (v_new, out["v8"], out["vs"])):
                for t in range(cap // block):
                    here = [(p, i) for i, p in enumerate(pos) if 0 <= p and p // block == t]
                    if not here:
                        continue
                    vals = np.stack([x[b, h, i] for _, i in here])
                    scale = block_scale(vals)
                    if first > t * block:
                        old = float(s[b, h, t])
                        if scale > old:
                            held = slice(t * block, first)
                            c[b, h, held] = codes(c[b, h, held] * (old / scale), 1.0)
                        scale = max(scale, old)
                    s[b, h, t] = scale
                    for p, i in here:
                        c[b, h, p] = codes(x[b, h, i], scale)
            for p in pos:
                if p >= 0:
                    out["w"][b, h, p] = 0.0
    return out


def seen(length, count, i, causal):
    """How many of the first keys row i sees (0 for a padding row)."""
    if i >= count:
        return 0
    return min(length, max(0, length - count + i + 1)) if causal else length


def _values(cache, which, b, h, m):
    c, s = cache[which + "8"], cache[which + "s"]
    block = c.shape[2] // s.shape[2]
    per = np.array([s[b, h, j // block] for j in range(m)], dtype=np.float64).reshape(m, 1)
    return c[b, h, :m] * per


def attend(cache, q, c, counts=None, causal=False):
    """O, LSE of q [B, H, n, d] over the cache, and per element sum_j P_ij |V_j|, per row the
    largest sum_r |q_r k_jr| c of a seen key, and sum_j |v8_j| times the largest V scale."""
    B, H, n, d = q.shape
    Hk = cache["k8"].shape[1]
    G = H // Hk
    O, L = np.zeros((B, H, n, d)), np.full((B, H, n), -np.inf)
    A, S, F = np.zeros((B, H, n, d)), np.zeros((B, H, n)), np.zeros((B, H, n, d))
    for b in range(B):
        length = int(cache["lengths"][b])
        cnt = n if counts is None else int(counts[b])
        for h in range(H):
            k, v = (_values(cache, x, b, h // G, length) for x in "kv")
            for i in range(n):
                m = seen(length, cnt, i, causal)
                if m == 0:
                    continue
                s = c * (k[:m] @ q[b, h, i])
                top = s.max()
                e = np.exp(s - top)
                p = e / e.sum()
                O[b, h, i] = (p[:, None] * v[:m]).sum(0)
                L[b, h, i] = top + math.log(e.sum()) if np.isfinite(top) else np.nan
                A[b, h, i] = (p[:, None] * np.abs(v[:m])).sum(0)
                S[b, h, i] = c * (np.abs(k[:m]) @ np.abs(q[b, h, i])).max()
                vs = cache["vs"][b, h // G, :(m - 1) * cache["vs"].shape[2] // cache["v8"].shape[2] + 1]
                F[b, h, i] = np.abs(cache["v8"][b, h // G, :m]).sum(0) * vs.max()
    return O, L, A, S, F


def add_weights(cache, q, c, lse, counts=None, causal=False):
    """The cache's weights plus, for each key, sum over the rows that see it of e^{s - LSE}."""
    B, H, n, d = q.shape
    G = H // cache["k8"].shape[1]
    w = np.array(cache["w"], dtype=np.float64, copy=True)
    for b in range(B):
        length = int(cache["lengths"][b])
        cnt = n if counts is None else int(counts[b])
        for h in range(H):
            k = _values(cache, "k", b, h // G, length)
            for i in range(n):
                m = seen(length, cnt, i, causal)
                if m and lse[b, h, i] != -np.inf:
                    w[b, h // G, :m] += np.exp(c * (k[:m] @ q[b, h, i]) - lse[b, h, i])
    return w


def kept_tokens(w, length, keep, sink, recent):
    """Positions kept of one head's ``length`` tokens, ascending."""
    if length <= keep:
        return list(range(length))
    safe = [j for j in range(length) if j < sink or j >= length - recent]
    rest = [j for j in range(length) if sink <= j < length - recent]
    key = lambda j: (-np.inf if np.isnan(w[j]) else w[j])
    rest.sort(key=lambda j: (-key(j), j))
    return sorted(safe + rest[:keep - len(safe)])


def evict(cache, out, keep, sink=0, recent=0):
    """Moves the kept tokens of ``cache`` into ``out`` (a new dict), and their positions."""
    out = {key: np.array(val, copy=True) for key, val in out.items()}
    B, Hk, cap, _ = cache["k8"].shape
    block = cap // cache["ks"].shape[2]
    kept = np.full((B, Hk, keep), -1, dtype=np.int64)
    for b in range(B):
        length = int(cache["lengths"][b])
        for h in range(Hk):
            at = kept_tokens(cache["w"][b, h], length, keep, sink, recent)
            kept[b, h, :len(at)] = at
            out["w"][b, h, :len(at)] = cache["w"][b, h, at]
            for x in "kv":
                vals = _values(cache, x, b, h, length)[at]
                for t in range(-(-len(at) // block)):
                    part = vals[t * block:(t + 1) * block]
                    s = block_scale(part)
                    out[x + "s"][b, h, t] = s
                    out[x + "8"][b, h, t * block:t * block + len(part)] = codes(part, s)
        out["lengths"][b] = min(length, keep)
    return out, kept
