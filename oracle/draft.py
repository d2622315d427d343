"""A decoding round over a tree of drafted tokens, in float64 or fractions (test infrastructure only).

Node 0 of a sequence is the token decided last, nodes 1 .. count - 1 are drafts, ``parents`` their
parents.  The cache is the dict of ``kv8``.  One node, one row, one token at a time.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from . import kv8


def ancestors(parents, i):
    """Node i and its ancestors; a parent that is no lower node is none."""
    out = {i}
    while 0 <= parents[i] < i:
        i = int(parents[i])
        out.add(i)
    return out


def sees(parents, counts=None):
    """[B, n, n] truth values: which nodes each node sees (rows from the count on: none)."""
    B, n = parents.shape
    out = np.zeros((B, n, n), bool)
    for b in range(B):
        for i in range(n if counts is None else int(counts[b])):
            out[b, i, sorted(ancestors(parents[b], i))] = True
    return out


def words(seen):
    """uint32 words [B, n, ceil(n / 32)] of [B, n, n] truth values, bit by bit."""
    B, n, m = seen.shape
    out = np.zeros((B, n, -(-m // 32)), np.uint32)
    for b, i, j in np.argwhere(seen):
        out[b, i, j // 32] |= np.uint32(1 << (j % 32))
    return out


def keys(length, count, row):
    """Positions that a row with the truth values ``row`` over the nodes sees."""
    base = length - count
    return [j for j in range(length) if j < base or row[j - base]]


def attend(cache, q, c, seen, counts=None):
    """As kv8.attend, with the keys of each row from ``seen`` [B, n, n]."""
    B, H, n, d = q.shape
    G = H // cache["k8"].shape[1]
    block = cache["k8"].shape[2] // cache["ks"].shape[2]
    O, L = np.zeros((B, H, n, d)), np.full((B, H, n), -np.inf)
    A, S, F = np.zeros((B, H, n, d)), np.zeros((B, H, n)), np.zeros((B, H, n, d))
    for b in range(B):
        length = int(cache["lengths"][b])
        cnt = n if counts is None else int(counts[b])
        for h in range(H):
            k, v = (kv8._values(cache, x, b, h // G, length) for x in "kv")
            for i in range(cnt):
                at = keys(length, cnt, seen[b, i])
                if not at:
                    continue
                s = c * (k[at] @ q[b, h, i])
                top = s.max()
                e = np.exp(s - top)
                p = e / e.sum()
                O[b, h, i] = (p[:, None] * v[at]).sum(0)
                L[b, h, i] = top + math.log(e.sum()) if np.isfinite(top) else np.nan
                A[b, h, i] = (p[:, None] * np.abs(v[at])).sum(0)
                S[b, h, i] = abs(c) * (np.abs(k[at]) @ np.abs(q[b, h, i])).max()
                F[b, h, i] = (np.abs(cache["v8"][b, h // G, at]).sum(0)
                              * cache["vs"][b, h // G, :(length - 1) // block + 1].max())
    return O, L, A, S, F


def _number(x, exact):
    """A probability as it counts, within [0, 1], NaN as 0."""
    x = float(x)
    x = 0.0 if math.isnan(x) else min(max(x, 0.0), 1.0)
    return Fraction(x) if exact else x


def verify(target, draft, tokens, parents, uniforms, count, exact=True):
    """One sequence: (accepted nodes, next token).  The residual is a normalised distribution that
    each refusal replaces; target and draft [n, V], draft None for drafts that were not drawn."""
    n, V = target.shape
    if count == 0:
        return [], -1
    node, path = 0, [0]
    while True:
        p = [_number(x, exact) for x in target[node]]
        q = None if draft is None else [_number(x, exact) for x in draft[node]]
        # r over `mass`: as p is given its mass counts as 1 until a refusal changes it.
        r, mass, child = list(p), 1, None
        for i in range(node + 1, count):
            if parents[i] != node:
                continue
            x, u = int(tokens[i]), _number(uniforms[i], exact)
            known = 0 <= x < V
            if q is None:
                if u * mass < (r[x] if known else 0):
                    child = i
                    break
                if known:
                    mass -= r[x]
                    r[x] = type(r[x])(0)
                continue
            if known and u * q[x] < r[x] / mass:
                child = i
                break
            left = [max(a / mass - b, 0) for a, b in zip(r, q)]
            if sum(left) > 0:
                r, mass = left, sum(left)
        if child is None:
            break
        node = child
        path.append(node)
    total, goal, cum = sum(r), None, 0
    if not total > 0:
        return path, -1
    goal = _number(uniforms[0], exact) * total
    for v in range(V):
        cum += r[v]
        if cum > goal:
            return path, v
    return path, max(v for v in range(V) if r[v] > 0)


def keep(cache, path, accepted, counts=None):
    """Moves the accepted nodes' tokens next to those before the tree (a new dict)."""
    out = {key: np.array(val, copy=True) for key, val in cache.items()}
    B, Hk, cap, _ = out["k8"].shape
    n, block = path.shape[1], cap // out["ks"].shape[2]
    for b in range(B):
        length = int(cache["lengths"][b])
        cnt = n if counts is None else int(counts[b])
        acc, base = min(max(int(accepted[b]), 0), cnt), length - cnt
        moves = [(base + i, base + min(max(int(path[b, i]), i), cnt - 1)) for i in range(acc) if base + i >= 0]
        out["lengths"][b] = max(base + acc, 0)
        for h in range(Hk):
            for to, src in moves:
                out["w"][b, h, to] = cache["w"][b, h, src]
            for x in "kv":
                c, s, c0, s0 = out[x + "8"], out[x + "s"], cache[x + "8"], cache[x + "s"]
                for t in range(cap // block):
                    here = [(to, src) for to, src in moves if to // block == t]
                    if not here:
                        continue
                    vals = np.stack([c0[b, h, src] * s0[b, h, src // block] for _, src in here])
                    scale = kv8.block_scale(vals)
                    if max(base, 0) > t * block:
                        old = float(s0[b, h, t])
                        if scale > old:
                            held = slice(t * block, max(base, 0))
                            c[b, h, held] = kv8.codes(c0[b, h, held] * (old / scale), 1.0)
                        scale = max(scale, old)
                    s[b, h, t] = scale
                    for (to, _), row in zip(here, vals):
                        c[b, h, to] = kv8.codes(row, scale)
    return out
