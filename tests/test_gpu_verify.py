"""Verification of drafted tokens where what a refusal leaves is a small part of what it was taken from.

A node's state is S and W, the residual max(p - S q, 0) and its mass.  Where p lies next to S q, what is left
may be all in the last places that S q is rounded at.  Expected values are fractions, exact; the kernel's S
and W are pairs of float32, 2^-44 off at most here, so at residuals of 2^-30 of p and more a border is known
to 2^-14 of itself.  Random numbers stand at 2^-10 of a border and further.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import exact_io_aware_gb300 as ea
from test_gpu_draft import check_verify
from test_gpu_kv8 import i32, status

pytestmark = pytest.mark.gpu

F32 = np.float32
BELOW_ONE = np.nextafter(F32(1), F32(0))


def left(p, q, S):
    return max(Fraction(float(p)) - S * Fraction(float(q)), Fraction(0))


def after_refusals(p, q, k):
    """S and W after k refusals."""
    S, W = Fraction(0), Fraction(1)
    for _ in range(k):
        mass = sum(left(a, b, S + W) for a, b in zip(p, q))
        if mass > 0:
            S, W = S + W, mass
    return S, W


def accepted(p, q, tokens, u):
    """How many nodes are accepted of roots with the rows p and q [B, V] whose children hold tokens [B, n]."""
    (B, n), V = tokens.shape, p.shape[1]
    rows = [torch.from_numpy(x)[:, None].expand(B, n, V).contiguous().cuda() for x in (p, q)]
    got = ea.attn_draft_verify(*rows, i32(tokens), i32(np.tile(np.r_[-1, np.zeros(n - 1, int)], (B, 1))),
                               torch.from_numpy(u).cuda())
    return got[1].cpu().numpy()


def next_to_nothing(rng, N):
    """Rows p and q [N, 4] whose residual at token 0 after two refusals is what is left of p beside S q, at most
    2^-22 of it.  Token 3 has no probability: a child that holds it is refused."""
    P, Q = [], []
    while len(P) < N:
        q = np.array([rng.uniform(0.05, 0.6), rng.uniform(0.01, 0.2), rng.uniform(0.05, 0.3), rng.uniform(0.05, 0.2)], F32)
        p = np.array([0.0, q[1] * F32(rng.uniform(2, 4)), q[2] * F32(rng.uniform(0.1, 0.9)), 0.0], F32)
        at = float(q[0])
        p[0] = at * (1 + float(p[1]) - float(q[1]) - at) / (1 - at)   # p = S q, as S = 1 + sum max(p - q, 0)
        p[0] += F32(rng.integers(-3, 4)) * np.spacing(p[0])
        if not 0 < p[0] < 1:
            continue
        S, W = after_refusals(p, q, 2)
        t = left(p[0], q[0], S)
        if 2.0 ** -30 * p[0] <= t <= 2.0 ** -22 * p[0] and t < W:
            P.append(p), Q.append(q)
    return np.stack(P), np.stack(Q)


@pytest.mark.parametrize("V", [4, 20000])
def test_a_probability_next_to_what_was_refused(V):
    """A third child with S q rounded, or a neighbour, as its probability: accepted below the exact border,
    next to it and far from it."""
    rng = np.random.default_rng(31)
    few_p, few_q = next_to_nothing(rng, 60)
    border = []
    for a, b in zip(few_p, few_q):
        S, W = after_refusals(a, b, 2)
        border.append(float(left(a[0], b[0], S) / (Fraction(float(b[0])) * W)))
    p, q = np.zeros((60, V), F32), np.zeros((60, V), F32)
    p[:, [0, 1, 2, V - 1]], q[:, [0, 1, 2, V - 1]] = few_p, few_q
    tokens = np.tile([0, V - 1, V - 1, 0], (60, 1))
    u = rng.random((60, 4)).astype(F32)
    for f in (1 - 2.0 ** -10, 1 + 2.0 ** -10, 0.5, 2.0, 2.0 ** -6, 2.0 ** -12, 0.0):
        u[:, 3] = np.minimum(np.array(border) * f, BELOW_ONE)
        assert (accepted(p, q, tokens, u) == 1 + (u[:, 3] < border)).all(), f
        if V == 4:
            rows = [torch.from_numpy(x)[:, None].expand(60, 4, 4).contiguous() for x in (p, q)]
            check_verify(*rows, tokens, np.tile([-1, 0, 0, 0], (60, 1)), u, None, True)
    status()


def test_a_ratio_that_refusals_approach():
    """p = 1.5 q on half the vocabulary and 0.5 q on the other: each refusal takes S half the way that is left to
    1.5, down to where the residuals of all tokens are one rounding of S q.  Children of tokens whose own
    ratio is 1.5 but for a rounding tell the border."""
    rng = np.random.default_rng(33)
    odd = rng.uniform(1e-4, 1.1e-4, 60).astype(F32)
    q = np.concatenate([np.full(300, 1 / 310, F32), odd, [F32(0.01)]]).astype(F32)
    p = np.concatenate([F32(1.5) * q[:150], F32(0.5) * q[150:300], F32(1.5) * odd, [F32(0)]]).astype(F32)
    tokens, u, want, n = [], [], [], 28
    for k in range(22, 26):
        S, W = after_refusals(p, q, k)
        for x in range(300, 360):
            border = float(left(p[x], q[x], S) / (Fraction(float(q[x])) * W))
            if not 2.0 ** -4 < border < 1 - 2.0 ** -4:
                continue
            for f in (1 - 2.0 ** -8, 1 + 2.0 ** -8):
                tokens.append([0] + [360] * k + [x] + [360] * (n - k - 2))
                u.append([0.5] * n)
                u[-1][k + 1] = border * f
                want.append(2 if f < 1 else 1)
    assert {t.index(x) - 1 for t in tokens for x in t if 300 <= x < 360} >= {24, 25} and len(want) > 60
    B = len(want)
    got = accepted(np.tile(p, (B, 1)), np.tile(q, (B, 1)), np.array(tokens), np.array(u, F32))
    # (a node that was accepted is asked for children; there are none)
    assert (got == want).all(), np.argwhere(got != np.array(want))[:5].tolist()
    status()


@pytest.mark.parametrize("V,exact", [(24, True), (3000, False)])
def test_many_refusals(V, exact):
    """Rows whose ratios lie at 1.5 within 2^-24 to 2^-12 on half the vocabulary: up to 23 refusals, then six
    children of such tokens, against the oracle."""
    rng = np.random.default_rng(32)
    B, n = 48, 40
    q = rng.uniform(0.5, 1.5, (B, V))
    q /= q.sum(-1, keepdims=True)
    near = 1.5 + rng.choice([-1, 0, 1], (B, V)) * 2.0 ** rng.uniform(-24, -12, (B, V))
    p = q * np.where(np.arange(V) < V // 2, near, 0.5)
    q[:, V - 1], p[:, V - 1] = 0.01, 0.0                              # refused whatever the random number
    target, given = (torch.from_numpy(x).float()[:, None].expand(B, n, V).contiguous() for x in (p, q))
    k = rng.integers(1, 24, B)
    tokens = np.where(np.arange(n) <= k[:, None], V - 1, rng.integers(0, V // 2, (B, n)))
    seen = check_verify(target, given, tokens, np.tile(np.r_[-1, np.zeros(n - 1, int)], (B, 1)),
                        rng.random((B, n)).astype(F32), [int(x) + 7 for x in k], exact)
    assert len(seen) > 1 and status() == ea.ATTN_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_mass_of_a_long_row(dtype):
    """2^26 equal probabilities: what the additions round off all has one sign.  A sum is off by at most
    2^-42 + 2^26 2^-48 of mass 1; the border of a child of the residual, of mass 0.7, by less than 2^-21 of itself."""
    V = 1 << 26
    target, given = (torch.zeros(1, 3, V, dtype=dtype, device="cuda") for _ in range(2))
    target[0, 0] = 0.7 / V
    target[0, 0, 5], given[0, 0, 5], target[0, 0, 7] = 0.2, 0.1875, 0.0
    (a, p), q = (Fraction(x) for x in target[0, 0, 4:6].tolist()), Fraction(given[0, 0, 5].item())
    border = float((p - q) / (q * ((V - 2) * a + p - q)))
    for f in (1 - 2.0 ** -18, 1 - 2.0 ** -20, 1 - 2.0 ** -21, 1 + 2.0 ** -21, 1 + 2.0 ** -20, 1 + 2.0 ** -18):
        u = F32(border * f)
        got = ea.attn_draft_verify(target, given, i32([[0, 7, 5]]), i32([[-1, 0, 0]]),
                                   torch.tensor([[0.5, 0.5, float(u)]], device="cuda"))
        assert got[1].tolist() == [2 if float(u) < border else 1], f
    status()
