"""Decoding by a tree of drafted tokens on the GPU, against its oracle.

Words, accepted nodes, tokens, codes, scales, weights and lengths are whole decisions and must be equal.
The oracle decides in fractions or 64 bits; the kernel's sums hold 2^-40, and no drawn number lies that
near a border unless a test puts it there, where both are exact.  Attention is held to the bounds
counted in test_gpu_kv8.py.
"""
import numpy as np
import pytest
import torch

import exact_io_aware_gb300 as ea
from oracle import draft, kv8
from test_gpu_kv8 import DT, Cache, i32, rounded, status

pytestmark = pytest.mark.gpu

PROB = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def trees(rng, B, n, kind):
    """Parents [B, n]: chains, stars, or each node's parent at most `kind` nodes back."""
    up = np.full((B, n), -1)
    for i in range(1, n):
        if kind == "chain":
            up[:, i] = i - 1
        elif kind == "star":
            up[:, i] = 0
        else:
            up[:, i] = np.maximum(0, i - rng.integers(1, kind + 1, B))
    return up


def tree_words(seen):
    return torch.from_numpy(draft.words(seen).view(np.int32)).cuda()


# ------------------------------------------------------------------ the words

@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 65, 200, 1024])
@pytest.mark.parametrize("kind", ["chain", "star", 3, 50])
def test_tree_mask(n, kind):
    rng = np.random.default_rng(n)
    B = 5 if n < 1024 else 2
    up = trees(rng, B, n, kind)
    counts = None if n % 2 else [int(x) for x in rng.integers(0, n + 1, B)]
    if counts:
        counts[0] = 0
    got = ea.attn_tree_mask(i32(up), counts=i32(counts))
    want = draft.words(draft.sees(up, counts)).view(np.int32)
    assert (got.cpu().numpy() == want).all()
    assert status() == ea.ATTN_OK


def test_tree_mask_out_of_range():
    """Parents that are no lower node count as none; counts are clamped; both are told."""
    up = np.array([[-1, 0, 2, 1, 3, -5, 5], [-1, 0, 1, 9, 3, 1 << 30, 5], [3, 0, 1, 2, 3, 4, 5]])
    for b in range(3):
        got = ea.attn_tree_mask(i32(up[b:b + 1]))
        assert (got.cpu().numpy() == draft.words(draft.sees(up[b:b + 1])).view(np.int32)).all()
        assert status() == ea.ATTN_WARN_CLAMPED
    good = trees(np.random.default_rng(0), 2, 7, "chain")
    got = ea.attn_tree_mask(i32(good), counts=i32([-4, 100]))
    assert (got.cpu().numpy() == draft.words(draft.sees(good, [0, 7])).view(np.int32)).all()
    assert status() == ea.ATTN_WARN_CLAMPED
    # What padding nodes hold does not matter.
    up = np.array([[-1, 0, 99, -7]])
    got = ea.attn_tree_mask(i32(up), counts=i32([2]))
    assert got.cpu().numpy()[0, :, 0].tolist() == [1, 3, 0, 0] and status() == ea.ATTN_OK


# ------------------------------------------------------------------ attention

def check_attend(ca, q, c, dtype, o, lse, seen, counts=None):
    O, L, A, S, F = draft.attend(ca.c, q.double().numpy(), c, seen, counts)
    d, cap = q.shape[3], ca.k8.shape[2]
    ds = (d + 16) * 2.0 ** -23 * (S + 32.0)
    sums = (cap / 8 + 64) * 2.0 ** -24
    info = torch.finfo(DT[dtype])
    tol = (info.eps / 2 * np.abs(O) * (1 + 2.0 ** -6) + info.smallest_normal * info.eps / 2
           + (1 + 2.0 ** -6) * A * (2.0 ** -11 + 2 * ds[..., None] + 2 * sums) + 2.0 ** -31 * F)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(L)
    ltol = ds + sums + 2.0 ** -22 * (np.where(empty, 0, np.abs(L)) + 32.0)
    assert (np.isneginf(lse) == empty).all() and (o[empty] == 0).all()
    assert np.isfinite(o).all() and np.isfinite(lse[~empty]).all()
    bad = np.abs(o - O) > tol
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), (np.abs(o - O) / tol).max())
    lerr = np.abs(np.where(empty, 0.0, lse) - np.where(empty, 0.0, L))
    assert (lerr <= ltol).all(), (np.argwhere(lerr > ltol)[:4].tolist(), lerr.max())
    return L


@pytest.mark.parametrize("dtype,d,block", [("bf16", 128, 64), ("bf16", 64, 16), ("f16", 128, 16),
                                           ("f16", 64, 128), ("bf16", 128, 128)])
@pytest.mark.parametrize("G,n", [(1, 1), (1, 7), (3, 3), (2, 8), (5, 5), (1, 16), (1, 33), (8, 11), (4, 32), (4, 75),
                                 (9, 31)])
def test_attend(dtype, d, block, G, n):
    """Trees, and words that are no tree's (with rows that see nothing of it), at lengths around the
    kernels' steps and below the number of nodes."""
    lengths = [0, 1, 15, 16, 33, 127, 128, 129, 255, 384]
    B = len(lengths)
    rng = np.random.default_rng(G * 100 + n)
    ca = Cache(rng, lengths, 2, 384, d, block, pow2=G % 2 == 0)
    counts = [int(rng.integers(0, n + 1)) for _ in lengths] if n > 1 and G % 2 else None
    seen = draft.sees(trees(rng, B, n, 3), counts)
    odd = rng.random((B, n, n)) < 0.4
    odd[:, n // 2] = False
    q = rounded(rng.normal(size=(B, 2 * G, n, d)), dtype)
    for s in (seen, odd):
        o, lse = ea.attn_fwd_kv8_tree(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, tree_words(s), d ** -0.5,
                                      counts=i32(counts))
        L = check_attend(ca, q, d ** -0.5, dtype, o, lse, s, counts)
        real = np.arange(n) < np.array(counts if counts else [n] * B)[:, None]
        assert status() == (ea.ATTN_WARN_EMPTY_ROW if (np.isneginf(L) & real[:, None]).any() else ea.ATTN_OK)


@pytest.mark.parametrize("G,n,cap,lengths", [
    (4, 2, 8192, [8191, 5, 3000]),       # runs that end inside a tile
    (1, 8, 32768, [32768]),              # one head over many CTAs
    (8, 6, 4096, [4096, 4001, 77]),
    (2, 200, 1024, [1000, 201, 150]),    # trees over two blocks of 128 keys and more
    (1, 300, 768, [700, 300, 129]),      # no key before the tree; fewer keys than nodes
])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
def test_attend_long(dtype, d, G, n, cap, lengths):
    rng = np.random.default_rng(cap + G)
    ca = Cache(rng, lengths, 1 if cap > 8192 else 2, cap, d, 64)
    Hk, B = ca.k8.shape[1], len(lengths)
    q = rounded(rng.normal(size=(B, Hk * G, n, d)), dtype)
    up = trees(rng, B, n, 20)
    seen = draft.sees(up)
    tree = ea.attn_tree_mask(i32(up))
    args = (q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, tree, d ** -0.5)
    o, lse = ea.attn_fwd_kv8_tree(*args)
    check_attend(ca, q, d ** -0.5, dtype, o, lse, seen)
    again = ea.attn_fwd_kv8_tree(*args)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    status()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", [(1, 5), (4, 4), (2, 16), (8, 12), (8, 30)])
def test_a_chain_and_a_full_square_are_the_masks_that_there_were(dtype, d, G, n):
    """Bit for bit, at sizes whose work both divide alike (no tile is cut: caches of at most 512 tokens for few
    rows, two blocks of 128 keys for many): the same rows, keys and order of sums."""
    rng = np.random.default_rng(n)
    lengths = [200, 131, 256, 129, 224]
    ca = Cache(rng, lengths, 2, 384, d, 32)
    q = rounded(rng.normal(size=(5, 2 * G, n, d)), dtype).cuda()
    args = (ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths)
    chain = ea.attn_tree_mask(i32(trees(rng, 5, n, "chain")))
    square = torch.full((5, n, (n + 31) // 32), -1, dtype=torch.int32, device="cuda")
    for tree, mask in ((chain, "causal"), (square, "none")):
        a = ea.attn_fwd_kv8(q, *args, d ** -0.5, mask=mask)
        b = ea.attn_fwd_kv8_tree(q, *args, tree, d ** -0.5)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), mask


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", [(1, 5), (4, 4), (2, 16), (8, 12), (8, 30)])
def test_chains_and_full_squares_whose_tiles_are_cut(dtype, d, G, n):
    """At sizes whose work the two divide differently, so that sums may be in another order: both masks
    against the oracle."""
    rng = np.random.default_rng(n)
    lengths = [n, 100, 256, 1000, 131]
    ca = Cache(rng, lengths, 2, 1024, d, 32)
    q = rounded(rng.normal(size=(5, 2 * G, n, d)), dtype)
    for seen in (draft.sees(trees(rng, 5, n, "chain")), np.ones((5, n, n), bool)):
        o, lse = ea.attn_fwd_kv8_tree(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, tree_words(seen), d ** -0.5)
        check_attend(ca, q, d ** -0.5, dtype, o, lse, seen)
    status()


@pytest.mark.parametrize("G,n", [(2, 3), (1, 24), (4, 40)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_reaches_only_the_rows_that_see_it(d, G, n):
    rng = np.random.default_rng(13)
    m = 100
    ca = Cache(rng, [m], 1, 128, d, 16)
    up = trees(rng, 1, n, 4)
    seen = draft.sees(up)
    bad = [(m - 2, 3), (m - 2, d - 1), (m - n + n // 2, 8)]
    for key, col in bad:
        ca.c["v8"][0, 0, key, col] = np.nan
    ca.load()
    q = rounded(rng.normal(size=(1, G, n, d)), "f16")
    tree = tree_words(seen)
    o, lse = ea.attn_fwd_kv8_tree(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, tree, 0.1)
    want = np.zeros((1, G, n, d), bool)
    for i in range(n):
        for key, col in bad:
            want[0, :, i, col] |= seen[0, i, key - (m - n)]
    got = torch.isnan(o).cpu().numpy()
    assert (got == want).all(), np.argwhere(got != want)[:5].tolist()
    assert torch.isfinite(lse).all()
    # A NaN key makes the rows that see it NaN, and no others.
    ca.c["v8"][np.isnan(ca.c["v8"]) & (np.arange(128) < m)[None, None, :, None]] = 1.0
    ca.c["k8"][0, 0, m - 2, 0] = np.nan
    ca.load()
    o, lse = ea.attn_fwd_kv8_tree(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, tree, 0.1)
    sick = torch.from_numpy(seen[0, :, n - 2]).cuda()
    assert torch.isnan(o[:, :, sick]).all() and torch.isnan(lse[:, :, sick]).all()
    assert torch.isfinite(o[:, :, ~sick]).all() and torch.isfinite(lse[:, :, ~sick]).all()


@pytest.mark.parametrize("G,n", [(1, 5), (4, 60)])
def test_padding_nodes_do_not_matter(G, n):
    """Whatever the padding rows of q and of the words, and the bits past the count, hold."""
    rng = np.random.default_rng(G * n)
    counts = [1, n - 1, n // 2, 0, n]
    ca = Cache(rng, [384, 17, 200, 0, 129], 2, 384, 128, 64)
    seen = draft.sees(trees(rng, 5, n, 3), counts)
    q = rounded(rng.normal(size=(5, 2 * G, n, 128)), "bf16")
    pad = np.arange(n) >= np.array(counts)[:, None]
    q[torch.from_numpy(np.broadcast_to(pad[:, None, :, None], q.shape).copy())] = 0.0
    call = lambda x, s: ea.attn_fwd_kv8_tree(x.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, tree_words(s), 0.1,
                                             counts=i32(counts))
    o, lse = call(q, seen)
    check_attend(ca, q, 0.1, "bf16", o, lse, seen, counts)
    sick = q.clone()
    sick[torch.from_numpy(np.broadcast_to(pad[:, None, :, None], q.shape).copy())] = float("nan")
    more = seen | pad[:, None, :] | pad[:, :, None]
    o2, lse2 = call(sick, more)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    status()


@pytest.mark.parametrize("dtype,d,block", [("bf16", 128, 32), ("f16", 64, 64), ("bf16", 64, 16), ("f16", 128, 128)])
@pytest.mark.parametrize("G,n", [(4, 200), (1, 129), (6, 50), (2, 33)])
def test_rows_of_few_nodes_among_many(dtype, d, block, G, n):
    """Counts from none to all, so that the real rows fill other tiles than all rows would: real rows
    as the oracle's, padding rows 0 and -inf wherever they lie."""
    rng = np.random.default_rng(G + n)
    counts = [0, 1, n, n // 2, n - 1, 3, n // 3, 0, 17]
    lengths = [300, 1, 900, 257, n - 1, 640, 0, 0, 17]
    ca = Cache(rng, lengths, 2, 1024, d, block)
    seen = draft.sees(trees(rng, 9, n, 7), counts)
    q = rounded(rng.normal(size=(9, 2 * G, n, d)), dtype)
    o, lse = torch.full(q.shape, 7.0, dtype=DT[dtype], device="cuda"), torch.full(q.shape[:3], 7.0, device="cuda")
    ea.attn_fwd_kv8_tree(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, tree_words(seen), d ** -0.5,
                         counts=i32(counts), o=o, lse=lse)
    check_attend(ca, q, d ** -0.5, dtype, o, lse, seen, counts)
    assert status() == ea.ATTN_WARN_EMPTY_ROW                         # sequence 6 has nodes and no keys


@pytest.mark.parametrize("dtype,d,block", [("bf16", 128, 32), ("f16", 64, 64), ("bf16", 64, 16), ("f16", 128, 128)])
@pytest.mark.parametrize("B,G,n", [(9, 4, 4), (9, 5, 3), (90, 2, 8), (90, 1, 16), (230, 1, 5)])
def test_few_rows_of_few_nodes_among_many(dtype, d, block, B, G, n):
    """The same for few rows, in caches that are cut: fewer heads than CTAs, about as many, and more."""
    rng = np.random.default_rng(G + n)
    counts = [(0, 1, n, n // 2, n - 1, 3, 2, 0, n)[b % 9] for b in range(B)]
    lengths = [(300, 1, 900, 257, n - 1, 640, 0, 0, n)[b % 9] for b in range(B)]
    ca = Cache(rng, lengths, 2, 1024, d, block)
    seen = draft.sees(trees(rng, B, n, 7), counts)
    q = rounded(rng.normal(size=(B, 2 * G, n, d)), dtype)
    o, lse = torch.full(q.shape, 7.0, dtype=DT[dtype], device="cuda"), torch.full(q.shape[:3], 7.0, device="cuda")
    ea.attn_fwd_kv8_tree(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, tree_words(seen), d ** -0.5,
                         counts=i32(counts), o=o, lse=lse)
    some = np.r_[0:9, B - 9:B]
    sub = type("Sub", (), {})()
    sub.c, sub.k8 = {key: val[some] for key, val in ca.c.items()}, ca.k8
    check_attend(sub, q[some], d ** -0.5, dtype, o[some], lse[some], seen[some], [counts[b] for b in some])
    pad = torch.from_numpy(np.arange(n) >= np.array(counts)[:, None]).cuda()[:, None, :].expand(lse.shape)
    assert (o[pad] == 0).all() and torch.isneginf(lse[pad]).all() and torch.isfinite(o).all()
    assert status() == ea.ATTN_WARN_EMPTY_ROW                         # sequence 6 has nodes and no keys


@pytest.mark.parametrize("B,G,n,lengths", [
    (100, 1, 4, [320]),             # more heads than CTAs, all alike: whole heads a CTA
    (100, 8, 5, [320]),
    (30, 8, 5, [320]),              # as many as CTAs, nearly
    (7, 8, 40, [1100]),             # equal parts of a head
    (7, 2, 4, [1100]),
    (11, 3, 50, [1100, 700, 130]),  # parts of unequal heads
    (40, 2, 3, [1100, 20, 600]),
])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
def test_every_way_work_is_divided(dtype, d, B, G, n, lengths):
    """Heads that CTAs take whole, in parts, or in runs across them: some sequences against the oracle, and
    the whole call the same once more."""
    rng = np.random.default_rng(B + G + n)
    lengths = [lengths[b % len(lengths)] for b in range(B)]
    ca = Cache(rng, lengths, 5, 1152 if max(lengths) > 320 else 640, d, 64)
    seen = draft.sees(trees(rng, B, n, 4))
    q = rounded(rng.normal(size=(B, 5 * G, n, d)), dtype)
    args = (q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, tree_words(seen), d ** -0.5)
    o, lse = ea.attn_fwd_kv8_tree(*args)
    again = ea.attn_fwd_kv8_tree(*args)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    some = rng.choice(B, min(B, 7), replace=False)
    sub = type("Sub", (), {})()
    sub.c, sub.k8 = {key: val[some] for key, val in ca.c.items()}, ca.k8
    check_attend(sub, q[some], d ** -0.5, dtype, o[some], lse[some], seen[some])
    assert torch.isfinite(o).all() and torch.isfinite(lse).all() and status() == ea.ATTN_OK


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,most", [(150, 140), (60, 1500)])
def test_tiles_of_more_and_of_fewer_real_rows_in_turn(dtype, B, most):
    """Many tiles in each CTA's run, of up to 180 real rows: with more than 128 and with fewer, whole and cut,
    some ending in a NaN value, some with nothing to see."""
    rng = np.random.default_rng(B)
    Hk, G, n, d = 5, 3, 60, 64
    lengths = [int(x) for x in rng.integers(0, most, B)]
    counts = [min(int(x), m) for x, m in zip(rng.integers(0, n + 1, B), lengths)]
    ca = Cache(rng, lengths, Hk, 1536, d, 32)
    seen = draft.sees(trees(rng, B, n, 9), counts)
    sick = [b for b in range(B) if b % 7 == 3 and counts[b] > 2]
    for b in sick:
        ca.c["v8"][b, :, lengths[b] - 1, 5] = np.nan                  # the last node's: a leaf
    ca.load()
    q = rounded(rng.normal(size=(B, Hk * G, n, d)), dtype)
    args = (q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, tree_words(seen), 0.125)
    o, lse = ea.attn_fwd_kv8_tree(*args, counts=i32(counts))
    again = ea.attn_fwd_kv8_tree(*args, counts=i32(counts))
    assert torch.equal(o.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])
    want = np.zeros(o.shape, bool)
    for b in sick:
        want[b, :, counts[b] - 1, 5] = True
    nan = torch.isnan(o).cpu().numpy()
    assert (nan == want).all(), np.argwhere(nan != want)[:5].tolist()
    for b in sick:
        ca.c["v8"][b, :, lengths[b] - 1, 5] = 0.0
    some = rng.choice(B, 10, replace=False)
    sub = type("Sub", (), {})()
    sub.c, sub.k8 = {key: val[some] for key, val in ca.c.items()}, ca.k8
    o2 = o[some].clone()
    O = draft.attend(sub.c, q[some].double().numpy(), 0.125, seen[some], [counts[b] for b in some])[0]
    fix = torch.from_numpy(want[some]).cuda()
    o2[fix] = torch.from_numpy(O).to(o2)[fix]
    check_attend(sub, q[some], 0.125, dtype, o2, lse[some], seen[some], [counts[b] for b in some])
    status()


def test_attend_clamps_and_tells():
    rng = np.random.default_rng(4)
    ca = Cache(rng, [32, 0, 20], 2, 32, 64, 16)
    seen = draft.sees(trees(rng, 3, 4, 2))
    q = rounded(rng.normal(size=(3, 2, 4, 64)), "f16")
    o, lse = ea.attn_fwd_kv8_tree(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, i32([40, -3, 20]), tree_words(seen), 0.1,
                                  counts=i32([4, 0, 9]))
    assert status() == ea.ATTN_WARN_CLAMPED
    check_attend(ca, q, 0.1, "f16", o, lse, seen, [4, 0, 4])


# ------------------------------------------------------------------ verification

def distributions(rng, shape, sharp, dtype):
    x = np.exp(sharp * rng.normal(size=shape))
    return torch.from_numpy(x / x.sum(-1, keepdims=True)).to(PROB[dtype])


def check_verify(target, given, tokens, up, u, counts, exact):
    got = ea.attn_draft_verify(target.cuda(), None if given is None else given.cuda(), i32(tokens), i32(up),
                               torch.from_numpy(u).cuda(), counts=i32(counts))
    path, accepted, token = (x.cpu().numpy() for x in got)
    t, q = target.double().numpy(), None if given is None else given.double().numpy()
    B, n = up.shape
    seen = set()
    for b in range(B):
        want, after = draft.verify(t[b], None if q is None else q[b], tokens[b], up[b], u[b],
                                   n if counts is None else counts[b], exact=exact)
        assert path[b].tolist() == want + [-1] * (n - len(want)), (b, want)
        assert accepted[b] == len(want) and token[b] == after, (b, token[b], after)
        seen.add(len(want))
    return seen


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V,n,kind", [(1, 3, 2), (2, 5, 3), (7, 1, 1), (7, 12, 4), (31, 8, "star"), (127, 9, "chain"),
                                      (129, 40, 6)])
def test_verify(dtype, drawn, V, n, kind):
    """Against fractions: small vocabularies, whose tokens come up again among a node's children."""
    rng = np.random.default_rng(V * n)
    B = 24
    up = trees(rng, B, n, kind)
    target, given = distributions(rng, (B, n, V), 1.0, dtype), distributions(rng, (B, n, V), 1.0, dtype)
    tokens = rng.integers(0, V, (B, n))
    counts = [int(x) for x in rng.integers(0, n + 1, B)] if n % 2 else None
    seen = check_verify(target, given if drawn else None, tokens, up, rng.random((B, n)).astype(np.float32), counts,
                        True)
    # (one of 129 tokens chosen at random is hardly ever accepted)
    assert V == 1 or n == 1 or len(seen) > 1 or (V == 129 and not drawn)
    assert status() == ea.ATTN_OK


@pytest.mark.parametrize("dtype,V,n", [("f32", 1001, 6), ("f32", 33333, 5), ("bf16", 4099, 7), ("f16", 100003, 4),
                                       ("f32", 131072, 3), ("bf16", 16, 70)])
@pytest.mark.parametrize("drawn", [True, False])
def test_verify_large_vocabularies(dtype, V, n, drawn):
    """Rows that start at every place of a 16-byte piece, shares of one warp to eight CTAs."""
    rng = np.random.default_rng(V + n)
    B = 3 if V > 2000 else 8
    up = trees(rng, B, n, 3)
    target = distributions(rng, (B, n, V), 2.0, dtype)
    given = torch.softmax(target.double().log() + 0.7 * torch.from_numpy(rng.normal(size=(B, n, V))), -1).to(PROB[dtype])
    tokens = np.zeros((B, n), int)
    for b in range(B):
        for i in range(1, n):
            p = given[b, up[b, i]].double().numpy()
            tokens[b, i] = min(V - 1, np.searchsorted(np.cumsum(p / p.sum()), rng.random()))
    for _ in range(2):
        check_verify(target, given if drawn else None, tokens, up, rng.random((B, n)).astype(np.float32), None, False)
    assert status() == ea.ATTN_OK


def test_verify_at_borders():
    """Random numbers on the borders themselves, where every value is exact: equality is refused, and the
    sum has to pass the drawn number."""
    p = torch.tensor([[0.5, 0.25, 0.25], [0.0, 1.0, 0.0], [0.25, 0.25, 0.5]])
    q = torch.tensor([[0.25, 0.5, 0.25], [0.5, 0.5, 0.0], [0.25, 0.25, 0.5]])
    up = np.array([[-1, 0, 0]])
    below = np.nextafter(np.float32(0.5), np.float32(0))
    for tokens in ([0, 1, 0], [0, 1, 2], [0, 0, 0], [0, 1, 1], [0, 2, 2]):
        for u in ([0.0, 0.5, 0.5], [0.5, below, 0.25], [0.75, 0.5, below], [0.25, 0.25, 1 / 3], [0.5, 0.75, 0.99],
                  [np.nextafter(np.float32(1), np.float32(0)), 0.5, 0.99], [0.0, 0.0, 0.0]):
            for given in (q, None):
                check_verify(p[None], given if given is None else given[None], np.array([tokens]), up,
                             np.array([u], np.float32), None, True)
    assert status() == ea.ATTN_OK


def test_verify_strange_probabilities():
    """NaN, negative and large values, zeros, rows that are equal, or sum to more or less than 1."""
    rng = np.random.default_rng(9)
    B, n, V = 40, 6, 11
    up = trees(rng, B, n, 3)
    x = rng.choice([0.0, 0.0, 0.125, 0.25, 0.5, 1.0, 3.0, -2.0, np.nan, np.inf, 1e-40], size=(2, B, n, V))
    x[1, :10] = x[0, :10]
    target, given = (torch.from_numpy(y).float() for y in x)
    target[20:24] = 0.0
    tokens, u = rng.integers(0, V, (B, n)), rng.random((B, n)).astype(np.float32)
    for g in (given, None):
        check_verify(target, g, tokens, up, u, None, True)
    assert status() == ea.ATTN_WARN_EMPTY_ROW


def test_verify_out_of_range():
    """Tokens past the vocabulary, parents that are no lower node, counts outside their range."""
    rng = np.random.default_rng(10)
    target, given = distributions(rng, (4, 5, 9), 1.0, "f32"), distributions(rng, (4, 5, 9), 1.0, "f32")
    up, u = trees(rng, 4, 5, "star"), np.zeros((4, 5), np.float32)
    tokens = rng.integers(0, 9, (4, 5))
    tokens[1, 1], tokens[2, 2], tokens[3, 3] = 9, -1, 1 << 30
    u[1:, 1] = u[1:, 2] = 0.999
    for g in (given, None):
        check_verify(target, g, tokens, up, u, None, True)
        assert status() == ea.ATTN_WARN_CLAMPED
    tokens %= 9
    for bad in (-2, 4, 77):
        up[2, 4] = bad
        check_verify(target, given, tokens, np.where((up < 0) | (up >= np.arange(5)), -1, up), u, None, True)
        status()
        got = ea.attn_draft_verify(target.cuda(), given.cuda(), i32(tokens), i32(up), torch.from_numpy(u).cuda())
        want = ea.attn_draft_verify(target.cuda(), given.cuda(), i32(tokens),
                                    i32(np.where((up < 0) | (up >= np.arange(5)), -1, up)), torch.from_numpy(u).cuda())
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and status() == ea.ATTN_WARN_CLAMPED
    up = trees(rng, 4, 5, "star")
    got = ea.attn_draft_verify(target.cuda(), given.cuda(), i32(tokens), i32(up), torch.from_numpy(u).cuda(),
                               counts=i32([-1, 9, 3, 0]))
    assert got[1].tolist()[0] == 0 and got[2].tolist()[0] == -1 and got[2].tolist()[3] == -1
    assert status() == ea.ATTN_WARN_CLAMPED


@pytest.mark.parametrize("drawn", [True, False])
def test_tokens_follow_the_targets_probabilities(drawn):
    """The first token after the root over 2^16 sequences with drafts of their own: each value's share
    within 5 sigma of its probability."""
    rng = np.random.default_rng(11)
    B, V, n = 1 << 16, 8, 4
    p, q = (x / x.sum() for x in np.exp(rng.normal(size=(2, V))).astype(np.float32))
    tokens = np.stack([rng.choice(V, n, p=q.astype(np.float64) / q.astype(np.float64).sum()) for _ in range(B)]) \
        if drawn else np.argsort(rng.random((B, V)), 1)[:, :n]
    rep = lambda x: torch.from_numpy(np.broadcast_to(x, (B, n, V)).copy()).cuda()
    path, accepted, token = ea.attn_draft_verify(rep(p), rep(q) if drawn else None, i32(tokens),
                                                 i32(np.tile([-1, 0, 0, 0], (B, 1))),
                                                 torch.from_numpy(rng.random((B, n)).astype(np.float32)).cuda())
    path, accepted, token = path.cpu().numpy(), accepted.cpu().numpy(), token.cpu().numpy()
    first = np.where(accepted > 1, tokens[np.arange(B), np.maximum(path[:, 1], 0)], token)
    share = np.bincount(first, minlength=V) / B
    want = p.astype(np.float64)
    assert (np.abs(share - want) <= 5 * np.sqrt(want * (1 - want) / B)).all(), (share, want)
    if drawn:
        assert (accepted > 1).mean() > 0.5
    else:  # a token is among three of eight chosen at random in 3/8 of the sequences, and then accepted by p
        assert abs((accepted > 1).mean() - 0.375) <= 5 * 0.5 / 256


def test_verify_deep_and_many():
    """1024 nodes, some accepted all the way down a chain; and more sequences than clusters at once."""
    rng = np.random.default_rng(12)
    n, V = 1024, 5
    up = trees(rng, 3, n, "chain")
    up[1] = trees(rng, 1, n, 2)[0]
    up[2] = trees(rng, 1, n, "star")[0]
    target = distributions(rng, (3, n, V), 0.5, "f32")
    tokens = rng.integers(0, V, (3, n))
    tokens[2] = 0
    target[2, 0] = torch.tensor([0.0, 0.5, 0.0, 0.5, 0.0])
    u = np.zeros((3, n), np.float32)
    u[1:] = rng.random((2, n))
    u[1] *= 0.2
    for given in (target, None):
        check_verify(target, given, tokens, up, u, None, False)
    up = trees(rng, 700, 4, 2)
    target = distributions(rng, (700, 4, 300), 1.0, "bf16")
    check_verify(target, target.roll(1, 0), rng.integers(0, 300, (700, 4)), up,
                 rng.random((700, 4)).astype(np.float32), None, False)


# ------------------------------------------------------------------ the cache of the accepted nodes

def paths(rng, up, counts):
    """A random node's branch in each sequence: [B, n] and how many."""
    B, n = up.shape
    path, acc = np.full((B, n), -1), np.zeros(B, int)
    for b in range(B):
        if counts[b] > 0:
            at = sorted(draft.ancestors(up[b], int(rng.integers(0, counts[b]))))
            path[b, :len(at)], acc[b] = at, len(at)
    return path, acc


def check_keep(ca, path, acc, counts, weights=True):
    ref = draft.keep(ca.c, path, acc, counts)
    got = ea.attn_kv8_keep(ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, i32(path), i32(acc), counts=i32(counts),
                           weights=ca.w if weights else None)
    if not weights:
        ref["w"] = ca.c["w"]
    assert ca.lengths.tolist() == list(ca.c["lengths"])               # an input
    assert got.tolist() == list(ref["lengths"])
    ca.lengths = got
    ca.check(ref)
    return ref


@pytest.mark.parametrize("d,block", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("n,kind,lengths", [
    (1, 1, [1, 17, 128, 300]),
    (6, 3, [6, 16, 129, 383]),
    (26, 6, [27, 129, 140, 384]),
    (33, "chain", [33, 64, 150, 290]),
    (200, 5, [200, 329, 384, 257]),
    (260, "chain", [261, 300, 384, 383]),
])
def test_keep(d, block, n, kind, lengths):
    rng = np.random.default_rng(n + d + block)
    ca = Cache(rng, lengths, 2, 384, d, block)
    up = trees(rng, 4, n, kind)
    counts = None if n % 2 else [n, n // 2, max(1, n - 1), 0]
    path, acc = paths(rng, up, counts or [n] * 4)
    if kind == "chain":
        path[0, :n], acc[0] = np.arange(n), n                         # all of them
    check_keep(ca, path, acc, counts, weights=n != 6)
    assert status() == ea.ATTN_OK


def test_keep_scales_far_apart():
    """Moved tokens that make their block's scale grow or shrink, at both ends of the scales' range, with
    zeros and NaN among them."""
    rng = np.random.default_rng(23)
    for low, high in ((-100, -60), (-20, 20), (80, 121)):
        ca = Cache(rng, [60, 64, 33, 50], 2, 64, 64, 16)
        for x in "kv":
            ca.c[x + "s"] = 2.0 ** rng.integers(low, high, size=ca.c[x + "s"].shape).astype(np.float64)
            c = ca.c[x + "8"]
            c[rng.random(c.shape[:3]) < 0.2] = 0.0
            small = rng.random(c.shape) < 0.1
            c[small] = kv8.codes(c[small] * 2.0 ** -9, 1.0)
            c[0, 0, 50:, 3] = np.nan
        ca.load()
        up = trees(rng, 4, 30, 4)
        path, acc = paths(rng, up, [30] * 4)
        check_keep(ca, path, acc, None)
        assert status() == ea.ATTN_OK


def test_keep_out_of_range():
    """Entries below their place or past the tree, counts and `accepted` outside their range, a tree longer
    than its sequence: clamped, and told."""
    rng = np.random.default_rng(24)
    path = np.array([[0, 0, 9, 3, -1, 2], [5, 1, 1, 4, 2, 0], [0, 2, 3, 4, 5, -1], [0, 1, 2, 3, 4, 5]])
    ca = Cache(rng, [40, 30, 4, 20], 2, 64, 64, 16)
    check_keep(ca, path, np.array([6, 6, 5, 9]), None)
    assert status() == ea.ATTN_WARN_CLAMPED
    ca = Cache(rng, [40, 30, 4, 0], 2, 64, 64, 16)
    check_keep(ca, path, np.array([-1, 0, 1, 6]), None)
    assert status() == ea.ATTN_WARN_CLAMPED
    ca = Cache(rng, [40, 30, 4, 20], 2, 64, 64, 16)
    ca.lengths = i32([90, -5, 4, 20])
    ref = dict(ca.c)
    ref["lengths"] = np.array([64, 0, 4, 20])
    # (the first sequence's tokens up to 64 are poison: none is accepted there)
    want = draft.keep(ref, path, [0, 0, 2, 3], [6, 6, 6, 0])
    got = ea.attn_kv8_keep(ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, i32(path), i32([0, 0, 2, 3]),
                           counts=i32([7, 6, 6, -1]), weights=ca.w)
    assert status() == ea.ATTN_WARN_CLAMPED
    ca.lengths = got
    ca.check(want)


# ------------------------------------------------------------------ as they are used

class Round:
    """A decoding round: tree mask, append, attention, verification, the cache of the accepted nodes."""

    def __init__(self, rng, B, Hk, G, n, d, cap, block, V, lengths):
        self.B, self.n, self.V, self.d = B, n, V, d
        self.ca = Cache(rng, lengths, Hk, cap, d, block)
        bf = torch.bfloat16
        self.k, self.v = (torch.zeros(B, Hk, n, d, dtype=bf, device="cuda") for _ in range(2))
        self.q = torch.zeros(B, Hk * G, n, d, dtype=bf, device="cuda")
        self.target, self.given = (torch.zeros(B, n, V, device="cuda") for _ in range(2))
        self.tokens, self.parents = (torch.zeros(B, n, dtype=torch.int32, device="cuda") for _ in range(2))
        self.counts = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.uniforms = torch.zeros(B, n, device="cuda")
        self.tree = torch.zeros(B, n, (n + 31) // 32, dtype=torch.int32, device="cuda")
        self.o, self.lse = torch.empty_like(self.q), torch.empty(B, Hk * G, n, device="cuda")
        self.ws = torch.empty(max(16, ea.attn_fwd_kv8_workspace_bytes(bf, B, Hk * G, Hk, n, d, cap)), dtype=torch.uint8,
                              device="cuda")
        self.path = torch.empty(B, n, dtype=torch.int32, device="cuda")
        self.accepted, self.token = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
        self.kept = torch.empty_like(self.counts)

    def fill(self, rng):
        self.up = trees(rng, self.B, self.n, 3)
        self.cnt = [int(x) for x in rng.integers(1, self.n + 1, self.B)]
        self.x = [rounded(rng.normal(size=t.shape), "bf16") for t in (self.k, self.v, self.q)]
        self.p = [distributions(rng, (self.B, self.n, self.V), 1.0, "f32") for _ in range(2)]
        self.tok = rng.integers(0, self.V, (self.B, self.n))
        self.u = rng.random((self.B, self.n)).astype(np.float32)
        for t, x in zip((self.k, self.v, self.q, self.target, self.given, self.tokens, self.parents, self.counts, self.uniforms),
                        (*self.x, *self.p, i32(self.tok), i32(self.up), i32(self.cnt), torch.from_numpy(self.u))):
            t.copy_(x)

    def run(self):
        ca = self.ca
        ca.lengths.add_(self.counts)
        ea.attn_tree_mask(self.parents, counts=self.counts, tree=self.tree)
        ea.attn_kv8_append(self.k, self.v, ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, counts=self.counts, weights=ca.w)
        ea.attn_fwd_kv8_tree(self.q, ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, self.tree, 0.125, counts=self.counts,
                             o=self.o, lse=self.lse, workspace=self.ws)
        ea.attn_draft_verify(self.target, self.given, self.tokens, self.parents, self.uniforms, counts=self.counts,
                             path=self.path, accepted=self.accepted, next_token=self.token)
        ea.attn_kv8_keep(ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, self.path, self.accepted, counts=self.counts,
                         weights=ca.w, lengths_out=self.kept)
        ca.lengths.copy_(self.kept)

    def check(self):
        ca = self.ca
        ca.c["lengths"] = ca.c["lengths"] + np.array(self.cnt)
        ca.c = kv8.append(ca.c, self.x[0].double().numpy(), self.x[1].double().numpy(), self.cnt)
        seen = draft.sees(self.up, self.cnt)
        check_attend(ca, self.x[2], 0.125, "bf16", self.o, self.lse, seen, self.cnt)
        path, acc = self.path.cpu().numpy(), self.accepted.tolist()
        for b in range(self.B):
            want, after = draft.verify(self.p[0][b].double().numpy(), self.p[1][b].double().numpy(), self.tok[b],
                                       self.up[b], self.u[b], self.cnt[b], exact=False)
            assert path[b, :acc[b]].tolist() == want and self.token[b].item() == after
        ca.c = draft.keep(ca.c, path, acc, self.cnt)
        ca.check(ca.c)


@pytest.mark.parametrize("captured", [False, True])
def test_rounds_over_one_cache(captured):
    """Rounds with trees, counts and lengths of their own, the cache carried along with the oracle's; as
    calls, and as two captured graphs replayed in turn."""
    rng = np.random.default_rng(71)
    r = Round(rng, 3, 2, 4, 9, 64, 256, 32, 50, [40, 100, 0])
    if not captured:
        for _ in range(8):
            r.fill(rng)
            r.run()
            r.check()
        assert status() == ea.ATTN_OK
        return
    start = r.ca.lengths.clone()
    r.fill(rng)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.run()
    torch.cuda.current_stream().wait_stream(side)
    r.ca.load()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            r.run()
    r.ca.lengths.copy_(start)
    for i in range(6):
        r.fill(rng)
        graphs[i % 2].replay()
        r.check()
    assert status() == ea.ATTN_OK


def test_weights_of_the_accepted_nodes():
    """After a round the accepted rows, gathered by their path, are the causal rows of the kept cache: their
    LSE is that of the tree's call where no scale moved, and their weights add up to one a row."""
    rng = np.random.default_rng(72)
    r = Round(rng, 2, 2, 2, 6, 128, 128, 32, 20, [50, 64])
    r.fill(rng)
    r.run()
    r.check()
    ca, acc = r.ca, r.accepted
    at = r.path.clamp(min=0).long()[:, None, :, None].expand(-1, 4, -1, 128)
    q = r.q.gather(2, at).contiguous()
    o, lse = ea.attn_fwd_kv8(q, ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.125, counts=acc, mask="causal")
    w = ea.attn_kv8_weights(q, ca.k8, ca.ks, ca.lengths, lse, None, 0.125, counts=acc, mask="causal")
    # A row's weights sum to 1 within (d + 16) 2^-23 (c sum |q k| + 32), c sum |q k| below 32 here, and sums.
    assert ((w.sum(-1) / (2.0 * acc[:, None])) - 1).abs().max() <= 2.0 ** -9
    old = r.lse.gather(2, at[..., 0])
    real = torch.arange(6, device="cuda") < acc[:, None]
    # A key requantized twice differs by half an E4M3 step, 2^-4 of its values: |ds| <= 2^-4 c |q| |k|.
    bound = 2.0 ** -4 * 0.125 * q.float().norm(dim=-1).max() * (ca.k8.float().nan_to_num() * ca.ks.nan_to_num(
        ).repeat_interleave(32, -1)[..., None]).norm(dim=-1).max()
    assert (lse - old).abs()[real[:, None].expand(-1, 4, -1)].max() <= bound


def test_calls_on_two_streams_at_once():
    rng = np.random.default_rng(51)
    ca = Cache(rng, [3000, 2500], 4, 4096, 128, 64)
    qs = [rounded(rng.normal(size=(2, 16, 5, 128)), "bf16").cuda() for _ in range(2)]
    tree = ea.attn_tree_mask(i32(trees(rng, 2, 5, 2)))
    target = [distributions(rng, (2, 5, 40000), 1.0, "f32").cuda() for _ in range(2)]
    tokens, up, u = i32(rng.integers(0, 40000, (2, 5))), i32(trees(rng, 2, 5, 2)), torch.rand(2, 5, device="cuda")
    call = lambda i, s=None: (*ea.attn_fwd_kv8_tree(qs[i], ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, tree, 0.1, stream=s),
                              *ea.attn_draft_verify(target[i], target[1 - i], tokens, up, u, stream=s))
    want = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [call(i, s) for i, s in enumerate(streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_past_32_bits():
    """Probabilities past 2^31 bytes and 2^31 values; a tree at the end of a cache past 2^31 bytes."""
    B, n, V = 9, 16, 1 << 24
    target = torch.zeros(B, n, V, dtype=torch.bfloat16, device="cuda")
    target[:, :, 5] = 0.5
    target[:, :, V - 1] = 0.5
    up, u = np.tile(np.arange(-1, n - 1), (B, 1)), torch.full((B, n), 0.75, device="cuda")
    tokens = torch.full((B, n), V - 1, dtype=torch.int32, device="cuda")
    u[:, 1:] = 0.25
    path, accepted, token = ea.attn_draft_verify(target, None, tokens, i32(up), u)
    assert accepted.tolist() == [n] * B and token.tolist() == [V - 1] * B
    path, accepted, token = ea.attn_draft_verify(target, target, tokens, i32(up), u)
    assert accepted.tolist() == [n] * B and token.tolist() == [V - 1] * B
    del target
    cap = (1 << 24) + 256
    k8 = torch.zeros(1, 1, cap, 128, dtype=torch.uint8, device="cuda")
    v8 = torch.full((1, 1, cap, 128), 0x38, dtype=torch.uint8, device="cuda")    # 1.0
    v8[0, 0, -2] = 0x7E                                                          # 448
    ks, vs = (torch.ones(1, 1, cap // 128, device="cuda") for _ in range(2))
    ks[0, 0, -1] = 1.0
    lens = i32([cap])
    q = torch.ones(1, 1, 3, 128, dtype=torch.bfloat16, device="cuda")
    k8[0, 0, -3:] = 0x48                                                         # 4.0: scores of 512 c
    tree = ea.attn_tree_mask(i32([[-1, 0, 0]]))
    o, lse = ea.attn_fwd_kv8_tree(q, k8, v8, ks, vs, lens, tree, 1.0)
    # The nodes' own keys outweigh all others (e^512): their values alone, node 1's of 448.
    assert o[0, 0, :, 0].tolist() == [1.0, 224.0, 1.0]                           # 224.5 rounds to even
    w = torch.zeros(1, 1, cap, device="cuda")
    w[0, 0, -2:] = torch.tensor([3.0, 7.0], device="cuda")
    new = ea.attn_kv8_keep(k8, v8, ks, vs, lens, i32([[0, 2, -1]]), i32([2]), weights=w)
    assert new.tolist() == [cap - 1] and w[0, 0, -3:].tolist() == [0.0, 7.0, 7.0]
    assert (v8[0, 0, -2:] == 0x38).all()


def test_runner(capsys):
    import json

    from exact_io_aware_gb300 import run

    rc = run.main("--kv8-tree --B 2 --H 8 --H-kv 2 --n 9 --n-kv 700 --d 64 --vocab 1000 --iters 2 --json".split())
    out = json.loads(capsys.readouterr().out)
    assert rc == 0 and all(out[f"{x}_us"] > 0 for x in ("mask", "append", "attend", "verify", "keep"))
