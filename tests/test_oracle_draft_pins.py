"""Pins of the oracle for trees of drafted tokens: hand values, the law of accepted tokens, and
reductions to what is pinned already."""
from fractions import Fraction as Fr
from itertools import product

import numpy as np
import pytest

from oracle import draft, kv8

PARENTS = np.array([[-1, 0, 0, 1, 1, 2, 4]])


def test_what_nodes_see_by_hand():
    got = draft.sees(PARENTS, [6])
    want = [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {0, 1, 4}, {0, 2, 5}, set()]
    assert [set(np.flatnonzero(r)) for r in got[0]] == want
    assert draft.words(draft.sees(PARENTS))[0, :, 0].tolist() == [1, 3, 5, 11, 19, 37, 83]
    chain = np.arange(-1, 39)[None]
    w = draft.words(draft.sees(chain))
    assert w.shape == (1, 40, 2) and w[0, 39].tolist() == [0xFFFFFFFF, 0xFF] and w[0, 31].tolist() == [0xFFFFFFFF, 0]


def test_a_parent_that_is_no_lower_node_is_none():
    assert draft.ancestors([-1, 1, 5, -3, 3], 1) == {1}
    assert draft.ancestors([-1, 1, 5, -3, 3], 2) == {2}
    assert draft.ancestors([-1, 1, 5, -3, 3], 4) == {3, 4}


def test_keys_by_hand():
    assert draft.keys(6, 3, [True, False, True]) == [0, 1, 2, 3, 5]
    assert draft.keys(2, 3, [True, False, True]) == [1]              # base -1: node 0 has no place
    assert draft.keys(0, 0, []) == []


def _cache(rng, lengths, cap=48, d=8, block=16):
    B = len(lengths)
    c = {x + "8": kv8.codes(rng.normal(size=(B, 1, cap, d)) * 100, 1.0) for x in "kv"}
    c.update({x + "s": 2.0 ** rng.integers(-9, -5, size=(B, 1, cap // block)) for x in "kv"})
    c.update(w=rng.random((B, 1, cap)), lengths=np.array(lengths))
    return c


def test_a_chain_attends_as_under_the_causal_mask():
    rng = np.random.default_rng(1)
    c = _cache(rng, [30, 17, 3])
    q = rng.normal(size=(3, 2, 5, 8))
    chain = np.tile(np.arange(-1, 4), (3, 1))
    for counts in (None, [5, 2, 3]):
        a = draft.attend(c, q, 0.3, draft.sees(chain, counts), counts)
        b = kv8.attend(c, q, 0.3, counts, True)
        for x, y in zip(a[:4], b[:4]):
            assert np.allclose(x, y, rtol=1e-13, atol=1e-13)


def test_a_node_attends_as_its_branch_alone_would():
    """A node's row over the whole tree is the last row of a chain whose cache holds its branch only."""
    rng = np.random.default_rng(2)
    c = _cache(rng, [20])
    for x in "kv":
        c[x + "s"][:] = 2.0 ** -7
    q = rng.normal(size=(1, 1, 7, 8))
    O, L = draft.attend(c, q, 0.3, draft.sees(PARENTS))[:2]
    for i in range(7):
        at = list(range(13)) + [13 + a for a in sorted(draft.ancestors(PARENTS[0], i))]
        own = {x: c[x].copy() for x in c}
        for x in ("k8", "v8"):
            own[x][0, 0, :len(at)] = c[x][0, 0, at]
        own["lengths"] = np.array([len(at)])
        o, l = kv8.attend(own, q[:, :, i:i + 1], 0.3)[:2]
        assert np.allclose(o[0, 0, 0], O[0, 0, i], atol=1e-13) and np.allclose(l[0, 0, 0], L[0, 0, i], atol=1e-13)


def _law(p, q, k):
    """Exact probabilities of the token after the root, over k children drawn from q (None: children
    with the tokens of the first k values of p) and all their random numbers, by the refusals' own
    probabilities."""
    V = len(p)
    out = [Fr(0)] * V
    for xs in product(range(V), repeat=k) if q is not None else [tuple(range(k))]:
        chance = Fr(1)
        for x in xs:
            chance *= q[x] if q is not None else 1
        r, mass = list(p), Fr(1)
        for x in xs:
            if chance == 0:
                break
            yes = min(Fr(1), r[x] / mass / (q[x] if q is not None else 1))
            out[x] += chance * yes
            chance *= 1 - yes
            if q is not None:
                r = [max(a / mass - b, Fr(0)) for a, b in zip(r, q)]
                mass = sum(r) or Fr(1)
            else:
                mass -= r[x]
                r[x] = Fr(0)
        if chance:
            for v in range(V):
                out[v] += chance * r[v] / mass
    return out


@pytest.mark.parametrize("drawn", [True, False])
def test_tokens_follow_the_targets_probabilities(drawn):
    """The rule that the oracle follows leaves the target's law, whatever the number of children: in
    fractions; and the oracle follows it: its tokens over many random numbers, within 5 sigma."""
    p = [Fr(x, 64) for x in (30, 2, 20, 12)]
    q = [Fr(x, 64) for x in (10, 30, 4, 20)]
    for k in range(4):
        assert _law(p, q if drawn else None, k) == p
    rng = np.random.default_rng(3)
    N, n = 6000, 4
    target = np.tile([float(x) for x in p], (n, 1))
    given = np.tile([float(x) for x in q], (n, 1))
    hits = np.zeros(4)
    for _ in range(N):
        tokens = rng.choice(4, size=n, p=given[0]) if drawn else rng.permutation(4)
        path, token = draft.verify(target, given if drawn else None, tokens, [-1, 0, 0, 0],
                                   rng.random(n).astype(np.float32), n, exact=False)
        hits[tokens[path[1]] if len(path) > 1 else token] += 1
    want = np.array([float(x) for x in p])
    assert (np.abs(hits / N - want) <= 5 * np.sqrt(want * (1 - want) / N)).all(), hits / N


def test_verify_by_hand():
    p = np.array([[0.5, 0.25, 0.25], [0.0, 1.0, 0.0], [0.25, 0.25, 0.5]])
    q = np.array([[0.25, 0.5, 0.25], [0.5, 0.5, 0.0], [0.25, 0.25, 0.5]])
    up = [-1, 0, 0]
    call = lambda u, x=(0, 1, 0), d=q: draft.verify(p, d, x, up, np.array(u), 3)
    # Token 1 at node 1: p / q = 1/2, so u decides at 1/2 (not accepted at the border).
    assert call([0.0, 0.49, 0.0])[0] == [0, 1]
    # Refused: the residual is (1/4, 0, 0), so token 0 at node 2 has probability 1 of mass against 1/4.
    assert call([0.0, 0.5, 0.9]) == ([0, 2], 0)
    # Token 2 at node 2 has no residual: refused as well, and token 0 is all that is left.
    assert call([0.99, 0.5, 0.0], (0, 1, 2)) == ([0], 0)
    # After node 1 (token 0 accepted there): its own probabilities.
    assert call([0.99, 0.1, 0.0], (0, 0, 0)) == ([0, 1], 1)
    # Not drawn: token 1 is accepted below 1/4, then token 2 below 1/4 of the 3/4 left.
    assert call([0.0, 0.24, 0.0], (0, 1, 2), None)[0] == [0, 1]
    assert call([0.0, 0.25, 0.33], (0, 1, 2), None)[0] == [0, 2]
    assert call([0.99, 0.25, 0.34], (0, 1, 2), None) == ([0], 0)
    assert call([0.0, 0.25, 0.0], (0, 1, 1), None) == ([0], 0)        # the same token again
    assert call([0.67, 0.25, 0.99], (0, 1, 1), None) == ([0], 2)      # 2/3 of the mass 3/4 is token 0's


def test_verify_at_the_edges():
    p = np.array([[0.5, 0.5, 0.0]])
    assert draft.verify(p, None, [0], [-1], np.array([0.0]), 1) == ([0], 0)
    assert draft.verify(p, None, [0], [-1], np.array([0.5]), 1) == ([0], 1)     # the sum has to pass it
    assert draft.verify(p, None, [0], [-1], np.array([0.9999]), 1) == ([0], 1)
    assert draft.verify(p, None, [0], [-1], np.array([0.5]), 0) == ([], -1)
    assert draft.verify(np.zeros((1, 3)), None, [0], [-1], np.array([0.5]), 1) == ([0], -1)
    assert draft.verify(np.array([[np.nan, -1.0, 7.0]]), None, [0], [-1], np.array([0.5]), 1) == ([0], 2)
    # p equal to q: a refusal (of a token neither has) would leave nothing, and changes nothing.
    two = np.tile([[0.5, 0.5, 0.0]], (2, 1))
    assert draft.verify(two, two, [0, 2], [-1, 0], np.array([0.6, 0.0]), 2) == ([0], 1)
    # A token past the vocabulary is refused.
    assert draft.verify(two, two, [0, 9], [-1, 0], np.array([0.2, 0.0]), 2) == ([0], 0)
    assert draft.verify(two, None, [0, -1], [-1, 0], np.array([0.2, 0.0]), 2) == ([0], 0)


def test_one_number_holds_a_residual():
    """max(r - q, 0) over its mass, again and again, is max(p - S q, 0) over its own with S the sum of
    the masses W: in fractions."""
    rng = np.random.default_rng(4)
    for _ in range(50):
        p, q = ([Fr(int(x)) / int(sum(w)) for x in w] for w in rng.integers(1, 50, size=(2, 6)))
        r, S, W = list(p), Fr(0), Fr(1)
        for _ in range(5):
            left = [max(a - b, Fr(0)) for a, b in zip(r, q)]
            if sum(left) == 0:
                break
            r = [a / sum(left) for a in left]
            S += W
            t = [max(a - S * b, Fr(0)) for a, b in zip(p, q)]
            W = sum(t)
            assert [a / W for a in t] == r


def test_keep_by_hand():
    c = dict(k8=np.zeros((1, 1, 32, 64)), v8=np.zeros((1, 1, 32, 64)), ks=np.array([[[1.0, 4.0]]]),
             vs=np.array([[[1.0, 2.0 ** -4]]]), w=np.arange(32.0).reshape(1, 1, 32), lengths=np.array([18]))
    c["k8"][0, 0, :18] = np.arange(1, 19)[:, None]
    c["v8"][0, 0, :18] = np.arange(1, 19)[:, None]
    got = draft.keep(c, np.array([[0, 2, 3, -1]]), [3])               # base 14: tokens 14, 16, 17
    assert got["lengths"].tolist() == [17]
    # 17 * 4 and 18 * 4 go to positions 15 and 16; block 0 keeps its scale, block 1 gets its least.
    assert got["ks"][0, 0].tolist() == [1.0, 2.0 ** -2]
    assert got["k8"][0, 0, :18, 0].tolist() == list(range(1, 16)) + [64.0, 288.0, 18.0]  # 68 ties to 64
    assert got["vs"][0, 0].tolist() == [1.0, 2.0 ** -8]
    assert got["v8"][0, 0, 15:17, 0].tolist() == [1.0, 288.0]         # 17/16 ties to 1
    assert got["w"][0, 0, :18].tolist() == list(range(15)) + [16.0, 17.0, 17.0]


def test_keep_of_all_nodes_changes_nothing_but_scales():
    rng = np.random.default_rng(6)
    c = _cache(rng, [40, 9])
    got = draft.keep(c, np.tile(np.arange(8), (2, 1)), [8, 8])
    for x in "kv":
        was, now = (np.repeat(y[x + "s"], 16, -1)[..., None] * y[x + "8"] for y in (c, got))
        assert (was == now).all()
    assert got["lengths"].tolist() == [40, 9] and (got["w"] == c["w"]).all()


def test_keep_is_an_append_of_the_tokens_values():
    rng = np.random.default_rng(7)
    c = _cache(rng, [41, 12, 30])
    path = np.array([[0, 3, 4, 9, -1, -1, -1, -1, -1, -1], list(range(10)), [0] + [-1] * 9])
    got = draft.keep(c, path, [4, 10, 1])
    for b, acc in enumerate([4, 10, 1]):
        base = int(c["lengths"][b]) - 10
        one = {key: val[b:b + 1] for key, val in c.items()}
        one["lengths"] = np.array([base + acc])
        new = {x: (np.repeat(c[x + "s"], 16, -1)[..., None] * c[x + "8"])[b:b + 1, :, base + path[b, :acc]]
               for x in "kv"}
        ref = kv8.append(one, new["k"], new["v"])
        for x in ("k8", "v8", "ks", "vs"):
            assert (got[x][b] == ref[x][0]).all()
