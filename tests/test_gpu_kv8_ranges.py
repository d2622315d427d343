"""The 8-bit cache's attention and weights over the whole range of values their inputs may have.

Bounds are those of test_gpu_kv8.py (counted from the roundings there), with a term of its own
where a test says so.
"""
import numpy as np
import pytest
import torch

import exact_io_aware_gb300 as ea
from oracle import kv8
from test_gpu_kv8 import DT, Cache, attend_bounds, check_attend, i32, rounded, status

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ padding rows

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,G,n", [(128, 1, 5), (128, 3, 5), (64, 4, 8), (128, 8, 6), (64, 5, 60)])
@pytest.mark.parametrize("cap", [384, 1024])
def test_what_padding_rows_hold_does_not_matter(dtype, d, G, n, cap):
    """Real rows come out bit for bit alike whatever the padding rows of q hold."""
    rng = np.random.default_rng(G * n)
    lengths = [cap, 17, 200, 0, 129]
    counts = [1, n - 1, n // 2, 0, n]
    ca = Cache(rng, lengths, 2, cap, d, 64)
    q = rounded(rng.normal(size=(5, 2 * G, n, d)), dtype)
    pad = (np.arange(n) >= np.array(counts)[:, None])[:, None, :, None]
    pad = torch.from_numpy(np.broadcast_to(pad, q.shape).copy())
    q[pad] = 0.0
    kw = dict(counts=i32(counts), mask="causal")
    args = (ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, d ** -0.5)
    o, lse = ea.attn_fwd_kv8(q.cuda(), *args, **kw)
    check_attend(ca, q, d ** -0.5, dtype, o, lse, counts, True)
    w = ea.attn_kv8_weights(q.cuda(), ca.k8, ca.ks, ca.lengths, lse, None, d ** -0.5, **kw)
    for bad in (torch.finfo(DT[dtype]).max, 2.0 ** 15 if dtype == "f16" else 2.0 ** 60, float("inf"),
                float("-inf"), float("nan")):
        sick = q.clone()
        sick[pad] = bad
        o2, lse2 = ea.attn_fwd_kv8(sick.cuda(), *args, **kw)
        assert torch.equal(o, o2) and torch.equal(lse, lse2), bad
        w2 = ea.attn_kv8_weights(sick.cuda(), ca.k8, ca.ks, ca.lengths, lse, None, d ** -0.5, **kw)
        assert torch.equal(w, w2), bad
    # the sequence of 17 has more than 17 queries where n is large: the first see no key
    assert status() == (ea.ATTN_WARN_EMPTY_ROW if n - 1 > 17 else ea.ATTN_OK)


# ------------------------------------------------------------------ rows of different sizes

@pytest.mark.parametrize("d,G,n", [(128, 4, 1), (128, 8, 2), (64, 8, 4)])
def test_each_row_keeps_its_bits_beside_much_larger_rows(d, G, n):
    """Rows of one head that differ by 2^45, the small ones' scores of size one: an attention of
    their own, and weights."""
    rng = np.random.default_rng(d + G)
    m = 300
    ca = Cache(rng, [m], 2, 384, d, 32)
    x = rng.normal(size=(1, 2 * G, n, d))
    x[:, ::4] *= 2.0 ** 45
    q = rounded(x, "bf16")
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, d ** -0.5)
    check_attend(ca, q, d ** -0.5, "bf16", o, lse)
    # The large rows count for nothing in the sums.
    _, L, _, S, _ = kv8.attend(ca.c, q.double().numpy(), d ** -0.5)
    L[:, ::4], S[:, ::4] = -np.inf, 0.0
    given = torch.from_numpy(L).float()
    ref = kv8.add_weights(ca.c, q.double().numpy(), d ** -0.5, given.double().numpy()) - ca.c["w"]
    w = ea.attn_kv8_weights(q.cuda(), ca.k8, ca.ks, ca.lengths, given.cuda(), None, d ** -0.5)
    rel = (d + 16) * 2.0 ** -23 * (S.max() + 32.0) + 2.0 ** -21 + G * n * 2.0 ** -24
    got = w.double().cpu().numpy()
    assert (np.abs(got - ref)[..., :m] <= rel * ref[..., :m]).all()
    status()


# ------------------------------------------------------------------ rows at the ends of the type

@pytest.mark.parametrize("d,G,n", [(128, 4, 1), (64, 8, 4), (128, 8, 6), (64, 4, 70)])
@pytest.mark.parametrize("exp", [124, 110, -100, -116])
def test_queries_at_the_ends_of_bf16(d, G, n, exp):
    """Rows of size 2^124 to 2^-116 under a c that makes their scores of size one."""
    rng = np.random.default_rng(d + n)
    m = 300
    ca = Cache(rng, [m], 1, 384, d, 32)
    q = rounded(np.clip(rng.normal(size=(1, G, n, d)), -4, 4) * 2.0 ** exp, "bf16")
    c = d ** -0.5 * 2.0 ** -exp
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, c)
    check_attend(ca, q, c, "bf16", o, lse)
    _, L, _, S, _ = kv8.attend(ca.c, q.double().numpy(), c)
    given = torch.from_numpy(L).float()
    ref = kv8.add_weights(ca.c, q.double().numpy(), c, given.double().numpy()) - ca.c["w"]
    w = ea.attn_kv8_weights(q.cuda(), ca.k8, ca.ks, ca.lengths, given.cuda(), None, c).double().cpu().numpy()
    rel = (d + 16) * 2.0 ** -23 * (S.max() + 32.0) + 2.0 ** -21 + G * n * 2.0 ** -24
    assert (np.abs(w - ref)[..., :m] <= rel * ref[..., :m]).all()
    assert status() == ea.ATTN_OK


# ------------------------------------------------------------------ large scores

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,G,n", [(128, 4, 1), (64, 8, 4), (128, 8, 6), (64, 4, 70)])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 27, 2.0 ** 45])
def test_scores_far_past_the_step_of_float32(dtype, d, G, n, size):
    """Scores so large that the step of float32 passes 2^14 in the exponent: the row's largest score
    is alone (the inputs are drawn until its lead is 2^-12 of the sums that make it, whose float32 error
    is below (d + 16) 2^-23), so O is that key's V, off by half a step of P in fp16 (2^-11; its sum l takes P
    unrounded) and half a step of the output, and LSE its score."""
    rng = np.random.default_rng(int(np.log2(size)) + d)
    m, c = 300, 0.1 * size
    ca = Cache(rng, [m], 1, 384, d, 32)
    x = rng.normal(size=(1, G, n, d))
    for g in range(G):
        for i in range(n):
            k = ca.c["k8"][0, 0, :m] * np.repeat(ca.c["ks"][0, 0], 32)[:m, None]
            while True:
                row = rounded(x[0, g, i], dtype).double().numpy()
                s = np.sort(k @ row)
                if s[-1] - s[-2] > 2.0 ** -12 * (np.abs(k) @ np.abs(row)).max():
                    break
                x[0, g, i] = rng.normal(size=d)
    q = rounded(x, dtype)
    O, L, A, S, _ = kv8.attend(ca.c, q.double().numpy(), c)
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, c)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (np.abs(o - O) <= (1.01 * torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -11) * np.abs(O) + 2.0 ** -25).all()
    assert (np.abs(lse - L) <= (d + 16) * 2.0 ** -23 * S + 2.0 ** -15).all()
    assert status() == ea.ATTN_OK


# ------------------------------------------------------------------ small values of a row

@pytest.mark.parametrize("dtype,lost", [("bf16", 2.0 ** -21), ("f16", 2.0 ** -24)])
@pytest.mark.parametrize("d,G,n", [(64, 8, 6), (128, 8, 6), (128, 4, 40), (64, 4, 1)])
@pytest.mark.parametrize("kind", ["ties", "random"])
def test_small_values_beside_a_large_one_in_a_row(dtype, lost, d, G, n, kind):
    """One value of each row 2^16 times the others, in a column where every key is zero: the others
    alone make the scores.  What a row's terms may lose of a value is `lost` of its largest, so a
    score is off by lost max|q| c sum_r |k_r| beside the usual bound."""
    rng = np.random.default_rng(d + n)
    m, c = 250, 0.1
    ca = Cache(rng, [m], 2, 256, d, 32)
    k = ca.c["k8"]
    if kind == "ties":  # one sign a key, so that what values lose adds up
        k[0, :, :m] = np.abs(k[0, :, :m]) * rng.choice([-1.0, 1.0], size=(2, m, 1))
    k[0, :, :m, 0] = 0.0
    ca.c["ks"][:, :, :8] = 2.0 ** -9
    ca.load()
    x = np.full((1, 2 * G, n, d), 0.3125) if kind == "ties" else rng.normal(size=(1, 2 * G, n, d)) / 4
    x[..., 0] = 2.0 ** 14
    q = rounded(x, dtype)
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, c)
    O, L, tol, ltol = attend_bounds(ca, q, c, dtype, None, False)
    A = kv8.attend(ca.c, q.double().numpy(), c)[2]
    off = lost * 2.0 ** 14 * c * np.abs(k[0, :, :m]).sum(-1).max() * 2.0 ** -9
    assert off < 0.05
    # P is off by e^off - 1 <= 1.1 off, numerator and denominator.
    assert (np.abs(o.double().cpu().numpy() - O) <= tol + 2.2 * off * A).all()
    assert (np.abs(lse.double().cpu().numpy() - L) <= ltol + off).all()
    ref = kv8.add_weights(ca.c, q.double().numpy(), c, lse.double().cpu().numpy()) - ca.c["w"]
    w = ea.attn_kv8_weights(q.cuda(), ca.k8, ca.ks, ca.lengths, lse, None, c).double().cpu().numpy()
    S = kv8.attend(ca.c, q.double().numpy(), c)[3]
    rel = (d + 16) * 2.0 ** -23 * (S.max() + 32.0) + 2.0 ** -21 + G * n * 2.0 ** -24
    assert (np.abs(w - ref)[..., :m] <= (rel + 1.1 * off) * ref[..., :m]).all()
    status()


# ------------------------------------------------------------------ probabilities

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", [(1, 1), (12, 1), (4, 6), (2, 40), (4, 75)])
def test_fp16_outputs_keep_more_of_p_than_half_a_step(d, G, n):
    """Two scores whose products with V all but cancel: P of 64 and of 38.421875, which lies in the
    middle between two fp16 values.  One fp16 value for P would leave 5 / 64 of 384; as a pair, half a
    step of P is 2^-22, beside float32 roundings of the score (values below 1) and the sums."""
    m = 96
    r = 38.421875 / 64
    ca = Cache(np.random.default_rng(1), [m], 1, 128, d, 16, spread=0)
    low = np.arange(m) % 8 < 5
    ca.c["k8"][0, 0, :m] = 0.0
    ca.c["k8"][0, 0, :m, 3] = np.where(low, -1.0, 0.0)
    ca.c["v8"][0, 0, :m] = np.where(low, -1.0, 1.0)[:, None]
    for x in ("ks", "vs"):
        ca.c[x][0, 0, :-(-m // 16)] = 1.0
    ca.load()
    q = torch.zeros(1, G, n, d, dtype=torch.float16)
    q[..., 3] = 1.0
    c = float(np.float32(-np.log(r)))
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, c)
    p = np.exp(-c)
    want = (3 - 5 * p) / (3 + 5 * p)
    assert np.abs(o.double().cpu().numpy() - want).max() <= 2.0 ** -11 * abs(want) + 2.0 ** -24 + 2.0 ** -18
    assert np.abs(lse.double().cpu().numpy() - np.log(m / 8 * (3 + 5 * p))).max() <= 2.0 ** -18
    status()


# ------------------------------------------------------------------ value scales

FEW_AND_MANY = [(4, 1), (4, 4), (8, 6), (4, 70)]


@pytest.mark.parametrize("G,n", FEW_AND_MANY)
@pytest.mark.parametrize("block", [16, 128])
@pytest.mark.parametrize("exps", [(-100, 40), (40, -100), (-100, 40, -100), (-100, 119), (119, -100, -20, 119),
                                  (0, -100), (-100, 0), (-100, -100), (60, -60), (-60, 60)])
def test_value_scales_at_both_ends(G, n, block, exps):
    """Blocks whose scales lie far apart, as those that hold only zeros (2^-100) and large values
    give; all scores are equal, so every key has the same weight."""
    m = block * len(exps) - 3
    cap = 128 * -(-m // 128)
    ca = Cache(np.random.default_rng(5), [m], 2, cap, 64, block)
    ca.c["k8"][0, :, :m] = 0.0
    for i, e in enumerate(exps):
        ca.c["vs"][0, :, i] = 2.0 ** e
        if e == -100:
            ca.c["v8"][0, :, i * block:min(m, (i + 1) * block)] = 0.0
    ca.load()
    q = rounded(np.random.default_rng(6).normal(size=(1, 2 * G, n, 64)), "bf16")
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.125)
    check_attend(ca, q, 0.125, "bf16", o, lse)
    assert np.abs(lse.double().cpu().numpy() - np.log(m)).max() <= 2.0 ** -14
    status()


@pytest.mark.parametrize("G,n", FEW_AND_MANY)
@pytest.mark.parametrize("lo,hi", [(-100, 100), (-100, -90), (90, 110), (-70, -50), (-20, 90)])
@pytest.mark.parametrize("pow2", [True, False])
def test_value_scales_over_the_whole_range(G, n, lo, hi, pow2):
    """Every block's scale drawn over a wide range, the scores random too.  A scale below 2^-70 counts as
    2^-70 and the values take the rest, in fp16: a value may lose 2^-25 (half a step below its normal
    values) of 2^-70, or a probability 2^-25 of a code over sums of at least 2^76."""
    rng = np.random.default_rng(abs(lo) + hi)
    lengths = [1000, 90]
    ca = Cache(rng, lengths, 2, 1024, 128, 16, pow2=pow2)
    for b, m in enumerate(lengths):
        e = rng.integers(lo, hi + 1, size=(2, -(-m // 16))) + (0.0 if pow2 else rng.random((2, -(-m // 16))))
        ca.c["vs"][b, :, :-(-m // 16)] = np.float32(2.0 ** e)
    ca.load()
    q = rounded(rng.normal(size=(2, 2 * G, n, 128)), "bf16")
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.3, mask="causal")
    O, L, tol, ltol = attend_bounds(ca, q, 0.3, "bf16", None, True)
    codes = np.where(np.isnan(ca.c["v8"]), 0.0, np.abs(ca.c["v8"])).sum(2).repeat(G, 1)[:, :, None]
    # log2 of the scale stands beside the score: float32 values up to 128 + |score|, rounded twice
    ds = 2.0 ** -16
    A = kv8.attend(ca.c, q.double().numpy(), 0.3, None, True)[2]
    assert (np.abs(o.double().cpu().numpy() - O) <= tol + 2 * ds * A + 2.0 ** -95 + 2.0 ** -101 * codes).all()
    assert (np.abs(lse.double().cpu().numpy() - L) <= ltol + ds).all()
    status()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("G,n", FEW_AND_MANY)
@pytest.mark.parametrize("first", [True, False])
def test_value_scales_far_apart_in_parts_of_a_long_sequence(dtype, G, n, first):
    """Half of the sequence holds zeros, the other large values: CTAs of each half join their parts."""
    rng = np.random.default_rng(8)
    cap, m = 8192, 8000
    ca = Cache(rng, [m], 1, cap, 64, 128)
    half = slice(0, 4096) if first else slice(4096, m)
    ca.c["v8"][0, :, half] = 0.0
    ca.c["vs"][0, :, :63] = 2.0 ** 40 if dtype == "bf16" else 0.125
    ca.c["vs"][0, :, 0 if first else 32:32 if first else 63] = 2.0 ** -100
    ca.load()
    q = rounded(rng.normal(size=(1, G, n, 64)), dtype)
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.125, mask="causal")
    check_attend(ca, q, 0.125, dtype, o, lse, None, True)
    status()


@pytest.mark.parametrize("G,n", [(1, 1), (8, 5)])
def test_a_long_sequence_of_zero_values(G, n):
    """2^22 tokens whose values are all zero (scale 2^-100), in every CTA's part and their join."""
    cap = 1 << 22
    codes = torch.zeros(1, 1, cap, 64, dtype=torch.uint8, device="cuda")
    ks, vs = torch.ones(1, 1, cap // 128, device="cuda"), torch.full((1, 1, cap // 128), 2.0 ** -100, device="cuda")
    q = torch.ones(1, G, n, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = ea.attn_fwd_kv8(q, codes, codes, ks, vs, i32([cap]), 1.0)
    assert (o == 0).all()
    # sums of 2^22 equal terms in float32 over the warps of every CTA
    assert (lse.double() - np.log(cap)).abs().max() <= 2.0 ** -12
    w = ea.attn_kv8_weights(q, codes, ks, i32([cap]), lse, None, 1.0)
    assert (w.double() * cap / (G * n) - 1).abs().max() <= 2.0 ** -11
    status()


# ------------------------------------------------------------------ many rows

@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("f16", 128)])
def test_more_than_2048_rows_a_head(dtype, d):
    """A prompt's chunk: 2404 rows of a key/value head (a last tile of 100), ragged, attention and weights."""
    rng = np.random.default_rng(d)
    G, n, lengths, counts = 4, 601, [1500, 601, 40], [601, 599, 33]
    ca = Cache(rng, lengths, 1, 1536, d, 64)
    q = rounded(rng.normal(size=(3, G, n, d)), dtype)
    kw = dict(counts=i32(counts), mask="causal")
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, d ** -0.5, **kw)
    check_attend(ca, q, d ** -0.5, dtype, o, lse, counts, True)
    w = ea.attn_kv8_weights(q.cuda(), ca.k8, ca.ks, ca.lengths, lse, None, d ** -0.5, **kw).double().cpu().numpy()
    ref = kv8.add_weights(ca.c, q.double().numpy(), d ** -0.5, lse.double().cpu().numpy(), counts, True) - ca.c["w"]
    S = kv8.attend(ca.c, q.double().numpy(), d ** -0.5, counts, True)[3]
    rel = (d + 16) * 2.0 ** -23 * (S.max() + 32.0) + 2.0 ** -21 + G * n * 2.0 ** -24
    for b, m in enumerate(lengths):
        assert (np.abs(w - ref)[b, :, :m] <= rel * ref[b, :, :m]).all()
    assert status() == ea.ATTN_OK
