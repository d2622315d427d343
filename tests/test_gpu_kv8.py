"""The 8-bit key/value cache on the GPU against its float64 oracle.

Codes, scales, weights moved or zeroed, lengths and kept positions are whole decisions and must be
equal.  Attention is held to bounds counted from its roundings:
  P to fp16, half a step              2^-11 sum_j P_ij |V_j|   (and 2^-31 sum |v8_j| max vs: the
                                      subnormal step 2^-24 below a largest P of at least 2^6)
  a score's products and sums         ds = (d + 16) 2^-23 (c sum_r |q_r k_r| + log2 range) on P
                                      twice (numerator and denominator), once on LSE
  float32 sums over keys and parts    (keys / 8 + 64) 2^-24
  the output's type                   eps / 2 of |O| (and half its subnormal step)
"""
import numpy as np
import pytest
import torch

import exact_io_aware_gb300 as ea
from oracle import kv8

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
F8 = torch.float8_e4m3fn


def gpu_codes(vals):
    """E4M3 tensor of the given E4M3 values (NaN: the NaN code)."""
    return torch.from_numpy(np.ascontiguousarray(vals)).float().to(F8).cuda()


def rounded(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype])


class Cache:
    """A cache on both sides.  Everything past the lengths is poison: NaN codes, NaN scales."""

    def __init__(self, rng, lengths, Hk, cap, d, block, spread=4, pow2=True):
        B = len(lengths)
        shape = (B, Hk, cap, d)
        c = {x + "8": kv8.codes(rng.normal(size=shape) * 60, 1.0) for x in "kv"}
        for x in "kv":
            e = rng.integers(-7 - spread, -5, size=(B, Hk, cap // block)).astype(np.float64)
            c[x + "s"] = 2.0 ** e if pow2 else np.float32(2.0 ** (e + rng.random(e.shape))).astype(np.float64)
        c["w"] = rng.random((B, Hk, cap)).astype(np.float32).astype(np.float64)
        c["lengths"] = np.array(lengths)
        for b, m in enumerate(lengths):
            for x in "kv":
                c[x + "8"][b, :, m:] = np.nan
                c[x + "s"][b, :, -(-m // block):] = np.nan
        self.c = c
        self.load()

    def load(self):
        c = self.c
        self.k8, self.v8 = gpu_codes(c["k8"]), gpu_codes(c["v8"])
        self.ks, self.vs, self.w = (torch.from_numpy(c[x]).float().cuda() for x in ("ks", "vs", "w"))
        self.lengths = torch.tensor(c["lengths"], dtype=torch.int32, device="cuda")

    def check(self, ref, what=""):
        for name, got in (("k8", self.k8), ("v8", self.v8), ("ks", self.ks), ("vs", self.vs), ("w", self.w)):
            got = got.float().double().cpu().numpy()
            same = (got == ref[name]) | (np.isnan(got) & np.isnan(ref[name]))
            assert same.all(), f"{what} {name}: {np.argwhere(~same)[:4].tolist()}"
        assert self.lengths.cpu().numpy().tolist() == list(ref["lengths"])


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    return ea.attn_device_status()


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,block", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("n,lengths,counts", [
    (1, [1, 17, 128, 300], None),
    (1, [16, 64, 129, 5], [1, 0, 1, 1]),
    (2, [129, 2, 384, 65], None),                 # straddles a span of 128
    (7, [7, 9, 250, 31], [7, 3, 0, 6]),
    (130, [257, 130, 384, 131], [130, 129, 130, 1]),
    (300, [300, 384, 301, 333], None),
])
def test_append(dtype, d, block, n, lengths, counts):
    rng = np.random.default_rng(n + d + block)
    ca = Cache(rng, [m - (n if counts is None else k) for m, k in zip(lengths, counts or [0] * 4)],
               2, 384, d, block)
    # Held blocks keep a defined scale; the new tokens differ in size, so some blocks grow.
    k, v = (rounded(rng.normal(size=(4, 2, n, d)) * 2.0 ** rng.integers(-4, 6, size=(4, 2, n, 1)), dtype)
            for _ in range(2))
    ca.c["lengths"] = np.array(lengths)
    ca.lengths = i32(lengths)
    ref = kv8.append(ca.c, k.double().numpy(), v.double().numpy(), counts)
    ea.attn_kv8_append(k.cuda(), v.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, counts=i32(counts),
                       weights=ca.w)
    ca.check(ref)
    assert status() == ea.ATTN_OK


def test_append_extremes():
    """Values that are not finite, all zeros, the types' largest and least, and growth over them."""
    rng = np.random.default_rng(3)
    ca = Cache(rng, [0, 0, 0, 0, 0], 1, 64, 64, 16)
    x = np.zeros((5, 1, 3, 64))
    x[0, 0, 0, :3] = [np.inf, -np.inf, np.nan]
    x[0, 0, 1, 5] = 1.5
    x[1, 0, :, 0] = [3.38e38, -1e-38, 1.0]
    x[2, 0, :, 1] = [2.0 ** -120, 0, 0]
    x[3, 0, 0, :] = np.nan
    x[4] = rng.normal(size=(3, 64))
    for step, cnt in enumerate(([3, 3, 3, 3, 3], [1, 2, 3, 0, 3])):
        y = rounded(x * 2.0 ** (8 * step), "bf16")
        ca.c["lengths"] = ca.c["lengths"] + np.array(cnt)
        ca.lengths = i32(ca.c["lengths"].tolist())
        ref = kv8.append(ca.c, y.double().numpy(), y.double().numpy(), cnt)
        ea.attn_kv8_append(y.cuda(), y.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, counts=i32(cnt))
        ref["w"] = ca.c["w"]  # no weights given: left alone
        ca.check(ref, f"step {step}")
        ca.c = ref
    assert status() == ea.ATTN_OK


def test_append_out_of_range_lengths_are_clamped():
    rng = np.random.default_rng(4)
    ca = Cache(rng, [30, 0, 0], 2, 32, 64, 16)
    x = rounded(rng.normal(size=(3, 2, 4, 64)), "f16")
    # Length 40 of 32 counts as 32; -3 as 0; 2 with 4 new tokens drops two.  A count of 9 is 4.
    ca.lengths = i32([40, -3, 2])
    ea.attn_kv8_append(x.cuda(), x.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, counts=i32([9, 4, 4]),
                       weights=ca.w)
    assert status() == ea.ATTN_WARN_CLAMPED
    ca.c["lengths"] = np.array([32, 0, 2])
    ref = kv8.append(ca.c, x.double().numpy(), x.double().numpy(), [4, 4, 4])
    ca.lengths = i32([32, 0, 2])
    ca.check(ref)


# ------------------------------------------------------------------ attention

def attend_bounds(ca, q, c, dtype, counts, causal):
    O, L, A, S, F = kv8.attend(ca.c, q.double().numpy(), c, counts, causal)
    d, cap = q.shape[3], ca.k8.shape[2]
    ds = (d + 16) * 2.0 ** -23 * (S + 32.0)
    sums = (cap / 8 + 64) * 2.0 ** -24
    info = torch.finfo(DT[dtype])
    half = info.eps / 2
    tol = (half * (np.abs(O) * (1 + 2.0 ** -6)) + info.smallest_normal * info.eps / 2
           + (1 + 2.0 ** -6) * A * (2.0 ** -11 + 2 * ds[..., None] + 2 * sums) + 2.0 ** -31 * F)
    ltol = ds + sums + 2.0 ** -22 * (np.where(np.isfinite(L), np.abs(L), 0) + 32.0)
    return O, L, tol, ltol


def check_attend(ca, q, c, dtype, o, lse, counts=None, causal=False):
    O, L, tol, ltol = attend_bounds(ca, q, c, dtype, counts, causal)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(L)
    assert (np.isneginf(lse) == empty).all() and (o[empty] == 0).all()
    assert np.isfinite(o).all() and np.isfinite(lse[~empty]).all()
    bad = np.abs(o - O) > tol
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), np.abs(o - O).max(), (np.abs(o - O) / tol).max())
    lerr = np.abs(np.where(empty, 0.0, lse) - np.where(empty, 0.0, L))
    assert (lerr <= ltol).all(), (np.argwhere(lerr > ltol)[:4].tolist(), lerr.max())
    return L


@pytest.mark.parametrize("dtype,d,block", [("bf16", 128, 64), ("bf16", 64, 16), ("f16", 128, 16),
                                           ("f16", 64, 128), ("bf16", 128, 128), ("bf16", 128, 32)])
@pytest.mark.parametrize("G,n", [(1, 1), (4, 1), (3, 3), (16, 1), (5, 5), (2, 16), (33, 1), (8, 11), (1, 70), (4, 75)])
@pytest.mark.parametrize("mask", ["none", "causal"])
def test_attend(dtype, d, block, G, n, mask):
    lengths = [0, 1, 15, 16, 33, 127, 128, 129, 255, 384]
    rng = np.random.default_rng(G * 100 + n)
    ca = Cache(rng, lengths, 2, 384, d, block, pow2=G % 2 == 0)
    counts = [int(rng.integers(0, n + 1)) for _ in lengths] if n > 1 and G % 2 else None
    q = rounded(rng.normal(size=(len(lengths), 2 * G, n, d)), dtype)
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, d ** -0.5,
                             counts=i32(counts), mask=mask)
    L = check_attend(ca, q, d ** -0.5, dtype, o, lse, counts, mask == "causal")
    real = np.arange(n) < np.array(counts if counts else [n] * len(lengths))[:, None]
    assert status() == (ea.ATTN_WARN_EMPTY_ROW if (np.isneginf(L) & real[:, None]).any() else ea.ATTN_OK)


@pytest.mark.parametrize("G,n,cap,lengths", [
    (4, 1, 8192, [8191, 5, 3000]),       # runs that end inside a tile
    (1, 1, 65536, [65536]),              # one head over many CTAs
    (8, 6, 4096, [4096, 4001, 77]),
    (4, 128, 4096, [4096, 2047]),
    (2, 200, 1024, [1000, 201, 150]),
])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
def test_attend_long(dtype, d, G, n, cap, lengths):
    rng = np.random.default_rng(cap + G)
    ca = Cache(rng, lengths, 1 if cap > 8192 else 2, cap, d, 64)
    Hk = ca.k8.shape[1]
    q = rounded(rng.normal(size=(len(lengths), Hk * G, n, d)), dtype)
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, d ** -0.5, mask="causal")
    check_attend(ca, q, d ** -0.5, dtype, o, lse, None, True)
    again = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, d ** -0.5, mask="causal")
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    status()


@pytest.mark.parametrize("n,G", [(1, 4), (40, 8)])
def test_attend_scales_far_apart_and_large_scores(n, G):
    """V scales over 2^40, and scores whose maximum rises along the keys (c = 3)."""
    rng = np.random.default_rng(11)
    ca = Cache(rng, [300, 90], 2, 320, 128, 16, spread=40)
    for b, m in enumerate([300, 90]):
        ca.c["ks"][b, :, :-(-m // 16)] = 2.0 ** -7
    ca.load()
    q = rounded(rng.normal(size=(2, 2 * G, n, 128)), "bf16")
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 3.0, mask="causal")
    check_attend(ca, q, 3.0, "bf16", o, lse, None, True)
    status()


@pytest.mark.parametrize("c", [-0.3, 0.0])
@pytest.mark.parametrize("dtype,G,n", [("bf16", 4, 1), ("f16", 3, 7), ("bf16", 5, 40)])
def test_scale_negative_and_zero(c, dtype, G, n):
    rng = np.random.default_rng(14)
    ca = Cache(rng, [200, 50], 2, 256, 128, 32)
    q = rounded(rng.normal(size=(2, 2 * G, n, 128)), dtype)
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, c, mask="causal")
    O, L, A, S, F = kv8.attend(ca.c, q.double().numpy(), c, None, True)
    ds = (128 + 16) * 2.0 ** -23 * (np.abs(S) + 32.0)
    tol = (2.0 ** -8 * np.abs(O) + 2.0 ** -25 + 1.1 * A * (2.0 ** -11 + 2 * ds[..., None] + 2.0 ** -16)
           + 2.0 ** -31 * F)
    assert (np.abs(o.double().cpu().numpy() - O) <= tol).all()
    # LSE: the scores' error and float32 sums and rounding of values up to 64
    assert (np.abs(lse.double().cpu().numpy() - L) <= ds + 2.0 ** -15).all()
    ref = kv8.add_weights(ca.c, q.double().numpy(), c, lse.double().cpu().numpy(), None, True)
    w = ea.attn_kv8_weights(q.cuda(), ca.k8, ca.ks, ca.lengths, lse, ca.w, c, mask="causal")
    held = (np.arange(256) < np.array([200, 50])[:, None])[:, None].repeat(2, 1)
    assert np.allclose(w.double().cpu().numpy()[held], ref[held], rtol=1e-3 if c else 1e-5, atol=0)


def test_attend_query_sizes():
    """Rows of one call whose queries differ by 2^60, and tiny and huge ones."""
    rng = np.random.default_rng(12)
    ca = Cache(rng, [200], 1, 256, 64, 64)
    x = rng.normal(size=(1, 4, 1, 64)) * 2.0 ** np.array([0, -30, -60, 3]).reshape(1, 4, 1, 1)
    q = rounded(x, "bf16")
    for c in (0.125, 2.0 ** -20):
        o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, c)
        check_attend(ca, q, c, "bf16", o, lse)


@pytest.mark.parametrize("G,n", [(2, 3), (1, 24), (4, 40)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_value_reaches_only_the_rows_that_see_it(d, G, n):
    rng = np.random.default_rng(13)
    m = 100
    ca = Cache(rng, [m], 1, 128, d, 16)
    bad = [(m - 1, 3), (m - 1, d - 1), (m - 2, 8), (m - n, 0)] if n == 3 else [(m - 2, 5), (m - n // 2, d - 2)]
    for key, col in bad:
        ca.c["v8"][0, 0, key, col] = np.nan
    ca.load()
    q = rounded(rng.normal(size=(1, G, n, d)), "f16")
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.1, mask="causal")
    want = np.zeros((1, G, n, d), bool)
    for i in range(n):
        for key, col in bad:
            if key <= m - n + i:
                want[0, :, i, col] = True
    got = torch.isnan(o).cpu().numpy()
    assert (got == want).all(), np.argwhere(got != want)[:5].tolist()
    assert torch.isfinite(lse).all()
    # A NaN key makes the rows that see it NaN, and no others.
    ca.c["v8"][np.isnan(ca.c["v8"]) & (np.arange(128) < m)[None, None, :, None]] = 1.0
    ca.c["k8"][0, 0, m - 1, 0] = np.nan
    ca.load()
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.1, mask="causal")
    assert torch.isnan(o[:, :, -1]).all() and torch.isnan(lse[:, :, -1]).all()
    assert torch.isfinite(o[:, :, :-1]).all() and torch.isfinite(lse[:, :, :-1]).all()


@pytest.mark.parametrize("B,Hk,G,n", [(170, 5, 17, 2), (150, 5, 66, 2)])
def test_many_short_tiles_a_cta(B, Hk, G, n):
    """Many tiles in each CTA's run (of 128 rows, and of 256), some ending in a NaN value or seeing
    no key, so that what the kernel keeps by tile number is used over and over."""
    rng = np.random.default_rng(15)
    lengths = [int(x) for x in rng.integers(0, 140, B)]
    ca = Cache(rng, lengths, Hk, 256, 64, 16)
    sick = [b for b in range(B) if b % 7 == 3 and lengths[b] > 2]
    for b in sick:
        ca.c["v8"][b, :, lengths[b] - 1, 5] = np.nan
    ca.load()
    q = rounded(rng.normal(size=(B, Hk * G, n, 64)), "bf16")
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.125, mask="causal")
    nan = torch.isnan(o).cpu().numpy()
    want = np.zeros_like(nan)
    want[sick, :, n - 1, 5] = True
    assert (nan == want).all(), np.argwhere(nan != want)[:5].tolist()
    for b in sick:
        ca.c["v8"][b, :, lengths[b] - 1, 5] = 0.0
    some = rng.choice(B, 12, replace=False)
    sub = type("Sub", (), {})()
    sub.c = {key: val[some] for key, val in ca.c.items()}
    sub.k8 = ca.k8
    o2 = o[some].clone()
    o2[torch.isnan(o2)] = 0.0
    O, L, tol, ltol = attend_bounds(sub, q[some], 0.125, "bf16", None, True)
    o2, l2 = o2.double().cpu().numpy(), lse[some].double().cpu().numpy()
    keep = ~want[some]
    assert (np.abs(o2 - O) <= tol)[keep].all()
    empty = np.isneginf(L)
    assert (np.isneginf(l2) == empty).all() and (np.abs(l2 - L)[~empty] <= ltol[~empty]).all()
    status()


@pytest.mark.parametrize("G,n", [(4, 1), (2, 6), (7, 5)])
def test_many_sequences(G, n):
    """More sequences than lanes of a warp, some empty: attention and weights over runs that cross
    many heads."""
    rng = np.random.default_rng(16)
    B = 75
    lengths = [int(x) for x in rng.integers(0, 1024, B)]
    lengths[5] = lengths[40] = lengths[74] = 0
    ca = Cache(rng, lengths, 2, 1024, 64, 64)
    counts = [min(n, m) for m in lengths]
    q = rounded(rng.normal(size=(B, 2 * G, n, 64)), "f16")
    o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.125, counts=i32(counts),
                             mask="causal")
    check_attend(ca, q, 0.125, "f16", o, lse, counts, True)
    w = ea.attn_kv8_weights(q.cuda(), ca.k8, ca.ks, ca.lengths, lse, ca.w, 0.125, counts=i32(counts),
                            mask="causal")
    ref = kv8.add_weights(ca.c, q.double().numpy(), 0.125, lse.double().cpu().numpy(), counts, True)
    held = (np.arange(1024) < np.array(lengths)[:, None])[:, None].repeat(2, 1)
    assert np.allclose(w.double().cpu().numpy()[held], ref[held], rtol=2e-4, atol=0)
    status()


def test_attend_offsets_past_32_bits():
    """One head of 2^24 + 256 tokens: codes past 2^31 bytes.  Zero keys: every weight is 1 / len."""
    cap = (1 << 24) + 256
    k8 = torch.zeros(1, 1, cap, 128, dtype=torch.uint8, device="cuda")
    v8 = torch.full((1, 1, cap, 128), 0x38, dtype=torch.uint8, device="cuda")    # 1.0
    v8[0, 0, -1] = 0x7E                                                          # 448
    ks = torch.ones(1, 1, cap // 128, device="cuda")
    vs = torch.ones(1, 1, cap // 128, device="cuda")
    vs[0, 0, -1] = 2.0 ** 20
    q = torch.ones(1, 2, 1, 128, dtype=torch.bfloat16, device="cuda")
    o, lse = ea.attn_fwd_kv8(q, k8, v8, ks, vs, i32([cap]), 1.0)
    want = ((cap - 128) + 2.0 ** 20 * (127 + 448)) / cap
    # Weights 2^-20 of the largest stay normal fp16; sums of 2^24 terms in float32 over 1,216 warps.
    assert (o.double() / want - 1).abs().max() <= 2.0 ** -8 + 2.0 ** -9
    assert (lse.double() - np.log(cap)).abs().max() <= 2.0 ** -9
    w = ea.attn_kv8_weights(q, k8, ks, i32([cap]), lse, None, 1.0)
    assert (w.double() * cap / 2 - 1).abs().max() <= 2.0 ** -8
    x = torch.full((1, 1, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    ea.attn_kv8_append(x, x, k8.view(F8), v8.view(F8), ks, vs, i32([cap]))
    assert (v8.view(F8)[0, 0, -2:].float() * vs[0, 0, -1] == 0).all()            # 3 / 2^20 rounds to 0
    assert (k8.view(F8)[0, 0, -2:].float() * ks[0, 0, -1] == 3).all()


# ------------------------------------------------------------------ weights

@pytest.mark.parametrize("dtype,d,block", [("bf16", 128, 64), ("f16", 64, 16), ("bf16", 64, 32)])
@pytest.mark.parametrize("G,n", [(1, 1), (4, 1), (3, 5), (4, 6), (33, 1), (4, 32), (5, 33), (5, 60), (8, 70)])
@pytest.mark.parametrize("mask", ["none", "causal"])
def test_weights(dtype, d, block, G, n, mask):
    lengths = [0, 1, 16, 33, 127, 129, 255, 384]
    rng = np.random.default_rng(G * 10 + n)
    ca = Cache(rng, lengths, 2, 384, d, block)
    counts = [int(rng.integers(0, n + 1)) for _ in lengths] if n > 1 and G % 2 else None
    q = rounded(rng.normal(size=(len(lengths), 2 * G, n, d)), dtype)
    _, L, _, S, _ = kv8.attend(ca.c, q.double().numpy(), d ** -0.5, counts, mask == "causal")
    lse = torch.from_numpy(L).float().cuda()
    ref = kv8.add_weights(ca.c, q.double().numpy(), d ** -0.5, lse.double().cpu().numpy(), counts,
                          mask == "causal")
    args = (q.cuda(), ca.k8, ca.ks, ca.lengths, lse)
    kw = dict(counts=i32(counts), mask=mask)
    w0 = ca.w.clone()
    out = torch.full_like(ca.w, -7.0)
    got = ea.attn_kv8_weights(*args, ca.w, d ** -0.5, out=out, **kw)
    assert got is out and torch.equal(ca.w, w0)
    held = (np.arange(384) < np.array(lengths)[:, None])[:, None].repeat(2, 1)
    given = ref - ca.c["w"]
    rel = (d + 16) * 2.0 ** -23 * (S.max() + 32.0) + 2.0 ** -21 + G * n * 2.0 ** -24
    tol = given * rel + np.abs(ref) * 2.0 ** -23
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err[held] <= tol[held]).all(), (err[held] / tol[held]).max()
    assert (got.cpu().numpy()[~held] == -7.0).all()
    none = ea.attn_kv8_weights(*args, None, d ** -0.5, **kw)
    assert (np.abs(none.double().cpu().numpy() - np.where(held, given, 0)) <= given * rel + 2.0 ** -126).all()
    same = ea.attn_kv8_weights(*args, ca.w, d ** -0.5, **kw)
    assert same is ca.w and torch.equal(torch.where(torch.from_numpy(held).cuda(), same, -7.0), got)
    status()


# ------------------------------------------------------------------ eviction

def evict_both(ca, keep, sink, recent, cap_out, rng, block):
    B, Hk, _, d = ca.k8.shape
    out = Cache(rng, [0] * B, Hk, cap_out, d, block)
    ref, kept = kv8.evict(ca.c, out.c, keep, sink, recent)
    got = ea.attn_kv8_evict(ca.k8, ca.v8, ca.ks, ca.vs, ca.w, ca.lengths, keep, out.k8, out.v8, out.ks,
                            out.vs, out.w, out.lengths, sink=sink, recent=recent)
    assert got.cpu().numpy().tolist() == kept.tolist()
    out.check(ref)
    return out, ref


@pytest.mark.parametrize("d,block", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("keep,sink,recent,cap_out", [
    (1, 0, 0, 128), (1, 1, 0, 128), (17, 0, 5, 128), (100, 4, 20, 128), (128, 64, 64, 128),
    (129, 0, 0, 256), (384, 4, 4, 384), (500, 4, 4, 512),
])
def test_evict(d, block, keep, sink, recent, cap_out):
    rng = np.random.default_rng(keep + d)
    ca = Cache(rng, [0, 1, 16, 99, 130, 384], 2, 384, d, block, pow2=block != 32)
    evict_both(ca, keep, sink, recent, cap_out, rng, block)
    assert status() == ea.ATTN_OK


@pytest.mark.parametrize("kind", ["ties", "nan", "signs", "close", "long"])
def test_evict_weights_that_are_hard_to_order(kind):
    rng = np.random.default_rng(21)
    cap = 4096 if kind == "long" else 384
    ca = Cache(rng, [cap, cap - 7], 2, cap, 64, 16)
    w = rng.random(ca.c["w"].shape)
    if kind == "ties":
        w = np.floor(w * 3)
    elif kind == "nan":
        w[rng.random(w.shape) < 0.4] = np.nan
        w[0, 0, :] = np.nan
    elif kind == "signs":
        w = rng.choice([0.0, -0.0, -1.0, 1.0, np.inf, -np.inf, 1e-40, -1e-40], size=w.shape)
    else:
        w = 1.0 + np.floor(w * 40) * 2.0 ** -23
    ca.c["w"] = w.astype(np.float32).astype(np.float64)
    ca.load()
    for keep, sink, recent in ((50, 0, 0), (cap // 2, 3, 30), (cap - 100, 0, 1)):
        evict_both(ca, keep, sink, recent, -(-keep // 16) * 16, rng, 16)


@pytest.mark.parametrize("kind", ["random", "ties", "nan"])
def test_evict_long_sequences(kind):
    """Sequences whose tokens several CTAs look at together (40960 tokens; one just over keep)."""
    rng = np.random.default_rng(22)
    cap, lengths = 40960, [40960, 33333, 9001]
    ca = Cache(rng, lengths, 1, cap, 64, 128)
    w = np.exp(2 * rng.normal(size=ca.c["w"].shape))
    if kind == "ties":
        w = np.floor(w)
    elif kind == "nan":
        w[rng.random(w.shape) < 0.5] = np.nan
    ca.c["w"] = w.astype(np.float32).astype(np.float64)
    ca.load()
    for keep, sink, recent in ((9000, 5, 100), (1, 0, 0), (128, 64, 64)):
        evict_both(ca, keep, sink, recent, -(-keep // 128) * 128, rng, 128)
    assert status() == ea.ATTN_OK


# ------------------------------------------------------------------ as they are used

def test_a_decoding_run_that_stays_within_its_bound():
    """Prompt, then tokens one by one: append, attend, weigh, and evict at the bound, every step
    against the oracle carried along with the GPU's own weights."""
    rng = np.random.default_rng(31)
    B, Hk, G, d, block, cap, keep = 3, 2, 4, 64, 16, 96, 48
    caches = [Cache(rng, [0] * B, Hk, cap, d, block) for _ in range(2)]
    ca, other = caches
    lens = np.zeros(B, int)
    evicted = 0
    for step in range(60):
        n = 40 if step == 0 else 1
        counts = [40, 17, 33] if step == 0 else None
        lens = lens + np.array(counts if counts else [1] * B)
        k, v = (rounded(rng.normal(size=(B, Hk, n, d)) * 2.0 ** (step % 5), "bf16") for _ in range(2))
        q = rounded(rng.normal(size=(B, Hk * G, n, d)), "bf16")
        ca.c["lengths"] = lens.copy()
        ca.lengths.copy_(i32(lens.tolist()))
        ca.c = kv8.append(ca.c, k.double().numpy(), v.double().numpy(), counts)
        ea.attn_kv8_append(k.cuda(), v.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, counts=i32(counts),
                           weights=ca.w)
        ca.check(ca.c, f"step {step}")
        o, lse = ea.attn_fwd_kv8(q.cuda(), ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.125,
                                 counts=i32(counts), mask="causal")
        check_attend(ca, q, 0.125, "bf16", o, lse, counts, True)
        ref = kv8.add_weights(ca.c, q.double().numpy(), 0.125, lse.double().cpu().numpy(), counts, True)
        ea.attn_kv8_weights(q.cuda(), ca.k8, ca.ks, ca.lengths, lse, ca.w, 0.125, counts=i32(counts),
                            mask="causal")
        got = ca.w.double().cpu().numpy()
        held = (np.arange(cap) < lens[:, None])[:, None].repeat(Hk, 1)
        assert np.allclose(got[held], ref[held], rtol=2e-4, atol=0)
        ca.c["w"] = got
        if lens.max() > 80:
            out, kept = kv8.evict(ca.c, other.c, keep, 4, 16)
            pos = ea.attn_kv8_evict(ca.k8, ca.v8, ca.ks, ca.vs, ca.w, ca.lengths, keep, other.k8, other.v8,
                                    other.ks, other.vs, other.w, other.lengths, sink=4, recent=16)
            assert pos.cpu().numpy().tolist() == kept.tolist()
            other.check(out, f"evict at {step}")
            other.c = out
            ca, other = other, ca
            lens = ca.c["lengths"].copy()
            evicted += 1
    assert evicted >= 1
    assert status() == ea.ATTN_OK


def test_captured_step_replays_with_new_lengths():
    """A captured append + attend + weights step; the lengths move on the device between replays."""
    rng = np.random.default_rng(41)
    B, Hk, G, d, cap = 2, 2, 4, 128, 256
    ca = Cache(rng, [10, 100], Hk, cap, d, 64)
    x = [rounded(rng.normal(size=(B, Hk, 1, d)), "bf16") for _ in range(2)]
    q = rounded(rng.normal(size=(B, Hk * G, 1, d)), "bf16")
    kd, vd, qd = x[0].cuda(), x[1].cuda(), q.cuda()
    o, lse = torch.empty_like(qd), torch.empty(B, Hk * G, 1, device="cuda")

    def step():
        ca.lengths.add_(1)
        ea.attn_kv8_append(kd, vd, ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, weights=ca.w)
        ea.attn_fwd_kv8(qd, ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.1, o=o, lse=lse)
        ea.attn_kv8_weights(qd, ca.k8, ca.ks, ca.lengths, lse, ca.w, 0.1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    ca.load()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    lengths = ca.lengths.clone()
    for gr in graphs:
        with torch.cuda.graph(gr):
            step()
    ca.lengths.copy_(lengths)
    for i in range(6):
        graphs[i % 2].replay()
        ca.c["lengths"] = ca.c["lengths"] + 1
        ca.c = kv8.append(ca.c, x[0].double().numpy(), x[1].double().numpy())
        check_attend(ca, q, 0.1, "bf16", o, lse)
        ref = kv8.add_weights(ca.c, q.double().numpy(), 0.1, lse.double().cpu().numpy())
        got = ca.w.double().cpu().numpy()
        held = (np.arange(cap) < ca.c["lengths"][:, None])[:, None].repeat(Hk, 1)
        assert np.allclose(got[held], ref[held], rtol=2e-4, atol=0)
        ca.c["w"] = got
        ca.check(ca.c)


def test_captured_eviction_replays_with_new_weights():
    rng = np.random.default_rng(42)
    ca = Cache(rng, [300, 64], 2, 320, 64, 32)
    out = Cache(rng, [0, 0], 2, 128, 64, 32)
    out.c["k8"][:], out.c["v8"][:], out.c["ks"][:], out.c["vs"][:] = 1.0, 1.0, 1.0, 1.0
    out.load()
    kept = torch.empty(2, 2, 100, dtype=torch.int32, device="cuda")
    call = lambda: ea.attn_kv8_evict(ca.k8, ca.v8, ca.ks, ca.vs, ca.w, ca.lengths, 100, out.k8, out.v8, out.ks,
                                     out.vs, out.w, out.lengths, sink=3, recent=20, kept=kept)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call_on_side = ea.attn_kv8_evict(ca.k8, ca.v8, ca.ks, ca.vs, ca.w, ca.lengths, 100, out.k8, out.v8, out.ks,
                                     out.vs, out.w, out.lengths, sink=3, recent=20, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        graph.replay()
        ref, pos = kv8.evict(ca.c, out.c, 100, 3, 20)
        assert kept.cpu().numpy().tolist() == pos.tolist()
        out.check(ref)
        w = rng.random(ca.c["w"].shape).astype(np.float32)
        ca.c["w"] = w.astype(np.float64)
        ca.w.copy_(torch.from_numpy(w))
    assert call_on_side.shape == kept.shape


def test_codes_as_bytes_are_the_same_cache():
    rng = np.random.default_rng(43)
    ca = Cache(rng, [90, 17], 2, 96, 128, 32)
    q = rounded(rng.normal(size=(2, 2, 1, 128)), "bf16").cuda()
    a = ea.attn_fwd_kv8(q, ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.1)
    b = ea.attn_fwd_kv8(q, ca.k8.view(torch.uint8), ca.v8.view(torch.uint8), ca.ks, ca.vs, ca.lengths, 0.1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_calls_on_two_streams_at_once():
    rng = np.random.default_rng(51)
    ca = Cache(rng, [3000, 2500], 4, 4096, 128, 64)
    qs = [rounded(rng.normal(size=(2, 16, 1, 128)), "bf16").cuda() for _ in range(2)]
    want = [ea.attn_fwd_kv8(q, ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.1) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [ea.attn_fwd_kv8(q, ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.1, stream=s)
               for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for (o, lse), (o2, lse2) in zip(want, got):
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_binding_refusals():
    rng = np.random.default_rng(61)
    ca = Cache(rng, [5], 2, 32, 64, 16)
    q = rounded(rng.normal(size=(1, 4, 1, 64)), "bf16").cuda()
    args = (ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths, 0.1)
    for bad in (q.float(), q[:, :3], q[..., :32], q.transpose(1, 2)):
        with pytest.raises(ValueError):
            ea.attn_fwd_kv8(bad, *args)
    with pytest.raises(ValueError):
        ea.attn_fwd_kv8(q, ca.k8, ca.v8[:, :1], *args[2:])
    with pytest.raises(ValueError):
        ea.attn_fwd_kv8(q, ca.k8, ca.v8, ca.ks, ca.vs, ca.lengths.long(), 0.1)
    with pytest.raises(ea.AttnError) as e:
        ea.attn_fwd_kv8(q, *args, mask="bitmap")
    assert e.value.code == ea.ATTN_ERR_UNSUPPORTED
    big = Cache(rng, [5], 2, 4096, 64, 16)
    with pytest.raises(ea.AttnError) as e:
        ea.attn_fwd_kv8(q, big.k8, big.v8, big.ks, big.vs, big.lengths, 0.1,
                        workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == ea.ATTN_ERR_WORKSPACE
    with pytest.raises(ea.AttnError) as e:  # the output cache may not be the input
        ea.attn_kv8_evict(ca.k8, ca.v8, ca.ks, ca.vs, ca.w, ca.lengths, 8, ca.k8, ca.v8, ca.ks, ca.vs, ca.w,
                          ca.lengths)
    assert e.value.code == ea.ATTN_ERR_INVALID_ARG


def test_runner(capsys):
    import json

    from exact_io_aware_gb300 import run

    rc = run.main("--kv8 --B 2 --H 8 --H-kv 2 --n 3 --n-kv 700 --d 64 --mask causal --iters 2 --json".split())
    out = json.loads(capsys.readouterr().out)
    assert rc == 0 and out["keep"] == 175 and all(out[f"{x}_us"] > 0 for x in ("append", "attend", "weights", "evict"))
