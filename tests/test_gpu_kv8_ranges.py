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
