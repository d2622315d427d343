"""Pins of the 8-bit cache's oracle: hand values, and reductions to the dense definition."""
import numpy as np
import pytest

from oracle import attention as ref
from oracle import kv8, masks


def test_block_scale_by_hand():
    assert kv8.block_scale([448.0]) == 1.0
    assert kv8.block_scale([448.5]) == 2.0
    assert kv8.block_scale([224.0, -1.0]) == 0.5
    assert kv8.block_scale([0.0]) == 2.0 ** -100
    assert kv8.block_scale([np.inf, np.nan, 3.5]) == 2.0 ** -7      # 448 / 128 = 3.5
    assert kv8.block_scale([3.4e38]) == 2.0 ** 120


def test_codes_by_hand():
    got = kv8.codes([1.0625, 1.1875, 500.0, np.inf, np.nan, 2.0 ** -10, 3 * 2.0 ** -11], 1.0)
    assert got[:3].tolist() == [1.0, 1.25, 448.0]                   # ties to even, saturation
    assert np.isnan(got[3:5]).all()
    assert got[5:].tolist() == [0.0, 2.0 ** -9]                     # half the least subnormal: even


def _cache(B=1, Hk=1, cap=32, d=64, block=16, lengths=(0,)):
    return dict(k8=np.zeros((B, Hk, cap, d)), v8=np.zeros((B, Hk, cap, d)),
                ks=np.ones((B, Hk, cap // block)), vs=np.ones((B, Hk, cap // block)),
                w=np.ones((B, Hk, cap)), lengths=np.array(lengths))


def test_append_grows_a_block_by_hand():
    c = _cache(lengths=(1,))
    c = kv8.append(c, np.full((1, 1, 1, 64), 1.0), np.full((1, 1, 1, 64), 448.0))
    assert c["ks"][0, 0, 0] == 2.0 ** -8 and (c["k8"][0, 0, 0] == 256.0).all()
    assert c["vs"][0, 0, 0] == 1.0 and (c["v8"][0, 0, 0] == 448.0).all()
    assert c["w"][0, 0].tolist() == [0.0] + [1.0] * 31
    c["lengths"][0] = 2
    c = kv8.append(c, np.full((1, 1, 1, 64), 7.0), np.full((1, 1, 1, 64), 0.5))
    assert c["ks"][0, 0, 0] == 2.0 ** -6                            # 7 = 448 / 64
    assert (c["k8"][0, 0, 0] == 64.0).all() and (c["k8"][0, 0, 1] == 448.0).all()
    assert c["vs"][0, 0, 0] == 1.0 and (c["v8"][0, 0, 1] == 0.5).all()
    assert (c["k8"][0, 0, 2:] == 0).all() and (c["ks"][0, 0, 1:] == 1).all()


def test_append_drops_tokens_before_the_start_and_pads():
    c = _cache(lengths=(2,))
    x = np.arange(1, 6, dtype=float).reshape(1, 1, 5, 1) * np.ones(64)
    got = kv8.append(c, x, x, counts=[4])                           # tokens 1, 2 at -2, -1
    assert (got["k8"][0, 0, 0] * got["ks"][0, 0, 0] == 3.0).all()
    assert (got["k8"][0, 0, 1] * got["ks"][0, 0, 0] == 4.0).all()
    assert (got["k8"][0, 0, 2:] == 0).all()


@pytest.mark.parametrize("causal", [False, True])
def test_attend_is_the_dense_forward_on_the_dequantized_cache(causal):
    rng = np.random.default_rng(5)
    c = _cache(B=2, Hk=2, lengths=(29, 17))
    for x in "kv":
        c[x + "8"] = kv8.codes(rng.normal(size=c["k8"].shape) * 100, 1.0)
        c[x + "s"] = 2.0 ** rng.integers(-9, -5, size=c["ks"].shape)
    q = rng.normal(size=(2, 4, 3, 64))
    O, L, A, _, _ = kv8.attend(c, q, 0.1, causal=causal)
    w = kv8.add_weights(c, q, 0.1, L, causal=causal)
    for b in range(2):
        m = int(c["lengths"][b])
        allowed = masks.causal_rect(3, m)(0, np.arange(3)) if causal else np.ones((3, m), bool)
        for h in range(4):
            k, v = (c[x + "8"][b, h // 2, :m] * np.repeat(c[x + "s"][b, h // 2], 16)[:m, None] for x in "kv")
            Y, lse, _, _ = ref.forward_rows(q[b, h], k, v, 0.1, allowed)
            assert np.allclose(O[b, h], Y, atol=1e-12) and np.allclose(L[b, h], lse, atol=1e-12)
            assert (np.abs(O[b, h]) <= A[b, h] + 1e-12).all()
    # Every row's weights sum to one: a head of G rows and n queries adds G n to its keys' sum.
    assert np.allclose((w - c["w"]).sum(-1), 2 * 3, atol=1e-12)


def test_attend_rows_that_see_nothing():
    c = _cache(B=2, lengths=(0, 2))
    O, L, _, _, _ = kv8.attend(c, np.ones((2, 1, 4, 64)), 1.0, counts=[4, 3], causal=True)
    assert (O == 0).all()
    assert np.isneginf(L[0]).all()
    assert np.isneginf(L[1, 0, [0, 3]]).all() and np.allclose(L[1, 0, 1:3], [0.0, np.log(2)])


def test_kept_tokens_by_hand():
    w = np.array([5.0, 1.0, 3.0, 3.0, np.nan, 3.0, 0.0, -0.0])
    assert kv8.kept_tokens(w, 8, 8, 0, 0) == list(range(8))
    assert kv8.kept_tokens(w, 8, 3, 0, 0) == [0, 2, 3]              # ties: lower position
    assert kv8.kept_tokens(w, 8, 4, 0, 1) == [0, 2, 3, 7]
    assert kv8.kept_tokens(w, 8, 4, 2, 2) == [0, 1, 6, 7]
    assert kv8.kept_tokens(w, 8, 7, 0, 0) == [0, 1, 2, 3, 5, 6, 7]  # NaN lowest
    assert kv8.kept_tokens(w, 8, 6, 0, 0) == [0, 1, 2, 3, 5, 6]     # -0 = +0: lower position


def test_evict_keeps_values_exactly_under_power_of_two_scales():
    rng = np.random.default_rng(6)
    c = _cache(cap=64, lengths=(50,))
    for x in "kv":
        c[x + "8"] = kv8.codes(rng.normal(size=c["k8"].shape) * 100, 1.0)
        c[x + "s"] = 2.0 ** rng.integers(-3, 0, size=c["ks"].shape)
    c["w"] = rng.random((1, 1, 64))
    out, kept = kv8.evict(c, _cache(cap=32), 20, sink=2, recent=5)
    at = kept[0, 0]
    assert at[:2].tolist() == [0, 1] and at[-5:].tolist() == list(range(45, 50))
    assert (np.diff(at) > 0).all() and out["lengths"][0] == 20
    for x in "kv":
        was = c[x + "8"][0, 0, at] * np.repeat(c[x + "s"][0, 0], 16)[at, None]
        now = out[x + "8"][0, 0, :20] * np.repeat(out[x + "s"][0, 0], 16)[:20, None]
        big = np.abs(was) > 2.0 ** -5 * 2.0 ** -1
        assert (was[big] == now[big]).all() and np.abs(was - now).max() <= 2.0 ** -10
    assert (out["k8"][0, 0, 20:] == 0).all() and (out["w"][0, 0, 20:] == 1).all()
