"""The 8-bit cache's entry points refuse bad arguments on the host, before any CUDA call."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_gb300.build import build

    build()
    import exact_io_aware_gb300 as ea

    return ea.load()


vp = ctypes.c_void_p
A = 1 << 20  # stand-in addresses, far apart; nothing is read before the checks refuse


def _append(lib, **kw):
    a = dict(dtype=2, B=2, Hk=2, n=3, d=64, cap=64, block=16, k=A, v=2 * A, lens=3 * A, cnt=0,
             k8=4 * A, v8=5 * A, ks=6 * A, vs=7 * A, w=8 * A)
    a.update(kw)
    return lib.attn_kv8_append(a["dtype"], a["B"], a["Hk"], a["n"], a["d"], a["cap"], a["block"],
                               *(vp(a[x]) for x in ("k", "v", "lens", "cnt", "k8", "v8", "ks", "vs", "w")),
                               vp(0))


COMMON = [
    (dict(B=0), -1), (dict(Hk=-1), -1), (dict(d=32), -2), (dict(d=96), -2), (dict(block=8), -2),
    (dict(block=48), -2), (dict(cap=0), -1), (dict(cap=72), -1), (dict(B=300, Hk=300), -2),
    (dict(k8=0), -1), (dict(k8=A + 8), -3), (dict(ks=0), -1), (dict(ks=6 * A + 2), -3),
    (dict(lens=0), -1), (dict(lens=3 * A + 1), -3), (dict(cnt=9 * A + 2), -3),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dtype=0), -2), (dict(dtype=3), -1), (dict(n=0), -1), (dict(k=0), -1), (dict(v=2 * A + 4), -3),
    (dict(v8=0), -1), (dict(vs=0), -1), (dict(w=8 * A + 1), -3),
])
def test_append_refuses(lib, kw, code):
    assert _append(lib, **kw) == code
    assert lib.attn_last_error().decode() != ""


def _attend(lib, **kw):
    a = dict(dtype=2, B=2, H=4, Hk=2, n=3, d=64, cap=64, block=16, q=A, k8=2 * A, v8=4 * A, ks=5 * A,
             vs=6 * A, lens=3 * A, cnt=0, mask=0, o=7 * A, lse=8 * A, ws=10 * A, ws_bytes=1 << 30)
    a.update(kw)
    return lib.attn_fwd_kv8(a["dtype"], a["B"], a["H"], a["Hk"], a["n"], a["d"], a["cap"], a["block"], 0.1,
                            *(vp(a[x]) for x in ("q", "k8", "v8", "ks", "vs", "lens", "cnt")), a["mask"],
                            vp(a["o"]), vp(a["lse"]), vp(a["ws"]), a["ws_bytes"], vp(0))


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dtype=0), -2), (dict(H=3), -1), (dict(H=0), -1), (dict(n=0), -1), (dict(mask=2), -2),
    (dict(mask=5), -1), (dict(q=0), -1), (dict(o=0), -1), (dict(lse=0), -1), (dict(o=7 * A + 2), -3),
    (dict(n=1 << 24), -2), (dict(ws=10 * A + 8), -3),
])
def test_attend_refuses(lib, kw, code):
    assert _attend(lib, **kw) == code
    assert lib.attn_last_error().decode() != ""


def _weights(lib, **kw):
    a = dict(dtype=2, B=2, H=4, Hk=2, n=3, d=64, cap=64, block=16, q=A, k8=2 * A, ks=5 * A, lens=3 * A,
             cnt=0, mask=0, lse=7 * A, w=8 * A, out=10 * A)
    a.update(kw)
    return lib.attn_kv8_weights(a["dtype"], a["B"], a["H"], a["Hk"], a["n"], a["d"], a["cap"], a["block"],
                                0.1, *(vp(a[x]) for x in ("q", "k8", "ks", "lens", "cnt")), a["mask"],
                                vp(a["lse"]), vp(a["w"]), vp(a["out"]), vp(0))


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dtype=0), -2), (dict(H=3), -1), (dict(n=0), -1), (dict(mask=2), -2), (dict(q=0), -1),
    (dict(lse=0), -1), (dict(out=0), -1), (dict(out=8 * A + 16), -1), (dict(w=8 * A + 2), -3),
])
def test_weights_refuses(lib, kw, code):
    assert _weights(lib, **kw) == code
    assert lib.attn_last_error().decode() != ""


def _evict(lib, **kw):
    a = dict(B=2, Hk=2, d=64, cap=64, block=16, k8=A, v8=2 * A, ks=3 * A, vs=4 * A, w=5 * A, lens=6 * A,
             keep=20, sink=4, recent=8, cap_out=32, k8o=7 * A, v8o=8 * A, kso=10 * A, vso=11 * A,
             wo=12 * A, lo=13 * A, kept=14 * A)
    a.update(kw)
    a.pop("cnt", None)
    return lib.attn_kv8_evict(a["B"], a["Hk"], a["d"], a["cap"], a["block"],
                              *(vp(a[x]) for x in ("k8", "v8", "ks", "vs", "w", "lens")), a["keep"],
                              a["sink"], a["recent"], a["cap_out"],
                              *(vp(a[x]) for x in ("k8o", "v8o", "kso", "vso", "wo", "lo", "kept")), vp(0))


@pytest.mark.parametrize("kw,code", [
    x for x in COMMON if "cnt" not in x[0] and "ks" not in x[0] and "lens" not in x[0]
] + [
    (dict(keep=0), -1), (dict(keep=33), -1), (dict(sink=-1), -1), (dict(recent=17), -1),
    (dict(cap_out=24), -1), (dict(cap_out=0), -1), (dict(kept=0), -1), (dict(lo=6 * A), -1),
    (dict(k8o=A), -1), (dict(wo=5 * A + 64), -1), (dict(k8o=8 * A), -1), (dict(w=0), -1), (dict(lens=0), -1),
    (dict(kso=10 * A + 1), -3), (dict(v8o=8 * A + 8), -3),
])
def test_evict_refuses(lib, kw, code):
    assert _evict(lib, **kw) == code
    assert lib.attn_last_error().decode() != ""


def test_workspace_query_refuses_sizes(lib):
    for bad in ((0, 1, 4, 2, 1, 64, 64), (2, 0, 4, 2, 1, 64, 64), (2, 1, 3, 2, 1, 64, 64),
                (2, 1, 4, 0, 1, 64, 64), (2, 1, 4, 2, 1, 32, 64), (2, 1, 4, 2, 0, 64, 64)):
        assert lib.attn_fwd_kv8_workspace_bytes(*bad) == 0


def test_binding_refuses_tensors_off_the_gpu(lib):
    import exact_io_aware_gb300 as ea

    f8 = torch.float8_e4m3fn
    k8 = torch.zeros(1, 2, 32, 64, dtype=torch.uint8).view(f8)
    s, lens = torch.ones(1, 2, 2), torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    for call in (lambda: ea.attn_kv8_append(x, x, k8, k8, s, s, lens),
                 lambda: ea.attn_fwd_kv8(x, k8, k8, s, s, lens, 0.1),
                 lambda: ea.attn_kv8_weights(x, k8, s, lens, s[..., 0:1], None, 0.1),
                 lambda: ea.attn_kv8_evict(k8, k8, s, s, s, lens, 8, k8, k8, s, s, s, lens)):
        with pytest.raises(ValueError):
            call()
