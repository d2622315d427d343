"""The entry points for trees of drafted tokens refuse bad arguments on the host, before any CUDA call."""
import ctypes

import pytest
import torch

from test_kv8_binding_cpu import OnGpu, StreamOf, cache


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_gb300.build import build

    build()
    import exact_io_aware_gb300 as ea

    return ea.load()


vp = ctypes.c_void_p
A = 1 << 20  # stand-in addresses, far apart; nothing is read before the checks refuse


def _mask(lib, **kw):
    a = dict(B=2, n=40, parents=A, counts=0, tree=2 * A)
    a.update(kw)
    return lib.attn_tree_mask(a["B"], a["n"], *(vp(a[x]) for x in ("parents", "counts", "tree")), vp(0))


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -1), (dict(n=0), -1), (dict(n=-3), -1), (dict(n=1025), -2), (dict(B=(1 << 24) + 1), -2),
    (dict(parents=0), -1), (dict(tree=0), -1), (dict(parents=A + 2), -3), (dict(tree=2 * A + 1), -3),
    (dict(counts=3 * A + 2), -3), (dict(tree=A), -1), (dict(tree=A + 316), -1), (dict(counts=2 * A + 8), -1),
])
def test_tree_mask_refuses(lib, kw, code):
    assert _mask(lib, **kw) == code
    assert lib.attn_last_error().decode() != ""


def _attend(lib, **kw):
    a = dict(dtype=2, B=2, H=4, Hk=2, n=3, d=64, cap=64, block=16, q=A, k8=2 * A, v8=4 * A, ks=5 * A,
             vs=6 * A, lens=3 * A, cnt=0, tree=9 * A, o=7 * A, lse=8 * A, ws=10 * A, ws_bytes=1 << 30)
    a.update(kw)
    return lib.attn_fwd_kv8_tree(a["dtype"], a["B"], a["H"], a["Hk"], a["n"], a["d"], a["cap"], a["block"], 0.1,
                                 *(vp(a[x]) for x in ("q", "k8", "v8", "ks", "vs", "lens", "cnt", "tree", "o",
                                                      "lse", "ws")), a["ws_bytes"], vp(0))


CACHE = [
    (dict(B=0), -1), (dict(Hk=-1), -1), (dict(d=32), -2), (dict(block=8), -2), (dict(cap=0), -1),
    (dict(cap=72), -1), (dict(B=300, Hk=300), -2), (dict(k8=0), -1), (dict(k8=A + 8), -3), (dict(ks=0), -1),
    (dict(ks=6 * A + 2), -3), (dict(lens=0), -1), (dict(lens=3 * A + 1), -3), (dict(cnt=11 * A + 2), -3),
]


@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(dtype=0), -2), (dict(dtype=7), -1), (dict(H=3), -1), (dict(H=0), -1), (dict(n=0), -1), (dict(q=0), -1),
    (dict(o=0), -1), (dict(lse=0), -1), (dict(o=7 * A + 2), -3), (dict(n=1 << 24), -2), (dict(tree=0), -1),
    (dict(tree=9 * A + 2), -3), (dict(ws=10 * A + 8), -3),
])
def test_attend_tree_refuses(lib, kw, code):
    assert _attend(lib, **kw) == code
    assert lib.attn_last_error().decode() != ""


def _verify(lib, **kw):
    a = dict(dtype=0, B=2, n=5, V=100, target=A, draft=2 * A, tokens=3 * A, parents=4 * A, counts=0,
             uniforms=5 * A, path=6 * A, accepted=7 * A, token=8 * A)
    a.update(kw)
    return lib.attn_draft_verify(a["dtype"], a["B"], a["n"], a["V"],
                                 *(vp(a[x]) for x in ("target", "draft", "tokens", "parents", "counts", "uniforms",
                                                      "path", "accepted", "token")), vp(0))


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(B=0), -1), (dict(n=0), -1), (dict(n=1025), -2), (dict(V=0), -1),
    (dict(V=(1 << 30) + 1), -2), (dict(target=0), -1), (dict(tokens=0), -1), (dict(parents=0), -1),
    (dict(uniforms=0), -1), (dict(path=0), -1), (dict(accepted=0), -1), (dict(token=0), -1),
    (dict(target=A + 4), -3), (dict(draft=2 * A + 8), -3), (dict(tokens=3 * A + 2), -3), (dict(counts=9 * A + 1), -3),
    (dict(path=3 * A), -1), (dict(path=A + 64), -1), (dict(accepted=6 * A + 36), -1), (dict(token=7 * A + 4), -1),
    (dict(counts=8 * A), -1), (dict(path=2 * A + 3996), -1),
])
def test_verify_refuses(lib, kw, code):
    assert _verify(lib, **kw) == code
    assert lib.attn_last_error().decode() != ""


def _keep(lib, **kw):
    a = dict(B=2, Hk=2, n=5, d=64, cap=64, block=16, k8=A, v8=2 * A, ks=3 * A, vs=4 * A, lens=5 * A, cnt=0,
             path=6 * A, acc=7 * A, w=8 * A, out=10 * A)
    a.update(kw)
    return lib.attn_kv8_keep(a["B"], a["Hk"], a["n"], a["d"], a["cap"], a["block"],
                             *(vp(a[x]) for x in ("k8", "v8", "ks", "vs", "lens", "cnt", "path", "acc", "w", "out")),
                             vp(0))


@pytest.mark.parametrize("kw,code", [x for x in CACHE if "lens" not in x[0]] + [
    (dict(n=0), -1), (dict(n=(1 << 30) + 1), -2), (dict(v8=0), -1), (dict(vs=0), -1), (dict(path=0), -1),
    (dict(acc=0), -1), (dict(out=0), -1), (dict(w=8 * A + 2), -3), (dict(path=6 * A + 1), -3), (dict(out=5 * A), -1),
    (dict(v8=A), -1), (dict(out=7 * A), -1), (dict(w=8 * A, out=8 * A + 4), -1), (dict(cnt=10 * A + 4), -1),
    (dict(lens=0), -1), (dict(lens=5 * A + 2), -3),
])
def test_keep_refuses(lib, kw, code):
    assert _keep(lib, **kw) == code
    assert lib.attn_last_error().decode() != ""


# ------------------------------------------------------------------ the binding

def tensors(B=1, n=3, V=8, dtype=torch.float32, **kw):
    i32 = torch.int32
    t = dict(target=OnGpu((B, n, V), dtype), draft=OnGpu((B, n, V), dtype), nodes=OnGpu((B, n), i32),
             uniforms=OnGpu((B, n), torch.float32), tree=OnGpu((B, n, -(-n // 32)), i32), one=OnGpu((B,), i32))
    c = cache(B=B)
    c["q"] = OnGpu((B, 4, n, 64), torch.bfloat16)
    c.update(t)
    c.update(kw)
    return c


def calls(c, **kw):
    import exact_io_aware_gb300 as ea

    return {
        "mask": lambda: ea.attn_tree_mask(c["nodes"], **kw),
        "attend": lambda: ea.attn_fwd_kv8_tree(c["q"], c["k8"], c["v8"], c["ks"], c["vs"], c["lens"], c["tree"], 0.1, **kw),
        "verify": lambda: ea.attn_draft_verify(c["target"], c["draft"], c["nodes"], c["nodes"], c["uniforms"], **kw),
        "keep": lambda: ea.attn_kv8_keep(c["k8"], c["v8"], c["ks"], c["vs"], c["lens"], c["nodes"], c["one"], **kw),
    }


OPS = ["mask", "attend", "verify", "keep"]


@pytest.fixture
def no_gpu(monkeypatch):
    def reached(*a, **kw):
        raise AssertionError("reached CUDA")

    for name in ("current_device", "set_device", "stream"):
        monkeypatch.setattr(torch.cuda, name, reached)


@pytest.mark.parametrize("op", OPS)
def test_a_stream_of_another_device_is_refused(no_gpu, op):
    with pytest.raises(ValueError, match="stream"):
        calls(tensors(), stream=StreamOf(1))[op]()
    with pytest.raises(AssertionError, match="reached CUDA"):  # its own device's is taken
        calls(tensors(), stream=StreamOf(0))[op]()


class Elsewhere(OnGpu):
    def get_device(self):
        return 1


class Strided(OnGpu):
    def is_contiguous(self):
        return False


@pytest.mark.parametrize("op,kw", [
    ("mask", dict(nodes=OnGpu((1, 3), torch.int64))), ("mask", dict(nodes=OnGpu((3,), torch.int32))),
    ("mask", dict(nodes=OnGpu((1, 0), torch.int32))), ("mask", dict(nodes=Strided((1, 3), torch.int32))),
    ("attend", dict(tree=None)), ("attend", dict(tree=OnGpu((1, 3, 2), torch.int32))),
    ("attend", dict(tree=OnGpu((1, 3, 1), torch.int64))), ("attend", dict(tree=Elsewhere((1, 3, 1), torch.int32))),
    ("attend", dict(q=OnGpu((1, 4, 3, 64), torch.float32))), ("attend", dict(q=OnGpu((1, 3, 3, 64), torch.bfloat16))),
    ("verify", dict(target=OnGpu((1, 3, 8), torch.float64))), ("verify", dict(target=OnGpu((1, 3, 0), torch.float32))),
    ("verify", dict(draft=OnGpu((1, 3, 8), torch.bfloat16))), ("verify", dict(draft=OnGpu((1, 3, 9), torch.float32))),
    ("verify", dict(draft=Elsewhere((1, 3, 8), torch.float32))), ("verify", dict(uniforms=OnGpu((1, 3), torch.float64))),
    ("verify", dict(nodes=OnGpu((1, 4), torch.int32))),
    ("keep", dict(nodes=OnGpu((2, 3), torch.int32))), ("keep", dict(nodes=OnGpu((1, 3), torch.int64))),
    ("keep", dict(one=OnGpu((3,), torch.int32))), ("keep", dict(k8=OnGpu((1, 2, 32, 64), torch.float32))),
])
def test_binding_refuses(no_gpu, op, kw):
    with pytest.raises(ValueError):
        calls(tensors(**kw))[op]()


def test_binding_refuses_tensors_off_the_gpu():
    import exact_io_aware_gb300 as ea

    i, p = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, 3, 8)
    k8, s, one = torch.zeros(1, 2, 32, 64, dtype=torch.uint8), torch.ones(1, 2, 2), torch.ones(1, dtype=torch.int32)
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    for call in (lambda: ea.attn_tree_mask(i), lambda: ea.attn_draft_verify(p, p, i, i, p[..., 0]),
                 lambda: ea.attn_fwd_kv8_tree(q, k8, k8, s, s, one, i[..., None], 0.1),
                 lambda: ea.attn_kv8_keep(k8, k8, s, s, one, i, one)):
        with pytest.raises(ValueError):
            call()
