"""The 8-bit cache's binding: what it checks before anything reaches the GPU."""
import pytest
import torch

import exact_io_aware_gb300 as ea


class OnGpu:
    """Stands in for a contiguous CUDA tensor of device 0."""

    is_cuda = True

    def __init__(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


class StreamOf:
    def __init__(self, device_index):
        self.device_index = device_index


def cache(B=1, Hk=2, cap=32, d=64, block=16):
    f8, f32, i32, bf = torch.uint8, torch.float32, torch.int32, torch.bfloat16
    codes, scales = OnGpu((B, Hk, cap, d), f8), OnGpu((B, Hk, cap // block), f32)
    return dict(k8=codes, v8=codes, ks=scales, vs=scales, w=OnGpu((B, Hk, cap), f32), lens=OnGpu((B,), i32),
                q=OnGpu((B, 2 * Hk, 1, d), bf), kv=OnGpu((B, Hk, 1, d), bf), lse=OnGpu((B, 2 * Hk, 1), f32))


def calls(c, **kw):
    return {
        "append": lambda: ea.attn_kv8_append(c["kv"], c["kv"], c["k8"], c["v8"], c["ks"], c["vs"], c["lens"], **kw),
        "attend": lambda: ea.attn_fwd_kv8(c["q"], c["k8"], c["v8"], c["ks"], c["vs"], c["lens"], 0.1, **kw),
        "weights": lambda: ea.attn_kv8_weights(c["q"], c["k8"], c["ks"], c["lens"], c["lse"], c["w"], 0.1, **kw),
        "evict": lambda: ea.attn_kv8_evict(c["k8"], c["v8"], c["ks"], c["vs"], c["w"], c["lens"], 8, c["k8"],
                                           c["v8"], c["ks"], c["vs"], c["w"], c["lens"], **kw),
    }


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    """Nothing here may reach the GPU: whatever would set a device or a stream fails the test."""
    def reached(*a, **kw):
        raise AssertionError("reached CUDA")

    monkeypatch.setattr(torch.cuda, "current_device", reached)
    monkeypatch.setattr(torch.cuda, "set_device", reached)
    monkeypatch.setattr(torch.cuda, "stream", reached)


@pytest.mark.parametrize("op", ["append", "attend", "weights", "evict"])
def test_a_stream_of_another_device_is_refused(op):
    with pytest.raises(ValueError, match="stream"):
        calls(cache(), stream=StreamOf(1))[op]()
    with pytest.raises(AssertionError, match="reached CUDA"):  # its own device's is taken
        calls(cache(), stream=StreamOf(0))[op]()


@pytest.mark.parametrize("op", ["append", "attend", "weights", "evict"])
@pytest.mark.parametrize("sizes", [dict(Hk=0), dict(cap=0)])
def test_a_cache_of_no_heads_or_no_room_is_refused(op, sizes):
    c = cache(**sizes)
    if "cap" in sizes:
        c["ks"] = c["vs"] = OnGpu((1, 2, 1), torch.float32)
    with pytest.raises(ValueError):
        calls(c)[op]()
