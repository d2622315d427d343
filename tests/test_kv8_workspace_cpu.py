"""attn_fwd_kv8_workspace_bytes answers 0 for the sizes that attn_fwd_kv8 refuses."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_gb300.build import build

    build()
    import exact_io_aware_gb300 as ea

    return ea.load()


vp = ctypes.c_void_p
A = 1 << 20  # stand-in addresses: nothing is read before the checks refuse


@pytest.mark.parametrize("sizes,code", [  # dtype, B, H, H_kv, n_q, d, cap
    ((2, 300, 300, 300, 1, 64, 1024), -2),              # more than 65535 heads
    ((1, 1, 4, 4, 1, 128, (1 << 30) + 16), -2),         # cap past 2^30
    ((2, 1, 4, 2, 1 << 24, 64, 1024), -2),              # more than 2^24 rows a key/value head
    ((2, 1, 2, 1, 1, 64, 1000), -1),                    # cap no multiple of any block
    ((0, 1, 4, 2, 1, 64, 1024), -2),
    ((2, 1, 4, 2, 1, 96, 1024), -2),
])
def test_zero_for_refused_sizes(lib, sizes, code):
    assert lib.attn_fwd_kv8_workspace_bytes(*sizes) == 0
    dtype, B, H, Hk, n, d, cap = sizes
    ptr = [vp(A * (i + 1)) for i in range(12)]
    rc = lib.attn_fwd_kv8(dtype, B, H, Hk, n, d, cap, 16, 0.1, *ptr[:6], vp(0), 0, *ptr[7:9], ptr[9], 1 << 40, vp(0))
    assert rc == code and lib.attn_last_error().decode() != ""


def test_zero_for_a_work_list_past_its_bound(lib):
    """2^14 heads x 2^16 tiles of 256 rows x 2^10 steps: refused at the launch, so no address is given."""
    assert lib.attn_fwd_kv8_workspace_bytes(2, 1 << 14, 1, 1, 1, 64, 1 << 17) > 0
    assert lib.attn_fwd_kv8_workspace_bytes(2, 1 << 14, 1 << 14, 1, 1 << 10, 64, 1 << 17) == 0
