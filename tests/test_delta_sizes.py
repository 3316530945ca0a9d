"""Sizes of delta-rule calls that no launch holds: refused, and so are their workspaces' sizes (whose bytes would
leave 64 bits)."""
import ctypes

import pytest

BF16, F32 = 1, 0


@pytest.fixture(scope="module")
def lib():
    from bayesian_scan_gb300 import build
    build.build()
    from bayesian_scan_gb300 import kdn
    return kdn.lib


def ask(f, *sizes):
    n = ctypes.c_longlong(-7)
    return f(*sizes, ctypes.byref(n)), n.value


# heads x tokens of 2^51 (4.3 KB each: over 2^63 bytes), 2^38 (2^32 chunks), packed ones of as many
@pytest.mark.parametrize("B,H,T,nseq", [(1 << 15, 1 << 15, 1 << 21, 0), (1 << 12, 1 << 10, 1 << 16, 0), (1, 1 << 12, 1 << 26, 1 << 20),
                                        (1, 1 << 20, 1 << 20, 64)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_too_many_chunks(lib, B, H, T, nseq, dtype):
    back, forth = lib.kdn_delta_scan_bwd_workspace, lib.kdn_delta_scan_fwd_workspace
    assert ask(back, B, H, T, 128, 128, nseq, dtype) == (-1, -7)
    # token by token the forward needs none
    assert ask(forth, B, H, T, 128, 128, nseq, dtype) == ((-1, -7) if dtype == BF16 else (0, 0))
    p = ctypes.c_void_p(0x10000)
    off = p if nseq else None
    args = [p, p, p, p, p, p, None, off, nseq]
    sizes = [B, H, T, 128, 128, dtype, dtype]
    assert lib.kdn_delta_scan_bwd(*args, p, None, p, p, p, p, p, p, None, *sizes, p, 1 << 62, None) == -1
    if dtype == BF16:
        assert lib.kdn_delta_scan_fwd(*args, p, None, *sizes, p, 1 << 62, None) == -1


@pytest.mark.parametrize("B,H,T,nseq", [(8, 16, 4096, 0), (1, 1 << 10, 1 << 26, 0), (1, 64, 1 << 20, 32)])
def test_the_rest_is_answered(lib, B, H, T, nseq):
    for dtype in (BF16, F32):
        st, n = ask(lib.kdn_delta_scan_bwd_workspace, B, H, T, 128, 128, nseq, dtype)
        assert st == 0 and n >= B * H * T * 128 * 8
    st, n = ask(lib.kdn_delta_scan_fwd_workspace, B, H, T, 128, 128, nseq, BF16)
    assert st == 0 and n >= B * H * T * 128 * 4
