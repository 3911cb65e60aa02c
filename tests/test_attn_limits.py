"""Host-side limits of include/gdr_attn.h (no GPU): sizes whose 32-bit places would wrap are refused."""
import ctypes

import numpy as np
import pytest

import chunked_gated_delta_04_gb300 as gdr
from chunked_gated_delta_04_gb300 import build as gbuild

FAKE = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdr.load()


def packed(Tq, Tk, window):
    return gdr.gdr_attn_problem(1, Tq, Tk, 1, 1, 16, 2, FAKE, FAKE, gdr.GDR_DTYPE_BF16, 1, window, 0.0, 0, 0, 0, 0)


def test_the_first_key_of_a_window_is_a_32_bit_number(lib):
    """Of a sequence with n queries and one key the first query's window begins at 1 - n - window + 1: beyond -2^31 it would
    wrap to a place behind the last key, and the window be empty."""
    n, window = 1200000000, 1100000000
    with np.errstate(over="ignore"):
        assert np.int32(1) - np.int32(n) - np.int32(window) + np.int32(1) > 0
    p = packed(n + 1, window + 2, window)
    assert lib.gdr_attn_fwd(ctypes.byref(p), *[FAKE] * 6, 1 << 40, 0) == gdr.GDR_ERR_UNSUPPORTED
    assert lib.gdr_attn_bwd(ctypes.byref(p), *[FAKE] * 10, 1 << 40, 0) == gdr.GDR_ERR_UNSUPPORTED
    assert lib.gdr_attn_fwd_workspace_bytes(ctypes.byref(p)) == 0 == lib.gdr_attn_bwd_workspace_bytes(ctypes.byref(p))


def test_what_does_not_wrap_is_taken(lib):
    n, window = 1200000000, 1100000000
    for p in (packed(n + 1, window + 2, 0),               # no window
              packed(n + 1, window + 2, window + 2),      # one that hides nothing
              packed(n + 1, window + 2, (1 << 31) - 1025 - n - 1)):
        assert lib.gdr_attn_fwd_workspace_bytes(ctypes.byref(p)) > 256 and lib.gdr_attn_bwd_workspace_bytes(ctypes.byref(p)) > 256
