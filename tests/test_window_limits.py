"""Size limits of the decoding entry points, at their edges (CPU: a call within
them goes on to the device, which is not there)."""
import ctypes
import os

import pytest
import torch

import exact_tiled_attention_14_gb300 as fa


@pytest.mark.parametrize("B,H,Nq,Nk,ok", [
    # rows times (key tiles of a cache + 1) stay below 2^31, so the tiles of all units fit in an int
    (1 << 10, 1 << 10, 1, 2047 * 128, False),
    (1 << 10, 1 << 10, 1, 2047 * 128 + 1, False),
    (1 << 10, 1 << 10, 1, 2046 * 128, True),
    (1 << 10, (1 << 10) - 1, 1, 2047 * 128, True),
    (1 << 7, 1 << 9, 16, 2047 * 128, False),
    (1 << 7, 1 << 9, 16, 2046 * 128, True),
])
def test_rows_times_tiles(B, H, Nq, Nk, ok):
    if not os.path.exists(fa.LIB_PATH):
        fa.build()
    fa.load_library()
    if ok and torch.cuda.is_available():
        pytest.skip("a GPU is present")
    fake = 0x10000   # never dereferenced
    code = fa.fa_decode_window(fake, fake, fake, fake, fake, B, H, H, Nq, Nk, 64, 100, 4, None, 0.125,
                               fa.FA_FP16, fake, 1 << 40)
    assert code == (fa.FA_ERR_DEVICE if ok else fa.FA_ERR_SHAPE)
    size = fa.load_library().fa_decode_window_workspace_size
    out = ctypes.c_size_t(0)
    assert size(B, H, H, Nq, Nk, 64, ctypes.byref(out)) == code
