"""The largest launches of nvfp4_mx_rms_norm and nvfp4_kv_write_rotated, on the host: a launch has fewer than 2^32 threads in
a dimension, and what would take more is refused as such, not by the runtime (no GPU, no kernel)."""
import os

import pytest

import nvfp4_block_scaled_amd as nv

UNSUP = nv.NVFP4_ERR_UNSUPPORTED
A, B, C, D, E, F = (0x10000 * i for i in range(1, 7))  # fake aligned addresses


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_block_scaled_amd import build
        build.build()
    lib = nv.load_library()
    lib.nvfp4_debug_set_arch_override(b"gfx942")  # nothing reaches a device
    yield lib
    lib.nvfp4_debug_set_arch_override(None)


@pytest.mark.parametrize("rows,k,packed,fits", [
    # 1024 threads a row from k 16385 on; packed rows in tiles of 32, eight tiles at a time
    (2 ** 22 - 255, 16416, 1, False), (2 ** 22 - 1, 1 << 20, 1, False), (2 ** 22 - 256, 16416, 1, True),
    (2 ** 22 - 1, 16384, 1, True), (2 ** 22 - 1, 1 << 20, 0, True), (2 ** 22, 32, 0, False)])
def test_norm(L, rows, k, packed, fits):
    assert L.nvfp4_mx_rms_norm(A, None, None, 2, 8, rows, k, 1e-6, packed, None, None, B, C, None) == UNSUP
    text = L.nvfp4_last_error().decode()
    assert ("gfx950" if fits else "too large") in text, text


@pytest.mark.parametrize("tokens,fits", [(2 ** 26 - 4, True), (2 ** 26 - 3, False), (2 ** 26, False)])
def test_rotation(L, tokens, fits):
    """256 threads take four tokens."""
    cache = nv._KVCacheStruct(A, B, C, D, None, None, 10, 16, 1, 16)
    assert L.nvfp4_kv_write_rotated(cache, A, B, 2, tokens, 16, 16, 16, 16, C, D, E, 100, 16, 0, None, 0, 0, 0, None, None) == UNSUP
    text = L.nvfp4_last_error().decode()
    assert ("gfx950" if fits else "too large") in text, text
