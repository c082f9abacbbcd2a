"""The largest launches of nvfp4_kv_tree_attention, on the host: its kernels count units of 256 keys of every sequence,
kv head and 128 rows in 32 bits, so calls that could have more than 2^30 of them are refused (no GPU, no kernel)."""
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


def says(L, seqs, heads, groups, queries, context, window=0, tokens=None):
    """What a call of these sizes is told, and the workspace that it is asked for."""
    page = 1 << 16
    cache = nv._KVCacheStruct(A, B, C, D, None, None, 64, page, heads, 16)
    tokens = queries if tokens is None else tokens
    sizes = tokens, heads * groups, seqs, queries, context, window
    need = L.nvfp4_kv_tree_attention_workspace_size(cache, *sizes)
    status = L.nvfp4_kv_tree_attention(cache, A, 2, tokens, heads * groups, 16 * heads * groups, 16, B, seqs, -(-context // page), C,
                                       E, queries, context, 0.1, F, -(-queries // 64), D, window, D, None, 0x100000, need, None)
    assert status == UNSUP
    return L.nvfp4_last_error().decode(), need


def units(seqs, heads, groups, queries, context, window=0):
    keys = min(context, window + queries) if window else context
    return seqs * heads * -(-queries * groups // 128) * (keys // 256 + 1)


@pytest.mark.parametrize("sizes", [
    (1023, 8, 8, 65, 1 << 24),               # 2^29 of a row tile, five row tiles
    (4096, 8, 8, 2048, 131072), (1, 1, 1, 2 ** 20, 1 << 25), (65535, 1024, 4, 2048, 0),
    (1024, 16, 8, 2048, 131072, 131071)])
def test_more_units_than_are_counted(L, sizes):
    assert units(*sizes) > 1 << 30 and sizes[0] * sizes[1] * (sizes[4] // 128 + 1) <= 1 << 30  # (nvfp4_kv_attention's limit)
    text, need = says(L, *sizes)
    assert "[kv_tree_attention]" in text and "too large" in text and need == 0, text


@pytest.mark.parametrize("sizes", [
    (16, 8, 4, 64, 16384), (1023, 2, 8, 64, (1 << 24) - 1), (16384, 64, 2, 17, 255 * 256 - 1), (1, 1, 1, 2 ** 20, (1 << 25) - 1),
    (1024, 16, 8, 2048, 131072, 1024),       # the window bounds the keys
    (65535, 1024, 4, 128, 0)])
def test_up_to_the_limit(L, sizes):
    assert units(*sizes) <= 1 << 30
    text, _ = says(L, *sizes)
    assert "gfx950" in text, text


def test_few_rows_have_no_row_tiles(L):
    """Up to 32 rows a head the limit is that of nvfp4_kv_attention."""
    for queries in (32, 33):
        text, _ = says(L, 8192, 4, 1, queries, (1 << 22) - 1)  # 2^29 units of 256, 2^30 of 128
        assert "gfx950" in text, text
    text, _ = says(L, 8193, 4, 1, 32, (1 << 22) - 1)
    assert "too large" in text, text


def test_workspace_is_that_of_the_workgroups(L):
    """A workgroup leaves two unfinished tiles at most, however many tiles there are: 512 workgroups of two parts of
    128 rows, not a part for every (sequence, head, 128 rows)."""
    cache = nv._KVCacheStruct(A, B, C, D, None, None, 64, 1 << 16, 8, 128)
    for seqs, queries in ((256, 64), (60000, 64), (16, 4096)):
        need = L.nvfp4_kv_tree_attention_workspace_size(cache, 2 ** 24, 32, seqs, queries, 4000, 0)
        assert 0 < need <= 2 * 512 * 128 * (4 * 128 + 8) + 512, (seqs, queries, need)
    one = L.nvfp4_kv_tree_attention_workspace_size(cache, 64, 32, 1, 64, 4000, 0)
    assert 0 < one <= (8 * 2 * 16 + 8 * 2) * 128 * (4 * 128 + 8) + 512  # units and tiles of a single sequence
