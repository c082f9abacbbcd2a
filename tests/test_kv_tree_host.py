"""Host-side refusals of nvfp4_kv_tree_attention, and kv_trees (no GPU, no kernel)."""
import os

import pytest
import torch

import nvfp4_block_scaled_amd as nv

INV, UNSUP = nv.NVFP4_ERR_INVALID_ARGUMENT, nv.NVFP4_ERR_UNSUPPORTED
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


def cache(pages=10, page_size=16, heads=2, dim=128):
    return nv._KVCacheStruct(A, B, C, D, None, None, pages, page_size, heads, dim)


def attend(L, c, q=A, dt=2, tokens=12, query_heads=8, qt=1024, qh=128, table=B, seqs=4, table_pages=8, lens=C, starts=E,
           max_queries=5, max_context=100, scale=0.1, tree=F, words=1, positions=None, window=0, out=D, lse=None, nbytes=None):
    need = L.nvfp4_kv_tree_attention_workspace_size(c, tokens, query_heads, seqs, max_queries, max_context, window)
    return L.nvfp4_kv_tree_attention(c, q, dt, tokens, query_heads, qt, qh, table, seqs, table_pages, lens, starts, max_queries,
                                     max_context, scale, tree, words, positions, window, out, lse, 0x70000,
                                     need if nbytes is None else nbytes, None)


@pytest.mark.parametrize("bad,status,says", [
    (dict(dt=9), INV, "dtype"), (dict(tokens=-1), INV, "tokens"), (dict(query_heads=7), INV, "multiple of heads"),
    (dict(max_queries=0), INV, "positive"), (dict(max_context=129), INV, "table_pages"), (dict(scale=0.0), INV, "scale"),
    (dict(window=-1), INV, "window"), (dict(qt=-1), INV, "strides"), (dict(starts=None), INV, "query_starts"),
    (dict(words=0), INV, "tree_words"), (dict(words=-1), INV, "tree_words"), (dict(words=1 << 25), INV, "tree_words"),
    (dict(max_queries=65), INV, "tree_words"), (dict(tree=None), INV, "NULL"), (dict(window=9), INV, "positions"),
    (dict(tree=F + 4), INV, "aligned"), (dict(positions=E + 2), INV, "aligned"), (dict(out=D + 8), INV, "aligned"),
    (dict(q=None), INV, "NULL"), (dict(starts=E + 1), INV, "aligned"), (dict(seqs=70000), UNSUP, "too large")])
def test_errors(L, bad, status, says):
    assert attend(L, cache(), **bad) == status, bad
    text = L.nvfp4_last_error().decode()
    assert "[kv_tree_attention]" in text and says in text, text


def test_accepts(L):
    for more in (dict(), dict(words=2, max_queries=100, tokens=200), dict(window=9, positions=E), dict(lse=A), dict(dt=0),
                 dict(tokens=0, tree=None, q=None), dict(seqs=0), dict(tree=F + 8)):
        assert attend(L, cache(), **more) == UNSUP and "gfx950" in L.nvfp4_last_error().decode(), more


def test_trees():
    tree, depths = nv.kv_trees([[-1, 0, 0, 1, -1], [], [-1]])
    assert tree.tolist() == [[1], [3], [5], [11], [16], [1]] and depths.tolist() == [0, 1, 1, 2, 0, 0]
    tree, depths = nv.kv_trees([list(range(-1, 129))])
    assert tree.shape == (130, 3) and depths.tolist() == list(range(130))
    assert tree[63].tolist() == [-1, 0, 0] and tree[129].tolist() == [-1, -1, 3]
    assert nv.kv_trees([])[0].shape == (0, 1) and nv.kv_trees([[]])[1].shape == (0,)
    for bad in ([[0]], [[-2]], [[-1, 1]], [[-1, 0, 3]]):
        with pytest.raises(ValueError):
            nv.kv_trees(bad)


def test_python_refusals():
    c = nv.kv_cache(2, 4, 3, 64, device="cpu")
    with pytest.raises(ValueError):  # host tensors
        nv.nvfp4_kv_tree_attention(torch.zeros(5, 6, 64), c, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                                   torch.zeros(2, dtype=torch.int32), torch.zeros(5, 1, dtype=torch.int64))
