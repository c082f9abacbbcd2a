"""Host-side refusals of the key/value cache calls (no GPU, no kernel): every
argument error is reported before any HIP call, with the call's name."""
import ctypes
import os

import pytest

import nvfp4_block_scaled_amd as nv

INV, UNSUP = nv.NVFP4_ERR_INVALID_ARGUMENT, nv.NVFP4_ERR_UNSUPPORTED
F32, F16, BF16 = 0, 1, 2
A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000  # fake aligned addresses


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_block_scaled_amd import build
        build.build()
    lib = nv.load_library()
    lib.nvfp4_debug_set_arch_override(b"gfx942")  # nothing reaches a device
    yield lib
    lib.nvfp4_debug_set_arch_override(None)


def err(L):
    return L.nvfp4_last_error().decode()


def cache(pages=10, page_size=16, heads=2, dim=128, k_codes=A, k_scales=B, v_codes=C, v_scales=D):
    return nv._KVCacheStruct(k_codes, k_scales, v_codes, v_scales, None, None, pages, page_size, heads, dim)


def write(L, c, k=A, v=B, dt=BF16, tokens=4, strides=(256, 128, 256, 128), slots=C):
    return L.nvfp4_kv_write(c, k, v, dt, tokens, *strides, slots, None)


def attend(L, c, q=A, dt=BF16, tokens=4, query_heads=8, qt=1024, qh=128, table=B, seqs=4, table_pages=8, lens=C,
           starts=None, max_queries=1, max_context=100, scale=0.1, causal=1, window=0, out=D, lse=None, nbytes=None):
    need = L.nvfp4_kv_attention_workspace_size(c, tokens, query_heads, seqs, max_queries, max_context, window)
    return L.nvfp4_kv_attention(c, q, dt, tokens, query_heads, qt, qh, table, seqs, table_pages, lens, starts,
                                max_queries, max_context, scale, causal, window, out, lse, 0x50000,
                                need if nbytes is None else nbytes, None)


@pytest.mark.parametrize("bad,status,says", [
    (dict(pages=0), INV, "positive"), (dict(page_size=-1), INV, "positive"), (dict(heads=0), INV, "positive"),
    (dict(dim=24), INV, "group size 16"), (dict(dim=0), INV, "group size 16"), (dict(dim=272), UNSUP, "above 256"),
    (dict(k_codes=None), INV, "NULL"), (dict(v_scales=None), INV, "NULL"), (dict(v_codes=C + 8), INV, "aligned"),
    (dict(k_scales=B + 4), INV, "aligned"), (dict(pages=1 << 28, page_size=16), UNSUP, "2^31"),
    (dict(heads=40000), UNSUP, "heads")])
def test_cache_errors(L, bad, status, says):
    for call in (write, lambda L, c: L.nvfp4_kv_read(c, A, 4, B, C, BF16, None)):
        assert call(L, cache(**bad)) == status and says in err(L), err(L)
    if "heads" not in bad:
        assert attend(L, cache(**bad)) == status and says in err(L), err(L)
    assert L.nvfp4_kv_attention_workspace_size(cache(**bad), 4, 8, 4, 1, 100, 0) == 0


def test_write_and_read_errors(L):
    c = cache()
    assert write(L, None) == INV and "cache" in err(L)
    assert write(L, c, dt=5) == INV and "dtype" in err(L)
    assert write(L, c, tokens=-1) == INV and "tokens" in err(L)
    assert write(L, c, k=None) == INV and write(L, c, v=None) == INV and write(L, c, slots=None) == INV
    assert write(L, c, k=A + 1) == INV and "aligned" in err(L)
    assert write(L, c, k=A + 2, dt=F32) == INV and write(L, c, slots=C + 4) == INV
    assert write(L, c, strides=(256, -1, 256, 128)) == INV and "strides" in err(L)
    assert write(L, c, tokens=1 << 28) == UNSUP and "too large" in err(L)
    assert write(L, c) == UNSUP and "gfx950" in err(L)
    assert write(L, c, k=A + 2) == UNSUP and "gfx950" in err(L)  # element alignment is enough
    assert write(L, c, k=None, v=None, slots=None, tokens=0) == UNSUP and "gfx950" in err(L)
    read = L.nvfp4_kv_read
    assert read(None, A, 4, B, C, BF16, None) == INV and read(c, A, 4, B, C, 3, None) == INV
    assert read(c, None, 4, B, C, BF16, None) == INV and read(c, A, 4, None, C, BF16, None) == INV
    assert read(c, A, 4, B, C + 8, BF16, None) == INV and "16-byte" in err(L)
    assert read(c, A, -4, B, C, BF16, None) == INV
    assert read(c, A, 4, B, C, BF16, None) == UNSUP and "gfx950" in err(L)


@pytest.mark.parametrize("bad,status,says", [
    (dict(dt=9), INV, "dtype"), (dict(tokens=-1), INV, "tokens"), (dict(query_heads=7), INV, "multiple of heads"),
    (dict(query_heads=0), INV, "positive"), (dict(seqs=-1), INV, ">= 0"), (dict(max_queries=0), INV, "positive"),
    (dict(max_context=-1), INV, ">= 0"), (dict(max_context=129), INV, "table_pages"), (dict(table_pages=-1), INV, "table_pages"),
    (dict(scale=0.0), INV, "scale"), (dict(scale=-1.0), INV, "scale"), (dict(scale=float("nan")), INV, "scale"),
    (dict(scale=float("inf")), INV, "scale"), (dict(window=-1), INV, "window"), (dict(window=5, causal=0), INV, "window"),
    (dict(qt=-1), INV, "strides"), (dict(tokens=5), INV, "query_starts"), (dict(max_queries=2), INV, "query_starts"),
    (dict(q=None), INV, "NULL"), (dict(out=None), INV, "NULL"), (dict(lens=None), INV, "NULL"), (dict(table=None), INV, "NULL"),
    (dict(q=A + 1), INV, "aligned"), (dict(out=D + 8), INV, "aligned"), (dict(lse=A + 2), INV, "aligned"),
    (dict(starts=A + 2), INV, "aligned"), (dict(query_heads=65536), UNSUP, "too large"),
    (dict(seqs=70000, tokens=70000), UNSUP, "too large"), (dict(tokens=1 << 28, starts=A, query_heads=16, max_queries=9), UNSUP, "too large")])
def test_attention_errors(L, bad, status, says):
    assert attend(L, cache(), **bad) == status and says in err(L), err(L)


def test_attention_accepts(L):
    for more in (dict(), dict(starts=A, tokens=9, max_queries=5), dict(window=7), dict(causal=0), dict(lse=A),
                 dict(max_context=0, table=None, table_pages=0), dict(qt=0, qh=0), dict(tokens=0, seqs=0, q=None),
                 dict(dt=F32), dict(dt=F16, q=A + 2)):
        assert attend(L, cache(), **more) == UNSUP and "gfx950" in err(L), (more, err(L))


def test_workspace(L):
    """The workspace that a long context needs is asked for, and its size checked."""
    c = cache(pages=1 << 16)
    need = L.nvfp4_kv_attention_workspace_size(c, 1, 8, 1, 1, 1 << 20, 0)
    args = dict(tokens=1, seqs=1, table_pages=1 << 16, max_context=1 << 20)
    assert attend(L, c, **args) == UNSUP and "gfx950" in err(L)
    if need:
        assert attend(L, c, nbytes=need - 1, **args) == INV and "workspace" in err(L)


def test_python_refusals():
    """The binding's own checks, on CPU tensors."""
    import torch
    held = dict(k_codes=torch.zeros(2, 3, 4, 32, dtype=torch.uint8), k_scales=torch.zeros(2, 3, 4, 4, dtype=torch.uint8),
                v_codes=torch.zeros(2, 3, 4, 32, dtype=torch.uint8), v_scales=torch.zeros(2, 3, 4, 4, dtype=torch.uint8))
    c = nv.KVCache(**held)
    assert (c.pages, c.heads, c.page_size, c.dim) == (2, 3, 4, 64)
    for change in (dict(v_codes=held["v_codes"][:1]), dict(k_scales=held["k_scales"][..., :2]),
                   dict(k_codes=held["k_codes"].int()), dict(k_codes=held["k_codes"][0]),
                   dict(v_scales=held["v_scales"].transpose(0, 1).contiguous().transpose(0, 1)),
                   dict(global_scale_k=torch.ones(2)), dict(global_scale_v=torch.ones(1, dtype=torch.float64))):
        with pytest.raises(ValueError):
            nv.KVCache(**{**held, **change})
    with pytest.raises(ValueError):
        nv.kv_cache(1, 1, 1, 40, device="cpu")
    k = torch.zeros(5, 3, 64)
    with pytest.raises(ValueError):  # host tensors
        nv.nvfp4_kv_write(c, k, k, torch.zeros(5, dtype=torch.int64))
    with pytest.raises(ValueError):
        nv.nvfp4_kv_write(c, k[..., :32], k, torch.zeros(5, dtype=torch.int64))
    with pytest.raises(ValueError):
        nv.nvfp4_kv_read(c, torch.zeros(5, dtype=torch.int32))
    with pytest.raises(ValueError):
        nv.nvfp4_kv_attention(torch.zeros(5, 6, 64), c, torch.zeros(5, 1, dtype=torch.int32),
                              torch.zeros(5, dtype=torch.int32))
