"""Host-side refusals of nvfp4_kv_write_rotated (no GPU, no kernel)."""
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


def cache(pages=10, page_size=16, heads=2, dim=128, k_codes=A):
    return nv._KVCacheStruct(k_codes, B, C, D, None, None, pages, page_size, heads, dim)


def write(L, c, k=A, v=B, dt=2, tokens=4, strides=(256, 128, 256, 128), slots=C, positions=D, table=E, rows=100, rotary=64,
          interleaved=0, q=F, query_heads=4, qt=512, qh=128, out=A):
    return L.nvfp4_kv_write_rotated(c, k, v, dt, tokens, *strides, slots, positions, table, rows, rotary, interleaved, q,
                                    query_heads, qt, qh, out, None)


@pytest.mark.parametrize("bad,status,says", [
    (dict(dt=9), INV, "dtype"), (dict(tokens=-1), INV, "tokens"), (dict(strides=(256, 128, -1, 128)), INV, "strides"),
    (dict(qt=-5), INV, "strides"), (dict(rotary=0), INV, "rotary_dim"), (dict(rotary=24), INV, "rotary_dim"),
    (dict(rotary=144), INV, "rotary_dim"), (dict(rotary=-16), INV, "rotary_dim"), (dict(rows=-1), INV, ">= 0"),
    (dict(query_heads=-1), INV, ">= 0"), (dict(k=None), INV, "NULL"), (dict(v=None), INV, "NULL"), (dict(slots=None), INV, "NULL"),
    (dict(positions=None), INV, "NULL"), (dict(table=None), INV, "NULL"), (dict(q=None), INV, "NULL"), (dict(out=None), INV, "NULL"),
    (dict(k=A + 1), INV, "aligned"), (dict(q=F + 1), INV, "aligned"), (dict(v=B + 2, dt=0), INV, "aligned"),
    (dict(slots=C + 4), INV, "aligned"), (dict(positions=D + 2), INV, "aligned"), (dict(table=E + 8), INV, "aligned"),
    (dict(out=A + 8), INV, "aligned"), (dict(tokens=1 << 26), UNSUP, "too large"), (dict(query_heads=65536), UNSUP, "too large"),
    (dict(rows=1 << 31), UNSUP, "too large")])
def test_errors(L, bad, status, says):
    assert write(L, cache(), **bad) == status, bad
    text = L.nvfp4_last_error().decode()
    assert "[kv_write_rotated]" in text and says in text, text


def test_cache_errors(L):
    for c in (None, cache(pages=0), cache(dim=24), cache(dim=272), cache(k_codes=None), cache(k_codes=A + 8)):
        assert write(L, c) != UNSUP or "gfx950" not in L.nvfp4_last_error().decode()


def test_accepts(L):
    for more in (dict(), dict(q=None, query_heads=0, out=None), dict(rows=0, table=None), dict(k=A + 2), dict(rotary=128),
                 dict(tokens=0, k=None, v=None, slots=None, positions=None), dict(dt=0), dict(interleaved=1)):
        assert write(L, cache(), **more) == UNSUP and "gfx950" in L.nvfp4_last_error().decode(), more


def test_python_refusals():
    c = nv.kv_cache(2, 4, 3, 64, device="cpu")
    k, i = torch.zeros(5, 3, 64), torch.zeros(5, dtype=torch.int64)
    with pytest.raises(ValueError):  # host tensors
        nv.nvfp4_kv_write_rotated(c, k, k, i, i.int(), torch.zeros(4, 64))
    for bad in (0, 8, 40, -16):
        with pytest.raises(ValueError):
            nv.rotation_table(4, bad, device="cpu")
    t = nv.rotation_table(3, 16, device="cpu")
    assert t.shape == (3, 16) and t.dtype == torch.float32
    assert (t[0, :8] == 1).all() and (t[0, 8:] == 0).all()
