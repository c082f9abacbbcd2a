"""Host-side refusals of nvfp4_moe (no GPU, no kernel)."""
import os

import pytest
import torch

import nvfp4_block_scaled_amd as nv

INV, UNSUP = nv.NVFP4_ERR_INVALID_ARGUMENT, nv.NVFP4_ERR_UNSUPPORTED
A, B, C, D, E, F, G, H = (0x10000 * i for i in range(1, 9))  # fake aligned addresses


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_block_scaled_amd import build
        build.build()
    lib = nv.load_library()
    lib.nvfp4_debug_set_arch_override(b"gfx942")  # nothing reaches a device
    yield lib
    lib.nvfp4_debug_set_arch_override(None)


def moe(L, x=A, dt=2, router=B, idx=C, weights=D, up=E, up_scales=F, up_g=None, down=G, down_scales=H, down_g=None, t=3, top_k=2,
        e=8, k=128, f=64, out=A + 0x8000, wsp=0x100000, nbytes=None):
    need = L.nvfp4_moe_workspace_size(dt, t, top_k, e, k, f)
    return L.nvfp4_moe(x, dt, router, idx, weights, 1, up, up_scales, up_g, down, down_scales, down_g, t, top_k, e, k, f, out, wsp,
                       need if nbytes is None else nbytes, None)


@pytest.mark.parametrize("bad,status,says", [
    (dict(dt=4), INV, "dtype"), (dict(t=-1), INV, ">= 0"), (dict(top_k=0), INV, "positive"), (dict(e=0), INV, "positive"),
    (dict(top_k=9), INV, "at most e"), (dict(k=120), INV, "group size 16"), (dict(f=0), INV, "group size 16"), (dict(f=72), INV, "group size 16"),
    (dict(t=65), UNSUP, "tokens"), (dict(top_k=33, e=40), UNSUP, "experts"), (dict(e=1025), UNSUP, "experts"),
    (dict(k=1 << 20), UNSUP, "too large"), (dict(f=1 << 20), UNSUP, "too large"),
    (dict(t=64, top_k=32, e=1024, f=(1 << 18)), UNSUP, "too large"), (dict(x=None), INV, "NULL"), (dict(idx=None), INV, "NULL"),
    (dict(weights=None), INV, "NULL"), (dict(up=None), INV, "NULL"), (dict(up_scales=None), INV, "NULL"), (dict(down=None), INV, "NULL"),
    (dict(down_scales=None), INV, "NULL"), (dict(out=None), INV, "NULL"), (dict(x=A + 8), INV, "aligned"), (dict(router=B + 2), INV, "aligned"),
    (dict(up=E + 8), INV, "aligned"), (dict(down=G + 4), INV, "aligned"), (dict(out=A + 4), INV, "aligned"), (dict(idx=C + 2), INV, "aligned"),
    (dict(weights=D + 1), INV, "aligned"), (dict(up_g=B + 2), INV, "aligned"), (dict(nbytes=16), INV, "workspace"),
    (dict(wsp=None), INV, "workspace"), (dict(wsp=0x100010), INV, "aligned")])
def test_errors(L, bad, status, says):
    assert moe(L, **bad) == status, bad
    text = L.nvfp4_last_error().decode()
    assert "[moe]" in text and says in text, text


def test_accepts(L):
    for more in (dict(), dict(router=None), dict(t=64, top_k=8), dict(t=0, x=None, idx=None), dict(dt=0), dict(dt=1), dict(e=1024, top_k=32),
                 dict(up_g=A, down_g=A + 4), dict(up_scales=F + 1, down_scales=H + 3), dict(k=16, f=16)):
        assert moe(L, **more) == UNSUP and "gfx950" in L.nvfp4_last_error().decode(), (more, L.nvfp4_last_error())


def test_workspace(L):
    for dt in (0, 1, 2):
        need = L.nvfp4_moe_workspace_size(dt, 7, 3, 11, 1040, 592)
        assert need > 0 and need % 256 == 0
        assert moe(L, dt=dt, t=7, top_k=3, e=11, k=1040, f=592, nbytes=need - 1) == INV
    assert L.nvfp4_moe_workspace_size(2, 0, 3, 11, 1040, 592) == 0
    assert L.nvfp4_moe_workspace_size(2, 65, 3, 11, 1040, 592) == 0
    assert L.nvfp4_moe_workspace_size(7, 1, 3, 11, 1040, 592) == 0


def test_python_refusals():
    with pytest.raises(ValueError, match="device tensor"):
        nv.nvfp4_moe(torch.zeros(2, 32), *(torch.zeros(1, dtype=torch.uint8),) * 4)
