"""Host-side refusals of nvfp4_mx_rms_norm (no GPU, no kernel)."""
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


def norm(L, x=A, residual=B, weight=C, dt=2, mode=8, rows=4, k=64, eps=1e-6, packed=0, sum=D, normed=E, codes=F, scales=F + 1):
    return L.nvfp4_mx_rms_norm(x, residual, weight, dt, mode, rows, k, eps, packed, sum, normed, codes, scales, None)


@pytest.mark.parametrize("bad,status,says", [
    (dict(dt=3), INV, "dtype"), (dict(mode=6), INV, "mx mode"), (dict(rows=-1), INV, "rows"), (dict(k=0), INV, "group size 32"),
    (dict(k=48), INV, "group size 32"), (dict(eps=0.0), INV, "eps"), (dict(eps=float("nan")), INV, "eps"),
    (dict(eps=float("inf")), INV, "eps"), (dict(x=None), INV, "NULL"), (dict(codes=None), INV, "NULL"),
    (dict(scales=None), INV, "NULL"), (dict(x=A + 8), INV, "aligned"), (dict(residual=B + 2), INV, "aligned"),
    (dict(weight=C + 4), INV, "aligned"), (dict(sum=D + 8), INV, "aligned"), (dict(normed=E + 8), INV, "aligned"),
    (dict(codes=F + 8), INV, "aligned"), (dict(sum=E), INV, "different"), (dict(rows=1 << 22), UNSUP, "too large"),
    (dict(k=(1 << 30) + 32), UNSUP, "too large")])
def test_errors(L, bad, status, says):
    assert norm(L, **bad) == status, bad
    text = L.nvfp4_last_error().decode()
    assert "[mx_rms_norm]" in text and says in text, text


def test_accepts(L):
    for more in (dict(), dict(residual=None, weight=None, sum=None, normed=None), dict(sum=A), dict(sum=B, normed=A), dict(packed=1),
                 dict(rows=0, x=None, codes=None, scales=None), dict(dt=0, mode=4), dict(rows=(1 << 22) - 1)):
        assert norm(L, **more) == UNSUP and "gfx950" in L.nvfp4_last_error().decode(), more


def test_python_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        nv.nvfp4_mx_rms_norm(x)
    with pytest.raises(ValueError, match="mx mode"):
        nv.nvfp4_mx_rms_norm(x, mode="nvfp4")
