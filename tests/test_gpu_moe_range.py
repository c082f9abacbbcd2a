"""The expert layer far from ordinary sizes, against 64 bits within the bounds of test_gpu_moe.py: rows and global scales
near the ends of float32, rows whose values are far apart, subnormal float16, gates whose exponential is infinite."""
import pytest
import torch

import nvfp4_block_scaled_amd as nv
from _parity import say
from test_gpu_moe import Weights, check, reference

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


def run(x, w, what, top_k=2, seed=1):
    """Every token with experts and weights of its own, ordinary ones."""
    gen = torch.Generator().manual_seed(seed)
    t = len(x)
    idx = torch.stack([torch.randperm(w.e, generator=gen)[:top_k] for _ in range(t)]).int()
    p = torch.rand(t, top_k, generator=gen) + 0.1
    args, more = w.args()
    got = nv.nvfp4_moe(x.cuda(), *args, expert_idx=idx.cuda(), expert_weights=p.cuda(), **more)[0]
    ref = reference(x, w, idx.long(), p.double())
    assert torch.isfinite(ref[0]).all() and (ref[0].abs() < torch.finfo(x.dtype).max / 2).all()
    check(got, ref, what)
    return got


def weights(e, k, f, seed, up, down):
    """Global scales of 2^up and 2^down."""
    w = Weights(e, k, f, seed)
    w.up = w.up[:2] + (torch.full((e,), 2.0 ** up),)
    w.down = w.down[:2] + (torch.full((e,), 2.0 ** down),)
    return w


@pytest.mark.parametrize("dtype,size,up,down", [
    (d, *s) for d in (BF16, F32) for s in ((-110, 106, 3), (-110, 118, 3), (30, -28, 2), (100, -99, 10), (0, 22, -40), (63, 1, -102),
                                           (-50, 1, 100), (-120, 120, -110), (0, 2, 2))] +
    [(F16, *s) for s in ((-20, 22, 2), (-23, 25, 2), (11, -8, -2), (0, 2, 1))])
@pytest.mark.parametrize("k,f", [(96, 80), (1040, 272)])
def test_sizes(dtype, size, up, down, k, f):
    """x of 2^size, weights of up to 2^up and 2^down: sums and factors apart pass float32's range, the layer does not."""
    say(f"moe {dtype} x 2^{size}, weights 2^{up} and 2^{down}, {k} x {f}")
    gen = torch.Generator().manual_seed(k + size)
    x = (torch.randn(5, k, generator=gen, dtype=torch.float64) * 2.0 ** size).to(dtype)
    run(x, weights(3, k, f, 7, up, down), f"{dtype} 2^{size}")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("t,k,f", [(5, 96, 80), (20, 320, 272)])
def test_rows_of_different_sizes(dtype, t, k, f):
    """A power of two of its own for every token, and values of a row up to 2^-45 (float16: its subnormals) of the largest."""
    gen = torch.Generator().manual_seed(t)
    low, wide = (-5.0, 18.0) if dtype == F16 else (-20.0, 45.0)
    rows = torch.rand(t, 1, generator=gen, dtype=torch.float64) * low
    within = torch.rand(t, k, generator=gen, dtype=torch.float64) * -wide
    x = (torch.randn(t, k, generator=gen, dtype=torch.float64) * torch.exp2(rows + within)).to(dtype)
    x[0, 3:] = 0  # one value alone
    x[1] = 0
    sizes = x[x != 0].abs().double()
    assert sizes.max() / sizes.min() > 2 ** 20
    got = run(x, weights(4, k, f, 9, 3, 3), f"{dtype} spread")
    assert not got[1].any()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_gates_far_from_zero(dtype):
    """Gates of +-2^17 and more: exp(-g) is infinite for half of them, whose h is 0 and no NaN."""
    t, k, f = 6, 64, 48
    gen = torch.Generator().manual_seed(2)
    x = (torch.randn(t, k, generator=gen) * 2.0 ** 10).to(dtype)
    w = weights(3, k, f, 11, 16, -40)
    both = torch.stack([w.values(w.up, e)[:f] @ x.double().T for e in range(3)])
    assert (both < -2.0 ** 17).any() and (both > 2.0 ** 17).any()
    run(x, w, f"{dtype} gates")
    x = x.abs()
    w.up[0][:, :f] = 0xFF  # gates that are all negative: zeros
    got = run(x, w, f"{dtype} closed")
    assert not got.any()
