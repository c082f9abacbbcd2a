"""The norm that encodes its output (nvfp4_mx_rms_norm) against its definition.

Reference: numpy on the CPU, the squares in float64, r rounded to float32, the
two products in float32, and the oracle's encode of the result.  All of it is
defined to the bit (the sum of squares up to its order, 2^-52 relative, which
moves r's float32 only if the exact value lies within about 2^-28 of a step of a
midpoint), so sums, codes and scales must be equal, and the normed values too
after their one rounding.  A row whose 64-bit r lies within 2^-20 of a step of
such a midpoint would be excused; none of these inputs has one (asserted)."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
from _parity import O, assert_bytes_equal, guarded, host, say

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


def reference(x, residual, weight, eps):
    """(h in x's type, float32 y) on the CPU."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    f = h.float().numpy()
    d = f.astype(np.float64)
    exact = 1.0 / np.sqrt((d * d).sum(-1, keepdims=True) / x.shape[-1] + eps)
    r = exact.astype(np.float32)
    fine = np.isfinite(exact)
    step = np.spacing(r[fine]).astype(np.float64)
    off = np.abs(np.abs(exact[fine] - r[fine]) / step - 0.5)
    assert (off > 2.0 ** -20).all(), "an input with an undecided r"
    y = (f * r).astype(np.float32)
    if weight is not None:
        y = (y * weight.float().numpy()).astype(np.float32)
    return h, y


def inputs(rows, k, dtype, seed, residual=True, weight=True, size=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, k, generator=gen) * size).to(dtype)
    res = (torch.randn(rows, k, generator=gen) * (1 + 30 * (torch.rand(k, generator=gen) < 0.02)) * size).to(dtype)
    w = (1 + 0.3 * torch.randn(k, generator=gen)).to(dtype)
    return x, res if residual else None, w if weight else None


def dev(t):
    return None if t is None else t.cuda()


def run(x, res, w, mode, packed, normed=True, eps=1e-6):
    rows, k = x.shape
    bits = nv.MX_MODES[mode]
    if packed:
        tiles, quads = -(-rows // 32), -(-k // 256)
        codes, scales = guarded((tiles * quads * 4 * bits // 2 * 512,), torch.uint8), guarded((tiles * quads * 256,), torch.uint8)
        out = nv.MxPacked(codes.t, scales.t, (rows, k), mode)
    else:
        codes, scales = guarded((rows, k * bits // 8), torch.uint8), guarded((rows, k // 32), torch.uint8)
        out = (codes.t, scales.t)
    codes.t.fill_(0x5A)
    scales.t.fill_(0x5A)
    total = guarded((rows, k), x.dtype)
    r = nv.nvfp4_mx_rms_norm(dev(x), dev(w), mode, residual=dev(res), eps=eps, packed=packed, normed=normed,
                             sum_out=total.t, out=out)
    torch.cuda.synchronize()
    for g, n in ((codes, "codes"), (scales, "scales"), (total, "sum")):
        g.check(n)
    return r


def check(x, res, w, mode, packed, eps=1e-6):
    h, y = reference(x, res, w, eps)
    r = run(x, res, w, mode, packed, True, eps)
    assert torch.equal(r.sum.cpu(), h), "sum"
    assert torch.equal(r.normed.cpu(), torch.from_numpy(y).to(x.dtype)), "normed"
    oc, os_ = O.mx_quantize(y, mode)
    if packed:
        want = nv.nvfp4_mx_pack(torch.from_numpy(oc).cuda(), torch.from_numpy(os_).cuda(), mode)
        assert torch.equal(r.quantized.scales, want.scales), "packed scales"
        assert torch.equal(r.quantized.codes, want.codes), "packed codes"
    else:
        assert_bytes_equal(r.quantized[1].cpu().numpy(), os_, "scales")
        assert_bytes_equal(r.quantized[0].cpu().numpy(), oc, "codes")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 64), (33, 96), (5, 1024), (2, 1056), (4, 4096), (31, 4128), (3, 16384), (2, 16416),
                                    (1, 32768), (2, 33024), (1025, 1056), (1100, 4096), (1031, 2080)])
def test_values(dtype, mode, packed, rows, k):
    """Row lengths on both sides of every launch shape, a few rows and many."""
    say(f"norm {dtype} {mode} packed={packed} {rows}x{k}")
    x, res, w = inputs(rows, k, dtype, rows + k, residual=(rows + k) % 3 != 0, weight=(rows + k) % 5 != 0)
    check(x, res, w, mode, packed)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", ["mxfp8", "mxfp4"])
def test_sizes_of_values(dtype, mode):
    """Rows of zeros, tiny and huge rows, groups of zeros, one value alone."""
    x, res, w = inputs(9, 256, dtype, 7)
    x[0] = 0
    res[0] = 0
    x[1], res[1] = x[1] * 1e-6, 0
    big = 1e30 if dtype != torch.float16 else 3e4
    x[2], res[2] = torch.sign(x[2].float()) * big, 0
    x[3, :64], res[3, :64] = 0, 0
    x[4], res[4] = 0, 0
    x[4, 100] = 1.0
    w[200:232] = 0
    for eps in (1e-6, 1e-12, 1.0):
        check(x, res, w, mode, False, eps)


def test_not_numbers():
    """A NaN or an infinity makes its row's groups NaN, and leaves the other rows as they are."""
    x, res, w = inputs(4, 128, torch.bfloat16, 11)
    clean = run(x, res, w, "mxfp8", False)
    for value in (float("nan"), float("inf"), float("-inf")):
        y = x.clone()
        y[1, 5] = value
        r = run(y, res, w, "mxfp8", False)
        got = nv.nvfp4_mx_dequantize(*r.quantized, "mxfp8", dtype=torch.float32).cpu()
        if value != value:
            assert got[1].isnan().all()  # r is NaN
        else:
            assert got[1, :32].isnan().all()  # inf * 0, in one group
            assert (got[1, 32:] == 0).all()
        for row in (0, 2, 3):
            for a, b in ((r.quantized[0], clean.quantized[0]), (r.quantized[1], clean.quantized[1]), (r.sum, clean.sum)):
                assert torch.equal(a[row], b[row])
    w2 = w.clone()
    w2[40] = float("nan")  # a NaN in one group of every row
    r = run(x, res, w2, "mxfp4", True)
    got = run(x, res, w2, "mxfp4", False).quantized
    want = nv.nvfp4_mx_pack(*got, "mxfp4")
    assert (got[1][:, 1] == 255).all() and (got[1][:, 0] != 255).all()
    assert torch.equal(r.quantized.scales, want.scales)


@pytest.mark.parametrize("k", [96, 4096, 40000])
def test_in_place(k):
    """The sum written over x or over the residual."""
    x, res, w = inputs(40, k, torch.bfloat16, k)
    want = run(x, res, w, "mxfp8", False)
    for which in (0, 1):
        xd, rd = x.cuda(), res.cuda()
        r = nv.nvfp4_mx_rms_norm(xd, w.cuda(), "mxfp8", residual=rd, sum_out=(xd, rd)[which], normed=True)
        assert r.sum is (xd, rd)[which] and torch.equal(r.sum, want.sum) and torch.equal(r.normed, want.normed)
        assert torch.equal(r.quantized[0], want.quantized[0]) and torch.equal(r.quantized[1], want.quantized[1])
    r = nv.nvfp4_mx_rms_norm(x.cuda(), None, "mxfp8")
    assert r.normed is None and torch.equal(r.sum.cpu(), x)


def test_product():
    """The packed output is an operand: its product equals that of the same codes packed by nvfp4_mx_pack."""
    x, res, w = inputs(70, 320, torch.bfloat16, 3)
    weight = nv.nvfp4_mx_pack(*nv.nvfp4_mx_quantize(torch.randn(96, 320).to(torch.bfloat16).cuda(), "mxfp8"), "mxfp8")
    a = run(x, res, w, "mxfp8", True).quantized
    b = nv.nvfp4_mx_pack(*run(x, res, w, "mxfp8", False).quantized, "mxfp8")
    assert torch.equal(nv.nvfp4_mx_mm_packed(a, weight), nv.nvfp4_mx_mm_packed(b, weight))


def test_empty_streams_and_graphs():
    e = nv.nvfp4_mx_rms_norm(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), None, "mxfp8")
    assert e.quantized[0].shape == (0, 64) and e.quantized[1].shape == (0, 2)
    x, res, w = inputs(50, 512, torch.float16, 5)
    want = run(x, res, w, "mxfp8", False)
    xd, rd, wd = x.cuda(), res.cuda(), w.cuda()
    out = (torch.empty_like(want.quantized[0]), torch.empty_like(want.quantized[1]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = nv.nvfp4_mx_rms_norm(xd, wd, "mxfp8", residual=rd, out=out)
        s.synchronize()
        assert torch.equal(out[0], want.quantized[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r = nv.nvfp4_mx_rms_norm(xd, wd, "mxfp8", residual=rd, out=out)
    for i in range(3):
        out[0].fill_(0)
        out[1].fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want.quantized[0]) and torch.equal(out[1], want.quantized[1]), i
        assert torch.equal(r.sum, want.sum)
        run(x, res, w, "mxfp4", True)
