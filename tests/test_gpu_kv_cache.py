"""The NVFP4 key/value cache on the GPU: writing tokens and reading them back.

Codes and scales equal the oracle's encode of the same rows byte for byte, the
values read equal the oracle's decode, tokens without a slot are skipped, and
no byte outside the written slots changes."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
import workloads as W
from _parity import O, assert_bytes_equal, assert_values_equal, guarded, host, oracle_dtype, say

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


def _slots(tokens, total, seed, padded):
    gen = torch.Generator().manual_seed(seed)
    slots = torch.randperm(total, generator=gen)[:tokens]
    for i, bad in zip(torch.randperm(tokens, generator=gen)[:padded].tolist(), (-1, total, -2 ** 40, 2 ** 40)):
        slots[i] = bad
    return slots


def _guarded_cache(pages, page, heads, dim, g_k, g_v):
    """A KVCache between canary bytes, filled with 0x5A, and its guards."""
    parts = {n: guarded((pages, heads, page, dim // per), torch.uint8)
             for n, per in (("k_codes", 2), ("k_scales", 16), ("v_codes", 2), ("v_scales", 16))}
    for p in parts.values():
        p.t.fill_(0x5A)
    return nv.KVCache(**{n: p.t for n, p in parts.items()}, global_scale_k=g_k, global_scale_v=g_v), parts


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,heads,dim,page,padded", [
    (1, 1, 16, 1, 0), (1, 8, 128, 16, 0), (7, 3, 80, 5, 2), (64, 8, 128, 16, 0), (33, 5, 96, 24, 1),
    (130, 2, 256, 64, 4), (257, 1, 64, 7, 3), (40, 2, 240, 16, 1)])
def test_write_and_read(dtype, tokens, heads, dim, page, padded):
    say(f"kv write/read {dtype} {tokens}x{heads}x{dim} page {page}")
    pages = -(-tokens // page) + 2
    total = pages * page
    k = W.normal((tokens, heads, dim), 1.0, 900 + dim, oracle_dtype(dtype), outlier_frac=0.02, outlier_mult=20.0)
    v = W.normal((tokens, heads, dim), 0.3, 901 + tokens, oracle_dtype(dtype))
    slots = _slots(tokens, total, 17 + tokens, padded)
    # both with a global scale, too small a one for the outliers (they saturate), then none
    for g_k, g_v in ((21.5, 1.25), (None, None), (21.5, None)):
        dg = [None if g is None else torch.tensor([g], device="cuda") for g in (g_k, g_v)]
        cache, parts = _guarded_cache(pages, page, heads, dim, *dg)
        nv.nvfp4_kv_write(cache, k.cuda(), v.cuda(), slots.cuda())
        rk, rv = guarded((tokens, heads, dim), dtype), guarded((tokens, heads, dim), dtype)
        nv.nvfp4_kv_read(cache, slots.cuda(), out=(rk.t, rv.t))
        torch.cuda.synchronize()
        for n, p in [*parts.items(), ("k", rk), ("v", rv)]:
            p.check(n)
        there = ((slots >= 0) & (slots < total)).numpy()
        at = slots.numpy()[there]
        for x, g, n, r in ((k, g_k, "k", rk), (v, g_v, "v", rv)):
            codes, scales = O.quantize(host(x).reshape(-1, dim), g)
            for got, want, per in ((parts[n + "_codes"].t, codes, 2), (parts[n + "_scales"].t, scales, 16)):
                whole = np.full((pages, heads, page, dim // per), 0x5A, np.uint8)
                whole[at // page, :, at % page] = want.reshape(tokens, heads, -1)[there]
                assert_bytes_equal(got.cpu().numpy(), whole, f"{n} /{per}")
            back = O.dequantize(codes, scales, g, dtype=oracle_dtype(dtype)).reshape(tokens, heads, dim).copy()
            back[~there] = 0.0
            assert_values_equal(host(r.t), back, f"{n} read")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("off", [0, 1])
def test_strided_views(dtype, off):
    """Keys and values as slices of one fused projection, also misaligned ones: the copies' bytes."""
    heads, dim, tokens, page = 3, 48, 50, 16
    fused = W.normal((tokens, 7 * heads * dim + 3), 1.0, 77, oracle_dtype(dtype)).cuda()
    k = fused[:, off:off + heads * dim].unflatten(1, (heads, dim))
    v = fused[:, off + 3 * heads * dim:off + 6 * heads * dim].unflatten(1, (3 * heads, dim))[:, ::3]
    slots = torch.arange(tokens, device="cuda") + 5
    g = torch.tensor([4.0], device="cuda")
    a, b = (nv.kv_cache(5, page, heads, dim, g, g) for _ in range(2))
    nv.nvfp4_kv_write(a, k, v, slots)
    nv.nvfp4_kv_write(b, k.contiguous(), v.contiguous(), slots)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    # keys shared by every head (stride 0)
    one = k[:, :1].expand(-1, heads, -1)
    nv.nvfp4_kv_write(a, one, v, slots)
    nv.nvfp4_kv_write(b, one.contiguous(), v.contiguous(), slots)
    assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.k_scales, b.k_scales)


def test_read_types_and_empty():
    """One cache read in each type equals nvfp4_dequantize of its rows; no tokens is a no-op."""
    heads, dim, page, pages = 4, 64, 8, 6
    g = torch.tensor([9.0], device="cuda")
    cache = nv.kv_cache(pages, page, heads, dim, g, None)
    x = W.normal((pages * page, heads, dim), 1.0, 5, "f32").cuda()
    slots = torch.arange(pages * page, device="cuda")
    nv.nvfp4_kv_write(cache, x, x * 0.5, slots)
    back = slots.flip(0).contiguous()
    for dtype in DTYPES:
        k, v = nv.nvfp4_kv_read(cache, back, dtype=dtype)
        for got, n, gs in ((k, "k", g), (v, "v", None)):
            rows = nv.nvfp4_dequantize(getattr(cache, n + "_codes"), getattr(cache, n + "_scales"), gs, dtype=dtype)
            assert torch.equal(got, rows.transpose(1, 2).reshape(-1, heads, dim).flip(0)), (dtype, n)
    none = torch.empty(0, heads, dim, device="cuda")
    nv.nvfp4_kv_write(cache, none, none, slots[:0])
    assert nv.nvfp4_kv_read(cache, slots[:0])[0].shape == (0, heads, dim)


def test_offsets_past_32_bits():
    """A cache whose codes pass 4 GiB: tokens in its last page are written there, and nowhere else."""
    heads, dim, page = 16, 256, 64
    pages = (1 << 32) // (heads * page * dim // 2) + 3
    cache = nv.kv_cache(pages, page, heads, dim)
    assert cache.k_codes.numel() > 1 << 32
    tokens = page
    k = W.normal((tokens, heads, dim), 1.0, 40, "bf16").cuda()
    v = W.normal((tokens, heads, dim), 1.0, 41, "bf16").cuda()
    slots = (pages - 1) * page + torch.arange(tokens, device="cuda")
    nv.nvfp4_kv_write(cache, k, v, slots)
    for x, n in ((k, "k"), (v, "v")):
        codes, scales = nv.nvfp4_quantize(x)
        assert torch.equal(getattr(cache, n + "_codes")[-1], codes.transpose(0, 1))
        assert torch.equal(getattr(cache, n + "_scales")[-1], scales.transpose(0, 1))
        assert int(torch.count_nonzero(getattr(cache, n + "_scales")[:-1])) == 0
        assert not getattr(cache, n + "_codes")[:-1].any()
    rk, rv = nv.nvfp4_kv_read(cache, slots)
    assert torch.equal(rk, nv.nvfp4_quant_dequant(k)) and torch.equal(rv, nv.nvfp4_quant_dequant(v))


def test_other_stream_and_graph():
    """Write and read on a side stream, and captured: every replay equals the eager result."""
    heads, dim, page, tokens = 8, 128, 16, 64
    g = torch.tensor([6.0], device="cuda")
    cache = nv.kv_cache(8, page, heads, dim, g, g)
    k = W.normal((tokens, heads, dim), 1.0, 50, "bf16").cuda()
    v = W.normal((tokens, heads, dim), 1.0, 51, "bf16").cuda()
    slots = torch.randperm(8 * page)[:tokens].cuda()
    rk, rv = torch.empty_like(k), torch.empty_like(v)

    def step():
        nv.nvfp4_kv_write(cache, k, v, slots)
        nv.nvfp4_kv_read(cache, slots, out=(rk, rv))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for i in range(4):
        k.copy_(W.normal((tokens, heads, dim), 1.0, 60 + i, "bf16"))
        rk.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rk, nv.nvfp4_quant_dequant(k, g)) and torch.equal(rv, nv.nvfp4_quant_dequant(v, g)), i
