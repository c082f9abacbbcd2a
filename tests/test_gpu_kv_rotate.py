"""nvfp4_kv_write_rotated on the GPU against its definition.

Each product and sum of the rotation is one float32 rounding, which numpy's
float32 arithmetic repeats exactly; the codes and scales are the oracle's encode
of those float32 rows.  So the cache's bytes and the rotated queries (after their
one rounding to T) must be equal, and no byte outside the slots may change."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
import workloads as W
from _parity import O, assert_bytes_equal, guarded, host, oracle_dtype, say

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


def rotated(x, row, rotary, interleaved):
    """float32 numpy x [tokens, heads, dim] rotated by row [tokens, rotary], one rounding an operation."""
    x, half = x.astype(np.float32), rotary // 2
    c, s = row[:, None, :half], row[:, None, half:]
    first, second = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, half), slice(half, rotary))
    a, b, out = x[..., first], x[..., second], x.copy()
    out[..., first] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
    out[..., second] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return out


def cache_of(pages, page, heads, dim, g_k, g_v):
    parts = {n: guarded((pages, heads, page, dim // per), torch.uint8)
             for n, per in (("k_codes", 2), ("k_scales", 16), ("v_codes", 2), ("v_scales", 16))}
    for p in parts.values():
        p.t.fill_(0x5A)
    g = [None if v is None else torch.tensor([v], device="cuda") for v in (g_k, g_v)]
    return nv.KVCache(**{n: p.t for n, p in parts.items()}, global_scale_k=g[0], global_scale_v=g[1]), parts


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,groups,dim,rotary,page", [
    (1, 1, 1, 16, 16, 1), (1, 8, 4, 128, 128, 16), (7, 3, 2, 80, 32, 5), (64, 2, 5, 128, 64, 16), (33, 5, 3, 96, 48, 24),
    (5, 2, 1, 256, 256, 64), (130, 1, 8, 64, 64, 7), (9, 2, 3, 240, 112, 16), (1031, 2, 1, 32, 32, 16), (4500, 1, 2, 48, 16, 32)])
def test_values(dtype, interleaved, tokens, heads, groups, dim, rotary, page):
    say(f"rotate {dtype} {tokens}x{heads}x{groups}x{dim} of {rotary} page {page} interleaved={interleaved}")
    pages, length = -(-tokens // page) + 2, 3000
    total = pages * page
    gen = torch.Generator().manual_seed(tokens + dim)
    slots = torch.randperm(total, generator=gen)[:tokens]
    positions = torch.randint(0, length, (tokens,), generator=gen).to(torch.int32)
    if tokens > 6:
        for i, bad in enumerate((-1, total, -2 ** 40)):
            slots[i] = bad
        positions[4], positions[5] = -1, length
        positions[6] = length - 1
    nq = heads * groups
    fused = W.normal((tokens, nq + 2 * heads, dim), 1.0, 400 + dim, oracle_dtype(dtype), outlier_frac=0.02, outlier_mult=15.0)
    table = nv.rotation_table(length, rotary)
    fd = fused.cuda()
    q, k, v = fd[:, :nq], fd[:, nq:nq + heads], fd[:, nq + heads:]
    g_k, g_v = (21.5, None) if tokens % 2 else (30.0, 2.0)
    cache, parts = cache_of(pages, page, heads, dim, g_k, g_v)
    out = guarded((tokens, nq, dim), dtype)
    out.t.fill_(float("nan"))
    r = nv.nvfp4_kv_write_rotated(cache, k, v, slots.cuda(), positions.cuda(), table, q=q, interleaved=interleaved, out=out.t)
    torch.cuda.synchronize()
    assert r is out.t
    for n, p in [*parts.items(), ("q", out)]:
        p.check(n)
    known = ((positions >= 0) & (positions < length)).numpy()
    there = ((slots >= 0) & (slots < total)).numpy() & known
    row = table.cpu().numpy()[positions.clamp(0, length - 1).numpy()]
    x = host(fused)
    want = torch.from_numpy(rotated(x[:, :nq], row, rotary, interleaved)).to(dtype)
    want[torch.from_numpy(~known)] = 0
    assert torch.equal(out.t.cpu(), want), "queries"
    for n, g, y in (("k", g_k, rotated(x[:, nq:nq + heads], row, rotary, interleaved)), ("v", g_v, x[:, nq + heads:])):
        codes, scales = O.quantize(np.ascontiguousarray(y).reshape(-1, dim), g)
        at = slots.numpy()[there]
        for got, enc, per in ((parts[n + "_codes"].t, codes, 2), (parts[n + "_scales"].t, scales, 16)):
            whole = np.full((pages, heads, page, dim // per), 0x5A, np.uint8)
            whole[at // page, :, at % page] = enc.reshape(tokens, heads, -1)[there]
            assert_bytes_equal(got.cpu().numpy(), whole, f"{n} /{per}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("off", [0, 1])
def test_strided_views(dtype, off):
    """Slices of one projection, also misaligned ones, and heads that share their keys: the copies' bytes."""
    heads, dim, tokens, page = 3, 48, 50, 16
    fused = W.normal((tokens, 9 * heads * dim + 3), 1.0, 77, oracle_dtype(dtype)).cuda()
    k = fused[:, off:off + heads * dim].unflatten(1, (heads, dim))
    v = fused[:, off + heads * dim:off + 4 * heads * dim].unflatten(1, (3 * heads, dim))[:, ::3]
    q = fused[:, off + 4 * heads * dim:off + 8 * heads * dim].unflatten(1, (4 * heads, dim))[:, ::2]
    slots, positions = torch.arange(tokens, device="cuda") + 5, torch.arange(tokens, device="cuda", dtype=torch.int32) * 7
    table = nv.rotation_table(400, 32)
    g = torch.tensor([4.0], device="cuda")
    for one in (False, True):
        if one:
            k = k[:, :1].expand(-1, heads, -1)
        a, b = (nv.kv_cache(5, page, heads, dim, g, g) for _ in range(2))
        qa = nv.nvfp4_kv_write_rotated(a, k, v, slots, positions, table, q=q)
        qb = nv.nvfp4_kv_write_rotated(b, k.contiguous(), v.contiguous(), slots, positions, table, q=q.contiguous())
        assert torch.equal(qa, qb)
        for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_without_queries_and_position_zero():
    """No queries; position 0 turns nothing: the bytes of nvfp4_kv_write."""
    heads, dim, tokens, page = 4, 128, 70, 16
    g = torch.tensor([5.0], device="cuda")
    k, v = (W.normal((tokens, heads, dim), 1.0, s, "bf16").cuda() for s in (1, 2))
    slots = torch.randperm(6 * page)[:tokens].cuda()
    a, b = (nv.kv_cache(6, page, heads, dim, g, g) for _ in range(2))
    table = nv.rotation_table(4, dim)
    zero = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    assert nv.nvfp4_kv_write_rotated(a, k, v, slots, zero, table) is None
    nv.nvfp4_kv_write(b, k, v, slots)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    none = torch.empty(0, heads, dim, dtype=torch.bfloat16, device="cuda")
    assert nv.nvfp4_kv_write_rotated(a, none, none, slots[:0], zero[:0], table, q=none).shape == (0, heads, dim)
    # a table without rows: every token is skipped
    q = nv.nvfp4_kv_write_rotated(a, v, k, slots, zero, table[:0], q=k)
    assert not q.any() and torch.equal(a.k_codes, b.k_codes)


def test_rotation_table():
    """Angles of far positions in 64 bits."""
    t = nv.rotation_table(200001, 64, base=5e5).cpu()
    p, i = 200000, torch.arange(0, 64, 2, dtype=torch.float64)
    angle = p * 5e5 ** (-i / 64)
    assert (t[p, :32].double() - angle.cos()).abs().max() <= 2.0 ** -24 + 2.0 ** -33  # half a step, and the angle's own 2^-53 p
    assert (t[p, 32:].double() - angle.sin()).abs().max() <= 2.0 ** -24 + 2.0 ** -33


def test_offsets_past_32_bits():
    """A cache whose codes pass 4 GiB, and strides that pass 2^31 elements."""
    heads, dim, page = 16, 256, 64
    pages = (1 << 32) // (heads * page * dim // 2) + 3
    cache = nv.kv_cache(pages, page, heads, dim)
    far = torch.empty(3, (1 << 30) + 4096, dtype=torch.bfloat16, device="cuda")  # token 2 starts past 2^31 elements
    x = W.normal((3, heads, dim), 1.0, 9, "bf16").cuda()
    k = far[:, :heads * dim].unflatten(1, (heads, dim))
    k.copy_(x)
    slots = torch.tensor([pages * page - 1, 0, pages * page - 3], device="cuda")
    positions = torch.tensor([3, 1, 2], dtype=torch.int32, device="cuda")
    table = nv.rotation_table(8, dim)
    q = nv.nvfp4_kv_write_rotated(cache, k, k, slots, positions, table, q=k)
    small = nv.kv_cache(1, 64, heads, dim)
    q2 = nv.nvfp4_kv_write_rotated(small, x, x, torch.arange(3, device="cuda"), positions, table, q=x)
    assert torch.equal(q, q2)
    for n in ("k_codes", "v_codes", "k_scales"):
        held = getattr(cache, n)
        for i, s in enumerate(slots.tolist()):
            assert torch.equal(held[s // page, :, s % page], getattr(small, n)[0, :, i]), n


def test_other_stream_and_graph():
    heads, dim, page, tokens = 8, 128, 16, 64
    g = torch.tensor([6.0], device="cuda")
    cache = nv.kv_cache(8, page, heads, dim, g, g)
    fused = W.normal((tokens, 6 * heads, dim), 1.0, 50, "bf16").cuda()
    slots = torch.randperm(8 * page)[:tokens].cuda()
    positions = torch.arange(tokens, dtype=torch.int32, device="cuda")
    table = nv.rotation_table(tokens, dim)
    out = torch.empty(tokens, 4 * heads, dim, dtype=torch.bfloat16, device="cuda")

    def step(c=cache, o=out):
        return nv.nvfp4_kv_write_rotated(c, fused[:, 4 * heads:5 * heads], fused[:, 5 * heads:], slots, positions, table,
                                         q=fused[:, :4 * heads], out=o)

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
        fused.copy_(W.normal((tokens, 6 * heads, dim), 1.0, 60 + i, "bf16"))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        other = nv.kv_cache(8, page, heads, dim, g, g)
        assert torch.equal(out, step(other, torch.empty_like(out))), i
        assert torch.equal(cache.k_codes, other.k_codes) and torch.equal(cache.v_scales, other.v_scales), i
