"""Attention over the NVFP4 key/value cache against the 64-bit reference of
_kv.py, within its derived bound: types, head layouts, lengths from none to
long ones, ragged batches, masks that leave rows empty, windows, pages that
end inside a tile, unwritten pages, strides, streams and graphs."""
import pytest
import torch

import nvfp4_block_scaled_amd as nv
import _kv
from _parity import guarded, guarded_workspace, say

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


def _batch(contexts, page, seed, spare=2, unwritten=1):
    """(page table, pages, unwritten pages): shuffled pages, -1 past each context."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-max(c, 0) // page) for c in contexts]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.full((len(contexts), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages, order[at:at + unwritten].tolist()


def _poison_tails(cache, table, contexts):
    """Bytes 255 in every slot past a context's end within its last page."""
    for b, c in enumerate(contexts):
        if c > 0 and c % cache.page_size:
            p = int(table[b, c // cache.page_size])
            for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
                getattr(cache, n)[p, :, c % cache.page_size:] = 255


def _run(contexts, queries, heads, groups, dim, page, dtype, seed, causal=True, window=0, scale=None, g=(20.0, 6.0),
         q_size=1.0, tail=0):
    table, pages, unwritten = _batch(contexts, page, seed)
    cache = _kv.random_cache(pages, page, heads, dim, seed, *g, unwritten=unwritten)
    _poison_tails(cache, table, contexts)
    starts = [0]
    for n in queries:
        starts.append(starts[-1] + n)
    tokens = starts[-1] + tail
    gen = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(tokens, heads * groups, dim, generator=gen) * q_size).to(dtype).cuda()
    table_d, lens = table.cuda(), torch.tensor(contexts, dtype=torch.int32, device="cuda")
    starts_d = torch.tensor(starts, dtype=torch.int32, device="cuda")
    plain = all(n == 1 for n in queries) and not tail and seed % 2 == 0
    most = max(max(queries), 1)
    top = max(max(contexts), 0) if seed % 3 else None
    out = guarded(tuple(q.shape), dtype)
    out.t.fill_(float("nan"))
    wsp, nbytes = nv.kv_attention_workspace(cache, tokens, heads * groups, len(contexts), most,
                                            table.shape[1] * page if top is None else top, window)
    wsp = guarded_workspace(nbytes)
    wsp.t.fill_(255)
    got, lse = nv.nvfp4_kv_attention(q, cache, table_d, lens, query_starts=None if plain else starts_d,
                                     max_queries=most, max_context=top, scale=scale, causal=causal, window=window,
                                     return_lse=True, out=out.t, workspace=wsp.t)
    torch.cuda.synchronize()
    out.check("out")
    wsp.check("workspace")
    ref = _kv.reference(q, cache, table, lens, starts, dim ** -0.5 if scale is None else scale, causal, window)
    _kv.check(got, lse, ref, f"{dtype} d{dim} g{groups} page {page}")
    return got, lse


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,groups,dim,page", [
    (1, 1, 16, 1), (2, 4, 128, 16), (1, 8, 128, 64), (3, 1, 64, 7), (2, 5, 96, 24), (1, 16, 256, 32), (2, 3, 80, 16),
    (1, 2, 192, 128), (1, 17, 128, 16), (1, 40, 64, 256), (2, 2, 240, 5), (1, 1, 48, 3)])
def test_single_tokens(dtype, heads, groups, dim, page):
    """One query a sequence; contexts of none, one, a few, around the tile sizes, and some hundred."""
    say(f"single {dtype} h{heads} g{groups} d{dim} page {page}")
    contexts = [0, 1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 129, 300, 701]
    _run(contexts, [1] * len(contexts), heads, groups, dim, page, dtype, 10 + dim + groups)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", [2, 3, 4, 5, 8, 13])
@pytest.mark.parametrize("window", [0, 1, 20, 200])
def test_few_tokens(dtype, queries, window):
    """Speculated tokens: a few queries a sequence, some without any, more than the context holds."""
    contexts = [0, 1, queries, queries + 1, 33, 64, 257, 130]
    counts = [queries, queries, queries, queries, 0, 1, queries, queries - 1]
    _run(contexts, counts, 2, 4, 128, 16, dtype, 500 + queries + window, window=window, tail=2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,groups,page", [(128, 4, 16), (64, 1, 64), (96, 5, 24), (256, 2, 32), (192, 1, 7), (80, 3, 16),
                                             (16, 1, 16), (128, 1, 1)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 37), (False, 0)])
def test_prompts(dtype, dim, groups, page, causal, window):
    """Whole prompts and chunks over a cached prefix, ragged, around the tile sizes."""
    contexts = [1, 70, 129, 200, 257, 64]
    counts = [1, 70, 65, 33, 130, 0]
    _run(contexts, counts, 1, groups, dim, page, dtype, 900 + dim + window, causal=causal, window=window, tail=3)


@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_rows_that_see_nothing(dtype):
    """More queries than cached tokens: the first ones stand before the context."""
    _run([20, 0, 100], [90, 70, 140], 2, 2, 128, 16, dtype, 31)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("groups", [1, 4, 12])
def test_long_contexts(dtype, groups):
    """Contexts that are split over many workgroups, next to short ones."""
    _run([9000, 3, 5123, 0, 2048], [1] * 5, 1, groups, 64, 16, dtype, 70 + groups)
    _run([6001], [3], 2, groups, 128, 64, dtype, 71 + groups, window=4500)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", [1, 40])
def test_peaked_and_flat(dtype, queries):
    """Large scores (one key takes all), and flat ones with a spike that comes last."""
    _run([600, 513], [queries] * 2, 1, 4, 128, 16, dtype, 81, q_size=60.0)
    _run([600, 513], [queries] * 2, 1, 4, 128, 16, dtype, 82, q_size=1e-3)
    _run([600, 513], [queries] * 2, 1, 4, 128, 16, dtype, 83, g=(None, None))
    _run([600, 513], [queries] * 2, 1, 4, 128, 16, dtype, 84, g=(1e-3, 5e4), scale=7.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", [1, 40])
def test_rising_scores(dtype, queries):
    """Scores that rise along the keys, so that the running maximum moves all the way, then fall."""
    dim, page, context = 64, 16, 1500
    cache = _kv.random_cache(100, page, 1, dim, 3)
    table = torch.arange(94, dtype=torch.int32).view(1, -1)
    ramp = torch.arange(1504).view(94, 1, page) / 1504.0
    scale_byte = (0x30 + ramp * 0x38).to(torch.uint8).cuda()
    for back in (False, True):
        cache.k_codes[:94] = 0x22  # every value 1
        cache.k_scales[:94] = (scale_byte.flip(0, 2) if back else scale_byte).unsqueeze(-1)
        q = torch.ones(queries, 4, dim).to(dtype).cuda()
        lens = torch.tensor([context], dtype=torch.int32, device="cuda")
        starts = torch.tensor([0, queries], dtype=torch.int32, device="cuda")
        got, lse = nv.nvfp4_kv_attention(q, cache, table.cuda(), lens, query_starts=starts, max_queries=queries,
                                         scale=0.5, return_lse=True)
        _kv.check(got, lse, _kv.reference(q, cache, table, lens, [0, queries], 0.5), f"{dtype} ramp back={back}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", [1, 50])
def test_pages_outside_the_cache(dtype, queries):
    """Page numbers outside [0, pages) hide their tokens; a whole context of them leaves zeros."""
    page, contexts = 16, [100, 90, 40]
    table, pages, _ = _batch(contexts, page, 5)
    table[0, 2], table[0, 5], table[1, 0] = -1, pages, 2 ** 31 - 1
    table[2, :] = -7
    cache = _kv.random_cache(pages, page, 2, 64, 6)
    q = torch.randn(3 * queries, 4, 64, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    lens = torch.tensor(contexts, dtype=torch.int32, device="cuda")
    starts = [0, queries, 2 * queries, 3 * queries]
    got, lse = nv.nvfp4_kv_attention(q, cache, table.cuda(), lens, max_queries=queries, return_lse=True,
                                     query_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    _kv.check(got, lse, _kv.reference(q, cache, table, lens, starts, 0.125), "holes")
    assert not got[2 * queries:].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", [1, 70])
def test_strided_queries(dtype, queries):
    """Queries as a slice of a fused projection, misaligned, and shared by heads: the copy's bits."""
    heads, groups, dim, page = 2, 3, 64, 16
    cache = _kv.random_cache(20, page, heads, dim, 8)
    table = torch.randperm(20, generator=torch.Generator().manual_seed(2)).to(torch.int32).view(2, 10).cuda()
    lens = torch.tensor([150, 77], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, queries, 2 * queries], dtype=torch.int32, device="cuda")
    fused = torch.randn(2 * queries, 10 * 6 * dim + 5, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    for off in (0, 1, 8):
        q = fused[:, off:off + 12 * dim].unflatten(1, (12, dim))[:, ::2]
        for x in (q, q[:, :1].expand(-1, heads * groups, -1)):
            a = nv.nvfp4_kv_attention(x, cache, table, lens, query_starts=starts, max_queries=queries)
            b = nv.nvfp4_kv_attention(x.contiguous(), cache, table, lens, query_starts=starts, max_queries=queries)
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", [1, 90])
def test_shared_pages_and_same_bits(dtype, queries):
    """Sequences that share their pages (a common prefix): each row's bits are those of the same call again."""
    cache = _kv.random_cache(40, 16, 2, 128, 9)
    table = torch.arange(40, dtype=torch.int32).view(1, 40).expand(3, 40).contiguous()
    lens = torch.tensor([640, 500, 640], dtype=torch.int32, device="cuda")
    starts = [0, queries, 2 * queries, 3 * queries]
    q = torch.randn(3 * queries, 8, 128, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    q[2 * queries:] = q[:queries]
    args = dict(query_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), max_queries=queries, return_lse=True)
    a, la = nv.nvfp4_kv_attention(q, cache, table.cuda(), lens, **args)
    b, lb = nv.nvfp4_kv_attention(q, cache, table.cuda(), lens, **args)
    assert torch.equal(a, b) and torch.equal(la, lb)
    assert torch.equal(a[:queries], a[2 * queries:])
    _kv.check(a, la, _kv.reference(q, cache, table, lens, starts, 128 ** -0.5), "shared")


def test_offsets_past_32_bits():
    """Pages at the far end of a cache whose codes pass 4 GiB."""
    heads, dim, page = 16, 256, 64
    pages = (1 << 32) // (heads * page * dim // 2) + 3
    small = _kv.random_cache(3, page, heads, dim, 12)
    cache = nv.kv_cache(pages, page, heads, dim, small.global_scale_k, small.global_scale_v)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        getattr(cache, n)[-3:] = getattr(small, n)
    lens = torch.tensor([page * 3 - 5], dtype=torch.int32, device="cuda")
    for queries in (1, 30):
        q = torch.randn(queries, 2 * heads, dim, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
        starts = torch.tensor([0, queries], dtype=torch.int32, device="cuda")
        t = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
        a = nv.nvfp4_kv_attention(q, small, t, lens, query_starts=starts, max_queries=queries)
        b = nv.nvfp4_kv_attention(q, cache, t + (pages - 3), lens, query_starts=starts, max_queries=queries)
        assert torch.equal(a, b) and a.any()


@pytest.mark.parametrize("queries", [1, 100])
def test_stream_and_graph(queries):
    """On a side stream, captured: every replay equals the eager call, with eager work in between."""
    cache = _kv.random_cache(200, 16, 2, 128, 13)
    table = torch.randperm(200, generator=torch.Generator().manual_seed(6)).to(torch.int32).view(2, 100).cuda()
    lens = torch.tensor([1600, 900], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, queries, 2 * queries], dtype=torch.int32, device="cuda")
    q = torch.randn(2 * queries, 8, 128, device="cuda").bfloat16()
    out = torch.empty_like(q)
    wsp, _ = nv.kv_attention_workspace(cache, 2 * queries, 8, 2, queries, 1600)

    def step():
        nv.nvfp4_kv_attention(q, cache, table, lens, query_starts=starts, max_queries=queries, max_context=1600,
                              out=out, workspace=wsp)

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
        q.copy_(torch.randn(2 * queries, 8, 128, generator=torch.Generator().manual_seed(20 + i)).bfloat16())
        lens.copy_(torch.tensor([1600 - 300 * i, 900 + 7 * i], dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        wsp.fill_(i)
        step()
        assert torch.equal(replayed, out), i


def test_write_then_attend():
    """Tokens written by nvfp4_kv_write, attended to as they were quantized: the dense attention
    over nvfp4_kv_read's values agrees within the bound."""
    heads, groups, dim, page = 2, 4, 128, 16
    g = torch.tensor([5.0], device="cuda")
    cache = nv.kv_cache(12, page, heads, dim, g, g)
    gen = torch.Generator().manual_seed(30)
    table = torch.randperm(12, generator=gen).to(torch.int32).view(1, 12)
    slots = table.long().repeat_interleave(page, 1).view(-1) * page + torch.arange(192) % page
    k = torch.randn(150, heads, dim, generator=gen).bfloat16().cuda()
    v = torch.randn(150, heads, dim, generator=gen).bfloat16().cuda()
    nv.nvfp4_kv_write(cache, k, v, slots[:150].cuda())
    q = torch.randn(20, heads * groups, dim, generator=gen).bfloat16().cuda()
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    got, lse = nv.nvfp4_kv_attention(q, cache, table.cuda(), lens, query_starts=starts, max_queries=20, return_lse=True)
    _kv.check(got, lse, _kv.reference(q, cache, table, lens, [0, 20], dim ** -0.5), "written")
    rk, rv = nv.nvfp4_kv_read(cache, slots[:150].cuda(), dtype=torch.float32)
    rk, rv = (t.repeat_interleave(groups, 1).transpose(0, 1) for t in (rk, rv))
    s = q.float().transpose(0, 1) @ rk.transpose(1, 2).contiguous() * dim ** -0.5
    i = torch.arange(20, device="cuda").view(-1, 1)
    s = s.masked_fill(torch.arange(150, device="cuda") > 130 + i, float("-inf"))
    dense = (torch.softmax(s, -1) @ rv).transpose(0, 1)
    assert (got.float() - dense).abs().max() <= 2.0 ** -7 * dense.abs().max()
