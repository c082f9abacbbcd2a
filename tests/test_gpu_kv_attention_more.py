"""Attention over the NVFP4 cache where its work is shared out: more sequences
than one wave scans, contexts whose page numbers are staged in several goes,
runs that end inside a pair, prompts whose keys are split, and queries that
are not finite.  The bound is that of _kv.py."""
import pytest
import torch

import nvfp4_block_scaled_amd as nv
import _kv
from _parity import say
from test_gpu_kv_attention import _batch, _run

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("seqs", [63, 64, 65, 130])
@pytest.mark.parametrize("longest", [90, 1500])
def test_many_sequences(seqs, longest):
    """Ragged batches around the 64 sequences of one scan; empty ones between; one launch and two."""
    say(f"sequences {seqs} longest {longest}")
    contexts = [(i * 37) % 91 for i in range(seqs)]
    contexts[seqs // 2] = longest
    counts = [0 if i % 11 == 5 else 1 for i in range(seqs)]
    _run(contexts, counts, 2, 2, 64, 16, torch.bfloat16, 301 + seqs, tail=1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [1, 2, 3])
def test_small_pages(dtype, page):
    """Pages of one to three tokens: page numbers are staged in several goes, also behind another run."""
    _run([1000, 0, 2600, 700], [1, 1, 1, 1], 1, 4, 64, page, dtype, 411 + page)
    _run([900], [1], 2, 2, 128, page, dtype, 412 + page)


@pytest.mark.parametrize("heads,groups", [(1, 1), (7, 3), (16, 1)])
def test_runs_across_pairs(heads, groups):
    """Pairs whose units do not divide evenly among the workgroups."""
    _run([1281, 1153, 2049, 1, 1407], [1] * 5, heads, groups, 64, 16, torch.float16, 501 + heads)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 80])
def test_split_prompts(dtype, dim):
    """Few tiles of rows over long contexts: the keys are split and joined."""
    _run([3000, 1200], [40, 9], 1, 1, dim, 16, dtype, 601 + dim)
    _run([2500], [45], 1, 2, dim, 32, dtype, 602 + dim, window=1900)
    _run([2600], [35], 1, 1, dim, 24, dtype, 603 + dim, causal=False)


@pytest.mark.parametrize("queries", [1, 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_queries_not_finite(queries, bad):
    """A query that is not finite gives NaN in its own row and nowhere else."""
    table, pages, _ = _batch([200], 16, 3)
    cache = _kv.random_cache(pages, 16, 1, 64, 4)
    lens = torch.tensor([200], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, queries], dtype=torch.int32, device="cuda")
    q = torch.randn(queries, 4, 64, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    args = (cache, table.cuda(), lens)
    more = dict(query_starts=starts, max_queries=queries, return_lse=True)
    want, want_lse = nv.nvfp4_kv_attention(q, *args, **more)
    q[queries // 2, 2, 7] = bad
    got, lse = nv.nvfp4_kv_attention(q, *args, **more)
    assert torch.isnan(got[queries // 2, 2]).all() and torch.isnan(lse[queries // 2, 2])
    got[queries // 2, 2], lse[queries // 2, 2] = want[queries // 2, 2], want_lse[queries // 2, 2]
    assert torch.equal(got, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -60, 2.0 ** 60, 2.0 ** 110])
def test_query_sizes(size):
    """bfloat16 queries of any size: a power of two on the queries is one on the scores, bit for bit
    where that product itself is exact (at 2^-120 some elements fall below bfloat16's normal range)."""
    table, pages, _ = _batch([300], 16, 3)
    cache = _kv.random_cache(pages, 16, 1, 64, 4)
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    for queries in (1, 40):
        starts = torch.tensor([0, queries], dtype=torch.int32, device="cuda")
        q = torch.randn(queries, 2, 64, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
        more = dict(query_starts=starts, max_queries=queries)
        want = nv.nvfp4_kv_attention(q, cache, table.cuda(), lens, scale=0.125, **more)
        got, lse = nv.nvfp4_kv_attention(q * size, cache, table.cuda(), lens, scale=0.125 / size, return_lse=True,
                                         **more)
        _kv.check(got, lse, _kv.reference(q * size, cache, table, lens, [0, queries], 0.125 / size), f"size {size}")
        if torch.equal((q * size) / size, q):
            assert torch.equal(got, want)
        else:
            assert size < 2.0 ** -100


def test_excess_device_sizes():
    """Query counts and contexts on the device beyond the stated bounds stay within memory: rows
    past max_queries are left alone and nothing else changes."""
    table, pages, _ = _batch([100, 100], 16, 3)
    cache = _kv.random_cache(pages, 16, 1, 64, 4)
    q = torch.randn(20, 2, 64, generator=torch.Generator().manual_seed(7)).half().cuda()
    lens = torch.tensor([100, 100], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    nv.nvfp4_kv_attention(q, cache, table.cuda(), lens, max_queries=4, out=out,
                          query_starts=torch.tensor([0, 10, 2 ** 30], dtype=torch.int32, device="cuda"))
    assert (out[4:10] == 7).all() and (out[14:] == 7).all()
    assert torch.isfinite(out).all() and not (out[:4] == 7).all() and not (out[10:14] == 7).all()
    big = torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32, device="cuda")
    got = nv.nvfp4_kv_attention(q, cache, table.cuda(), big, max_queries=10, causal=False,
                                query_starts=torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda"))
    assert torch.isfinite(got).all() and not got[10:].any()
