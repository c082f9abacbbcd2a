"""Attention over the NVFP4 cache where the size of the scores, of their factor
or of what a mask hides could spoil a result.  The bound is that of _kv.py."""
import pytest
import torch

import nvfp4_block_scaled_amd as nv
import _kv
from _parity import say
from test_gpu_kv_attention import _batch, _run

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
MASKS = [(True, 0), (True, 37), (False, 0)]  # causal, window
ROWS = [1, 17]  # queries: few rows a kv head, and many


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("queries", ROWS)
@pytest.mark.parametrize("causal,window", MASKS)
def test_zero_global_scales(dtype, dim, queries, causal, window):
    """A global scale of 0 (the largest magnitude of keys or values that are all 0): every score is 0 and the
    output the mean of what is seen, or every output is 0."""
    say(f"global scale 0 {dtype} d{dim} queries {queries} causal {causal} window {window}")
    contexts, counts = [130, 64, queries, 0], [queries, queries, queries, queries]
    for g in ((0.0, 6.0), (20.0, 0.0), (0.0, 0.0)):
        _run(contexts, counts, 1, 2, dim, 16, dtype, 2000 + dim + queries, causal=causal, window=window, g=g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("queries", ROWS)
@pytest.mark.parametrize("causal,window", MASKS)
def test_tiny_queries(dtype, dim, queries, causal, window):
    """Queries around and below the smallest normal number, the scale as usual: the scores are as good as 0."""
    say(f"tiny queries {dtype} d{dim} queries {queries} causal {causal} window {window}")
    contexts, counts = [130, 64, queries, 0], [queries, queries, queries, queries]
    for size, g_k in ((2.0 ** -124, 4.0), (2.0 ** -130, 20.0), (2.0 ** -134, 6.0), (2.0 ** -140, 22.0)):
        _run(contexts, counts, 1, 2, dim, 16, dtype, 2100 + dim + queries, causal=causal, window=window, g=(g_k, 6.0),
             q_size=size)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", ROWS)
def test_other_global_scales(dtype, queries):
    """Negative global scales are factors like others; one that is NaN makes NaN of every query that sees a key,
    and of no other."""
    say(f"global scales below 0 and NaN {dtype} queries {queries}")
    contexts, counts = [130, 64, max(queries - 5, 0), 0], [queries] * 4
    for causal, window in MASKS:
        _run(contexts, counts, 1, 2, 64, 16, dtype, 2300, causal=causal, window=window, g=(-20.0, -6.0))
    table, pages, _ = _batch(contexts, 16, 5)
    cache = _kv.random_cache(pages, 16, 1, 64, 2301, float("nan"), 6.0)
    q = torch.randn(4 * queries, 2, 64, generator=torch.Generator().manual_seed(2302)).to(dtype).cuda()
    starts = torch.arange(5, dtype=torch.int32, device="cuda") * queries
    got, lse = nv.nvfp4_kv_attention(q, cache, table.cuda(), torch.tensor(contexts, dtype=torch.int32, device="cuda"),
                                     query_starts=starts, max_queries=queries, return_lse=True)
    sees = torch.cat([torch.arange(c - queries, c) >= 0 for c in contexts]).cuda()
    assert torch.isnan(got[sees]).all() and torch.isnan(lse[sees]).all()
    assert not got[~sees].any() and (lse[~sees] == float("-inf")).all() and not sees.all()
