"""Attention over the NVFP4 cache near the limits of its sizes: contexts of more than 2^30 keys on pages of millions
of tokens (the page table names two pages again and again, so that little memory is needed)."""
import math

import pytest
import torch

import nvfp4_block_scaled_amd as nv
import _kv
from _parity import say

pytestmark = pytest.mark.gpu

PAGE, DIM = 1 << 22, 16
MOST = 2 ** 31 - 4096  # the longest context


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


@pytest.fixture(scope="module")
def cache():
    """Page 0: keys of 0 and values of -1.  Page 1: keys of 1, values 0.5 to 6 by the element, small ones up to 8
    tokens.  No global scales."""
    c = nv.kv_cache(2, PAGE, 1, DIM)
    for x in (c.k_scales, c.v_scales):
        x.fill_(0x38)  # 1
    c.v_codes[0] = 0xAA
    c.k_codes[1] = 0x22
    c.v_codes[1] = torch.tensor([0x21, 0x43, 0x65, 0x17] * 2, dtype=torch.uint8, device="cuda")
    yield c


VALUES = [0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 0.5] * 2


@pytest.mark.parametrize("queries", [1, 45])
@pytest.mark.parametrize("context", [257 * PAGE - 12345, MOST])
def test_contexts_past_2_30(cache, queries, context):
    """All pages but the last are page 0, scores 0; the last is page 1, scores 24, so that the output is its values.
    The sums are float32 and add up to 2^21 weights one after the other: 2^-3 of each sum at most, for the output
    and for lse's argument; the flat pages weigh 2^31 e^-24 / 2^21, less than 2^-24 of it."""
    say(f"context {context} queries {queries}")
    pages = -(-context // PAGE)
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    q = torch.full((queries, 1, DIM), 1.5, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([context], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, queries], dtype=torch.int32, device="cuda")
    got, lse = nv.nvfp4_kv_attention(q, cache, table, lens, query_starts=starts, max_queries=queries, scale=1.0,
                                     max_context=context, return_lse=True)
    torch.cuda.synchronize()
    want = torch.tensor(VALUES).double()
    assert ((got[:, 0].cpu().double() - want).abs() <= (2 * 2.0 ** -3 + 2.0 ** -8) * want).all(), got[0, 0]
    n = context - (pages - 1) * PAGE - queries + 1 + torch.arange(queries)
    assert ((lse[:, 0].cpu().double() - (24 + n.double().log())).abs() <= -math.log(1 - 2.0 ** -3) + 1e-4).all()


@pytest.mark.parametrize("queries", [1, 3, 45])
@pytest.mark.parametrize("window", [0, MOST - 1, 50])
def test_short_contexts_under_the_longest_bound(queries, window):
    """max_context as large as it may be, contexts and queries as usual, also more queries than tokens."""
    say(f"short contexts, queries {queries} window {window}")
    small = _kv.random_cache(2, PAGE, 1, DIM, 3, None, None)
    table = torch.tensor([[0, 1] + [-1] * 510, [1, 0] + [-1] * 510], dtype=torch.int32)
    lens = torch.tensor([130, 2], dtype=torch.int32, device="cuda")
    starts = [0, queries, 2 * queries]
    q = torch.randn(2 * queries, 2, DIM, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    got, lse = nv.nvfp4_kv_attention(q, small, table.cuda(), lens, max_queries=queries, max_context=MOST, window=window,
                                     query_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), return_lse=True)
    _kv.check(got, lse, _kv.reference(q, small, table, lens, starts, DIM ** -0.5, True, window), "short")


def test_longest_context_is_refused_beyond():
    c = nv.kv_cache(1, PAGE, 1, DIM)
    table = torch.zeros(1, 512, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 1, DIM, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_kv_attention(q, c, table, torch.ones(1, dtype=torch.int32, device="cuda"), max_context=MOST + 1)
