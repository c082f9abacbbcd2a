"""Attention over the NVFP4 cache on both sides of the rule that leaves a
context to one workgroup (1024 keys and 6 more a pair of sequence and kv head,
at most 4096), and shared out among more sequences than one wave scans.  The
bound is that of _kv.py."""
import pytest
import torch

import nvfp4_block_scaled_amd as nv
from _parity import say
from test_gpu_kv_attention import _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


def test_workspace_follows_the_rule():
    cache = nv.kv_cache(300, 16, 8, 64)

    def size(seqs, context):
        return nv.kv_attention_workspace(cache, seqs, 8, seqs, 1, context)[1]

    assert size(1, 1024 + 48) == 0 and size(1, 1024 + 49) > 0
    assert size(16, 1024 + 768) == 0 and size(16, 1024 + 769) > 0
    assert size(64, 4096) == 0 and size(64, 4097) > 0 and size(256, 4097) > 0


@pytest.mark.parametrize("page", [1, 5, 16])
@pytest.mark.parametrize("longest", [4096, 4097])
def test_many_pairs(page, longest):
    """512 pairs, contexts around the limit, pages staged in several goes by a workgroup alone."""
    say(f"page {page} longest {longest}")
    contexts = [longest, 1, 0, 2049, 513, 3000, 128, 129, 1025, 700, 4000, 31, 512, 2048, 1537, 96]
    _run(contexts, [1] * 16, 32, 1, 16, page, torch.bfloat16, 701 + page)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_several_tokens_alone(dtype):
    """Up to 32 rows a pair, a window, sequences without queries."""
    contexts = [1900, 2000, 7, 0, 1100, 1500, 64, 1999]
    _run(contexts, [4, 1, 4, 3, 0, 2, 4, 4], 24, 8, 32, 16, dtype, 721)
    _run(contexts, [4, 1, 4, 3, 0, 2, 4, 4], 24, 4, 48, 24, dtype, 722, window=1500)


@pytest.mark.parametrize("seqs", [65, 130])
def test_many_sequences_shared_out(seqs):
    """More sequences than one wave scans, one context past the limit for all: shared out."""
    say(f"sequences {seqs}")
    contexts = [(i * 577) % 1500 for i in range(seqs)]
    contexts[seqs // 2] = 5000
    counts = [0 if i % 11 == 5 else 1 for i in range(seqs)]
    _run(contexts, counts, 2, 2, 64, 16, torch.bfloat16, 731 + seqs, tail=1)
