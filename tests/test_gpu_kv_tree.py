"""Attention of drafted trees (nvfp4_kv_tree_attention) against 64 bits on the CPU, within the bound that _kv.py
derives (the arithmetic is that of nvfp4_kv_attention): types, head layouts, trees of one draft to several words,
masks that leave rows empty, windows, contexts shorter than the drafts, pages that end inside a tile, held values
that are no number, strides, streams and graphs."""
import pytest
import torch

import nvfp4_block_scaled_amd as nv
import _kv
from _parity import guarded, guarded_workspace, say
from test_gpu_kv_attention import _batch, _poison_tails

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


def random_trees(counts, seed):
    gen = torch.Generator().manual_seed(seed)
    return [[int(torch.randint(max(-1, d - 9), d, (1,), generator=gen)) if d else -1 for d in range(n)] for n in counts]


def visible(tree_row, context, n, position, window, j):
    """Which keys j a query with this row of the masks sees."""
    base = context - n
    see = j < base
    if window:
        see &= j > min(max(position, base), context - 1) - window
    words = [int(w) for w in tree_row]
    bits = torch.tensor([(words[d // 64] >> (d % 64)) & 1 if d // 64 < len(words) else 0 for d in (j - base).clamp(min=0).tolist()],
                        dtype=torch.bool)
    return see | ((j >= base) & bits)


def reference(q, cache, table, lens, starts, scale, tree, positions, window):
    """As _kv.reference, with the keys that visible() gives."""
    c = {n: getattr(cache, n).cpu() for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    g = {n: None if getattr(cache, "global_scale_" + n) is None else getattr(cache, "global_scale_" + n).item() for n in "kv"}
    dtype, u = q.dtype, _kv.UNIT[q.dtype]
    p_round = 2.0 ** -22 if dtype == torch.float32 else 2.0 ** -11
    x = q.detach().cpu().double()
    tokens, hq, dim = x.shape
    groups = hq // cache.heads
    out = torch.full((tokens, hq, dim), float("nan"), dtype=torch.float64)
    lse = torch.full((tokens, hq), float("nan"), dtype=torch.float64)
    bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    tree = tree.cpu()
    for b, context in enumerate(lens):
        first, last = starts[b], starts[b + 1]
        n = last - first
        rows = table[b].tolist()
        j = [i for i in range(max(context, 0)) if 0 <= rows[i // cache.page_size] < cache.pages]
        pages = torch.tensor([rows[i // cache.page_size] for i in j], dtype=torch.long)
        offs = torch.tensor([i % cache.page_size for i in j], dtype=torch.long)
        key = torch.tensor(j, dtype=torch.long)
        sees = [visible(tree[i], context, n, int(positions[i]), window, key) for i in range(first, last)]
        for h in range(cache.heads if n else 0):
            k = _kv.values(c["k_codes"][pages, h, offs], c["k_scales"][pages, h, offs], g["k"])
            v = _kv.values(c["v_codes"][pages, h, offs], c["v_scales"][pages, h, offs], g["v"])
            for i in range(first, last):
                see = sees[i - first]
                for a in range(h * groups, (h + 1) * groups):
                    if not see.any():
                        out[i, a], lse[i, a] = 0.0, float("-inf")
                        continue
                    ks, vs = k[see], v[see]
                    s = ks @ x[i, a] * scale
                    lse[i, a] = torch.logsumexp(s, 0)
                    w = torch.exp(s - lse[i, a])
                    out[i, a] = w @ vs
                    size = (ks.abs() @ x[i, a].abs() * scale).max().item()
                    e = (dim + 8) * 2.0 ** -24 * size + (2.0 ** -22 * size if dtype == torch.float32 else 0.0)
                    more = len(s) * 2.0 ** -24
                    bound[i, a] = u * out[i, a].abs() + _kv.TINY[dtype] + \
                        (p_round + 4 * e + 2.0 ** -18 + 2 * more) * (w @ vs.abs()) * (1 + 2 * u)
                    lse_bound[i, a] = e + 2.0 ** -20 + more + 2.0 ** -22 * abs(lse[i, a].item())
    return out, lse, bound, lse_bound


def setup(contexts, counts, heads, groups, dim, page, dtype, seed, tail=0):
    table, pages, unwritten = _batch(contexts, page, seed)
    cache = _kv.random_cache(pages, page, heads, dim, seed, unwritten=unwritten)
    _poison_tails(cache, table, contexts)
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    gen = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(starts[-1] + tail, heads * groups, dim, generator=gen).to(dtype).cuda()
    return table, cache, starts, q


def run(contexts, counts, heads, groups, dim, page, dtype, seed, window=0, tail=0, masks=None, words=None):
    table, cache, starts, q = setup(contexts, counts, heads, groups, dim, page, dtype, seed, tail)
    tree, depths = nv.kv_trees(random_trees(counts, seed))
    if masks is not None:
        tree = masks(tree)
    if words is not None:
        tree = torch.cat([tree, torch.full((len(tree), words - tree.shape[1]), -1)], 1)  # bits that count for nothing
    positions = torch.cat([torch.tensor([contexts[b] - n], dtype=torch.int32).expand(n) for b, n in enumerate(counts)]) + depths
    tree = torch.cat([tree, torch.full((tail, tree.shape[1]), -1)])
    positions = torch.cat([positions, torch.zeros(tail, dtype=torch.int32)])
    lens = torch.tensor(contexts, dtype=torch.int32, device="cuda")
    out = guarded(tuple(q.shape), dtype)
    out.t.fill_(float("nan"))
    most, top = max(max(counts), 1), max(max(contexts), 0)
    _, nbytes = nv.kv_tree_attention_workspace(cache, len(q), heads * groups, len(contexts), most, top, window)
    wsp = guarded_workspace(nbytes)
    wsp.t.fill_(255)
    got, lse = nv.nvfp4_kv_tree_attention(
        q, cache, table.cuda(), lens, torch.tensor(starts, dtype=torch.int32, device="cuda"), tree.cuda(), max_queries=most,
        max_context=top, positions=positions.cuda() if window else None, window=window, return_lse=True, out=out.t,
        workspace=wsp.t)
    torch.cuda.synchronize()
    out.check("out")
    wsp.check("workspace")
    ref = reference(q, cache, table, contexts, starts, dim ** -0.5, tree, positions, window)
    _kv.check(got, lse, ref, f"{dtype} d{dim} g{groups} page {page}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,groups,dim,page", [
    (1, 1, 16, 1), (2, 4, 128, 16), (1, 8, 64, 64), (3, 1, 64, 7), (2, 2, 96, 24), (1, 2, 256, 32), (2, 3, 80, 16),
    (1, 2, 192, 128), (1, 17, 128, 16), (2, 1, 240, 5)])
def test_few_rows(dtype, heads, groups, dim, page):
    """Small trees: contexts of none, shorter than the drafts, around the tile sizes."""
    say(f"tree few {dtype} h{heads} g{groups} d{dim} page {page}")
    n = max(1, 32 // groups)
    contexts = [0, 1, n, n + 1, 33, 64, 65, 129, 257, 300, 40]
    counts = [n, n, n, n, 1, n, max(1, n - 1), n, n, 0, min(2, n)]
    run(contexts, counts, heads, groups, dim, page, dtype, 20 + dim + groups, tail=2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,groups,dim,page", [
    (1, 1, 16, 1), (2, 4, 128, 16), (1, 8, 64, 64), (1, 5, 96, 24), (1, 2, 256, 32), (1, 3, 192, 7), (2, 1, 80, 16)])
@pytest.mark.parametrize("window", [0, 1, 40])
def test_many_rows(dtype, heads, groups, dim, page, window):
    """Trees of 33 to 130 drafts (masks of up to three words), ragged."""
    contexts = [70, 129, 200, 260, 64, 20]
    counts = [33, 65, 130, 64, 0, 40]
    run(contexts, counts, heads, groups, dim, page, dtype, 50 + dim + window, window=window, tail=3)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window", [1, 2, 17, 33, 200])
def test_windows(dtype, window):
    run([0, 1, 7, 8, 33, 64, 257, 130], [7, 7, 7, 7, 0, 1, 7, 6], 2, 4, 128, 16, dtype, 500 + window, window=window)


@pytest.mark.parametrize("counts,contexts", [([5, 8, 1], [2100, 4500, 1200]), ([60, 20, 64], [3000, 1100, 700])])
@pytest.mark.parametrize("window", [0, 1000])
def test_long_contexts(counts, contexts, window):
    """Contexts whose keys several workgroups share."""
    run(contexts, counts, 1, 4, 128, 16, torch.bfloat16, 70 + window, window=window)


@pytest.mark.parametrize("n", [6, 50])
def test_any_masks(n):
    """Masks that are no trees: none set, all set, random ones, and words more than needed."""
    contexts, counts = [n, 90, n + 1, 10], [n, n, n, n]
    gen = torch.Generator().manual_seed(n)
    run(contexts, counts, 2, 2, 64, 16, torch.bfloat16, 81, masks=lambda t: torch.zeros_like(t))
    run(contexts, counts, 2, 2, 64, 16, torch.bfloat16, 82, masks=lambda t: torch.full_like(t, -1), words=3)
    run(contexts, counts, 2, 2, 64, 16, torch.float32, 83, words=2,
        masks=lambda t: torch.randint(-2 ** 62, 2 ** 62, t.shape, generator=gen))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,groups", [(7, 4), (40, 4), (1, 1)])
def test_chain_is_causal(dtype, n, groups):
    """A chain of drafts is a sequence's next tokens: the bits of nvfp4_kv_attention, but for other tiles of keys."""
    contexts = [n, 100 + n, 1500, 77 + n]
    table, cache, starts, q = setup(contexts, [n] * 4, 2, groups, 128, 16, dtype, 90 + n)
    tree, depths = nv.kv_trees([list(range(-1, n - 1))] * 4)
    assert depths.tolist() == list(range(n)) * 4
    lens = torch.tensor(contexts, dtype=torch.int32, device="cuda")
    s = torch.tensor(starts, dtype=torch.int32, device="cuda")
    for window in (0, 50):
        positions = (torch.repeat_interleave(lens.cpu() - n, n) + depths).int().cuda() if window else None
        a, la = nv.nvfp4_kv_tree_attention(q, cache, table.cuda(), lens, s, tree.cuda(), max_queries=n, positions=positions,
                                           window=min(window, n + 43), return_lse=True)
        b, lb = nv.nvfp4_kv_attention(q, cache, table.cuda(), lens, s, max_queries=n, window=min(window, n + 43), return_lse=True)
        if n * groups > 32:
            # More than 32 rows a head: the keys are shared out among the workgroups by another rule than a
            # sequence's next tokens' (and with a window their ranges begin elsewhere).  Other parts, another order of
            # the sums: each answer is within its bound of the 64-bit one, so the two within twice that of each other.
            ref = reference(q, cache, table, contexts, starts, 128 ** -0.5, tree,
                            depths if positions is None else positions.cpu(), min(window, n + 43))
            assert ((a.double() - b.double()).abs().cpu() <= 2 * ref[2]).all()
            assert ((la.double() - lb.double()).abs().cpu() <= 2 * ref[3]).all()
        else:
            assert torch.equal(a, b) and torch.equal(la, lb), window


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,groups,dim", [(6, 4, 128), (1, 1, 64), (50, 4, 128), (40, 2, 96)])
def test_values_that_are_no_number(dtype, n, groups, dim):
    """A held value that is NaN reaches the queries that see its key, and no other; an unseen key's NaN nothing."""
    contexts, page = [n + 45, n], 16
    table, cache, starts, q = setup(contexts, [n, n], 1, groups, dim, page, dtype, 130 + n)
    tree, _ = nv.kv_trees([[-1] * n] * 2)  # each draft sees itself alone, besides the context
    args = (q, cache, table.cuda(), torch.tensor(contexts, dtype=torch.int32, device="cuda"),
            torch.tensor(starts, dtype=torch.int32, device="cuda"))
    want = nv.nvfp4_kv_tree_attention(*args, tree.cuda(), max_queries=n)
    for b, d in ((0, 0), (0, n - 1), (1, n // 2)):
        at = contexts[b] - n + d
        scales = cache.v_scales[table[b, at // page], 0, at % page]
        before = scales.clone()
        scales[1] = 127
        got = nv.nvfp4_kv_tree_attention(*args, tree.cuda(), max_queries=n)
        clean = torch.ones(2 * n, dtype=torch.bool)
        clean[b * n + d] = False
        assert torch.equal(got[clean], want[clean]), (b, d)
        row = got[b * n + d].float().cpu()
        assert row[:, 16:32].isnan().all() and torch.equal(row[:, :16], want[b * n + d].float().cpu()[:, :16])
        none = nv.nvfp4_kv_tree_attention(*args, torch.zeros_like(tree).cuda(), max_queries=n)
        assert torch.isfinite(none).all()
        k_scales = cache.k_scales[table[b, at // page], 0, at % page]
        k_before = k_scales.clone()
        scales.copy_(before)
        k_scales.fill_(255)
        got = nv.nvfp4_kv_tree_attention(*args, tree.cuda(), max_queries=n)
        assert torch.equal(got[clean], want[clean]) and got[b * n + d].isnan().all()
        k_scales.copy_(k_before)


def test_strides_streams_graphs():
    n, contexts = 9, [200, 31, 64]
    table, cache, starts, _ = setup(contexts, [n] * 3, 2, 4, 64, 16, torch.bfloat16, 150)
    fused = torch.randn(3 * n, 12, 65, device="cuda").to(torch.bfloat16)
    tree = nv.kv_trees(random_trees([n] * 3, 5))[0].cuda()
    lens = torch.tensor(contexts, dtype=torch.int32, device="cuda")
    s = torch.tensor(starts, dtype=torch.int32, device="cuda")

    def call(q, out=None):
        return nv.nvfp4_kv_tree_attention(q, cache, table.cuda() if out is None else table_d, lens, s, tree, max_queries=n, out=out)

    table_d = table.cuda()
    q = fused[:, 2:10, 1:]
    want = call(q.contiguous())
    assert torch.equal(call(q), want)
    assert nv.nvfp4_kv_tree_attention(q[:0], cache, table_d, lens, s * 0, tree[:0]).shape == (0, 8, 64)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(q, out)
        side.synchronize()
        assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(q, out)
    for i in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        call(q.flip(0))
