"""Attention of drafted trees where workgroups share the work out: more units of keys than workgroups, so that each
takes several, its runs begin and end inside tiles and cross from one tile, head and sequence to the next; more than
64 sequences; graphs replayed on other contents.  Against 64 bits on the CPU within the bound of _kv.py."""
import pytest
import torch

import nvfp4_block_scaled_amd as nv
import _kv
from _parity import guarded, guarded_workspace, say
from test_gpu_kv_tree import random_trees, reference as row_reference, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


def sees(tree, context, n, positions, window, key):
    """[n, keys]: which of the keys `key` the queries see."""
    base = context - n
    low = positions.long().clamp(min=base).clamp(max=context - 1)[:, None]
    old = (key < base) & ((key > low - window) if window else True)
    d = (key - base).clamp(min=0)
    word = (d // 64).clamp(max=tree.shape[1] - 1)
    bits = (tree[:, word] >> (d % 64)) & 1
    return old | ((key >= base) & (d < 64 * tree.shape[1]) & (bits == 1))


def reference(q, cache, table, lens, starts, scale, tree, positions, window):
    """test_gpu_kv_tree.reference, all rows of a head at a time."""
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
    for b, context in enumerate(lens):
        first, last = starts[b], starts[b + 1]
        n = last - first
        if n == 0:
            continue
        j = torch.arange(max(context, 0))
        row = table[b].long()[j // cache.page_size]
        j = j[(row >= 0) & (row < cache.pages)]
        pages, offs = table[b].long()[j // cache.page_size], j % cache.page_size
        see = sees(tree[first:last], context, n, positions[first:last], window, j)[:, None]  # [n, 1, keys]
        any_seen = see.any(-1)
        seen = see.sum(-1).double()
        for h in range(cache.heads):
            k = _kv.values(c["k_codes"][pages, h, offs], c["k_scales"][pages, h, offs], g["k"])
            v = _kv.values(c["v_codes"][pages, h, offs], c["v_scales"][pages, h, offs], g["v"])
            at = slice(h * groups, (h + 1) * groups)
            r = x[first:last, at]
            hidden = ~see.expand(n, groups, len(j))
            # (a value that is no number and that no row sees counts for nothing)
            s = (r @ k.nan_to_num().T * scale).masked_fill(hidden, float("-inf"))
            z = torch.logsumexp(s, -1) if len(j) else torch.full((n, groups), float("-inf"), dtype=torch.float64)
            w = torch.where(hidden, 0.0, torch.exp(s - z.clamp(min=-1e300)[..., None]))
            o, size_v = w @ v.nan_to_num(), w @ v.nan_to_num().abs()
            sizes = (r.abs() @ k.nan_to_num().abs().T * scale).masked_fill(hidden, 0.0)
            size = sizes.amax(-1) if len(j) else torch.zeros(n, groups, dtype=torch.float64)
            e = (dim + 8) * 2.0 ** -24 * size + (2.0 ** -22 * size if dtype == torch.float32 else 0.0)
            more = seen * 2.0 ** -24
            out[first:last, at], lse[first:last, at] = o, z
            there = any_seen.double()
            bound[first:last, at] = there[..., None] * (u * o.abs() + _kv.TINY[dtype] + (
                p_round + 4 * e + 2.0 ** -18 + 2 * more)[..., None] * size_v * (1 + 2 * u))
            lse_bound[first:last, at] = there * (e + 2.0 ** -20 + more + 2.0 ** -22 * z.abs().nan_to_num(posinf=0.0))
    return out, lse, bound, lse_bound


def most_groups(dim, dtype):
    """Workgroups of more than 32 rows a head that run at once."""
    wide = (dim + 63) // 64 * (2 if dtype == torch.float32 else 1)
    return torch.cuda.get_device_properties(0).multi_processor_count * (2 if wide <= 2 else 1)


def many_units(contexts, counts, heads, groups, window=0):
    """Units of 256 keys of every (sequence, kv head, 128 rows)."""
    total = 0
    for c, n in zip(contexts, counts):
        low = max(0, max(c - n, 0) - window + 1) if window else 0
        total += heads * -(-n * groups // 128) * max(1, -(-(c - low) // 256)) if n else 0
    return total


def batch(contexts, counts, heads, groups, dim, page, dtype, seed, holes=True, tail=3):
    table, cache, starts, q = setup(contexts, counts, heads, groups, dim, page, dtype, seed, tail)
    if holes:  # pages that are not there, one in some hundred
        gen = torch.Generator().manual_seed(seed + 7)
        gone = torch.rand(table.shape, generator=gen) < 0.01
        table = torch.where(gone, torch.where(torch.rand(table.shape, generator=gen) < 0.5, -1, 2 ** 31 - 1), table.long()).int()
    tree, depths = nv.kv_trees(random_trees(counts, seed))
    base = torch.cat([torch.tensor([contexts[b] - n], dtype=torch.int32).expand(n) for b, n in enumerate(counts)])
    tree = torch.cat([tree, torch.full((tail, tree.shape[1]), -1)])
    positions = torch.cat([base + depths, torch.zeros(tail, dtype=torch.int32)])
    return table, cache, starts, q, tree, positions


def call(q, cache, table, contexts, starts, tree, positions, window, most=None, top=None, **more):
    counts = [b - a for a, b in zip(starts, starts[1:])]
    return nv.nvfp4_kv_tree_attention(
        q, cache, table.cuda(), torch.tensor(contexts, dtype=torch.int32, device="cuda"),
        torch.tensor(starts, dtype=torch.int32, device="cuda"), tree.cuda(), max_queries=most or max(counts),
        max_context=top or max(contexts), positions=positions.cuda() if window else None, window=window, return_lse=True, **more)


def run(contexts, counts, heads, groups, dim, page, dtype, seed, window=0):
    table, cache, starts, q, tree, positions = batch(contexts, counts, heads, groups, dim, page, dtype, seed)
    out = guarded(tuple(q.shape), dtype)
    out.t.fill_(float("nan"))
    _, nbytes = nv.kv_tree_attention_workspace(cache, len(q), heads * groups, len(contexts), max(counts), max(contexts), window)
    wsp = guarded_workspace(nbytes)
    wsp.t.fill_(255)
    got, lse = call(q, cache, table, contexts, starts, tree, positions, window, out=out.t, workspace=wsp.t)
    torch.cuda.synchronize()
    out.check("out")
    wsp.check("workspace")
    ref = reference(q, cache, table, contexts, starts, dim ** -0.5, tree, positions, window)
    _kv.check(got, lse, ref, f"{dtype} d{dim} h{heads} g{groups}")
    return table, cache, starts, q, tree, positions, got, lse


def ragged(seqs, longest, fewest, most, seed):
    gen = torch.Generator().manual_seed(seed)
    contexts = torch.randint(1, longest + 1, (seqs,), generator=gen).tolist()
    contexts[seqs // 2], contexts[-1] = longest, 0
    counts = torch.randint(fewest, most + 1, (seqs,), generator=gen).tolist()
    counts[1], counts[seqs // 3] = most, 0
    return contexts, counts


def test_the_references_agree():
    contexts, counts = [70, 20, 0, 150], [33, 40, 5, 0]
    for window, dtype in ((0, torch.bfloat16), (9, torch.float32)):
        table, cache, starts, q, tree, positions = batch(contexts, counts, 2, 2, 32, 16, dtype, 3)
        one = row_reference(q, cache, table, contexts, starts, 0.2, tree, positions, window)
        two = reference(q, cache, table, contexts, starts, 0.2, tree, positions, window)
        for a, b in zip(one, two):
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.isinf(), b.isinf())
            fine = torch.isfinite(a)
            assert torch.allclose(a[fine], b[fine], rtol=1e-9, atol=1e-300)


@pytest.mark.parametrize("dtype,heads,groups,dim,page,window", [
    (torch.bfloat16, 8, 4, 64, 16, 0), (torch.bfloat16, 8, 4, 64, 16, 700), (torch.float16, 4, 8, 128, 64, 0),
    (torch.float32, 8, 4, 16, 7, 300), (torch.float32, 4, 2, 128, 16, 0), (torch.float16, 4, 4, 256, 32, 0),
    (torch.bfloat16, 8, 3, 80, 24, 999)])
def test_more_units_than_workgroups(dtype, heads, groups, dim, page, window):
    """Runs of several units a workgroup, over the ends of tiles, heads and sequences."""
    say(f"tree shared {dtype} h{heads} g{groups} d{dim} page {page} window {window}")
    contexts, counts = ragged(24, 3000, 33, 130, dim + window)
    units, most = many_units(contexts, counts, heads, groups, window), most_groups(dim, dtype)
    assert units > 2 * most, (units, most)
    run(contexts, counts, heads, groups, dim, page, dtype, 700 + dim, window)


@pytest.mark.parametrize("dtype,window", [(torch.bfloat16, 0), (torch.float32, 200)])
def test_more_than_64_sequences(dtype, window):
    """The sequences' units are summed 64 at a time; several have no queries, among them all of a block's."""
    contexts, counts = ragged(203, 900, 0, 40, 5)
    counts[64:130] = [0] * 66
    counts[140] = 40
    heads, groups, dim = 4, 4, 32
    assert many_units(contexts, counts, heads, groups, window) > most_groups(dim, dtype)
    run(contexts, counts, heads, groups, dim, 16, dtype, 41, window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_short_contexts_without_parts(dtype):
    """Contexts of one unit, more tiles than workgroups that run at once: nothing is split, nothing joined."""
    contexts, counts = ragged(90, 256, 33, 64, 6)
    heads, groups, dim = 8, 4, 16
    assert many_units(contexts, counts, heads, groups) > 2 * most_groups(dim, dtype)
    cache = run(contexts, counts, heads, groups, dim, 16, dtype, 43)[1]
    assert nv.kv_tree_attention_workspace(cache, sum(counts), 32, 90, 64, 256)[1] == 0


def test_many_sequences_of_short_contexts():
    """65535 sequences of 64 heads, four million tiles of one unit: a workgroup each, all of which count the sequences,
    would take minutes.  Only the last few have queries."""
    seqs, heads, dim, page = 65535, 64, 16, 16
    few, n = 9, 40
    contexts, counts = [0] * (seqs - few) + [200] * few, [0] * (seqs - few) + [n] * few
    table = torch.full((seqs, 16), -1, dtype=torch.int32)
    table[-few:, :13] = torch.randperm(13 * few, generator=torch.Generator().manual_seed(1)).view(few, 13).int()
    cache = _kv.random_cache(13 * few, page, heads, dim, 47)
    q = torch.randn(few * n, heads, dim, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    starts = [0] * (seqs - few) + [n * i for i in range(few + 1)]
    tree, depths = nv.kv_trees(random_trees([n] * few, 3))
    got, lse = call(q, cache, table, contexts, starts, tree, depths, 0, most=n, top=256)
    ref = reference(q, cache, table[-few:], contexts[-few:], starts[-few - 1:], dim ** -0.5, tree, depths, 0)
    _kv.check(got, lse, ref, "65535 sequences")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("seqs", [40, 150])
def test_few_rows_shared_out(dtype, seqs):
    """Up to 32 rows a head: runs of the streaming kernel over pairs and sequences, also more than 64 of them."""
    contexts, counts = ragged(seqs, 4500, 0, 8, seqs)
    run(contexts, counts, 2, 4, 32, 16, dtype, 45, 0)
    run(contexts, counts, 2, 4, 32, 16, dtype, 46, 3000)


@pytest.mark.parametrize("dtype,groups", [(torch.bfloat16, 4), (torch.float32, 4), (torch.bfloat16, 1)])
def test_values_that_are_no_number_in_later_runs(dtype, groups):
    """The first draft's value is no number in every sequence: its descendants' outputs are NaN there, in whichever
    run of a workgroup they are, and the others keep their bits."""
    contexts, counts = ragged(24, 3000, 33, 70, 9)
    contexts = [max(c, n) for c, n in zip(contexts, counts)]
    heads, dim, page = 8, 64, 16
    assert many_units(contexts, counts, heads, groups) > (2 if groups > 1 else 1) * most_groups(dim, dtype)
    table, cache, starts, q, tree, positions = batch(contexts, counts, heads, groups, dim, page, dtype, 51, holes=False, tail=0)
    want, want_lse = call(q, cache, table, contexts, starts, tree, positions, 0)
    for b, n in enumerate(counts):
        if n:
            at = contexts[b] - n
            cache.v_scales[table[b, at // page], :, at % page, 2] = 127
    got, lse = call(q, cache, table, contexts, starts, tree, positions, 0)
    hit = (tree[:, 0] & 1).bool().cuda()
    assert hit.any() and not hit.all()
    assert torch.equal(got[~hit], want[~hit]) and torch.equal(lse, want_lse)
    assert got[hit][..., 32:48].isnan().all()
    rest = torch.ones(dim, dtype=torch.bool)
    rest[32:48] = False
    assert torch.equal(got[hit][..., rest.cuda()], want[hit][..., rest.cuda()])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,groups", [(7, 4), (70, 4), (130, 1)])
@pytest.mark.parametrize("window", [1, 3, 65, 150])
def test_a_chain_with_a_window_is_causal(dtype, n, groups, window):
    """A chain of drafts behind a window, also one shorter than the chain, is nvfp4_kv_attention's: each answer is
    within its bound of the 64-bit one."""
    contexts = [n, 100 + n, 1500, 77 + n]
    table, cache, starts, q = setup(contexts, [n] * 4, 2, groups, 64, 16, dtype, 90 + n)
    tree, depths = nv.kv_trees([list(range(-1, n - 1))] * 4, window)
    positions = (torch.repeat_interleave(torch.tensor(contexts) - n, n) + depths).int()
    got, lse = call(q, cache, table, contexts, starts, tree, positions, window)
    ref = _kv.reference(q, cache, table, torch.tensor(contexts), starts, 0.125, window=window)
    _kv.check(got, lse, ref, f"chain {n} window {window}")
    same, same_lse = nv.nvfp4_kv_attention(
        q, cache, table.cuda(), torch.tensor(contexts, dtype=torch.int32, device="cuda"),
        torch.tensor(starts, dtype=torch.int32, device="cuda"), max_queries=n, window=window, return_lse=True)
    _kv.check(same, same_lse, ref, f"tokens {n} window {window}")


@pytest.mark.parametrize("counts,contexts", [([40, 64, 50], [2600, 5000, 900]), ([4, 8, 2], [2600, 9000, 900])])
def test_graphs_on_other_contents(counts, contexts):
    """A captured launch with its parts and join, replayed on other queries, codes, lengths and masks."""
    heads, groups, dim, page = 2, 4, 64, 16
    most, top = max(counts), max(contexts)
    state = batch(contexts, counts, heads, groups, dim, page, torch.bfloat16, 61, tail=0)
    table, cache, starts, q, tree, positions = state
    wsp, nbytes = nv.kv_tree_attention_workspace(cache, len(q), heads * groups, 3, most, top, 2000)
    assert nbytes > 0
    lens = torch.tensor(contexts, dtype=torch.int32, device="cuda")
    starts_d = torch.tensor(starts, dtype=torch.int32, device="cuda")
    table_d, tree_d, positions_d = table.cuda(), tree.cuda(), positions.cuda()
    out, lse = torch.empty_like(q), None

    def step(**more):
        return nv.nvfp4_kv_tree_attention(q, cache, table_d, lens, starts_d, tree_d, max_queries=most, max_context=top,
                                          positions=positions_d, window=2000, return_lse=True, **more)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out=out, workspace=wsp)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            _, lse = step(out=out, workspace=wsp)
    gen = torch.Generator().manual_seed(8)
    for i in range(4):
        now = [int(torch.randint(n, c + 1, (1,), generator=gen)) for n, c in zip(counts, contexts)]
        q.copy_(torch.randn(q.shape, generator=gen))
        for name in ("k_codes", "v_codes"):
            codes = getattr(cache, name)
            codes.copy_(torch.randint(0, 256, codes.shape, dtype=torch.uint8, generator=gen))
        tree, depths = nv.kv_trees(random_trees(counts, 70 + i))
        base = torch.repeat_interleave(torch.tensor(now) - torch.tensor(counts), torch.tensor(counts))
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        tree_d.copy_(tree)
        positions_d.copy_((base + depths).int())
        out.fill_(float("nan"))
        wsp.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        eager, eager_lse = step()
        assert torch.equal(out, eager) and torch.equal(lse, eager_lse), i
        ref = reference(q, cache, table, now, starts, dim ** -0.5, tree, (base + depths).int(), 2000)
        _kv.check(out, lse, ref, f"replay {i}")
