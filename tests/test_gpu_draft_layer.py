"""The norm, the rotation, the attention over trees and the expert layer in one step, as a layer that checks
drafted tokens runs them (examples/draft_tree_layer.py).

Each operator's output is held against 64 bits over what the step handed it, with the bounds derived beside
each operator's own tests: the norm's values and the rotation's are equal to the bit, the attention and the
expert layer lie within their rounding.  A captured step gives on every replay what an eager one gives, to the bit."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
import _kv
import test_gpu_kv_rotate as rotate
import test_gpu_kv_tree as trees
import test_gpu_moe as experts
import test_gpu_mx_norm as norms
from _parity import O, assert_bytes_equal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_tree_layer.py")
    spec = importlib.util.spec_from_file_location("draft_tree_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def held(m, layer):
    """The experts' weights as the expert layer's reference takes them."""
    w = experts.Weights.__new__(experts.Weights)
    w.e, w.k, w.f = m.EXPERTS, m.HIDDEN, m.INNER
    w.up, w.down = (tuple(t.cpu() for t in part) for part in (layer.gate_up, layer.down))
    return w


def inputs(m, n, seed):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(n, m.HIDDEN, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]


SETTLED, COUNTS = [37, 0, 150, 16], [9, 5, 1, 16]


def layer_of(m, seed):
    """A layer whose cache holds SETTLED tokens of each sequence, and its pages."""
    per_seq = -(-(max(SETTLED) + max(COUNTS)) // m.PAGE)
    gen = torch.Generator().manual_seed(seed)
    pages = torch.randperm(len(SETTLED) * per_seq, generator=gen).to(torch.int32).view(len(SETTLED), per_seq)
    layer = m.Layer(pages.numel())
    kv = torch.randn(sum(SETTLED), 2 * m.HEADS, m.DIM, generator=gen).to(torch.bfloat16).cuda()
    slots = torch.cat([pages[b, torch.arange(n) // m.PAGE].long() * m.PAGE + torch.arange(n) % m.PAGE
                       for b, n in enumerate(SETTLED)])
    nv.nvfp4_kv_write(layer.cache, kv[:, :m.HEADS], kv[:, m.HEADS:], slots.cuda())
    return layer, pages


def test_step(example):
    m = example
    layer, pages = layer_of(m, 3)
    parents = trees.random_trees(COUNTS, 4)
    plan = m.batch(pages, SETTLED, parents)
    x, residual = inputs(m, sum(COUNTS), 5)
    got = layer(x, residual, **plan)
    torch.cuda.synchronize()

    # both norms: sums and values to the bit
    for name, source, res, weight in (("n1", x, residual, layer.norms[0]), ("n2", got["projected"], got["n1"].sum, layer.norms[1])):
        h, y = norms.reference(source.cpu(), res.cpu(), weight.cpu(), 1e-6)
        assert torch.equal(got[name].sum.cpu(), h), name
        if got[name].normed is not None:
            assert torch.equal(got[name].normed.cpu(), torch.from_numpy(y).to(torch.bfloat16)), name
        else:
            want = nv.nvfp4_mx_pack(*(torch.from_numpy(t).cuda() for t in O.mx_quantize(y, "mxfp8")), "mxfp8")
            assert torch.equal(got[name].quantized.codes, want.codes) and torch.equal(got[name].quantized.scales, want.scales)

    # the rotation: queries to the bit, and the codes in their slots
    row = layer.table.cpu().numpy()[plan["positions"].cpu().numpy()]
    qkv = got["qkv"].float().cpu().numpy()
    nq = m.QUERY_HEADS
    assert torch.equal(got["rotated"].cpu(), torch.from_numpy(rotate.rotated(qkv[:, :nq], row, m.DIM, False)).to(torch.bfloat16))
    at = plan["slots"].cpu()
    for n, y in (("k", rotate.rotated(qkv[:, nq:nq + m.HEADS], row, m.DIM, False)), ("v", qkv[:, nq + m.HEADS:])):
        want = O.quantize(np.ascontiguousarray(y).reshape(-1, m.DIM), 16.0)
        for part, w in zip(("codes", "scales"), want):
            t = getattr(layer.cache, f"{n}_{part}").cpu()[at // m.PAGE, :, at % m.PAGE]
            assert_bytes_equal(t.numpy().reshape(w.shape), w, f"{n}_{part}")

    # the attention over what the cache holds now
    lens = [s + n for s, n in zip(SETTLED, COUNTS)]
    ref = trees.reference(got["rotated"], layer.cache, pages, lens, plan["starts"].tolist(), m.DIM ** -0.5, plan["tree"].cpu(),
                          plan["positions"].cpu(), 0)
    _kv.check(got["attention"], got["lse"], ref, "attention")

    # the experts
    n2 = got["n2"].normed.cpu()
    index, p = experts.choose(n2, layer.router.cpu(), m.TOP_K, True)
    assert torch.equal(got["chosen"].cpu().long(), index)
    assert ((got["weights"].cpu().double() - p).abs() <= 2.0 ** -23 * p).all()
    experts.check(got["out"], experts.reference(n2, held(m, layer), index, p), "experts")


def test_captured_step(example):
    """Two layers' steps, one after the other on the same tokens, captured; every replay is given other tokens."""
    m = example
    layer, pages = layer_of(m, 7)
    other, _ = layer_of(m, 7)
    plan = m.batch(pages, SETTLED, trees.random_trees(COUNTS, 8))
    x, residual = inputs(m, sum(COUNTS), 9)

    def both():
        one = layer(x, residual, **plan)
        two = other(one["out"], one["n2"].sum, **plan)
        return [one["out"], two["out"], two["n2"].sum, two["attention"], two["chosen"], two["weights"], layer.cache.k_codes,
                other.cache.v_codes]

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        both()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    for seed in (11, 12, 13, 14):
        a, b = inputs(m, sum(COUNTS), seed)
        x.copy_(a)
        residual.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in kept]
        for t in kept[:6]:
            t.zero_()
        eager = both()
        torch.cuda.synchronize()
        for i, (r, e) in enumerate(zip(replayed, eager)):
            assert torch.equal(r, e), i


@pytest.mark.parametrize("prompts,drafts,steps", [((13, 1, 20), 6, 3), ((1,), 1, 2), ((30, 2), 20, 2)])
def test_example(example, prompts, drafts, steps):
    lengths, out = example.run(prompts, drafts, steps)
    assert len(lengths) == len(prompts) and torch.isfinite(out).all()
