"""The norm and the rotation captured into graphs and replayed on other inputs, also where the norm's sum is written
over its input: every replay gives what an eager call on the same inputs gives, to the bit."""
import pytest
import torch

import nvfp4_block_scaled_amd as nv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


def capture(call):
    """(graph, what its call returned); the call has run once before."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = call()
    torch.cuda.synchronize()
    return graph, got


def parts(n, packed):
    return (n.quantized.codes, n.quantized.scales) if packed else n.quantized


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mode,packed", [("mxfp8", True), ("mxfp4", False)])
@pytest.mark.parametrize("rows,k", [(1, 64), (37, 1056), (70, 5120), (9, 20000)])
def test_norm(dtype, mode, packed, rows, k):
    gen = torch.Generator(device="cuda").manual_seed(k)

    def some(*shape):
        return torch.randn(*shape, device="cuda", generator=gen).to(dtype)

    x, res, w = some(rows, k), some(rows, k), some(k)
    graph, got = capture(lambda: nv.nvfp4_mx_rms_norm(x, w, mode, res, packed=packed, normed=True))
    for i in range(4):
        x.copy_(some(rows, k) * 2.0 ** i)
        res.copy_(some(rows, k))
        w.copy_(some(k))
        for t in (*parts(got, packed), got.sum, got.normed):
            t.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        want = nv.nvfp4_mx_rms_norm(x, w, mode, res, packed=packed, normed=True)
        assert torch.equal(got.sum, want.sum) and torch.equal(got.sum, x + res) and torch.equal(got.normed, want.normed), i
        assert all(torch.equal(a, b) for a, b in zip(parts(got, packed), parts(want, packed))), i


@pytest.mark.parametrize("k", [512, 8192, 20000])
@pytest.mark.parametrize("over", ["x", "residual"])
def test_norm_over_its_input(k, over):
    """The residual stream kept in one tensor: each replay adds to what the last one left."""
    gen = torch.Generator(device="cuda").manual_seed(k)
    x, res = (torch.randn(33, k, device="cuda", generator=gen).to(torch.bfloat16) for _ in range(2))
    into = x if over == "x" else res
    first = into.clone()
    graph, got = capture(lambda: nv.nvfp4_mx_rms_norm(x, None, "mxfp8", res, packed=True, sum_out=into))
    into.copy_(first)
    for i in range(4):
        a, b = x.clone(), res.clone()
        graph.replay()
        torch.cuda.synchronize()
        want = nv.nvfp4_mx_rms_norm(a, None, "mxfp8", b, packed=True)
        assert got.sum.data_ptr() == into.data_ptr() and torch.equal(into, want.sum), i
        assert all(torch.equal(c, d) for c, d in zip(parts(got, True), parts(want, True))), i


@pytest.mark.parametrize("dtype,interleaved", [(torch.bfloat16, False), (torch.float32, True)])
def test_rotation(dtype, interleaved):
    gen = torch.Generator(device="cuda").manual_seed(6)
    tokens, heads, dim, pages, page = 29, 3, 96, 7, 16
    one = torch.tensor([5.0], device="cuda")
    cache, other = (nv.kv_cache(pages, page, heads, dim, global_scale_k=one, global_scale_v=one) for _ in range(2))
    both = torch.empty(tokens, 4 * heads, dim, dtype=dtype, device="cuda")
    slots = torch.empty(tokens, dtype=torch.int64, device="cuda")
    positions = torch.empty(tokens, dtype=torch.int32, device="cuda")
    table = nv.rotation_table(500, 64)

    def call(cache):
        return nv.nvfp4_kv_write_rotated(cache, both[:, 2 * heads:3 * heads], both[:, 3 * heads:], slots, positions, table,
                                         q=both[:, :2 * heads], interleaved=interleaved)

    def fill():
        both.copy_(torch.randn(both.shape, device="cuda", generator=gen))
        slots.copy_(torch.randperm(pages * page, device="cuda", generator=gen)[:tokens])
        slots[3] = -1
        positions.copy_(torch.randint(-3, 503, (tokens,), device="cuda", generator=gen))

    fill()
    graph, q = capture(lambda: call(cache))
    for c in (cache, other):
        for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
            getattr(c, name).zero_()
    for i in range(4):
        fill()
        q.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = call(other)
        assert torch.equal(q, want), i
        for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert torch.equal(getattr(cache, name), getattr(other, name)), (i, name)
