"""The expert layer (nvfp4_moe) against 64 bits on the CPU.

The choice of experts is that of float64 logits, whose order no other float64
sum can change unless two lie within 2^-45 of their terms' sizes of each other
(asserted not to happen): indices must be equal.  Bounds (u: the output type's
unit roundoff, K and F the inner sizes):
    weights   float64 arithmetic rounded once: 2^-23 of the value
    x         as float16 pieces times a power of two that brings the row's largest
              X to 2^13 .. 2^14: below the smallest normal number a step is
              2^-24, so at most 2^-25 2^-13 X = 2^-38 X is lost; bfloat16's 8 bits
              fit the 11, float16 is used as it lies, and float32's two pieces
              leave 2^-11 2^-11 / 2 of a value: dx = 2^-38 X, 0, 2^-23 |x| + 2^-38 X
    g, u      float32 sums of exact products, in any order, and one factor:
              e_g = (K + 8) 2^-24 (|x| . |w|) + dx . |w|
    h         = g s(g) u, s the logistic: |dh| <= 1.1 |u| e_g + |g s(g)| e_u (the
              slope of g s(g) is below 1.1) + 2^-20 |h| (exponential, division,
              products) + its pieces, H the pair's largest: 2^-11 |h| + 2^-38 H
              (bfloat16: one), 2^-22 |h| + 2^-38 H (two)
    out       sum_j p_j (|W_d| . dh + (F + 8) 2^-24 |W_d| . |h|) + 2^-22 of
              sum_j p_j |W_d| . |h|, and u |out| for the last rounding."""
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


class Weights:
    def __init__(self, e, k, f, seed, with_global=True):
        gen = torch.Generator().manual_seed(seed)

        def held(n, inner):
            codes = torch.randint(0, 256, (e, n, inner // 2), dtype=torch.uint8, generator=gen)
            scales = torch.randint(0x30, 0x58, (e, n, inner // 16), dtype=torch.uint8, generator=gen)
            return codes, scales, (0.5 + torch.rand(e, generator=gen)) * 4 if with_global else None

        self.e, self.k, self.f = e, k, f
        self.up, self.down = held(2 * f, k), held(k, f)
        if not with_global:  # scales small enough for ordinary sums
            self.up[1].sub_(0x28)
            self.down[1].sub_(0x28)

    def args(self):
        u, d = self.up, self.down
        return (u[0].cuda(), u[1].cuda(), d[0].cuda(), d[1].cuda()), dict(
            global_scale_gate_up=None if u[2] is None else u[2].cuda(), global_scale_down=None if d[2] is None else d[2].cuda())

    def values(self, which, e):
        c, s, g = which
        return _kv.values(c[e], s[e], None if g is None else g[e].item())


def choose(x, router, top_k, normalize):
    """(indices, weights float64) by float64 logits."""
    logits = (x.double()[:, None, :] * router.double()[None]).sum(-1)
    value, index = torch.sort(logits, dim=-1, descending=True, stable=True)
    size = (x.double().abs() @ router.double().abs().T).max()
    gap = (value[:, :-1] - value[:, 1:])[:, :top_k]
    assert ((gap == 0) | (gap > 2.0 ** -45 * size)).all(), "undecided logits"
    p = (value - value[:, :1]).exp()
    p = p[:, :top_k] / (p[:, :top_k] if normalize else p).sum(-1, keepdim=True)
    return index[:, :top_k], p


def reference(x, w, index, p):
    """(out, bound) in float64; index -1: none."""
    dtype, u = x.dtype, _kv.UNIT[x.dtype]
    x = x.double()
    t, k = x.shape
    out, bound = torch.zeros(t, k, dtype=torch.float64), torch.zeros(t, k, dtype=torch.float64)
    for e in set(index.flatten().tolist()):
        if not 0 <= e < w.e:
            continue
        up, down = w.values(w.up, e), w.values(w.down, e)
        for i, j in (index == e).nonzero().tolist():
            both, size = up @ x[i], up.abs() @ x[i].abs()
            g, v = both[:w.f], both[w.f:]
            dx = (0.0 if dtype == torch.float16 else 2.0 ** -38 * x[i].abs().max()) + \
                (2.0 ** -23 * x[i].abs() if dtype == torch.float32 else torch.zeros(k, dtype=torch.float64))
            e_both = (k + 8) * 2.0 ** -24 * size + up.abs() @ dx
            s = torch.sigmoid(g)
            h = g * s * v
            dh = 1.1 * v.abs() * e_both[:w.f] + (g * s).abs() * e_both[w.f:] + 1.1 * e_both[:w.f] * e_both[w.f:] + \
                (2.0 ** -20 + (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22)) * h.abs() + 2.0 ** -38 * h.abs().max() + 2.0 ** -126
            out[i] += p[i, j] * (down @ h)
            sizes = down.abs() @ h.abs()
            bound[i] += p[i, j].abs() * (down.abs() @ dh + ((w.f + 8) * 2.0 ** -24 + 2.0 ** -22) * sizes)
    return out, bound + u * (out.abs() + bound) + _kv.TINY[dtype]


def check(got, ref, what):
    out, bound = ref
    off = ((got.detach().cpu().double() - out).abs() / bound.clamp(min=1e-300))
    say(f"  {what}: worst error / bound = {off.max().item():.3f}")
    assert torch.isfinite(got).all() and off.max() <= 1.0, what


def inputs(t, e, k, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(t, k, generator=gen).to(dtype), (torch.randn(e, k, generator=gen) * k ** -0.5).to(dtype)


def run(t, e, top_k, k, f, dtype, seed, normalize=True, with_global=True):
    x, router = inputs(t, e, k, dtype, seed)
    w = Weights(e, k, f, seed, with_global)
    args, more = w.args()
    out = guarded((t, k), dtype)
    out.t.fill_(float("nan"))
    _, nbytes = nv.moe_workspace(t, top_k, e, k, f, dtype, "cuda")
    wsp = guarded_workspace(nbytes)
    wsp.t.fill_(255)
    idx, p = guarded((t, top_k), torch.int32), guarded((t, top_k), torch.float32)
    got, gi, gp = nv.nvfp4_moe(x.cuda(), *args, router=router.cuda(), top_k=top_k, normalize=normalize, out=out.t,
                               expert_idx=idx.t, expert_weights=p.t, workspace=wsp.t, **more)
    torch.cuda.synchronize()
    for g, n in ((out, "out"), (wsp, "workspace"), (idx, "idx"), (p, "weights")):
        g.check(n)
    index, weight = choose(x, router, top_k, normalize)
    assert torch.equal(gi.cpu().long(), index)
    assert ((gp.cpu().double() - weight).abs() <= 2.0 ** -23 * weight).all()
    check(got, reference(x, w, index, weight), f"{dtype} {t} of {e} top {top_k} {k}x{f}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,e,top_k,k,f", [
    (1, 1, 1, 16, 16), (1, 8, 2, 128, 64), (1, 64, 8, 512, 256), (3, 5, 5, 48, 80), (7, 11, 3, 1040, 592), (16, 8, 2, 256, 272),
    (17, 8, 2, 320, 144), (32, 40, 4, 64, 32), (33, 3, 1, 272, 64), (64, 6, 2, 128, 304), (2, 300, 6, 80, 48), (5, 1024, 32, 32, 16)])
def test_values(dtype, t, e, top_k, k, f):
    say(f"moe {dtype} {t} tokens, {top_k} of {e}, {k} x {f}")
    run(t, e, top_k, k, f, dtype, 100 + t + e, normalize=(t + e) % 2 == 0, with_global=(t + f) % 3 != 0)


def test_ties_and_equal_rows():
    """Equal logits: the lower index; zeros of both signs are equal."""
    t, e, k, f = 3, 9, 32, 16
    x, router = inputs(t, e, k, torch.bfloat16, 4)
    router[3:7] = router[2]
    x[1] = 0
    x[2] = -x[2].abs()
    router[8] = 0
    w = Weights(e, k, f, 4)
    args, more = w.args()
    _, idx, p = nv.nvfp4_moe(x.cuda(), *args, router=router.cuda(), top_k=6, **more)
    index, weight = choose(x, router, 6, True)
    assert torch.equal(idx.cpu().long(), index) and idx[1].tolist() == list(range(6))
    assert ((p.cpu().double() - weight).abs() <= 2.0 ** -23 * weight).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,e,top_k,k,f", [
    (16, 2, 2, 1040, 144), (31, 3, 2, 832, 6160), (9, 2, 1, 64, 6400), (2, 4, 2, 1024, 6208), (40, 2, 1, 784, 4112),
    (64, 1, 1, 1088, 112), (13, 3, 3, 784, 32)])
def test_many_tokens_an_expert(dtype, t, e, top_k, k, f):
    """More tokens of an expert than are met at a time, by long and short rows of either product."""
    say(f"moe {dtype} {t} tokens, {top_k} of {e}, {k} x {f}")
    run(t, e, top_k, k, f, dtype, 300 + t + e, normalize=(t + e) % 2 == 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,f", [(3, 128, 64), (12, 1024, 832), (1, 192, 128)])
def test_scales_anywhere(dtype, t, k, f):
    """Scales that begin at any byte, before rows of whole 64s: as those that begin at a dword."""
    e, top_k = 4, 2
    x, router = inputs(t, e, k, dtype, 21)
    w = Weights(e, k, f, 21)
    (uc, us, dc, ds), more = w.args()

    def moved(s, by):
        room = torch.zeros(s.numel() + 8, dtype=torch.uint8, device="cuda")
        there = room[by:by + s.numel()].view(s.shape)
        there.copy_(s)
        return there

    want = nv.nvfp4_moe(x.cuda(), uc, us, dc, ds, router=router.cuda(), top_k=top_k, **more)
    index, p = choose(x, router, top_k, True)
    ref = reference(x, w, index, p)
    check(want[0], ref, "at dwords")
    for by in (1, 2, 3):
        got = nv.nvfp4_moe(x.cuda(), uc, moved(us, by), dc, moved(ds, by), router=router.cuda(), top_k=top_k, **more)
        torch.cuda.synchronize()
        check(got[0], ref, f"{by} behind")
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("dtype", DTYPES)
def test_given_experts(dtype):
    """Without a router: indices outside the experts, the same expert twice, tokens without any."""
    t, e, k, f, top_k = 20, 6, 144, 80, 4
    x, _ = inputs(t, e, k, dtype, 8)
    w = Weights(e, k, f, 8)
    args, more = w.args()
    gen = torch.Generator().manual_seed(1)
    idx = torch.randint(-2, e + 2, (t, top_k), generator=gen, dtype=torch.int32)
    idx[3] = -1
    idx[4] = 2
    idx[5] = torch.tensor([1, 5, 1, 5], dtype=torch.int32)
    idx[6] = torch.tensor([2 ** 31 - 1, -2 ** 31, e, 0], dtype=torch.int32)
    p = torch.rand(t, top_k, generator=gen) - 0.3
    out, i, q = nv.nvfp4_moe(x.cuda(), *args, expert_idx=idx.cuda(), expert_weights=p.cuda(), **more)
    assert torch.equal(i.cpu(), idx) and torch.equal(q.cpu(), p) and not out[3].any()
    check(out, reference(x, w, idx.long(), p.double()), f"given {dtype}")
    idx.fill_(-1)
    assert not nv.nvfp4_moe(x.cuda(), *args, expert_idx=idx.cuda(), expert_weights=p.cuda(), **more)[0].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_not_numbers_stay_with_their_token(dtype):
    """A NaN or an infinity in a token, or in an expert's weights, reaches the tokens it belongs to alone."""
    t, e, k, f = 18, 5, 96, 48
    x, router = inputs(t, e, k, dtype, 12)
    w = Weights(e, k, f, 12)
    args, more = w.args()
    call = lambda x, a=args: nv.nvfp4_moe(x.cuda(), *a, router=router.cuda(), top_k=2, **more)  # noqa: E731
    want, idx, p = call(x)
    for value in (float("nan"), float("inf"), float("-inf")):
        y = x.clone()
        y[7, 30] = value
        got, i, q = call(y)
        rest = torch.arange(t) != 7
        assert torch.equal(got[rest], want[rest]) and torch.equal(i[rest], idx[rest]) and torch.equal(q[rest], p[rest])
        assert not torch.isfinite(got[7]).any()
        assert (i[7] >= 0).all() and (i[7] < e).all() and i[7, 0] != i[7, 1]
    for part in (1, 3):  # scales of gate/up rows, of down rows
        scales = args[part].clone()
        scales[2, 5, 1] = 127
        got, i, _ = call(x, args[:part] + (scales,) + args[part + 1:])
        hit = (idx == 2).any(-1)
        assert torch.equal(i, idx) and torch.equal(got[~hit], want[~hit])
        if part == 3:
            assert got[hit][:, 5].isnan().all() and torch.isfinite(got[hit][:, :5]).all()
        else:
            assert got[hit].isnan().all()
    # exponents at their ends: gates so negative that exp(-g) is infinite give 0, not NaN
    big = torch.full((1, k), 3e4).to(dtype)
    got, _, _ = call(torch.cat([big, -big]))
    assert torch.isfinite(got).all() or dtype == torch.float16


def test_offsets_past_32_bits():
    """Weights whose codes pass 4 GiB: the last expert's."""
    e, k, f, t = 1024, 4096, 1040, 2
    up_codes = torch.zeros(e, 2 * f, k // 2, dtype=torch.uint8, device="cuda")
    up_scales = torch.zeros(e, 2 * f, k // 16, dtype=torch.uint8, device="cuda")
    down_codes = torch.zeros(e, k, f // 2, dtype=torch.uint8, device="cuda")
    down_scales = torch.zeros(e, k, f // 16, dtype=torch.uint8, device="cuda")
    assert up_codes.numel() > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(3)
    for c, s in ((up_codes, up_scales), (down_codes, down_scales)):
        c[-1] = torch.randint(0, 256, c.shape[1:], dtype=torch.uint8, device="cuda", generator=gen)
        s[-1] = torch.randint(0x08, 0x30, s.shape[1:], dtype=torch.uint8, device="cuda", generator=gen)
    x, _ = inputs(t, 1, k, torch.bfloat16, 5)
    p = torch.ones(t, 1, device="cuda")
    at = torch.full((t, 1), e - 1, dtype=torch.int32, device="cuda")
    got = nv.nvfp4_moe(x.cuda(), up_codes, up_scales, down_codes, down_scales, expert_idx=at, expert_weights=p)[0]
    alone = nv.nvfp4_moe(x.cuda(), up_codes[-1:].contiguous(), up_scales[-1:].contiguous(), down_codes[-1:].contiguous(),
                         down_scales[-1:].contiguous(), expert_idx=at * 0, expert_weights=p)[0]
    assert torch.equal(got, alone) and got.any()


def test_repeats_streams_graphs():
    """The same bits in every call; on another stream; captured, replayed between eager calls on other inputs."""
    t, e, k, f = 9, 16, 512, 256
    x, router = inputs(t, e, k, torch.bfloat16, 21)
    w = Weights(e, k, f, 21)
    args, more = w.args()
    xd, rd = x.cuda(), router.cuda()
    want = nv.nvfp4_moe(xd, *args, router=rd, top_k=4, **more)
    for _ in range(5):
        again = nv.nvfp4_moe(xd, *args, router=rd, top_k=4, **more)
        assert all(torch.equal(a, b) for a, b in zip(again, want))
    assert nv.nvfp4_moe(xd[:0], *args, router=rd, top_k=4, **more)[0].shape == (0, k)
    out, wsp = torch.empty_like(xd), nv.moe_workspace(t, 4, e, k, f, torch.bfloat16, "cuda")[0]
    idx, p = torch.empty_like(want[1]), torch.empty_like(want[2])

    def call():
        nv.nvfp4_moe(xd, *args, router=rd, top_k=4, out=out, workspace=wsp, expert_idx=idx, expert_weights=p, **more)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        assert torch.equal(out, want[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    for i in range(4):
        xd.copy_(inputs(t, e, k, torch.bfloat16, 30 + i)[0])
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        eager = nv.nvfp4_moe(xd, *args, router=rd, top_k=4, **more)
        assert torch.equal(out, eager[0]) and torch.equal(idx, eager[1]) and torch.equal(p, eager[2]), i


def test_two_streams_at_once():
    """Calls on two streams at the same time, each with its own workspace."""
    t, e, k, f = 4, 8, 1024, 512
    w = Weights(e, k, f, 31)
    args, more = w.args()
    xs = [inputs(t, e, k, torch.bfloat16, s)[0].cuda() for s in (1, 2)]
    rd = inputs(t, e, k, torch.bfloat16, 3)[1].cuda()
    want = [nv.nvfp4_moe(x, *args, router=rd, top_k=2, **more)[0] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(nv.nvfp4_moe(xs[i], *args, router=rd, top_k=2, **more)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_refusals():
    """The binding's checks that need device tensors."""
    w = Weights(4, 64, 32, 1)
    args, more = w.args()
    x, router = (v.cuda() for v in inputs(3, 4, 64, torch.bfloat16, 1))
    ok = dict(router=router, top_k=2)
    nv.nvfp4_moe(x, *args, **ok, **more)
    bad = [dict(ok, router=router.float()), dict(ok, router=router[:3]), dict(top_k=2), dict(ok, top_k=None),
           dict(ok, expert_idx=torch.zeros(3, 2, dtype=torch.int64, device="cuda")), dict(ok, top_k=5), dict(ok, top_k=0),
           dict(ok, out=torch.empty(3, 64, device="cuda")), dict(ok, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
           dict(ok, global_scale_gate_up=torch.ones(3, device="cuda"))]
    for b in bad:
        with pytest.raises(ValueError):
            nv.nvfp4_moe(x, *args, **{**more, **b})
    with pytest.raises(ValueError):
        nv.nvfp4_moe(x[:, :48].contiguous(), *args, **ok, **more)
    with pytest.raises(ValueError):
        nv.nvfp4_moe(x, args[0][:, :-2].contiguous(), *args[1:], **ok, **more)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_moe(torch.zeros(65, 64, dtype=torch.bfloat16, device="cuda"), *args, **ok, **more)
