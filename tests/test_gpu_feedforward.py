"""The feed-forward operators together, on streams of the caller's, captured
into graphs, and past 31 bits of bytes and elements."""
import pytest

import feedforward_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_experts import make as make_experts  # noqa: E402
from test_gpu_kv_streams import busy_then  # noqa: E402
from test_gpu_linear import handle, make as make_linear  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


class Layer:
    """Norms around a block, routing, experts and a product, with random weights."""

    def __init__(self, tokens, hidden, inner, experts, k, out, layout):
        g = torch.Generator().manual_seed(tokens + hidden)
        rnd = lambda *s: torch.randn(*s, generator=g)
        self.x, self.block = rnd(2, tokens, hidden).bfloat16().unbind(0)
        self.w, self.bw, self.gate = (1 + 0.2 * rnd(3, hidden)).bfloat16().unbind(0)
        self.router = rnd(hidden, experts) * hidden ** -0.5
        self.bias = 0.1 * rnd(experts)
        self.parts = [R.weight_bytes(g, (experts,), 2 * inner, hidden, layout),
                      R.weight_bytes(g, (experts,), hidden, inner, layout),
                      R.weight_bytes(g, (), out, hidden, layout)]
        self.case = dict(top_k=k, scores="sigmoid", groups=1, top_groups=1, group_top=1,
                         renormalize=True, scale=1.5)
        self.values = [R.values(p, layout) for p in self.parts]
        self.gu, self.dn, self.lin = map(handle, self.parts)
        for n in ("x", "block", "w", "bw", "gate", "router", "bias"):
            setattr(self, n + "_d", getattr(self, n).cuda())

    def run(self):
        """Every operator's results, with nothing between the launches."""
        y, z = fp4.residual_norm(self.x_d, self.block_d, self.w_d, self.bw_d, self.gate_d, 0.5)
        logits = z.float() @ self.router_d
        weights, ids = fp4.expert_route(logits, self.case["top_k"], "sigmoid", self.bias_d, scale=1.5)
        o = fp4.fp4_experts(self.gu, self.dn, z, weights, ids)
        y2, z2 = fp4.residual_norm(y, o, self.w_d)
        return y, z, logits, weights, ids, o, y2, z2, fp4.fp4_linear(self.lin, z2, dtype=F32)

    def check(self, got):
        """Each operator's results against 64 bits of what it was given."""
        y, z, logits, weights, ids, o, y2, z2, last = (t.cpu() for t in got)
        d = lambda t: t.double()
        # as in the norms' and the routing's own tests: runs of fp32 steps
        c = (self.x.shape[1] / 64 + 40) * R.U
        for (a, b), (p, q), args in (((y, z), (self.x, self.block), (self.bw, self.gate, 0.5)),
                                     ((y2, z2), (y, o), (None, None, 1.0))):
            bw, gate, scale = args
            wy, wz = R.residual(d(p), d(q), d(self.w), None if bw is None else d(bw),
                                None if gate is None else d(gate), scale, 1e-6)
            ey = c * ((scale * d(p)).abs() + (wy - scale * d(p)).abs())
            r = 1 / torch.sqrt(wy.square().mean(-1, keepdim=True) + 1e-6)
            ez = d(self.w).abs() * r * (ey + wy.abs() * r * ey.square().mean(-1, keepdim=True).sqrt())
            R.close(a, wy, ey)
            R.close(b, wz, ez + c * wz.abs())
        rw, re = R.route(self.case, logits, d(self.bias).tolist())
        assert torch.equal(ids, re)
        room = (2 * logits.shape[1] / 64 + 24 + 4 * float(logits.abs().max())) * R.U
        assert ((d(weights) - rw).abs() <= room * rw).all()
        R.close(o, *R.experts(z, self.values[0], self.values[1], weights, ids))
        R.close(last, *R.linear(z2, self.values[2]))


SIZES = [(1, 128, 64, 16, 4, 256, "tensor"), (7, 256, 128, 32, 4, 512, "mx"),
         (33, 288, 96, 20, 3, 1000, "rows"), (150, 256, 160, 6, 2, 8208, "tiles"),
         (700, 512, 96, 8, 2, 304, "mx")]


@pytest.mark.parametrize("size", SIZES)
def test_together(size):
    m = Layer(*size)
    m.check(m.run())


@pytest.mark.parametrize("size", SIZES)
def test_together_captured(size):
    """One graph of all of them, replayed on other inputs, with eager work between."""
    m = Layer(*size)
    m.run()                                     # nothing is loaded first inside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = m.run()
    for i in range(4):
        m.x_d.copy_(m.x * (1 + i))
        m.block_d.copy_(m.block.flip(0) if i % 2 else m.block)
        want = [t.clone() for t in m.run()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(held, want)), i


def test_two_graphs():
    """Two captured graphs of one set of weights, replayed on two streams at once."""
    m = Layer(40, 256, 128, 16, 4, 512, "tensor")
    want = [t.clone() for t in m.run()]
    torch.cuda.synchronize()
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            held.append(m.run())
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, sides):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for h in held:
        assert all(same(a, b) for a, b in zip(h, want))


def test_gradients_captured():
    """Forward and backward of fresh leaves in one captured graph."""
    g = torch.Generator().manual_seed(4)
    logits = torch.randn(60, 48, generator=g).cuda()
    x, b, dy, dz = torch.randn(4, 60, 512, generator=g).bfloat16().cuda().unbind(0)
    w, bw, gate = (1 + 0.1 * torch.randn(3, 512, generator=g)).bfloat16().cuda().unbind(0)
    dw = torch.randn(60, 5, generator=g).cuda()

    def back(leaves):
        weights, _ = fp4.expert_route(leaves[0], 5)
        y, z = fp4.residual_norm(*leaves[1:], scale=0.5)
        return torch.autograd.grad((weights, y, z), leaves, (dw, dy, dz))

    plain = [logits, x, b, w, bw, gate]
    back([v.clone().requires_grad_() for v in plain])
    leaves = [v.clone().requires_grad_() for v in plain]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = back(leaves)
    for i in range(3):
        with torch.no_grad():
            for leaf, v in zip(leaves, plain):
                leaf.copy_(v * (1 + i))
        ids = fp4.expert_route(leaves[0].detach(), 5)[1]
        now = [v.detach() for v in leaves]
        want = [fp4.expert_route_backward(dw, now[0], ids)]
        want += [t.bfloat16() for t in fp4.residual_norm_backward(dy, dz, *now[1:], scale=0.5)]
        want[3], want[4] = want[4], want[3]          # dweight before dblock_weight
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(held, want)), i


@pytest.mark.parametrize("tokens", [1, 30, 700])
def test_streams(tokens):
    """Calls on a stream of the caller's while the current one is busy."""
    gu, dn, x, w, ids = (v if isinstance(v, dict) else v.cuda()
                         for v in make_experts(3, tokens, 12, 3, 256, 128))
    gu, dn = handle(gu), handle(dn)
    b = x.flip(0).contiguous()
    nw = torch.ones(256, dtype=BF, device="cuda")
    logits = x.float()[:, :40].contiguous()
    busy_then(lambda s: [fp4.fp4_experts(gu, dn, x, w, ids, stream=s)])
    busy_then(lambda s: fp4.expert_route(logits, 6, stream=s))
    busy_then(lambda s: fp4.residual_norm(x, b, nw, stream=s))
    busy_then(lambda s: fp4.residual_norm_backward(b, x, x, b, nw, nw, nw, stream=s))
    dw, e = fp4.expert_route(logits, 6)
    busy_then(lambda s: [fp4.expert_route_backward(dw, logits, e, stream=s)])
    lw, lx = make_linear(4, tokens, 528, 288, "mx")
    lw, lx = handle(lw), lx.cuda()
    busy_then(lambda s: [fp4.fp4_linear(lw, lx, stream=s)])


@pytest.mark.parametrize("tokens", [1, 3, 16, 40, 700])
@pytest.mark.parametrize("hidden,inner", [(128, 256), (96, 32)])
def test_experts_named_twice(tokens, hidden, inner):
    """An expert in several places of a token, with and without streams of codes."""
    gu, dn, x, w, ids = make_experts(tokens, tokens, 9, 4, hidden, inner)
    ids[:] = 5
    ids[::2, 1] = 2
    ids[1::3, 2] = -1
    ids[0, 3] = 9
    want, err = R.experts(x, R.values(gu, "tensor"), R.values(dn, "tensor"), w, ids)
    R.close(fp4.fp4_experts(handle(gu), handle(dn), x.cuda(), w.cuda(), ids.cuda()), want, err)


def test_experts_over_a_long_batch():
    """More hidden values than 2^31 bytes: slices of tokens, as each alone."""
    tokens, k = 33100, 8
    gu, dn, x, w, _ = make_experts(1, tokens, 16, k, 32, 4096)
    ids = torch.randint(-1, 16, (tokens, k), generator=torch.Generator().manual_seed(1)).int()
    a = (handle(gu), handle(dn))
    got = fp4.fp4_experts(*a, x.cuda(), w.cuda(), ids.cuda())
    some = torch.cat([torch.arange(20), torch.arange(32750, 32790), torch.arange(33080, 33100)])
    want, err = R.experts(x[some], R.values(gu, "tensor"), R.values(dn, "tensor"), w[some], ids[some])
    R.close(got[some.cuda()], want, err)


@pytest.mark.parametrize("tokens", [20, 150, 300])
def test_rows_far_apart(tokens):
    """x and outputs of more than 2^31 elements from the first row to the last."""
    stride = (1 << 23) - 8
    big = torch.empty(tokens * stride, dtype=BF, device="cuda")
    wide = big.as_strided((tokens, 96), (stride, 1))
    away = big.as_strided((tokens, 528), (stride, 1), 4096)
    gu, dn, x, w, ids = make_experts(2, tokens, 4, 2, 96, 64)
    wide.copy_(x)
    want, err = R.experts(x, R.values(gu, "tensor"), R.values(dn, "tensor"), w, ids)
    out = away[:, :96]
    fp4.fp4_experts(handle(gu), handle(dn), wide, w.cuda(), ids.cuda(), out=out)
    R.close(out, want, err)
    lw, _ = make_linear(2, 1, 528, 96, "rows")
    want, err = R.linear(x, R.values(lw, "rows"))
    fp4.fp4_linear(handle(lw), wide, out=away)
    R.close(away, want, err)
    nw = torch.ones(96, dtype=BF, device="cuda")
    y, z = away[:, :96], away[:, 104:200]
    fp4.residual_norm(wide, wide, nw, out=(y, z))
    for a, b in zip((y, z), fp4.residual_norm(x.cuda(), x.cuda(), nw)):
        assert same(a, b)
    far = big.as_strided((tokens, 40), (stride, 1))
    far.normal_()
    for a, b in zip(fp4.expert_route(far, 4), fp4.expert_route(far.contiguous(), 4)):
        assert same(a, b)


@pytest.mark.parametrize("tokens", [1, 5, 40, 200])
def test_codes_past_31_bits(tokens):
    """A matrix of more than 2^31 bytes of codes: its first rows, some in between, its last."""
    rows, cols = (1 << 20) + 75, 4160
    g = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.randint(8, 0x70, (rows, cols // 16), generator=g, dtype=torch.uint8, device="cuda")
    alpha = torch.rand(rows, generator=g, device="cuda")
    x = torch.randn(tokens, cols, generator=g, device="cuda").bfloat16()
    got = fp4.fp4_linear(fp4.Fp4Weights(codes, scales, alpha), x)
    for first in (0, (1 << 19) - 7, rows - 90):
        part = slice(first, first + 90)
        v = R.values(dict(codes=codes[part].cpu(), scales=scales[part].cpu(), alpha=alpha[part].cpu()),
                     "rows")
        R.close(got[:, part], *R.linear(x.cpu(), v))


@pytest.mark.parametrize("tokens", [1, 3, 40, 400, 4000])
def test_experts_past_31_bits(tokens):
    """The first and the last of experts of more than 2^31 bytes of codes."""
    e, hidden, inner = 140, 8192, 2048
    g = torch.Generator(device="cuda").manual_seed(6)
    part = lambda *s: dict(
        codes=torch.randint(0, 256, (e, s[0], s[1] // 2), generator=g, dtype=torch.uint8, device="cuda"),
        scales=torch.randint(115, 122, (e, s[0], s[1] // 32), generator=g, dtype=torch.uint8, device="cuda"),
        alpha=None)
    gu, dn = part(2 * inner, hidden), part(hidden, inner)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    ids = torch.tensor([[0, e - 1]] * tokens, dtype=torch.int32, device="cuda")
    w = torch.rand(tokens, 2, generator=g, device="cuda")
    got = fp4.fp4_experts(*(fp4.Fp4Weights(fmt=fp4.FORMAT_MXFP4, **p) for p in (gu, dn)), x, w, ids)
    ends = [R.values({k: None if v is None else v[[0, e - 1]].cpu() for k, v in p.items()}, "mx")
            for p in (gu, dn)]
    some = sorted({0, tokens // 2, tokens - 1})
    want, err = R.experts(x[some].cpu(), *ends, w[some].cpu(), ids[some].cpu().clamp(max=1))
    R.close(got[some], want, err)


@pytest.mark.parametrize("tokens,experts,k", [(5, 17, 16), (9, 64, 17), (3, 256, 64), (20, 1000, 15),
                                              (7, 1024, 64), (300, 128, 16)])
def test_many_choices(tokens, experts, k):
    case = dict(top_k=k, scores="softmax", groups=1, top_groups=1, group_top=1, renormalize=False, scale=2.0)
    logits = 3 * torch.randn(tokens, experts, generator=torch.Generator().manual_seed(k))
    w, e = fp4.expert_route(logits.cuda(), k, renormalize=False, scale=2.0)
    rw, re = R.route(case, logits, None)
    assert torch.equal(e.cpu(), re)
    room = (2 * experts / 64 + 24 + 4 * float(logits.abs().max())) * R.U
    assert ((w.double().cpu() - rw).abs() <= room * rw + 1e-37).all()
