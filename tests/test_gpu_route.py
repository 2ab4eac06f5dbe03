"""expert_route and its gradient against 64 bits: every kind of score, groups,
ties, masked tokens, sizes around a wave's width."""
import math

import pytest

import feedforward_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402


def case(top_k, scores="softmax", groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0):
    return dict(top_k=top_k, scores=scores, groups=groups, top_groups=top_groups,
                group_top=group_top, renormalize=renormalize, scale=scale)


def check(c, logits, bias=None, stride=None):
    x = logits.cuda()
    if stride:
        wide = torch.zeros(logits.shape[0], stride, dtype=logits.dtype, device="cuda")
        wide[:, :logits.shape[1]] = x
        x = wide[:, :logits.shape[1]]
    w, e = fp4.expert_route(x, bias=None if bias is None else bias.cuda(), **c)
    want_w, want_e = R.route(c, logits, None if bias is None else bias.double().tolist())
    assert torch.equal(e.cpu(), want_e)
    # a score is off by exp (2 u and u |x - m|), the sum, a division and two products
    n = logits.shape[1]
    finite = torch.where(logits.double().abs() < 1e3, logits.double().abs(), 0.0)
    room = (2 * n / 64 + 24 + 4 * float(finite.max())) * R.U
    assert ((w.double().cpu() - want_w).abs() <= room * want_w + 1e-37).all()
    return w, e


SIZES = [(1, 1, 1), (3, 5, 2), (9, 8, 8), (33, 60, 4), (7, 64, 6), (12, 65, 3), (6, 128, 8),
         (10, 200, 8), (5, 256, 8), (4, 300, 20), (3, 512, 64), (3, 1000, 10), (2, 1024, 1)]


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("tokens,experts,k", SIZES)
def test_choice(scores, with_bias, tokens, experts, k):
    g = torch.Generator().manual_seed(tokens + experts + k)
    logits = torch.randn(tokens, experts, generator=g)
    bias = 0.1 * torch.randn(experts, generator=g) if with_bias else None
    check(case(k, scores), logits, bias)
    check(case(k, scores, renormalize=False, scale=2.5), logits.bfloat16(), bias, experts + 3)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("experts,groups,top_groups,k", [
    (8, 8, 3, 3), (24, 4, 2, 5), (60, 3, 1, 4), (64, 8, 4, 8), (100, 10, 7, 8), (256, 8, 4, 8),
    (320, 64, 5, 12), (512, 2, 1, 7)])
def test_groups(scores, group_top, with_bias, experts, groups, top_groups, k):
    g = torch.Generator().manual_seed(experts + groups + top_groups)
    logits = torch.randn(13, experts, generator=g)
    logits[3, :experts // 2] = -math.inf
    logits[4] = -math.inf
    logits[5, 1:] = -math.inf
    bias = 0.1 * torch.randn(experts, generator=g) if with_bias else None
    check(case(k, scores, groups, top_groups, group_top), logits, bias)


def test_ties_go_to_the_lower_index():
    logits = torch.zeros(6, 200)
    logits[1, ::3] = 1.0
    logits[2, 100:] = 0.5
    logits[3] = torch.arange(200) // 7
    logits[4, 64] = logits[4, 128] = logits[4, 0] = 2.0
    logits[5, 1::2] = -0.0
    for scores in ("softmax", "sigmoid"):
        check(case(9, scores), logits)
        check(case(9, scores), logits.bfloat16(), torch.zeros(200))
        check(case(9, scores, 20, 6, 1), logits)
        check(case(9, scores, 20, 6, 2), logits, torch.zeros(200))


def test_scores_next_to_each_other():
    """Sums that are equal in fp32 are told apart."""
    n = 64
    logits = torch.zeros(1, n)
    bias = torch.full((n,), 0.25)
    logits[0] = torch.linspace(-1e-7, 1e-7, n)
    check(case(8, "sigmoid"), logits, bias)
    check(case(8, "softmax"), logits, bias)


def test_masked():
    """-inf and NaN are no candidates; the type's lowest value is one."""
    low = torch.finfo(torch.float32).min
    logits = torch.full((5, 70), -math.inf)
    logits[1, 65] = 3.0
    logits[2, :3] = low
    logits[3] = low
    logits[4, 7] = low
    logits[4, 9] = 1.0
    for scores in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            for bias in (None, torch.zeros(70)):
                check(case(4, scores, renormalize=renormalize), logits, bias)
    w, e = fp4.expert_route(logits.cuda(), 4)
    assert (e[0] == -1).all() and (w[0] == 0).all() and e[1].tolist() == [65, -1, -1, -1]
    x = torch.randn(2, 64)
    x[0, 3] = math.nan
    w, e = fp4.expert_route(x.cuda(), 64, scores="sigmoid")
    assert 3 not in e[0].tolist() and sorted(e[0].tolist())[0] == -1 and w.isfinite().all()
    w, e = fp4.expert_route(x.cuda(), 4)
    assert w[0].isnan().all() and w[1].isfinite().all()
    assert len(set(e[0].tolist())) == 4 and 3 not in e[0].tolist()
    b = torch.zeros(64)
    b[11], b[12], b[13] = -math.inf, math.nan, math.inf
    w, e = fp4.expert_route(x[1:].cuda(), 64, bias=b.cuda())
    assert e[0, 0] == 13 and sorted(e[0].tolist())[:2] == [-1, -1]


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,experts,k", SIZES)
def test_gradient(scores, renormalize, dtype, tokens, experts, k):
    g = torch.Generator().manual_seed(experts * 3 + k)
    c = case(k, scores, renormalize=renormalize, scale=1.5)
    logits = torch.randn(tokens, experts, generator=g).to(dtype)
    logits[0, experts // 2] = -math.inf
    dw = torch.randn(tokens, k, generator=g)
    _, ids = fp4.expert_route(logits.cuda(), **c)
    how = dict(scores=scores, renormalize=renormalize, scale=1.5)
    got = fp4.expert_route_backward(dw.cuda(), logits.cuda(), ids, **how)
    x = logits.double().requires_grad_()
    (R.route_weights(c, x, ids.cpu()) * dw.double()).sum().backward()
    # dl is at most 2 scale s max|g|, its terms off by the scores' error and their sums
    room = (2 * experts / 64 + 4 * k + 60) * R.U * 3 * dw.double().abs().max()
    half = R.HALF[dtype] if dtype is torch.bfloat16 else 0.0
    assert ((got.double().cpu() - x.grad).abs() <= room + half * x.grad.abs()).all()


def test_gradient_against_differences():
    g = torch.Generator().manual_seed(4)
    logits, dw = torch.randn(5, 40, generator=g), torch.randn(5, 6, generator=g)
    for scores in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            c = case(6, scores, renormalize=renormalize)
            _, ids = fp4.expert_route(logits.cuda(), **c)
            got = fp4.expert_route_backward(dw.cuda(), logits.cuda(), ids, scores, renormalize)
            f = lambda x: (R.route_weights(c, x, ids.cpu()) * dw.double()).sum(1)
            x, h = logits.double(), 1e-4
            for i in range(40):
                d = torch.zeros(40, dtype=torch.float64)
                d[i] = h
                slope = (f(x + d) - f(x - d)) / (2 * h)
                assert ((got[:, i].double().cpu() - slope).abs() < 1e-5).all()


def test_gradient_of_any_experts():
    """Numbers outside the experts, the same one twice, tokens without any."""
    g = torch.Generator().manual_seed(8)
    logits, dw = torch.randn(4, 50, generator=g), torch.randn(4, 3, generator=g)
    ids = torch.tensor([[7, 7, 1], [-1, 50, 3], [-1, -1, -1], [49, 0, 49]], dtype=torch.int32)
    for scores in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            c = case(3, scores, renormalize=renormalize)
            x = logits.double().requires_grad_()
            (R.route_weights(c, x, ids) * dw.double()).sum().backward()
            got = fp4.expert_route_backward(dw.cuda(), logits.cuda(), ids.cuda(), scores, renormalize)
            assert ((got.double().cpu() - x.grad).abs() <= 200 * R.U * 3 * dw.abs().max()).all()


def test_autograd():
    g = torch.Generator().manual_seed(5)
    logits = torch.randn(20, 30, generator=g).cuda().requires_grad_()
    w, e = fp4.expert_route(logits, 4, scores="sigmoid", bias=torch.zeros(30, device="cuda"))
    assert w.requires_grad and not e.requires_grad
    dw = torch.randn(20, 4, generator=g).cuda()
    (w * dw).sum().backward()
    assert torch.equal(logits.grad, fp4.expert_route_backward(dw, logits.detach(), e, "sigmoid"))
    with pytest.raises(RuntimeError, match="out"):
        fp4.expert_route(logits, 4, out=(w.detach(), e))
    with pytest.raises(RuntimeError, match="bias"):
        fp4.expert_route(logits, 4, bias=torch.zeros(30, device="cuda", requires_grad=True))
    with torch.no_grad():
        assert not fp4.expert_route(logits, 4)[0].requires_grad


def test_empty():
    w, e = fp4.expert_route(torch.empty(0, 8, device="cuda"), 2)
    assert w.shape == (0, 2) and e.shape == (0, 2)
    d = fp4.expert_route_backward(w, torch.empty(0, 8, device="cuda"), e)
    assert d.shape == (0, 8)
