"""Renormalized routing weights and their gradient where the chosen scores lie
below the range of fp32: the weights are quotients of them, which do not."""
import math

import pytest

import feedforward_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_route import case, check  # noqa: E402

# (tokens, experts, k): 16 lanes a token, a wave a token, the long way (too many choices)
SIZES = [(9, 8, 8), (33, 60, 4), (5, 256, 8), (4, 300, 20), (3, 90, 64), (2, 1024, 3)]


def backward(c, logits, ids):
    """expert_route_backward against autograd in 64 bits."""
    dw = torch.randn(ids.shape, generator=torch.Generator().manual_seed(3))
    how = dict(scores=c["scores"], renormalize=True, scale=c["scale"])
    got = fp4.expert_route_backward(dw.cuda(), logits.cuda(), ids, **how)
    x = logits.double().requires_grad_()
    (R.route_weights(c, x, ids.cpu()) * dw.double()).sum().backward()
    k, experts = ids.shape[1], logits.shape[1]
    # as in the gradient's own tests; |l| in expf's argument is the distance to the largest chosen
    room = (2 * experts / 64 + 4 * k + 60 + 40) * R.U * 3 * c["scale"] * dw.double().abs().max()
    half = R.HALF[logits.dtype] if logits.dtype is torch.bfloat16 else 0.0
    assert ((got.double().cpu() - x.grad).abs() <= room + half * x.grad.abs()).all()
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("middle", [-80.0, -88.0, -100.0, -300.0, -600.0])
@pytest.mark.parametrize("tokens,experts,k", SIZES)
def test_sigmoid(dtype, with_bias, middle, tokens, experts, k):
    g = torch.Generator().manual_seed(experts + k)
    logits = (middle + 3 * torch.randn(tokens, experts, generator=g)).to(dtype)
    logits[0, experts // 2] = -math.inf
    logits[1, 1] = logits[1, 0]                    # a tie
    bias = 0.1 * torch.randn(experts, generator=g) if with_bias else None
    c = case(k, "sigmoid", scale=2.5)
    w, e = check(c, logits, bias)
    assert float(w.sum(1).min()) > 2.4
    backward(c, logits, e)


@pytest.mark.parametrize("far", [90.0, 104.0, 300.0, 600.0])
@pytest.mark.parametrize("tokens,experts,k", SIZES[1:])
def test_softmax_of_chosen_by_bias(far, tokens, experts, k):
    """The bias picks experts far below the largest logit."""
    g = torch.Generator().manual_seed(experts + k)
    logits = torch.randn(tokens, experts, generator=g)
    bias = torch.zeros(experts)
    low = torch.randperm(experts, generator=g)[:min(k + 3, experts - 1)]
    logits[:, low] -= far
    bias[low] = 2.0 + 0.1 * torch.randn(len(low), generator=g)
    c = case(k, scale=2.5)
    w, e = check(c, logits, bias)
    assert float(w.sum(1).min()) > 2.4
    backward(c, logits, e)


@pytest.mark.parametrize("experts,k,groups", [(64, 4, 8), (60, 5, 3), (300, 20, 3), (66, 3, 11)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_groups(scores, experts, k, groups):
    g = torch.Generator().manual_seed(experts + k)
    logits = torch.randn(7, experts, generator=g) - 200
    bias = 0.1 * torch.randn(experts, generator=g)
    bias[experts // groups:] += 1
    if scores == "softmax":
        logits[:, 0] = 0.0
    c = case(k, scores, groups, groups - 1, 2)
    w, e = check(c, logits, bias)
    assert float(w.sum(1).min()) > 0.9
    backward(c, logits, e)


@pytest.mark.parametrize("experts,k", [(12, 4), (300, 20), (90, 64)])
def test_below_64_bits(experts, k):
    """Sigmoids below e^-708 have weight 0 and no gradient, beside larger ones too."""
    logits = torch.full((3, experts), -800.0)
    logits[1] = torch.finfo(torch.float32).min
    logits[2, 5] = -100.0
    w, e = fp4.expert_route(logits.cuda(), k, "sigmoid")
    d = fp4.expert_route_backward(torch.randn(3, k).cuda(), logits.cuda(), e, "sigmoid")
    assert (w[:2] == 0).all() and (e >= 0).all() and (d == 0).all()
    assert w[2, 0] == 1 and e[2, 0] == 5 and (w[2, 1:] == 0).all()
