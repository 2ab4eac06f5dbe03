"""Routing by groups at the ends of the numbers: tokens whose scores are NaN,
groups' sizes in which large numbers cancel or stand apart."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_route import case, check  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts,groups,top_groups,k", [
    (64, 8, 4, 6), (60, 5, 2, 4), (256, 8, 3, 15), (128, 8, 2, 20), (320, 64, 5, 12), (18, 6, 2, 3)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_scores_that_are_nan(dtype, renormalize, experts, groups, top_groups, k, bad):
    """Sums of NaN scores are equal: the first groups with a candidate stay, the logits choose
    among their experts, and the weights are NaN.  Other tokens do not notice."""
    g = torch.Generator().manual_seed(experts + k)
    logits = torch.randn(6, experts, generator=g).to(dtype)
    per = experts // groups
    logits[1, per + 1] = bad
    logits[2, -1] = bad                                  # in the last group
    logits[4, :per] = -math.inf                          # the first group has no candidate
    logits[4, -2] = bad
    how = dict(groups=groups, top_groups=top_groups, group_top=2, renormalize=renormalize)
    w, e = fp4.expert_route(logits.cuda(), k, **how)
    fine = [0, 3, 5]
    w0, e0 = fp4.expert_route(logits[fine].cuda(), k, **how)
    assert torch.equal(e[fine], e0) and torch.equal(w[fine], w0) and w0.isfinite().all()
    for t, first in ((1, 0), (2, 0), (4, 1)):
        x = logits[t].double().tolist()
        mine = [i for i in range(first * per, (first + top_groups) * per) if x[i] > -math.inf]
        want = sorted(mine, key=lambda i: (-x[i], i))[:k]
        want += [-1] * (k - len(want))
        assert e[t].tolist() == want
        there = e[t] >= 0
        assert w[t][there].isnan().all() and (w[t][~there] == 0).all()


def sized(seed, tokens, experts, groups, far):
    """Logits, and a bias by which a group's two largest sums are far from 0 and cancel."""
    g = torch.Generator().manual_seed(seed)
    per = experts // groups
    bias = torch.full((groups, per), -far)
    bias[:, 0] = far
    return torch.randn(tokens, experts, generator=g), bias.flatten()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("far", [1.0, 40.0, 3e3, 1e6])
@pytest.mark.parametrize("experts,groups,top_groups,k", [
    (64, 8, 4, 4), (64, 8, 4, 6), (60, 5, 2, 2), (256, 8, 3, 3), (256, 8, 3, 15), (128, 8, 2, 20),
    (320, 64, 5, 5), (512, 32, 7, 7), (512, 32, 7, 9)])
def test_sizes_that_cancel(scores, far, experts, groups, top_groups, k):
    logits, bias = sized(experts + k, 40, experts, groups, far)
    check(case(k, scores, groups, top_groups, 2), logits, bias)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("far", [1e9, 3e38, math.inf])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_far_away(scores, far, group_top):
    """Whole groups that a bias puts last or first."""
    logits, bias = sized(7, 30, 256, 8, 0.25)
    bias[32:64] = -far
    bias[96] = far
    if math.isfinite(far):
        bias[100] = far
    check(case(6, scores, 8, 3, group_top), logits, bias)
