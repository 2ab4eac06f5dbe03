"""Refusals of feed-forward calls that would lose a gradient.  They come before
any GPU call, so no GPU is needed."""
import os

import pytest

import block_scaled_fp4_reduce_amd as fp4

torch = pytest.importorskip("torch")
from torch._subclasses.fake_tensor import FakeTensorMode  # noqa: E402

BF, I32, F32, U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(fp4.LIB_PATH):
        from block_scaled_fp4_reduce_amd import build
        build.build()


def weights(alpha, lead=(), rows=64, cols=96):
    with FakeTensorMode(allow_non_fake_inputs=True):
        new = lambda *s: torch.empty(s, dtype=U8, device="cuda:0")
        return fp4.Fp4Weights(new(*lead, rows, cols // 2), new(*lead, rows, cols // 16), alpha)


def ones(*shape):
    with FakeTensorMode():
        return torch.empty(shape, dtype=F32, device="cuda:0")


@pytest.mark.parametrize("later", [False, True])
@pytest.mark.parametrize("rows", [False, True])
def test_alpha_of_a_product(later, rows):
    """An alpha that requires a gradient when the handle is made, or from then on."""
    alpha = ones(64 if rows else 1)
    alpha.requires_grad_(not later)
    w = weights(alpha)
    alpha.requires_grad_()
    x = torch.zeros(5, 96, dtype=BF)
    with pytest.raises(RuntimeError, match="no backward"):
        fp4.fp4_linear(w, x)
    with torch.no_grad(), pytest.raises(ValueError):             # a host tensor
        fp4.fp4_linear(w, x)
    with pytest.raises(ValueError):
        fp4.fp4_linear(weights(alpha.detach()), x)


@pytest.mark.parametrize("which", [0, 1])
def test_alpha_of_experts(which):
    alphas = [ones(4), ones(4)]
    alphas[which].requires_grad_()
    w = weights(alphas[0], (4,), 128, 96), weights(alphas[1], (4,), 96, 64)
    rest = torch.zeros(5, 96, dtype=BF), torch.zeros(5, 2), torch.zeros(5, 2, dtype=I32)
    with pytest.raises(RuntimeError, match="no backward"):
        fp4.fp4_experts(*w, *rest)
    with torch.no_grad(), pytest.raises(ValueError):
        fp4.fp4_experts(*w, *rest)
