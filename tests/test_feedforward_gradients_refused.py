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


# calls of host tensors, of which one has a tangent of forward-mode differentiation
def at(which, *tensors):
    made = [t() for t in tensors]
    made[which] = torch.autograd.forward_ad.make_dual(made[which], torch.ones_like(made[which]))
    return made


bf = lambda *s: lambda: torch.zeros(s, dtype=BF)
f32 = lambda *s: lambda: torch.zeros(s)
i32 = lambda *s: torch.zeros(s, dtype=I32)
i64 = lambda *s: torch.zeros(s, dtype=torch.int64)
TABLE = torch.zeros(9, 32, 2)


def pick(*a):
    return fp4.expert_route(a[0], 2, bias=a[1], out=(a[2], i32(5, 2)))


TANGENTS = {
    "linear": (lambda *a: fp4.fp4_linear(weights(ones(1)), a[0], out=a[1]), bf(5, 96), bf(5, 64)),
    "experts": (lambda *a: fp4.fp4_experts(weights(ones(4), (4,), 128, 96), weights(ones(4), (4,), 96, 64),
                                           a[0], a[1], i32(5, 2), out=a[2]),
                bf(5, 96), f32(5, 2), bf(5, 96)),
    "route": (pick, f32(5, 8), f32(8), f32(5, 2)),
    "route_backward": (lambda *a: fp4.expert_route_backward(a[0], a[1], i32(5, 2), out=a[2]),
                       f32(5, 2), f32(5, 8), f32(5, 8)),
    "residual": (lambda *a: fp4.residual_norm(*a[:5], out=a[5:]), bf(5, 64), bf(5, 64), bf(64), bf(64),
                 bf(64), bf(5, 64), bf(5, 64)),
    "residual_backward": (lambda *a: fp4.residual_norm_backward(*a[:7], out=a[7:]), bf(5, 64), bf(5, 64),
                          bf(5, 64), bf(5, 64), bf(64), bf(64), bf(64), bf(5, 64), bf(5, 64)),
    "qk_norm_rope": (lambda *a: fp4.qk_norm_rope(*a[:4], i64(3), TABLE, out=a[4:]), bf(3, 2, 64),
                     bf(3, 1, 64), bf(64), bf(64), bf(3, 2, 64), bf(3, 1, 64)),
    "qk_norm_rope_backward": (
        lambda *a: fp4.qk_norm_rope_backward(*a[:6], i64(3), TABLE, out=a[6:]), bf(3, 2, 64), bf(3, 1, 64),
        bf(3, 2, 64), bf(3, 1, 64), bf(64), bf(64), bf(3, 2, 64), bf(3, 1, 64)),
}


@pytest.mark.parametrize("name,which", [(n, i) for n, t in TANGENTS.items() for i in range(len(t) - 1)])
def test_tangents(name, which):
    call, *tensors = TANGENTS[name]
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises(RuntimeError, match="gradient"):
            call(*at(which, *tensors))
        with torch.no_grad(), pytest.raises(RuntimeError, match="gradient"):
            call(*at(which, *tensors))
    with pytest.raises(ValueError):                              # host tensors
        call(*[t() for t in tensors])


def test_tangent_of_alpha():
    with torch.autograd.forward_ad.dual_level():
        alpha = torch.autograd.forward_ad.make_dual(torch.ones(1), torch.ones(1))
        at_ = fp4._Address(fp4._CWeights(0x10000, 0x10000, 0x10000, 1, 64, 96, 0, 0), 0, alpha)
        with pytest.raises(RuntimeError, match="gradient"):
            fp4._binding().linear(at_, torch.zeros(5, 96, dtype=BF), False, None, None, None)
