"""Refusals of calls that would lose a gradient.  They come before any GPU call,
so no GPU is needed."""
import os

import pytest

import block_scaled_fp4_reduce_amd as fp4

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(fp4.LIB_PATH):
        from block_scaled_fp4_reduce_amd import build
        build.build()


def bf(*shape, grad=False):
    return torch.zeros(shape, dtype=torch.bfloat16, requires_grad=grad)


REST = torch.zeros(3, dtype=torch.int64), torch.zeros(9, 32, 2)


@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_norm_refuses_given_outputs(which):
    x = [bf(3, 2, 64), bf(3, 1, 64), bf(64), bf(64)]
    x[which] = x[which].requires_grad_()
    out = bf(3, 2, 64), bf(3, 1, 64)
    with pytest.raises(RuntimeError, match="gradient"):
        fp4.qk_norm_rope(*x, *REST, out=out)
    with torch.no_grad(), pytest.raises(ValueError):         # host tensors
        fp4.qk_norm_rope(*x, *REST, out=out)


def test_norm_refuses_outputs_that_require_gradients():
    with pytest.raises(RuntimeError, match="gradient"):
        fp4.qk_norm_rope(bf(3, 2, 64), bf(3, 1, 64), None, None, *REST,
                         out=(bf(3, 2, 64, grad=True), bf(3, 1, 64)))


def test_norm_refuses_a_gradient_of_the_table():
    with pytest.raises(RuntimeError, match="table"):
        fp4.qk_norm_rope(bf(3, 2, 64), bf(3, 1, 64), None, None, REST[0], REST[1].clone().requires_grad_())


def test_other_refusals_come_through_autograd():
    with pytest.raises(ValueError):
        fp4.qk_norm_rope(bf(3, 2, 64, grad=True), bf(3, 1, 64), None, None, *REST)
    with pytest.raises(TypeError):
        fp4.qk_norm_rope(bf(3, 2, 64, grad=True).float(), bf(3, 1, 64), None, None, *REST)


class Handle:
    """A cache handle that was never allocated: only its numbers are read."""

    def __init__(self):
        p = 0x10000
        self._c = fp4._CCache(p, p, p, p, p, p, 4, 16, 2, 64, fp4.FORMAT_NVFP4, 0)
        self._at = fp4.C.addressof(self._c)


def test_attention_refuses_queries_that_require_gradients():
    args = torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    q = bf(3, 4, 64, grad=True)
    with pytest.raises(RuntimeError, match="no backward"):
        fp4.fp4_kv_attention(Handle(), q, *args)
    with pytest.raises(RuntimeError, match="no backward"):
        fp4.fp4_kv_attention(Handle(), q.detach(), *args, out=q)
    for x in (q.detach(), bf(3, 4, 64)):
        with pytest.raises(ValueError):                      # host tensors
            fp4.fp4_kv_attention(Handle(), x, *args)
    with torch.no_grad(), pytest.raises(ValueError):
        fp4.fp4_kv_attention(Handle(), q, *args)
