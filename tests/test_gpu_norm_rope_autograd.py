"""qk_norm_rope inside torch's autograd: outputs of inputs that require
gradients carry them, and the gradients are those of qk_norm_rope_backward
(which test_gpu_qk_norm_rope checks against the formula and differences)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_qk_norm_rope import make, tensor  # noqa: E402


def setup(t=70, hq=4, hk=2, d=64, rot=32):
    rng = np.random.default_rng(t)
    q, k, qw, kw, dq, dk, table, pos = make(rng, t, hq, hk, d, rot)
    return [tensor(x) for x in (q, k, qw, kw)], [tensor(x) for x in (dq, dk)], (
        torch.from_numpy(pos).cuda(), table)


def same(a, b):
    return a.dtype == b.dtype and torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("weights", [True, False])
def test_gradients(inter, weights):
    x, dy, rest = setup()
    if not weights:
        x[2] = x[3] = None
    want_y = fp4.qk_norm_rope(*x, *rest, interleaved=inter)
    want = fp4.qk_norm_rope_backward(*dy, *x, *rest, interleaved=inter)
    leaves = [None if v is None else v.clone().requires_grad_() for v in x]
    y = fp4.qk_norm_rope(*leaves, *rest, interleaved=inter)
    assert all(v.requires_grad for v in y)
    assert all(same(a, b) for a, b in zip(y, want_y))
    torch.autograd.backward(y, dy)
    torch.cuda.synchronize()
    for leaf, g in zip(leaves, want):
        if leaf is None:
            assert g is None
        else:
            assert same(leaf.grad, g.to(torch.bfloat16))


@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_any_one_input(which):
    """Each of the four alone; one output used, its gradient an expanded scalar."""
    x, dy, rest = setup(t=9)
    x[which] = x[which].clone().requires_grad_()
    y = fp4.qk_norm_rope(*x, *rest)
    out = which % 2                             # queries with their weight, keys with theirs
    y[out].sum().backward()
    ones = [torch.ones_like(v) if i == out else torch.zeros_like(v) for i, v in enumerate(dy)]
    plain = [v.detach() for v in x]
    want = fp4.qk_norm_rope_backward(*ones, *plain, *rest)[which]
    torch.cuda.synchronize()
    assert same(x[which].grad, want.to(torch.bfloat16))


def test_slices_of_a_projection_and_turned_gradients():
    """Queries and keys as slices of one tensor; gradients arrive transposed."""
    x, dy, rest = setup(t=33)
    qkv = torch.cat((x[0], x[1], x[1]), 1).requires_grad_()
    y = fp4.qk_norm_rope(qkv[:, :4], qkv[:, 4:6], x[2], x[3], *rest)
    turned = [g.transpose(0, 1).contiguous().transpose(0, 1) for g in dy]
    torch.autograd.backward(y, turned)
    want = fp4.qk_norm_rope_backward(*dy, *x, *rest)
    torch.cuda.synchronize()
    assert same(qkv.grad[:, :4], want[0]) and same(qkv.grad[:, 4:6], want[1])
    assert not qkv.grad[:, 6:].any()


def test_without_gradients():
    x, dy, rest = setup(t=5)
    leaves = [v.clone().requires_grad_() for v in x]
    with torch.no_grad():
        y = fp4.qk_norm_rope(*leaves, *rest)
    assert not any(v.requires_grad for v in y)
    y = fp4.qk_norm_rope(*x, *rest)
    assert not any(v.requires_grad for v in y)


def test_outputs_given():
    """Given outputs cannot carry a history: refused where one is wanted."""
    x, dy, rest = setup(t=5)
    leaves = [v.clone().requires_grad_() for v in x]
    out = [torch.empty_like(v) for v in x[:2]]
    with pytest.raises(RuntimeError, match="gradient"):
        fp4.qk_norm_rope(*leaves, *rest, out=out)
    with torch.no_grad():
        fp4.qk_norm_rope(*leaves, *rest, out=out)
    assert all(same(a, b) for a, b in zip(out, fp4.qk_norm_rope(*x, *rest)))


def test_refused():
    """A gradient of the table, and of the gradients."""
    x, dy, rest = setup(t=5)
    with pytest.raises(RuntimeError, match="table"):
        fp4.qk_norm_rope(*x, rest[0], rest[1].clone().requires_grad_())
    q = x[0].clone().requires_grad_()
    y = fp4.qk_norm_rope(q, *x[1:], *rest)
    g, = torch.autograd.grad(y[0].float().square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()


def test_captured_into_a_graph():
    """Forward and backward of fresh leaves in one captured graph."""
    x, dy, rest = setup(t=50)
    fp4.qk_norm_rope_backward(*dy, *x, *rest)   # nothing is loaded first inside the capture
    leaves = [v.clone().requires_grad_() for v in x]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = fp4.qk_norm_rope(*leaves, *rest)
        held = torch.autograd.grad(y, leaves, dy)
    for i in range(3):
        with torch.no_grad():
            leaves[0].copy_(x[0] * (i + 1))
        plain = [v.detach() for v in leaves]
        want = fp4.qk_norm_rope_backward(*dy, *plain, *rest)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(same(a, b.to(torch.bfloat16)) for a, b in zip(held, want)), i
