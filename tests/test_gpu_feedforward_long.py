"""Batches of so many tokens that one launch would have 2^32 threads or more."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402

BF, I32 = torch.bfloat16, torch.int32


def test_norms():
    """67 million rows of 8 channels: equal rows with a gate of their own, a few others among them."""
    n = (1 << 26) + 5
    g = torch.Generator(device="cuda").manual_seed(1)
    some = torch.randn(7, 8, generator=g, device="cuda").bfloat16()
    rows = torch.tensor([0, 1, (1 << 26) - 5, (1 << 26) - 4, (1 << 26) - 1, 1 << 26, n - 1], device="cuda")
    x = torch.ones(n, 8, dtype=BF, device="cuda")
    x[rows] = some
    gate = torch.ones(n, 1, dtype=BF, device="cuda")
    gate[rows] = some[:, :1]
    w = torch.ones(8, dtype=BF, device="cuda")
    y, z = torch.zeros_like(x), torch.zeros_like(x)
    fp4.residual_norm(x, x, w, None, gate, out=(y, z))
    want = fp4.residual_norm(some, some, w, None, some[:, :1].contiguous())
    assert torch.equal(y[rows], want[0]) and torch.equal(z[rows], want[1])
    y[rows], z[rows] = 2.0, 1.0
    assert (y == 2).all() and (z == 1).all()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_routing(scores):
    """268 million tokens of one expert, forward and backward."""
    n = (1 << 28) + 5
    x = torch.zeros(n, 1, device="cuda")
    out = torch.zeros_like(x), torch.full((n, 1), -7, dtype=I32, device="cuda")
    w, e = fp4.expert_route(x, 1, scores, renormalize=False, out=out)
    s = 1.0 if scores == "softmax" else 0.5
    assert (w == s).all() and (e == 0).all()
    w[-1] = 3.0
    d = torch.full_like(x, 7.0)
    fp4.expert_route_backward(w, x, e, scores, renormalize=False, out=d)
    want = s * (1 - s)
    assert (d[:-1] == s * want).all() and d[-1] == 3 * want


@pytest.mark.parametrize("rows,cols,tokens", [(16, 32, (1 << 27) + 5), (208, 32, (1 << 24) + 3),
                                              (200, 128, (1 << 24) + 200)])
def test_products(rows, cols, tokens):
    """Sums of equal values, and of a few other rows."""
    x = torch.ones(tokens, cols, dtype=BF, device="cuda")
    at = torch.tensor([0, (1 << 24) - 1, 1 << 24, tokens - 1], device="cuda")
    x[at] = torch.arange(2, 6, device="cuda", dtype=BF)[:, None].expand(4, cols)
    codes = torch.full((rows, cols // 2), 0x22, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, cols // 32), 127, dtype=torch.uint8, device="cuda")
    out = torch.zeros(tokens, rows, dtype=BF, device="cuda")
    fp4.fp4_linear(fp4.Fp4Weights(codes, scales, fmt=fp4.FORMAT_MXFP4), x, out=out)
    for i, t in enumerate(at.tolist()):
        assert (out[t] == (i + 2) * cols).all()
    out[at] = cols
    assert (out == cols).all()
