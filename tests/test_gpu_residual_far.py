"""Gradients of residual_norm where squares of y or of the block leave the range
of fp32, against 64 bits: rows that are scaled before their squares are summed."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import feedforward_reference as R  # noqa: E402
from test_gpu_residual_norm import check, make  # noqa: E402

CLOSE = R.close


def close_or_infinite(got, want, err):
    """A value past the largest number of its type is an infinity of its sign.  The row whose
    block is 0 has some: 1 / sqrt(eps) = 1e19 = 2^63 times a gate of 2^70 times dY is past 2^128.
    From half a step above bf16's largest, 2^128 (1 - 2^-9), a number rounds to infinity; one
    that its error may bring there may be either."""
    edge = 2.0 ** 128 * (1 - 2.0 ** -9)
    flat = got.double().cpu()
    sure = want.abs() - err > edge
    infinite = flat == torch.sign(want) * float("inf")
    assert infinite[sure].all()
    skip = sure | (infinite & (want.abs() + err >= edge))
    zero = torch.zeros((), dtype=torch.float64)
    CLOSE(torch.where(skip, zero, flat).to(got.dtype), torch.where(skip, zero, want), err)


@pytest.mark.parametrize("size", [2.0 ** -55, 2.0 ** 70])
@pytest.mark.parametrize("dim", [64, 1032, 2048, 8200])
@pytest.mark.parametrize("post,gate", [(False, "none"), (False, "channel"), (False, "token"),
                                       (True, "channel"), (True, "token")])
@pytest.mark.parametrize("with_dy", [False, True])
def test_far_gradients(size, dim, post, gate, with_dy, monkeypatch):
    """y is of this size, and so is the block; without dy the gradients are as far the other way."""
    d, dy, dz = make(dim, 5, dim, post, gate, size)
    if post:
        d["gate"] = (d["gate"].double() * size).bfloat16()
    d["x"][1] = 0
    d["block"][2] = 0
    if not with_dy:
        dy.zero_()
    monkeypatch.setattr(R, "close", close_or_infinite)
    check(d, dy, dz, 0.75, 1e-38)
