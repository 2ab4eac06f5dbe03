"""Forward-mode differentiation of calls that have a gradient: none of them has
its form for tangents, and torch's autograd says so."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402

dual = torch.autograd.forward_ad


@pytest.mark.parametrize("name", ["route", "residual", "rope"])
def test_refused(name):
    x = torch.randn(6, 64, device="cuda")
    b = x.bfloat16()
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(6, device="cuda")
    table = torch.randn(6, 32, 2, device="cuda")
    calls = {"route": (x, lambda x: fp4.expert_route(x, 3)),
             "residual": (b, lambda x: fp4.residual_norm(x, b, w)),
             "rope": (b.view(6, 1, 64), lambda x: fp4.qk_norm_rope(x, b.view(6, 1, 64), w, w, at, table))}
    v, call = calls[name]
    with dual.dual_level():
        for mode in (torch.enable_grad, torch.no_grad):
            with mode(), pytest.raises((RuntimeError, NotImplementedError), match="jvp"):
                call(dual.make_dual(v, torch.ones_like(v)))
        call(v)                                        # tensors without one are as before
    call(v)
