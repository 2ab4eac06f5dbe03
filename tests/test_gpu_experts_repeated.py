"""fp4_experts where tokens name an expert in several of their places: more rows
of an expert than there are tokens, with activations of one segment and of
several, hidden rows long and short."""
import pytest

import feedforward_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_experts import make  # noqa: E402
from test_gpu_linear import handle  # noqa: E402


def check(gu, dn, x, w, ids, layout):
    """Against 64 bits, from a workspace of NaN."""
    want, err = R.experts(x, R.values(gu, layout), R.values(dn, layout), w, ids)
    a, b = handle(gu), handle(dn)
    need = fp4.fp4_experts_workspace_bytes(a, b, *ids.shape)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    R.close(fp4.fp4_experts(a, b, x.cuda(), w.cuda(), ids.cuda(), ws=ws), want, err)


@pytest.mark.parametrize("layout", ["tensor", "mx"])
@pytest.mark.parametrize("hidden,inner", [(2048, 128), (4096, 128), (8192, 64), (128, 4096), (16384, 32)])
@pytest.mark.parametrize("tokens,k", [(1, 2), (1, 6), (2, 4), (3, 6), (4, 2), (7, 6), (8, 3), (9, 5), (15, 6)])
def test_long_rows(layout, hidden, inner, tokens, k):
    gu, dn, x, w, ids = make(hidden + tokens + k, tokens, 6, k, hidden, inner, layout)
    check(gu, dn, x, w, torch.full_like(ids, 4), layout)         # everyone names one expert only
    ids[:, 1:] = ids[:, :1]                                      # each token its own
    ids[::3, k // 2:] = -1
    check(gu, dn, x, w, ids, layout)


@pytest.mark.parametrize("tokens,k", [(9, 60), (10, 64), (15, 40)])
@pytest.mark.parametrize("hidden,inner", [(4096, 32), (256, 2048)])
def test_many_places(tokens, k, hidden, inner):
    """Sorted by a launch of its own: more than 512 assignments."""
    gu, dn, x, w, _ = make(tokens, tokens, 40, 1, hidden, inner)
    g = torch.Generator().manual_seed(k)
    w = torch.softmax(torch.randn(tokens, k, generator=g), 1)
    check(gu, dn, x, w, torch.randint(-1, 5, (tokens, k), generator=g).int() * 9, "tensor")


@pytest.mark.parametrize("layout", ["rows", "mx"])
@pytest.mark.parametrize("hidden,inner", [(96, 160), (256, 128), (128, 96), (4096, 128)])
@pytest.mark.parametrize("experts,k", [(1, 2), (1, 64), (3, 4), (4, 5), (4, 6), (4, 33), (20, 64)])
def test_more_places_than_experts(layout, hidden, inner, experts, k):
    """One token: experts that come late among its places, behind repeated ones and none."""
    gu, dn, x, w, ids = make(k + hidden, 1, experts, 1, hidden, inner, layout)
    w = torch.softmax(torch.randn(1, k, generator=torch.Generator().manual_seed(k)), 1)
    late = torch.arange(k, dtype=torch.int32)[None] - (k - experts)      # each once, at the end
    check(gu, dn, x, w, late.clamp(min=-1), layout)
    check(gu, dn, x, w, late.clamp(min=0), layout)
    check(gu, dn, x, w, late % experts, layout)
