"""fp4_experts against 64 bits: few assignments and many, experts without
tokens and with most of them, numbers outside the experts, every layout."""
import math

import pytest

import feedforward_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_linear import handle  # noqa: E402

BF = torch.bfloat16


def make(seed, tokens, experts, k, hidden, inner, layout="tensor"):
    g = torch.Generator().manual_seed(seed)
    gu = R.weight_bytes(g, (experts,), 2 * inner, hidden, layout)
    dn = R.weight_bytes(g, (experts,), hidden, inner, layout)
    x = torch.randn(tokens, hidden, generator=g).bfloat16()
    ids = torch.rand(tokens, experts, generator=g).topk(k, 1).indices.int()
    w = torch.softmax(torch.randn(tokens, k, generator=g), 1)
    return gu, dn, x, w, ids


def check(gu, dn, x, w, ids, layout="tensor"):
    want, err = R.experts(x, R.values(gu, layout), R.values(dn, layout), w, ids)
    got = fp4.fp4_experts(handle(gu), handle(dn), x.cuda(), w.cuda(), ids.cuda())
    R.close(got, want, err)
    return got


@pytest.mark.parametrize("layout", ["tensor", "rows", "tiles", "mx"])
@pytest.mark.parametrize("tokens,experts,k,hidden,inner", [
    (1, 1, 1, 32, 32), (1, 8, 2, 256, 96), (2, 5, 5, 64, 160), (7, 16, 4, 288, 64),
    (16, 64, 6, 128, 224), (17, 4, 2, 320, 96), (40, 8, 8, 160, 128), (64, 128, 8, 96, 32),
    (130, 6, 3, 512, 288), (300, 3, 2, 96, 352), (513, 2, 1, 64, 64), (520, 40, 4, 256, 128)])
def test_against_64_bits(layout, tokens, experts, k, hidden, inner):
    check(*make(tokens + experts + hidden, tokens, experts, k, hidden, inner, layout), layout)


@pytest.mark.parametrize("tokens", [3, 100, 700])
def test_uneven(tokens):
    """One expert has nearly everything, some have nothing; the same one twice; nobody."""
    gu, dn, x, w, ids = make(tokens, tokens, 12, 3, 128, 96)
    ids[:] = 5
    ids[::3, 1] = 11
    ids[1::3, 2] = -1
    ids[1, :] = torch.tensor([-1, 12, 1 << 30], dtype=torch.int32)
    ids[2, 0] = -(1 << 31)
    got = check(gu, dn, x, w, ids)
    assert (got[1] == 0).all()


@pytest.mark.parametrize("tokens", [5, 600])
def test_nobody(tokens):
    gu, dn, x, w, ids = make(1, tokens, 4, 2, 64, 32)
    assert (check(gu, dn, x, w, torch.full_like(ids, -1)) == 0).all()


@pytest.mark.parametrize("tokens", [6, 40, 400])
def test_values_that_are_not_finite(tokens):
    """A token's NaN and a weight's NaN stay with their token."""
    gu, dn, x, w, ids = make(tokens, tokens, 8, 2, 160, 64)
    x[1, 7] = math.nan
    w[3, 1] = math.nan
    got = fp4.fp4_experts(handle(gu), handle(dn), x.cuda(), w.cuda(), ids.cuda()).cpu()
    fine = [t for t in range(tokens) if t not in (1, 3)]
    assert got[1].isnan().all() and got[3].isnan().all()
    want, err = R.experts(x[fine], R.values(gu, "tensor"), R.values(dn, "tensor"), w[fine], ids[fine])
    R.close(got[fine], want, err)


@pytest.mark.parametrize("tokens", [4, 300])
def test_strides(tokens):
    gu, dn, x, w, ids = make(3, tokens, 6, 2, 96, 64)
    want = fp4.fp4_experts(handle(gu), handle(dn), x.cuda(), w.cuda(), ids.cuda())
    wide = torch.full((tokens, 120), 3.0, dtype=BF, device="cuda")
    wide[:, 16:112] = x.cuda()
    out = torch.full((tokens, 136), 7.0, dtype=BF, device="cuda")
    fp4.fp4_experts(handle(gu), handle(dn), wide[:, 16:112], w.cuda(), ids.cuda(), out=out[:, 8:104])
    assert torch.equal(out[:, 8:104], want)
    assert (out[:, :8] == 7).all() and (out[:, 104:] == 7).all()


def test_mixed_formats():
    """gate_up and down need not be of one format."""
    g = torch.Generator().manual_seed(2)
    gu = R.weight_bytes(g, (4,), 128, 96, "mx")
    dn = R.weight_bytes(g, (4,), 96, 64, "tiles")
    x = torch.randn(21, 96, generator=g).bfloat16()
    ids = torch.randint(0, 4, (21, 2), generator=g).int()
    w = torch.rand(21, 2, generator=g)
    want, err = R.experts(x, R.values(gu, "mx"), R.values(dn, "tiles"), w, ids)
    R.close(fp4.fp4_experts(handle(gu), handle(dn), x.cuda(), w.cuda(), ids.cuda()), want, err)


@pytest.mark.parametrize("tokens", [1, 60, 900])
def test_equal_calls_give_equal_bits(tokens):
    gu, dn, x, w, ids = make(9, tokens, 16, 4, 256, 128)
    a = (handle(gu), handle(dn), x.cuda(), w.cuda(), ids.cuda())
    first = fp4.fp4_experts(*a)
    ws = torch.full((fp4.fp4_experts_workspace_bytes(a[0], a[1], tokens, 4),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    for _ in range(4):
        assert torch.equal(fp4.fp4_experts(*a, ws=ws), first)


def test_empty():
    gu, dn, x, w, ids = make(9, 3, 4, 2, 64, 32)
    got = fp4.fp4_experts(handle(gu), handle(dn), x[:0].cuda(), w[:0].cuda(), ids[:0].cuda())
    assert got.shape == (0, 64)


def test_gradients_are_refused():
    gu, dn, x, w, ids = make(9, 3, 4, 2, 64, 32)
    a = [handle(gu), handle(dn), x.cuda(), w.cuda(), ids.cuda()]
    for i in (2, 3):
        b = list(a)
        b[i] = a[i].clone().requires_grad_()
        with pytest.raises(RuntimeError, match="no backward"):
            fp4.fp4_experts(*b)


@pytest.mark.parametrize("layout", ["rows", "mx"])
@pytest.mark.parametrize("tokens,experts,k", [
    (16, 1, 1), (10, 1, 1), (16, 2, 2), (4, 20, 8), (5, 20, 8), (11, 3, 3), (60, 8, 2), (80, 8, 2),
    (81, 8, 2), (128, 8, 2), (129, 8, 2), (64, 2, 2), (256, 12, 2), (257, 12, 2)])
def test_sizes_next_to_each_other(layout, tokens, experts, k):
    """Around the numbers of assignments at which another kernel takes the call."""
    check(*make(tokens + experts, tokens, experts, k, 256, 128, layout), layout)
