"""The gate of fp4_experts far below zero, where e^-g leaves fp32 and silu(g) u does not."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402

GATES = [-300.0, -170.0, -120.5, -96.0, -90.0, -89.0, -88.5, -88.0, -87.0, -60.0, -3.0, -0.0, 5.0, 100.0]


@pytest.mark.parametrize("hidden", [32, 128])               # by columns, by streams
@pytest.mark.parametrize("tokens", [1, 3, 14, 40, 700])
def test_far_gates(hidden, tokens):
    """Sums of one product each: silu(x0) * (2^60 x1 2^s) in every place, s by the size of silu."""
    inner = 32
    one = 127
    x = torch.zeros(tokens, hidden, dtype=torch.bfloat16)
    g = torch.tensor([GATES[(5 * t + 3) % len(GATES)] for t in range(tokens)])
    x[:, 0] = g
    # up so large that the product is near 1 where it can be
    size = torch.ceil((-g.clamp(max=0.0) / 0.6931)).clamp(max=126.0)
    x[:, 1] = torch.exp2(size - 60)
    codes = torch.zeros(1, 2 * inner, hidden // 2, dtype=torch.uint8)
    codes[0, :inner, 0] = 0x02                                # 1 at column 0
    codes[0, inner:, 0] = 0x20                                # 1 at column 1
    scales = torch.full((1, 2 * inner, hidden // 32), one, dtype=torch.uint8)
    scales[0, inner:] = one + 60
    down = torch.zeros(1, hidden, inner // 2, dtype=torch.uint8)
    down[0, :, 0] = 0x02
    mx = lambda c, s: fp4.Fp4Weights(c.cuda(), s.cuda(), fmt=fp4.FORMAT_MXFP4)
    gu, dn = mx(codes, scales), mx(down, torch.full((1, hidden, 1), one, dtype=torch.uint8))
    got = fp4.fp4_experts(gu, dn, x.cuda(), torch.ones(tokens, 1).cuda(),
                          torch.zeros(tokens, 1, dtype=torch.int32).cuda()).double().cpu()
    v = x[:, 0].double()
    want = (v * torch.sigmoid(v) * x[:, 1].double() * 2.0 ** 60)[:, None].expand(got.shape)
    # roundings to bf16 of the hidden value and the sum, exp of a rounded half of its argument
    room = (2 * 2.0 ** -8 + 400 * 2.0 ** -24) * want.abs() + 2.0 ** -126
    assert ((got - want).abs() <= room).all()
