"""fp4_linear against 64 bits: every layout of the weights, odd sizes, strides,
both output types, values that are not finite, handles made by the quantizers."""
import math

import pytest

import feedforward_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def handle(w):
    return fp4.Fp4Weights(**{k: v.cuda() if torch.is_tensor(v) else v for k, v in w.items()})


def make(seed, tokens, rows, cols, layout):
    gen = torch.Generator().manual_seed(seed)
    w = R.weight_bytes(gen, (), rows, cols, layout)
    x = (torch.randn(tokens, cols, generator=gen) * torch.exp(torch.randn(cols, generator=gen))).bfloat16()
    return w, x


@pytest.mark.parametrize("layout", ["tensor", "rows", "tiles", "mx"])
@pytest.mark.parametrize("tokens,rows,cols", [
    (1, 16, 32), (1, 4096, 4096), (2, 48, 96), (5, 1024, 2080), (15, 112, 160), (16, 64, 512),
    (17, 160, 544), (31, 32, 288), (33, 320, 1056), (64, 256, 256), (65, 80, 64), (130, 272, 800),
    (257, 528, 320), (600, 1040, 416)])
def test_against_64_bits(layout, tokens, rows, cols):
    w, x = make(tokens * 7 + rows + cols, tokens, rows, cols, layout)
    want, err = R.linear(x, R.values(w, layout))
    h = handle(w)
    R.close(fp4.fp4_linear(h, x.cuda()), want, err)
    R.close(fp4.fp4_linear(h, x.cuda(), dtype=F32), want, err)


@pytest.mark.parametrize("layout", ["tensor", "rows", "mx"])
@pytest.mark.parametrize("rows", [1, 2, 3, 7, 15, 17, 100, 129, 255, 257, 1001])
@pytest.mark.parametrize("tokens", [1, 3, 40, 150])
def test_odd_rows(layout, rows, tokens):
    w, x = make(rows + tokens, tokens, rows, 352, layout)
    want, err = R.linear(x, R.values(w, layout))
    h = handle(w)
    for dtype in (BF, F32):
        R.close(fp4.fp4_linear(h, x.cuda(), dtype=dtype), want, err)


@pytest.mark.parametrize("tokens", [1, 9, 70, 200])
def test_strides(tokens):
    """Rows inside wider tensors; what lies between the output's rows stays."""
    w, x = make(3, tokens, 96, 320, "tensor")
    wide = torch.full((tokens, 480), math.nan, dtype=BF)
    wide[:, 64:384] = x
    want, err = R.linear(x, R.values(w, "tensor"))
    for dtype in (BF, F32):
        for first, width in ((0, 96), (3, 101), (8, 128)):
            out = torch.full((tokens, width + first), 7.0, dtype=dtype, device="cuda")
            got = fp4.fp4_linear(handle(w), wide.cuda()[:, 64:384], dtype=dtype, out=out[:, first:first + 96])
            R.close(got, want, err)
            assert (out[:, :first] == 7).all() and (out[:, first + 96:] == 7).all()


@pytest.mark.parametrize("layout", ["tensor", "mx"])
@pytest.mark.parametrize("tokens", [3, 20, 300])
def test_values_that_are_not_finite(layout, tokens):
    """They reach their own token's outputs, as the sum says, and no other's."""
    w, x = make(5, tokens, 64, 288, layout)
    bad = {1: math.nan, 2: math.inf}
    for t, v in bad.items():
        x[t, 17 * t] = v
    wv = R.values(w, layout)
    got = fp4.fp4_linear(handle(w), x.cuda(), dtype=F32).double().cpu()
    fine = [t for t in range(tokens) if t not in bad]
    want, err = R.linear(x[fine], wv)
    R.close(got[fine].float(), want, err)
    assert got[1].isnan().all()
    col = wv[:, 34]
    assert torch.equal(got[2][col > 0], torch.full_like(got[2][col > 0], math.inf))
    assert torch.equal(got[2][col < 0], torch.full_like(got[2][col < 0], -math.inf))
    assert got[2][col == 0].isnan().all()


def test_weights_of_the_quantizers():
    """Handles of what the library's quantizers return decode as fp4_dequantize does."""
    g = torch.Generator().manual_seed(9)
    m = torch.randn(160, 512, generator=g).bfloat16().cuda()
    x = torch.randn(37, 512, generator=g).bfloat16()
    made = []
    for flags in (fp4.RTN6, fp4.FOUR_OVER_SIX, fp4.BLOCK2D | fp4.FOUR_OVER_SIX):
        q = fp4.nvfp4_quantize(m, flags)
        d = fp4.fp4_dequantize(fp4.FORMAT_NVFP4, q["codes"], q["scales"], q["alpha"], 160, 512,
                               flags & fp4.BLOCK2D)
        made.append((fp4.Fp4Weights(q["codes"], q["scales"], q["alpha"]), d))
    q = fp4.nvfp4_quantize_rows(m, fp4.FOUR_OVER_SIX)
    d = torch.cat([fp4.fp4_dequantize(fp4.FORMAT_NVFP4, q["codes"][i:i + 1], q["scales"][i:i + 1],
                                      q["alpha"][i:i + 1], 1, 512) for i in range(160)])
    made.append((fp4.Fp4Weights(q["codes"], q["scales"], q["alpha"]), d))
    q = fp4.mxfp4_quantize(m, fp4.ROWWISE)
    d = fp4.fp4_dequantize(fp4.FORMAT_MXFP4, q["codes_r"], q["scales_r"], None, 160, 512)
    made.append((fp4.Fp4Weights(q["codes_r"], q["scales_r"], fmt=fp4.FORMAT_MXFP4), d))
    for h, d in made:
        want, err = R.linear(x, d.double().cpu())      # d is rounded to fp32 itself
        R.close(fp4.fp4_linear(h, x.cuda(), dtype=F32), want, err)


def test_empty():
    w, x = make(1, 3, 32, 64, "tensor")
    h = handle(w)
    assert fp4.fp4_linear(h, x[:0].cuda()).shape == (0, 32)
    none = fp4.Fp4Weights(torch.empty(0, 32, dtype=torch.uint8, device="cuda"),
                          torch.empty(0, 4, dtype=torch.uint8, device="cuda"),
                          torch.ones(1, device="cuda"))
    assert fp4.fp4_linear(none, x.cuda()).shape == (3, 0)
    flat = fp4.Fp4Weights(torch.empty(32, 0, dtype=torch.uint8, device="cuda"),
                          torch.empty(32, 0, dtype=torch.uint8, device="cuda"),
                          torch.ones(1, device="cuda"))
    assert (fp4.fp4_linear(flat, x.cuda()[:, :0]) == 0).all()


@pytest.mark.parametrize("tokens", [1, 48, 300])
def test_equal_calls_give_equal_bits(tokens):
    w, x = make(2, tokens, 1040, 2080, "rows")
    h, x = handle(w), x.cuda()
    first = fp4.fp4_linear(h, x, dtype=F32)
    for _ in range(5):
        assert torch.equal(fp4.fp4_linear(h, x, dtype=F32), first)


def test_gradients_are_refused():
    w, x = make(1, 3, 32, 64, "tensor")
    x = x.cuda().requires_grad_()
    with pytest.raises(RuntimeError, match="no backward"):
        fp4.fp4_linear(handle(w), x)
    with torch.no_grad():
        fp4.fp4_linear(handle(w), x)


@pytest.mark.parametrize("layout", ["tensor", "rows", "tiles", "mx"])
@pytest.mark.parametrize("tokens,rows,cols", [
    (9, 8208, 320), (16, 9008, 1024),                                     # streams
    (33, 7008, 544), (40, 8208, 160), (100, 4112, 1056), (150, 4112, 352),   # 32 to 64 tokens at once
    (1030, 7024, 160), (4200, 1504, 416), (300, 20016, 96), (700, 12320, 32)])   # 128 tokens, 256 rows
def test_large(layout, tokens, rows, cols):
    w, x = make(tokens + rows + cols, tokens, rows, cols, layout)
    want, err = R.linear(x, R.values(w, layout))
    h = handle(w)
    R.close(fp4.fp4_linear(h, x.cuda()), want, err)
    R.close(fp4.fp4_linear(h, x.cuda(), dtype=F32), want, err)


@pytest.mark.parametrize("layout", ["rows", "mx"])
@pytest.mark.parametrize("tokens,rows,cols", [
    (13, 8193, 256), (50, 6001, 288), (70, 9001, 544), (1025, 7003, 288)])
def test_large_odd_rows_and_strides(layout, tokens, rows, cols):
    """Rows inside wider tensors; what lies between and behind the output's rows stays."""
    w, x = make(tokens + rows, tokens, rows, cols, layout)
    wide = torch.full((tokens, cols + 24), math.nan, dtype=BF)
    wide[:, 16:16 + cols] = x
    want, err = R.linear(x, R.values(w, layout))
    for dtype in (BF, F32):
        for first, width in ((0, rows), (1, rows + 4)):
            out = torch.full((tokens + 2, width + first), 7.0, dtype=dtype, device="cuda")
            R.close(fp4.fp4_linear(handle(w), wide.cuda()[:, 16:16 + cols], dtype=dtype,
                                   out=out[:tokens, first:first + rows]), want, err)
            out[:tokens, first:first + rows] = 7.0
            assert (out == 7.0).all()


@pytest.mark.parametrize("tokens,rows,cols", [(60, 6000, 320), (1025, 7008, 160)])
def test_large_values_that_are_not_finite(tokens, rows, cols):
    w, x = make(5, tokens, rows, cols, "tensor")
    x[1, 17], x[2, 33] = math.nan, math.inf
    got = fp4.fp4_linear(handle(w), x.cuda(), dtype=F32).cpu()
    fine = [t for t in range(tokens) if t not in (1, 2)]
    wv = R.values(w, "tensor")
    R.close(got[fine], *R.linear(x[fine], wv))
    assert got[1].isnan().all()
    col = wv[:, 33]
    assert (got[2][col > 0] == math.inf).all() and (got[2][col < 0] == -math.inf).all()
    assert got[2][col == 0].isnan().all()


@pytest.mark.parametrize("layout", ["tensor", "tiles", "mx"])
@pytest.mark.parametrize("tokens,rows", [(4, 8176), (4, 8192), (5, 8960), (5, 8944), (16, 28672), (17, 4096),
                                         (64, 4112), (65, 4112), (16, 6144)])
def test_sizes_next_to_each_other(layout, tokens, rows):
    """Around the sizes at which another kernel takes the call."""
    w, x = make(tokens + rows, tokens, rows, 256, layout)
    want, err = R.linear(x, R.values(w, layout))
    R.close(fp4.fp4_linear(handle(w), x.cuda()), want, err)


@pytest.mark.parametrize("tokens", [1, 30, 300])
@pytest.mark.parametrize("rows", [48, 9008])
def test_no_columns(tokens, rows):
    """Empty sums are zeros."""
    empty = lambda: torch.empty(rows, 0, dtype=torch.uint8, device="cuda")
    out = torch.full((tokens, rows), 7.0, dtype=BF, device="cuda")
    h = fp4.Fp4Weights(empty(), empty(), torch.ones(1, device="cuda"))
    fp4.fp4_linear(h, torch.empty(tokens, 0, dtype=BF, device="cuda"), out=out)
    assert (out == 0).all()


@pytest.mark.parametrize("layout", ["rows", "mx"])
@pytest.mark.parametrize("cols", [128, 160, 192, 224, 256, 480, 512, 544, 608, 1024, 1056])
@pytest.mark.parametrize("tokens", [17, 40, 64])
def test_ends_of_rows(layout, cols, tokens):
    """Rows that end anywhere within a run of values, and whose neighbours' scales are far larger."""
    w, x = make(cols + tokens, tokens, 6000, cols, layout)
    w["scales"][1::2] = 0x7E if layout == "rows" else 180
    want, err = R.linear(x, R.values(w, layout))
    R.close(fp4.fp4_linear(handle(w), x.cuda(), dtype=F32), want, err)
