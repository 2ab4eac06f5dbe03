"""The example layer: norm with rotation, cache write and attention together
against dense attention over the unquantized keys and values.  FP4 keeps a
value to about 2^-3 of its size: with E = 0.13 the root mean square of the
rounding of keys and values relative to them (NVFP4 0.09 to 0.1, MXFP4 0.12),
the output of a softmax over random keys is off by E from the values and by at
most as much again from the scores (|s| is of order 1), 2 E in all; a wrong
page, position or head would be off by about 1.4."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import fp4_attention_layer as layer  # noqa: E402


@pytest.mark.parametrize("fmt,flags", [(fp4.FORMAT_NVFP4, fp4.FOUR_OVER_SIX), (fp4.FORMAT_NVFP4, 0),
                                       (fp4.FORMAT_MXFP4, 0)])
@pytest.mark.parametrize("kw", [dict(lens=(300, 77, 1), chunk=100), dict(lens=(130,), chunk=130),
                                dict(lens=(65, 64), chunk=1, q_heads=4, kv_heads=4, dim=64, page=16)])
def test_layer(fmt, flags, kw):
    print("layer", fmt, flags, kw, flush=True)
    errors = layer.run(decode=4, hidden=256, fmt=fmt, flags=flags, **kw)
    assert max(errors) < 0.26, errors
