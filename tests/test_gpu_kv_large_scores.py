"""Scores far past the usual sizes, up to the end of fp32: finite, and keys of
equal score share the weight evenly.

All keys of the context are the same, so all scores of a row are the same
number whatever their rounding, and the output is the mean of the values: its
bound is that of test_gpu_kv_attention without the scores' part.  The log of
the sum is off by the scores' rounding, D u sum |q k| scale, and 4 u of itself."""
import numpy as np
import pytest

import kv_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_kv_attention import MODES, U, build, run  # noqa: E402


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,grp,n", [(1, 4, 70), (5, 5, 70), (30, 4, 70), (1, 4, 3000), (40, 4, 3000)])
@pytest.mark.parametrize("size", [1e3, 1e6, 3e7, 1e9, 1e15, 1e30])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_equal_scores_of_any_size(mode, d, new, grp, n, size, sign):
    print("large scores", mode, d, new, grp, n, size, sign, flush=True)
    fmt, flags = MODES[mode]
    rng = np.random.default_rng(new + d)
    ref, ka, pt, cu, qb = build(rng, mode, [n], [new], 1, grp, d, 64)
    kb = R.bf16_bits(np.repeat(rng.standard_normal((1, 1, d)), n, 0))
    vb = R.bf16_bits(rng.standard_normal((n, 1, d)))
    j = np.arange(n)
    ka = np.array([4.0], np.float32)
    R.write(ref, fmt, flags, kb, vb, pt[0][j // 64].astype(np.int64) * 64 + j % 64, ka, ka)
    scale = float(np.float32(sign * size))
    got = run(mode, ref, ka, pt, [n], cu, qb, max_q=new, scale=scale)
    out, lse, mean, mag = R.attention(ref, fmt, flags, ka, ka, R.bf16_values(qb), pt, [n], cu, scale,
                                      0.0, 0)
    weight = 2.0 ** -11 if fmt == 0 else 2.0 ** -8
    o, l = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(out) + (weight + (n + 16) * U) * mean + 1e-30
    assert (np.abs(o - out) <= tol).all(), (np.abs(o - out) / tol).max()
    assert (np.abs(l - lse) <= d * U * np.abs(mag) + (n + 16) * U + 4 * U * np.abs(lse)).all()
