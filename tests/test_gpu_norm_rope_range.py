"""Norm with rotation over the whole range of bf16: rows whose squares leave the
range of fp32.  Bounds as in test_gpu_qk_norm_rope, and the factor 1 / rms may be
a subnormal with 21 bits: 2^-21 more of each term.  A gradient below 2^-126 is a
subnormal, whose rounding is 2^-134 at most."""
import numpy as np
import pytest

import kv_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_qk_norm_rope import U, make, pair_size, tensor  # noqa: E402


def near(got, want, size, what):
    g = got.double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(want) + (40 * U + 2.0 ** -21) * size + 2.0 ** -133
    bad = np.argwhere(~(np.abs(g - want) <= tol))
    assert not len(bad), "%s off at %d of %d, first %s: %r for %r" % (
        what, len(bad), g.size, bad[0], g[tuple(bad[0])], want[tuple(bad[0])])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 32), (16, 16), (256, 256), (96, 96)])
@pytest.mark.parametrize("power,eps", [(62, 1e-6), (64, 1e-6), (90, 1e-6), (124, 1e-6), (64, 0.0), (124, 0.0),
                                       (-55, 0.0), (-66, 0.0), (-80, 0.0), (-110, 0.0), (-70, 1e-40),
                                       (-40, 1e-30)])
def test_sizes(inter, d, rot, power, eps):
    print("norm rope range", inter, d, rot, power, eps, flush=True)
    rng = np.random.default_rng(abs(power) + d)
    t, hq, hk = 19, 3, 2
    q, k, qw, kw, dq, dk, table, pos = make(rng, t, hq, hk, d, rot)
    shrink = lambda b: R.bf16_bits(np.clip(R.bf16_values(b), -8, 8) * 2.0 ** power)
    q[::2], k[::3] = shrink(q[::2]), shrink(k[::3])          # usual rows between them
    if eps == 0.0:
        q[np.abs(R.bf16_values(q)) == 0], k[np.abs(R.bf16_values(k)) == 0] = 1, 1
    a = (tensor(qw), tensor(kw), torch.from_numpy(pos).cuda(), table)
    yq, yk = fp4.qk_norm_rope(tensor(q), tensor(k), *a, eps=eps, interleaved=inter)
    grads = fp4.qk_norm_rope_backward(tensor(dq), tensor(dk), tensor(q), tensor(k), *a, eps=eps,
                                      interleaved=inter)
    torch.cuda.synchronize()
    cs = table.double().cpu().numpy()[pos]
    eps = float(np.float32(eps))
    for x, w, dy, y, dx, dw, what in ((q, qw, dq, yq, grads[0], grads[2], "q"),
                                      (k, kw, dk, yk, grads[1], grads[3], "k")):
        x, dy, w = R.bf16_values(x), R.bf16_values(dy), R.bf16_values(w)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        near(y, R.norm_rope(x, w, cs, rot, inter, eps), pair_size(x * r * w, rot, inter), "y " + what)
        want, want_w = R.norm_rope_backward(dy, x, w, cs, rot, inter, eps)
        g, n = pair_size(dy, rot, inter), np.abs(x) * r
        gw = g * np.abs(w)
        near(dx, want, r * (gw + n * (gw * n).mean(-1, keepdims=True)), "dx " + what)
        off = np.abs(dw.double().cpu().numpy() - want_w)
        assert (off <= (64 * U + 2.0 ** -21) * (g * n).sum((0, 1)) + 1e-30).all(), "dw " + what
