"""Capped scores c tanh(s / c) over the whole range of caps, against 64-bit
attention on the same bytes.

Bounds as in test_gpu_kv_attention, but for the cap's own error, which follows
the score and not the cap.  In units u = 2^-24 and with t = s / c: where t is
small the cap is a polynomial of four terms, 4 u of its value for the
roundings and 1 u for the terms left out; elsewhere tanh t = 1 - 2 / (e + 1)
from an exponential and a reciprocal good to 2 u each is off by
(1 - tanh^2 t)(1 + t) u + 6 u / (e + 1) + u tanh t, 16 u of tanh t from
t = 0.3 on.  Caps up to 64 may take the latter form for every score, which
leaves an absolute error of 8 u c."""
import numpy as np
import pytest

import kv_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_kv_attention import MODES, U, build, run  # noqa: E402


def check_capped(mode, got, ref, ka, pt, lens, cu, qb, cap, window=0, scale=None):
    fmt, flags = MODES[mode]
    d = qb.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    cap = float(np.float32(cap))
    out, lse, size, mag = R.attention(ref, fmt, flags, ka, ka, R.bf16_values(qb), pt, lens, cu,
                                      scale, cap, window)
    n = max(lens)
    score = (d + 16) * U * mag + 8 * U * min(cap, 64.0)
    weight = 2.0 ** -11 if fmt == 0 else 2.0 ** -8
    o, l = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(out) + (weight + 2 * score[..., None] + (n + 16) * U) * size + 1e-30
    bad = np.argwhere(~(np.abs(o - out) <= tol))
    assert not len(bad), "out off at %d of %d, first %s: %r for %r (bound %r)" % (
        len(bad), o.size, bad[0], o[tuple(bad[0])], out[tuple(bad[0])], tol[tuple(bad[0])])
    bad = np.argwhere(~(np.abs(l - lse) <= score + (n + 16) * U + 4 * U * np.abs(lse)))
    assert not len(bad), "lse off at %d of %d, first %s: %r for %r" % (
        len(bad), l.size, bad[0], l[tuple(bad[0])], lse[tuple(bad[0])])


CAPS = [1e-45, 1e-39, 1e-20, 1e-3, 1.0, 30.0, 64.0, 65.0, 1e3, 1e4, 1e6, 1e8, 1e30, 3.4e38]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("new", [1, 5, 40])
@pytest.mark.parametrize("cap", CAPS)
def test_every_cap(mode, new, cap):
    """Scores of usual size under caps from the least to the largest number."""
    print("cap", mode, new, cap, flush=True)
    rng = np.random.default_rng(new)
    lens, news = [260, 77], [new, new]
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, 1, 4, 128, 32)
    got = run(mode, ref, ka, pt, lens, cu, qb, max_q=new, softcap=cap)
    check_capped(mode, got, ref, ka, pt, lens, cu, qb, cap)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("grp", [4, 20, 40])
@pytest.mark.parametrize("cap", [1e-39, 1e-3, 20.0, 64.0, 65.0, 200.0, 1e4, 1e9, 1e30])
@pytest.mark.parametrize("ratio", [1e-4, 0.05, 0.4, 3.0, 100.0])
def test_one_key(mode, grp, cap, ratio):
    """The log of a single exponential is the capped score itself: scores of
    about `ratio` caps, where the cap bends little, about as much as it can, and
    where nothing but the cap is left."""
    print("one key", mode, grp, cap, ratio, flush=True)
    rng = np.random.default_rng(grp)
    lens = [1] * 40
    ref, ka, pt, cu, qb = build(rng, mode, lens, lens, 1, grp, 64, 16)
    scale = ratio * cap / 8                    # |q k| is of the order of 8 here
    if not 0 < np.float32(scale) < 1e36:
        pytest.skip("the scale is no ordinary number")
    scale = float(np.float32(scale))
    got = run(mode, ref, ka, pt, lens, cu, qb, max_q=1, softcap=cap, scale=scale)
    check_capped(mode, got, ref, ka, pt, lens, cu, qb, cap, scale=scale)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("cap", CAPS)
def test_zero_scores(mode, new, cap):
    """Scores of zero stay zero under every cap: the plain mean of the values."""
    print("zero scores", mode, new, cap, flush=True)
    rng = np.random.default_rng(new + 2)
    lens, news = [90], [new]
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, 1, 4, 64, 16)
    qb[:, ::2] = 0
    got = run(mode, ref, ka, pt, lens, cu, qb, max_q=new, softcap=cap)
    check_capped(mode, got, ref, ka, pt, lens, cu, qb, cap)
