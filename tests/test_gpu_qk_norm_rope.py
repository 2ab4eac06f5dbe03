"""Norm of queries and keys with the rotation, and its gradient, against the
64-bit formulas and against differences.

Bounds: one rounding to bf16 (2^-8 relative); before it fp32 arithmetic, at
most 32 roundings of terms no larger than the vector's (|x| r |w| for the
output; r (|w g| + |n| mean|w g n|) for dx).  A weight gradient is a sum of
fp32 terms of either sign: N terms in short fp32 runs, then 64 bits, bounded
by 64 u sum |g n| (a lane's run has at most 64 terms at these sizes)."""
import numpy as np
import pytest

import kv_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402

U = 2.0 ** -24
EPS = 1e-6


def tensor(b):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).cuda().view(torch.bfloat16)


def make(rng, t, hq, hk, d, rot, size=1.0):
    q, k = (R.bf16_bits(size * rng.standard_normal((t, h, d)) *
                        np.exp(0.5 * rng.standard_normal((t, h, 1)))) for h in (hq, hk))
    qw, kw = (R.bf16_bits(1 + 0.2 * rng.standard_normal(d)) for _ in range(2))
    dq, dk = (R.bf16_bits(rng.standard_normal((t, h, d))) for h in (hq, hk))
    rows = 5000
    table = fp4.rope_table(rows, rot)
    pos = rng.integers(0, rows, t).astype(np.int64)
    return q, k, qw, kw, dq, dk, table, pos


def pair_size(x, rot, inter):
    """Sum of the magnitudes of each pair: the size of the terms that a rotation adds."""
    a = np.abs(x)
    out = a.copy()
    if inter:
        s = a[..., 0:rot:2] + a[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = s, s
    else:
        s = a[..., :rot // 2] + a[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = s, s
    return out


def near(got, want, size, what, extra=32):
    g = got.double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(want) + extra * U * size + 1e-38
    bad = np.argwhere(~(np.abs(g - want) <= tol))
    assert not len(bad), "%s off at %d of %d, first %s: %r for %r" % (
        what, len(bad), g.size, bad[0], g[tuple(bad[0])], want[tuple(bad[0])])


CASES = [  # tokens, q heads, k heads, dim, rot
    (1, 1, 1, 64, 64), (3, 4, 1, 128, 128), (17, 5, 3, 128, 64), (33, 2, 2, 256, 256),
    (130, 7, 1, 64, 32), (9, 3, 2, 96, 96), (40, 1, 1, 80, 16), (25, 2, 1, 72, 32),
    (500, 8, 2, 128, 128), (6, 1, 1, 16, 16), (21, 2, 2, 128, 0), (700, 32, 8, 64, 64),
]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("normed", ["both", "queries", "none"])
@pytest.mark.parametrize("t,hq,hk,d,rot", CASES)
def test_forward_and_backward(inter, normed, t, hq, hk, d, rot):
    print("norm rope", inter, normed, t, hq, hk, d, rot, flush=True)
    rng = np.random.default_rng(t + d)
    q, k, qw, kw, dq, dk, table, pos = make(rng, t, hq, hk, d, rot)
    tqw = tensor(qw) if normed != "none" else None
    tkw = tensor(kw) if normed == "both" else None
    a = (tqw, tkw, torch.from_numpy(pos).cuda(), table)
    yq, yk = fp4.qk_norm_rope(tensor(q), tensor(k), *a, eps=EPS, interleaved=inter)
    grads = fp4.qk_norm_rope_backward(tensor(dq), tensor(dk), tensor(q), tensor(k), *a, eps=EPS,
                                      interleaved=inter)
    torch.cuda.synchronize()
    cs = table.double().cpu().numpy()[pos]
    for x, w, on, dy, y, dx, dw, what in ((q, qw, tqw, dq, yq, grads[0], grads[2], "q"),
                                          (k, kw, tkw, dk, yk, grads[1], grads[3], "k")):
        x, dy = R.bf16_values(x), R.bf16_values(dy)
        w = None if on is None else R.bf16_values(w)
        plain = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * w
        near(y, R.norm_rope(x, w, cs, rot, inter, EPS), pair_size(plain, rot, inter), "y " + what)
        want, want_w = R.norm_rope_backward(dy, x, w, cs, rot, inter, EPS)
        g = pair_size(dy, rot, inter)
        if w is None:
            near(dx, want, g, "dx " + what)
            assert dw is None
            continue
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
        n = np.abs(x) * r
        gw = g * np.abs(w)
        near(dx, want, r * (gw + n * (gw * n).mean(-1, keepdims=True)), "dx " + what)
        off = np.abs(dw.double().cpu().numpy() - want_w)
        assert (off <= 64 * U * (g * n).sum((0, 1)) + 1e-30).all(), "dw " + what


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_differences(inter):
    """<grad, e> equals the difference quotient of <dy, y> in 64 bits along
    random directions, up to the gradient's roundings."""
    rng = np.random.default_rng(31)
    t, hq, hk, d, rot = 6, 3, 2, 64, 32
    q, k, qw, kw, dq, dk, table, pos = make(rng, t, hq, hk, d, rot)
    got = fp4.qk_norm_rope_backward(tensor(dq), tensor(dk), tensor(q), tensor(k), tensor(qw),
                                    tensor(kw), torch.from_numpy(pos).cuda(), table, eps=EPS,
                                    interleaved=inter)
    cs = table.double().cpu().numpy()[pos]
    for x, w, dy, dx, dw in ((q, qw, dq, got[0], got[2]), (k, kw, dk, got[1], got[3])):
        x, w, dy = R.bf16_values(x), R.bf16_values(w), R.bf16_values(dy)
        f = lambda x, w: (dy * R.norm_rope(x, w, cs, rot, inter, EPS)).sum()
        h = 1e-5
        for _ in range(4):
            e = rng.standard_normal(x.shape)
            diff = (f(x + h * e, w) - f(x - h * e, w)) / (2 * h)
            dxn = dx.double().cpu().numpy()
            assert abs((dxn * e).sum() - diff) <= 2.0 ** -8 * np.abs(dxn * e).sum() + 1e-5
            e = rng.standard_normal(w.shape)
            diff = (f(x, w + h * e) - f(x, w - h * e)) / (2 * h)
            dwn = dw.double().cpu().numpy()
            assert abs((dwn * e).sum() - diff) <= 1e-4 * np.abs(dwn * e).sum() + 1e-5


def test_strided_in_place_and_far_positions():
    """Slices of a fused projection, rotated in place; positions outside the
    table take its nearest row."""
    rng = np.random.default_rng(7)
    t, hq, hk, d, rot = 50, 4, 2, 128, 128
    q, k, qw, kw, _, _, table, pos = make(rng, t, hq, hk, d, rot)
    x = torch.zeros(t, hq + 2 * hk, d, dtype=torch.bfloat16, device="cuda")
    x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:] = tensor(q), tensor(k), 5.0
    pos[:3] = [-4, 1 << 40, 5000]
    a = (tensor(qw), tensor(kw), torch.from_numpy(pos).cuda(), table)
    qs, ks = x[:, :hq], x[:, hq:hq + hk]
    fp4.qk_norm_rope(qs, ks, *a, eps=EPS, out=(qs, ks))
    fresh = fp4.qk_norm_rope(tensor(q), tensor(k), tensor(qw), tensor(kw),
                             torch.from_numpy(np.clip(pos, 0, 4999)).cuda(), table, eps=EPS)
    torch.cuda.synchronize()
    assert torch.equal(qs, fresh[0]) and torch.equal(ks, fresh[1])
    assert (x[:, hq + hk:] == 5).all()


def test_special_rows():
    """Zero rows stay zero; a row of Inf or NaN leaves the others alone; rows
    of extreme size are normed."""
    rng = np.random.default_rng(17)
    t, d = 12, 128
    q, k, qw, kw, dq, dk, table, pos = make(rng, t, 2, 1, d, d)
    a = lambda: (tensor(qw), tensor(kw), torch.from_numpy(pos).cuda(), table)
    base = fp4.qk_norm_rope(tensor(q), tensor(k), *a(), eps=EPS)
    q2 = q.copy()
    q2[0], q2[1, 0], q2[2, 1, 5], q2[3, 0, 9] = 0, 0x8000, 0x7F80, 0x7FC0
    got = fp4.qk_norm_rope(tensor(q2), tensor(k), *a(), eps=EPS)
    torch.cuda.synchronize()
    assert (got[0][0] == 0).all() and (got[0][1, 0] == 0).all()
    assert torch.equal(got[0][4:], base[0][4:]) and torch.equal(got[1], base[1])
    assert torch.equal(got[0][2, 0], base[0][2, 0]) and torch.equal(got[0][3, 1], base[0][3, 1])
    big = R.bf16_bits(R.bf16_values(q) * 2.0 ** 50)
    cs = table.double().cpu().numpy()[pos]
    y = fp4.qk_norm_rope(tensor(big), tensor(k), *a(), eps=EPS)[0]
    x, w = R.bf16_values(big), R.bf16_values(qw)
    plain = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * w
    near(y, R.norm_rope(x, w, cs, d, False, EPS), pair_size(plain, d, False), "large rows")


def test_no_tokens_and_same_bits_in_a_graph():
    rng = np.random.default_rng(23)
    q, k, qw, kw, dq, dk, table, pos = make(rng, 200, 4, 2, 128, 128)
    w = (tensor(qw), tensor(kw))
    none = fp4.qk_norm_rope_backward(tensor(dq[:0]), tensor(dk[:0]), tensor(q[:0]), tensor(k[:0]),
                                     *w, torch.from_numpy(pos[:0]).cuda(), table)
    assert none[0].shape == (0, 4, 128) and not none[2].any() and not none[3].any()
    tq, tk, tdq, tdk = tensor(q), tensor(k), tensor(dq), tensor(dk)
    p = torch.from_numpy(pos).cuda()

    def both():
        y = fp4.qk_norm_rope(tq, tk, *w, p, table)
        return y + fp4.qk_norm_rope_backward(tdq, tdk, tq, tk, *w, p, table)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = both()
    for i in range(3):
        tq.copy_(tensor(q) * (i + 1))
        want = both()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(held, want):
            assert torch.equal(x, y), i
