"""residual_norm and its gradient against 64 bits: with and without the block's
norm, every kind of gate, rows of one wave to sixteen, far values."""
import math

import pytest

import feedforward_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402

BF, F64 = torch.bfloat16, torch.float64
NAMES = ("x", "block", "weight", "block_weight", "gate")


def make(seed, tokens, dim, post, gate, size=1.0):
    g = torch.Generator().manual_seed(seed)
    new = lambda *s: torch.randn(*s, generator=g)
    d = dict(x=(4 * size * new(tokens, dim)).to(BF), block=(size * new(tokens, dim)).to(BF),
             weight=(1 + 0.2 * new(dim)).to(BF), block_weight=(1 + 0.2 * new(dim)).to(BF),
             gate=(0.5 + 0.3 * new(*((dim,) if gate == "channel" else (tokens, 1)))).to(BF))
    if not post:
        d["block_weight"] = None
    if gate == "none":
        d["gate"] = None
    return d, new(tokens, dim).to(BF), new(tokens, dim).to(BF)


def run(d, dy, dz, scale, eps):
    dev = {k: None if v is None else v.cuda() for k, v in d.items()}
    y, z = fp4.residual_norm(**dev, scale=scale, eps=eps)
    return (y, z) + fp4.residual_norm_backward(dy.cuda(), dz.cuda(), **dev, scale=scale, eps=eps)


def check(d, dy, dz, scale=0.9, eps=1e-6):
    tokens, dim = d["x"].shape
    y, z, dx, db, dbw, dw, dg = run(d, dy, dz, scale, eps)
    v = {k: None if t is None else t.double().requires_grad_() for k, t in d.items()}
    wy, wz = R.residual(scale=scale, eps=eps, **v)
    ((wy * dy.double()).sum() + (wz * dz.double()).sum()).backward()
    with torch.no_grad():
        # a mean of dim squares: its run of dim / 64 terms a lane at least, the joins, the
        # root and the products come to c u of the value
        c = (dim / 64 + 40) * R.U
        one = torch.ones((), dtype=F64)
        x, b = v["x"], v["block"]
        gate = one if v["gate"] is None else v["gate"]
        n, rb = b, one
        if v["block_weight"] is not None:
            rb = 1 / torch.sqrt(b.square().mean(-1, keepdim=True) + eps)
            n = b * rb * v["block_weight"]
        parts = (scale * x).abs() + (gate * n).abs()
        ey = c * parts
        R.close(y, wy, ey)
        r = 1 / torch.sqrt(wy.square().mean(-1, keepdim=True) + eps)
        # y's own error reaches z directly and through the mean of its square
        ez = v["weight"].abs() * r * (ey + wy.abs() * r * ey.square().mean(-1, keepdim=True).sqrt())
        ez = ez + c * wz.abs()
        R.close(z, wz, ez)
        if tokens == 0:
            return
        yh, u = wy * r, v["weight"] * dz.double()
        eh = (r * (ey + wy.abs() * r * ey.square().mean(-1, keepdim=True).sqrt())) + c * yh.abs()
        m = (u * yh).abs().mean(-1, keepdim=True)
        em = (u.abs() * eh).mean(-1, keepdim=True) + 2 * c * m
        ddy = dy.double() + r * (u - yh * (u * yh).mean(-1, keepdim=True))
        rel = r * (wy.abs() * r * r * ey).mean(-1, keepdim=True)          # of r itself
        e_dy = (r + rel) * (eh * m + yh.abs() * em) + (rel + 4 * c * r) * (u.abs() + yh.abs() * m)
        e_dy = e_dy + 4 * c * dy.double().abs()
        R.close(dx, v["x"].grad, abs(scale) * e_dy)
        w_b = one if v["block_weight"] is None else v["block_weight"]
        h, eh2 = gate * w_b * ddy, (gate * w_b).abs() * (e_dy + 4 * c * ddy.abs())
        bh = b * rb
        e_db = eh2
        if v["block_weight"] is not None:
            mean = (h * bh).abs().mean(-1, keepdim=True)
            e_mean = (eh2 * bh.abs()).mean(-1, keepdim=True) + 4 * c * mean
            e_db = rb * (eh2 + bh.abs() * e_mean) + 6 * c * rb * (h.abs() + bh.abs() * mean)
        R.close(db, v["block"].grad, e_db)
        # the tokens' sums: fp32 runs of tokens / 512 terms, joined in 64 bits
        run_ = (2 * tokens / 512 + 24) * R.U
        R.close(dw, v["weight"].grad, (dz.double().abs() * (eh + run_ * yh.abs())).sum(0))
        term = e_dy + (run_ + 4 * c) * ddy.abs()
        if v["block_weight"] is not None:
            R.close(dbw, v["block_weight"].grad, ((gate * bh).abs() * term).sum(0))
        else:
            assert dbw is None
        if v["gate"] is None:
            assert dg is None
        elif v["gate"].dim() == 1:
            R.close(dg, v["gate"].grad, (n.abs() * term).sum(0))
        else:
            R.close(dg, v["gate"].grad, (n.abs() * (term + 2 * c * ddy.abs())).sum(1, keepdim=True))


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("tokens,dim", [
    (1, 8), (2, 16), (7, 104), (5, 512), (9, 520), (6, 1024), (3, 1032), (33, 2048), (2, 2056),
    (5, 4096), (3, 4104), (2, 8192), (3, 8200), (2, 16384), (700, 256), (1100, 2056)])
def test_against_64_bits(post, gate, tokens, dim):
    check(*make(tokens + dim, tokens, dim, post, gate))


@pytest.mark.parametrize("size", [2.0 ** -70, 2.0 ** 70, 2.0 ** 100])
@pytest.mark.parametrize("dim", [64, 2048])
def test_far_values(size, dim):
    """Squares that leave the range of fp32."""
    d, dy, dz = make(3, 4, dim, True, "channel", size)
    d["x"][1] = 0
    d["block"][2] = 0
    y, z, dx, db, dbw, dw, dg = run(d, dy, dz, 1.0, 1e-30)
    v = {k: t.double().requires_grad_() for k, t in d.items()}
    wy, wz = R.residual(scale=1.0, eps=1e-30, **v)
    for got, want in ((y, wy), (z, wz)):
        assert ((got.double().cpu() - want).abs() <= 1.01 * 2.0 ** -8 * want.abs() + 2.0 ** -120).all()
    assert all(t.isfinite().all() for t in (dw, dbw))


def test_rows_of_zeros():
    d, dy, dz = make(1, 4, 128, True, "none")
    d["x"][:2] = 0
    d["block"][:2] = 0
    check(d, dy, dz)
    y, z = fp4.residual_norm(d["x"].cuda(), d["block"].cuda(), d["weight"].cuda(), eps=0.0)
    assert (y[:2] == 0).all() and z[:2].isnan().all() and z[2:].isfinite().all()


def test_values_that_are_not_finite():
    """They stay in their row."""
    d, dy, dz = make(1, 6, 2048, True, "channel")
    d["x"][1, 5] = math.nan
    d["block"][3, 7] = math.inf
    dev = {k: v.cuda() for k, v in d.items()}
    y, z = fp4.residual_norm(**dev)
    fine = [0, 2, 4, 5]
    assert y[fine].isfinite().all() and z[fine].isfinite().all()
    assert z[1].isnan().all() and y[1].isnan().sum() == 1 and not y[3].isfinite().all()


@pytest.mark.parametrize("tokens,dim", [(5, 96), (6, 1040), (4, 4096)])
def test_strides_and_places(tokens, dim):
    """Rows of wider tensors, and outputs in the inputs' own memory."""
    d, dy, dz = make(2, tokens, dim, True, "token")
    want = run(d, dy, dz, 0.9, 1e-6)
    dev = {k: v.cuda() for k, v in d.items()}

    def wide(t):
        w = torch.full((tokens, dim + 24), 5.0, dtype=BF, device="cuda")
        w[:, 8:8 + dim] = t
        return w, w[:, 8:8 + dim]
    (fx, x), (fb, b) = wide(dev["x"]), wide(dev["block"])
    (fy, gy), (fz, gz) = wide(dy.cuda()), wide(dz.cuda())
    rest = {k: dev[k] for k in ("weight", "block_weight", "gate")}
    got = fp4.residual_norm_backward(gy, gz, x, b, **rest, scale=0.9, out=(gy, gz))
    for g, w in zip(got, want[2:]):
        assert torch.equal(g, w)
    assert fp4.residual_norm(x, b, **rest, scale=0.9, out=(x, b))[0].data_ptr() == x.data_ptr()
    assert torch.equal(x, want[0]) and torch.equal(b, want[1])
    for f in (fx, fb, fy, fz):
        assert (f[:, :8] == 5).all() and (f[:, 8 + dim:] == 5).all()


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_autograd(post, gate):
    d, dy, dz = make(6, 9, 136, post, gate)
    dev = {k: None if v is None else v.cuda().requires_grad_() for k, v in d.items()}
    y, z = fp4.residual_norm(**dev, scale=0.7)
    torch.autograd.backward((y, z), (dy.cuda(), dz.cuda().t().contiguous().t()))
    dx, db, dbw, dw, dg = run(d, dy, dz, 0.7, 1e-6)[2:]
    for name, g in zip(NAMES, (dx, db, dw, dbw, dg)):
        if dev[name] is not None:
            assert torch.equal(dev[name].grad, g.to(BF)), name
    with pytest.raises(RuntimeError, match="out"):
        fp4.residual_norm(**dev, out=(y.detach(), z.detach()))


def test_gradient_against_differences():
    """Of the formula that the bounds above are taken from, in 64 bits."""
    d, dy, dz = make(6, 3, 24, True, "channel")
    v = {k: t.double() for k, t in d.items()}

    def f(w):
        y, z = R.residual(scale=0.9, eps=1e-6, **w)
        return float((y * dy.double()).sum() + (z * dz.double()).sum())
    got = dict(zip(("x", "block", "block_weight", "weight", "gate"), run(d, dy, dz, 0.9, 1e-6)[2:]))
    g = torch.Generator().manual_seed(1)
    for name in NAMES:
        way = torch.randn(v[name].shape, generator=g, dtype=F64)
        h = 1e-5
        slope = (f({**v, name: v[name] + h * way}) - f({**v, name: v[name] - h * way})) / (2 * h)
        mine = (got[name].double().cpu() * way)
        room = 2.0 ** -8 * float(mine.abs().sum()) + 1e-4
        assert abs(float(mine.sum()) - slope) <= room, name


def test_equal_calls_give_equal_bits():
    d, dy, dz = make(6, 1500, 1024, True, "channel")
    first = run(d, dy, dz, 0.9, 1e-6)
    for _ in range(3):
        for a, b in zip(run(d, dy, dz, 0.9, 1e-6), first):
            assert torch.equal(a, b)


def test_empty():
    d, dy, dz = make(6, 0, 64, True, "channel")
    y, z, dx, db, dbw, dw, dg = run(d, dy, dz, 0.9, 1e-6)
    assert y.shape == z.shape == dx.shape == db.shape == (0, 64)
    assert all((t == 0).all() and t.shape == (64,) for t in (dbw, dw, dg))
