"""Plain 64-bit references of the feed-forward operators, with the bounds of
what fp32 sums and the stated roundings may change.

u = 2^-24 is half a step of fp32, relative to the value.  A sum of n terms in
fp32, in any order and with a rounding of at most a whole step at every addition
(the matrix instructions may cut off), is off by at most 2 n u sum |term|."""
import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}          # half a step
E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
NVFP4, MXFP4 = 0, 1
F64 = torch.float64


def weight_bytes(gen, lead, rows, cols, layout):
    """Random codes, scales and alpha of layout "tensor", "rows", "tiles" (NVFP4) or "mx"."""
    byte = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, dtype=torch.uint8)
    codes = byte(0, 256, *lead, rows, cols // 2)
    if layout == "mx":
        return dict(codes=codes, scales=byte(110, 130, *lead, rows, cols // 32), alpha=None, fmt=MXFP4)
    tall = 16 if layout == "tiles" else 1
    scales = byte(0, 0x7F, *lead, rows // tall, cols // 16)          # subnormals among them
    scales |= byte(0, 2, *scales.shape) << 7                        # the sign bit does not count
    alpha = torch.exp(torch.randn(lead + ((rows,) if layout == "rows" else ()) or (1,), generator=gen))
    return dict(codes=codes, scales=scales, alpha=alpha * 2e-3, fmt=NVFP4)


def values(w, layout):
    """The weights in 64 bits."""
    c = torch.stack((w["codes"] & 15, w["codes"] >> 4), -1).flatten(-2).long()
    v = torch.tensor(E2M1 + [-x for x in E2M1], dtype=F64)[c]
    b = w["scales"].long()
    if layout == "mx":
        return v * torch.ldexp(torch.ones((), dtype=F64), b - 127).repeat_interleave(32, -1)
    b = b & 127
    s = torch.where(b >> 3 > 0, torch.ldexp(8.0 + (b & 7).double(), (b >> 3) - 10), (b & 7) / 512.0)
    s = s.repeat_interleave(16, -1)
    if layout == "tiles":
        s = s.repeat_interleave(16, -2)
    a = w["alpha"].double().reshape(w["codes"].shape[:-2] + (-1, 1))
    return v * s * a


def linear(x, w):
    """x @ w.T and the bound of its error before the output's rounding."""
    x, n = x.double(), x.shape[-1]
    return x @ w.T, 2 * (n + 2) * U * (x.abs() @ w.abs().T)


def experts(x, gate_up, down, weights, ids):
    """The routed experts' sum and its bound (before the output's rounding)."""
    x, t, f = x.double(), x.shape[0], down.shape[-1]
    out = torch.zeros(x.shape, dtype=F64)
    err = torch.zeros(x.shape, dtype=F64)
    for e in range(gate_up.shape[0]):
        tok, place = torch.nonzero(ids == e, as_tuple=True)
        if not len(tok):
            continue
        y, dy = linear(x[tok], gate_up[e])
        g, u = y[:, :f], y[:, f:]
        dg, du = dy[:, :f], dy[:, f:]
        s = g * torch.sigmoid(g)
        h = s * u
        # silu's slope is below 1.1; 8 u for exp, division and products
        dh = 1.1 * dg * (u.abs() + du) + s.abs() * du + 8 * U * h.abs()
        dh += 2.0 ** -8 * (h.abs() + dh)                       # h is rounded to bf16
        d = down[e]
        o = h @ d.T
        do = dh @ d.abs().T + 2 * (f + 2) * U * ((h.abs() + dh) @ d.abs().T)
        c = weights[tok, place].double()[:, None]
        out.index_add_(0, tok, c * o)
        err.index_add_(0, tok, c.abs() * (do + (ids.shape[1] + 2) * 2 * U * (o.abs() + do)))
    return out, err


def close(got, want, err):
    """got (bf16 or fp32) within the bound and the output's rounding of want, everywhere."""
    half = HALF[got.dtype]
    got = got.double().cpu()
    room = err * (1 + half) + half * want.abs() + 2.0 ** -133
    off = (got - want).abs()
    bad = ~(off <= room)
    assert not bad.any(), "%d of %d outside, worst %.3g of its room" % (
        int(bad.sum()), bad.numel(), float((off / room).nan_to_num(math.inf).max()))


def scores(case, x):
    """Scores of logits x [experts] (floats)."""
    if case["scores"] == "sigmoid":
        return [0.0 if v == -math.inf else 1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 for v in x]
    m = max(x)
    if m == -math.inf:
        return [0.0] * len(x)
    e = [math.exp(v - m) if v - m > -745 else 0.0 for v in x]
    t = math.fsum(e)
    return [v / t for v in e]


def route(case, logits, bias):
    """(weights, experts) as lists, token by token, from the definition."""
    out_w, out_e = [], []
    for x in logits.double().tolist():
        s = scores(case, x)
        n = len(x)
        c = [s[i] + bias[i] if bias is not None else x[i] for i in range(n)]
        open_ = [i for i in range(n) if x[i] > -math.inf and c[i] > -math.inf]
        g = case["groups"]
        if case["top_groups"] < g:
            per, sizes = n // g, []
            for j in range(g):
                mine = [i for i in open_ if i // per == j]
                if not mine:
                    continue
                if case["group_top"] == 1:
                    size = max(c[i] for i in mine)
                else:
                    by = sorted((c[i] if bias is not None else s[i] for i in mine), reverse=True)
                    size = sum(by[:2])
                sizes.append((-size, j))
            kept = {j for _, j in sorted(sizes)[:case["top_groups"]]}
            open_ = [i for i in open_ if i // per in kept]
        ids = sorted(open_, key=lambda i: (-c[i], i))[:case["top_k"]]
        w = [s[i] for i in ids]
        if case["renormalize"]:
            t = math.fsum(w)
            w = [v / t if t > 0 else 0.0 for v in w]
        pad = case["top_k"] - len(ids)
        out_w.append([case["scale"] * v for v in w] + [0.0] * pad)
        out_e.append(ids + [-1] * pad)
    return torch.tensor(out_w, dtype=F64), torch.tensor(out_e, dtype=torch.int32)


def route_weights(case, logits, ids):
    """Weights of given experts in 64 bits, by torch, differentiable in the logits."""
    open_ = logits > -math.inf
    z = torch.where(open_, logits, -1e300)
    s = torch.sigmoid(z) if case["scores"] == "sigmoid" else torch.softmax(z, 1)
    s = torch.where(open_, s, 0.0)
    there = (ids >= 0) & (ids < logits.shape[1])
    w = torch.where(there, s.gather(1, torch.where(there, ids, 0).long()), 0.0)
    if case["renormalize"]:
        t = w.sum(1, keepdim=True)
        w = w / torch.where(t > 0, t, 1.0)
    return case["scale"] * w


def residual(x, block, weight, block_weight, gate, scale, eps):
    """(y, z) in 64 bits, by torch."""
    def normed(v, w):
        return v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps) * w
    n = block if block_weight is None else normed(block, block_weight)
    y = scale * x + (n if gate is None else gate * n)
    return y, normed(y, weight)
