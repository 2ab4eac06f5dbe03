"""Cases of the feed-forward operators of a model whose weights are held in
block-scaled FP4.

The operators: the product of activations with FP4 weights, routing to experts
(forward and backward), the routed experts' gated products with FP4 weights,
and the norms around a block with its gate and residual scale (forward and
backward).  ``run`` computes each in plain torch (``own`` false) or through
``block_scaled_fp4_reduce_amd`` (``own`` true) on the same state.

Weights [rows][cols], G values per scale (16 for NVFP4, 32 for MXFP4):
  codes  [rows][cols/2]   two codes per byte, the even value in the low nibble
  scales [rows][cols/G]   E4M3 or UE8M0 bytes; NVFP4 in 16x16 tiles: [rows/16][cols/16]
  alpha  NVFP4 only: a float for the tensor, or one for every row
and with experts all of these once more in front.
"""
import math

import torch

own = False

NVFP4, MXFP4 = 0, 1
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _linear(name, tokens, rows, cols, fmt, layout, f32):
    """layout of the weights: "tensor" or "rows" (one alpha, one a row), "tiles" (16x16)."""
    return dict(name=name, op="linear", tokens=tokens, rows=rows, cols=cols, fmt=fmt,
                layout=layout, f32=f32)


def _route(name, tokens, experts, top_k, scores, bias, groups, top_groups, group_top, renormalize,
           scale, bf16, masked, train):
    return dict(name=name, op="route", tokens=tokens, experts=experts, top_k=top_k, scores=scores,
                bias=bias, groups=groups, top_groups=top_groups, group_top=group_top,
                renormalize=renormalize, scale=scale, bf16=bf16, masked=masked, train=train)


def _experts(name, tokens, experts, top_k, hidden, inner, fmt, layout, padded):
    return dict(name=name, op="experts", tokens=tokens, experts=experts, top_k=top_k,
                hidden=hidden, inner=inner, fmt=fmt, layout=layout, padded=padded)


def _norm(name, tokens, dim, post, gate, scale, train):
    return dict(name=name, op="norm", tokens=tokens, dim=dim, post=post, gate=gate, scale=scale,
                train=train)


def listed():
    return [
        # one token through a square projection: the smallest call, latency counts
        _linear("linear_decode_one", 1, 4096, 4096, NVFP4, "tensor", False),
        # a decoding batch through a feed-forward projection, power-of-two scales
        _linear("linear_decode_batch", 48, 14336, 4096, MXFP4, "tensor", False),
        # odd sizes, an alpha for every row, scores in float32 as a head gives them
        _linear("linear_ragged", 333, 1001, 2080, NVFP4, "rows", True),
        # a prompt through a feed-forward projection, weights in 16x16 tiles
        _linear("linear_prompt", 8192, 14336, 4096, NVFP4, "tiles", False),
        # one decoding step of a small batch
        _route("route_decode", 32, 128, 8, "softmax", False, 1, 1, 1, True, 1.0, False, False,
               False),
        # odd counts, bf16 scores, some experts masked; forward and backward
        _route("route_ragged", 1021, 60, 4, "softmax", False, 1, 1, 1, False, 1.0, True, True,
               True),
        # a training batch: sigmoid scores, balancing bias, groups; forward and backward
        _route("route_train", 16384, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, False, False,
               True),
        # one token through its experts
        _experts("experts_decode_one", 1, 64, 6, 2048, 1408, NVFP4, "tensor", False),
        # a decoding batch that wakes nearly every expert, a few tokens each
        _experts("experts_decode_batch", 64, 128, 8, 4096, 1024, MXFP4, "tensor", False),
        # a prompt, padded: the last tokens have no expert
        _experts("experts_prompt", 4096, 64, 6, 2048, 1408, NVFP4, "rows", True),
        # one decoding step: residual sum and the next block's norm
        _norm("norm_decode", 32, 4096, False, "none", 1.0, False),
        # a training step: norms on both sides, a gate for every channel; forward and backward
        _norm("norm_train", 8192, 4096, True, "channel", 0.9, True),
    ]


def _span(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(["linear", "linear", "route", "experts", "experts", "norm"])
    fmt = rng.choice([NVFP4, MXFP4])
    layout = rng.choice(["tensor", "rows"]) if fmt == NVFP4 else "tensor"
    if op == "linear":
        cols, rows = 32 * _span(rng, 2, 448), _span(rng, 16, 14336)
        if fmt == NVFP4 and rows % 16 == 0 and rng.random() < 0.5:
            layout = "tiles"
        tokens = _span(rng, 1, max(1, min(8192, 8192 * 14336 * 4096 // (rows * cols))))
        return _linear("", tokens, rows, cols, fmt, layout, rng.random() < 0.3)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _span(rng, max(1, 8 // groups), 256 // groups)
        top_groups = rng.randint(1, groups)
        most = min(8, experts // groups * top_groups)
        scores = rng.choice(["softmax", "sigmoid"])
        return _route("", _span(rng, 1, 16384), experts, rng.randint(1, most), scores,
                      rng.random() < 0.5, groups, top_groups, rng.choice([1, 2]),
                      rng.random() < 0.6, rng.choice([1.0, 2.5]), rng.random() < 0.3,
                      rng.random() < 0.3, rng.random() < 0.5)
    if op == "experts":
        experts = _span(rng, 4, 128)
        hidden = 32 * _span(rng, 8, 128)
        inner = 32 * _span(rng, 4, min(64, 4096 * 1024 // (32 * hidden)))
        top_k = rng.randint(1, min(8, experts))
        tokens = _span(rng, 1, min(4096, 4096 * 6 * 2048 * 1408 // (top_k * hidden * inner)))
        return _experts("", tokens, experts, top_k, hidden, inner, fmt, layout,
                        rng.random() < 0.4)
    dim = 8 * _span(rng, 16, 1024)
    tokens = _span(rng, 1, min(8192, 8192 * 4096 // dim))
    return _norm("", tokens, dim, rng.random() < 0.6, rng.choice(["none", "channel", "token"]),
                 rng.choice([1.0, 0.9]), rng.random() < 0.6)


# ------------------------------------------------------------------ inputs
def _group(fmt):
    return 16 if fmt == NVFP4 else 32


def _weights(gen, lead, rows, cols, fmt, layout):
    """FP4 weights of normal values: blocks drawn from a store of quantized ones."""
    dev = "cuda"
    g = _group(fmt)
    tall = 16 if layout == "tiles" else 1
    store = 4096 if tall == 16 else 32768
    y = torch.randn(store, tall, g, generator=gen, device=dev)
    top = y.abs().amax((1, 2), keepdim=True)
    if fmt == MXFP4:                                   # values scaled to the size of 1/sqrt(cols)
        e = torch.floor(torch.log2(top)) - 2
        t = y * torch.exp2(-e)
        byte = (e + 127 - round(math.log2(cols) / 2)).to(torch.uint8)
    else:                                              # a tensor's maximum at 5 and 4/6's constant
        byte = (top * (256.0 / 5.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        t = y / (byte.float() * (5.0 / (6 * 256.0)))
        byte = byte.view(torch.uint8)
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
    m = torch.bucketize(t.abs().contiguous(), edge).to(torch.uint8)
    c = m | (torch.signbit(t).to(torch.uint8) << 3)
    c = c[..., 0::2] | (c[..., 1::2] << 4)             # [store][tall][g/2]
    at = torch.randint(0, store, lead + (rows // tall, cols // g), generator=gen, device=dev)
    codes = c[at]                                      # [...][rows/tall][cols/g][tall][g/2]
    codes = codes.transpose(-3, -2).reshape(lead + (rows, cols // 2)).contiguous()
    scales = byte[:, 0, 0][at].contiguous()
    alpha = None
    if fmt == NVFP4:
        size = 5.0 / (6 * 256.0) / math.sqrt(cols)
        shape = lead + ((rows,) if layout == "rows" else ())
        alpha = size * torch.exp(0.2 * torch.randn(shape or (1,), generator=gen, device=dev))
    return {"codes": codes, "scales": scales, "alpha": alpha}


def _activations(gen, tokens, cols):
    """Rows as a model makes them: channels of unequal size, heavy tails."""
    dev = "cuda"
    x = torch.randn(tokens, cols, generator=gen, device=dev)
    x *= torch.exp(0.5 * torch.randn(cols, generator=gen, device=dev))
    x *= torch.exp(0.3 * torch.randn(tokens, 1, generator=gen, device=dev))
    return x.to(torch.bfloat16)


def _real_tokens(case):
    """Tokens of a batch before its padding."""
    return case["tokens"] - case["tokens"] // 8 if case["padded"] else case["tokens"]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 2 + 1)
    st = {"case": case}
    t = case["tokens"]
    if case["op"] == "linear":
        st["w"] = _weights(gen, (), case["rows"], case["cols"], case["fmt"], case["layout"])
        st["x"] = _activations(gen, t, case["cols"])
    elif case["op"] == "route":
        e = case["experts"]
        logits = torch.randn(t, e, generator=gen, device=dev)
        logits += 0.5 * torch.randn(e, generator=gen, device=dev)
        if case["masked"]:                             # experts that a token may not use
            hide = torch.rand(t, e, generator=gen, device=dev) < 0.1
            logits = logits.masked_fill(hide, -math.inf)
        st["logits"] = logits.bfloat16() if case["bf16"] else logits
        st["bias"] = 0.1 * torch.randn(e, generator=gen, device=dev) if case["bias"] else None
        if case["train"]:
            st["dweights"] = torch.randn(t, case["top_k"], generator=gen, device=dev)
    elif case["op"] == "experts":
        e, d, f = case["experts"], case["hidden"], case["inner"]
        st["gate_up"] = _weights(gen, (e,), 2 * f, d, case["fmt"], case["layout"])
        st["down"] = _weights(gen, (e,), d, f, case["fmt"], case["layout"])
        st["x"] = _activations(gen, t, d)
        logits = torch.randn(t, e, generator=gen, device=dev)
        logits += 0.5 * torch.randn(e, generator=gen, device=dev)    # some experts are liked more
        top, ids = torch.topk(logits, case["top_k"], dim=1)
        ids[_real_tokens(case):] = -1
        st["experts"] = ids.int()
        st["weights"] = torch.softmax(top, 1)
        # tokens of the busiest expert, which sizes the plain form's padded batch
        st["most"] = int(torch.bincount(ids[ids >= 0], minlength=e).max())
    else:
        d = case["dim"]
        size = torch.exp(0.5 * torch.randn(d, generator=gen, device=dev))
        st["x"] = (4.0 * size * torch.randn(t, d, generator=gen, device=dev)).bfloat16()
        st["block"] = _activations(gen, t, d)
        w = 1.0 + 0.2 * torch.randn(2, d, generator=gen, device=dev)
        st["block_weight"] = w[0].bfloat16() if case["post"] else None
        st["weight"] = w[1].bfloat16()
        gate = {"none": None, "channel": (d,), "token": (t, 1)}[case["gate"]]
        st["gate"] = None if gate is None else (
            0.5 + 0.3 * torch.randn(gate, generator=gen, device=dev)).bfloat16()
        if case["train"]:
            st["dy"] = torch.randn(t, d, generator=gen, device=dev).bfloat16()
            st["dz"] = torch.randn(t, d, generator=gen, device=dev).bfloat16()
    return st


# ------------------------------------------------------------------ plain forms
def _values(w, fmt, layout):
    """float32 values [...][rows][cols] of FP4 weights."""
    codes, byte = w["codes"], w["scales"]
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    q = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), -1).flatten(-2)
    if fmt == MXFP4:
        s = (byte.int() << 23).view(torch.float32)
    else:
        alpha = w["alpha"].reshape(codes.shape[:-2] + (-1, 1))
        s = alpha * byte.view(torch.float8_e4m3fn).float()
    if layout == "tiles":
        s = s.repeat_interleave(16, -2)
    return q.unflatten(-1, (-1, _group(fmt))).mul_(s[..., None]).flatten(-2)


def _linear_plain(st):
    case = st["case"]
    y = st["x"].float() @ _values(st["w"], case["fmt"], case["layout"]).T
    return y if case["f32"] else y.bfloat16()


def _scores64(case, logits):
    x = logits.double()
    if case["scores"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0)


def _route_plain(st):
    """(weights, experts): 64 bits, since two scores next to each other decide the choice."""
    case, x = st["case"], st["logits"].double()
    s = _scores64(case, st["logits"])
    c = s + st["bias"].double() if case["bias"] else x
    c = c.masked_fill(x == -math.inf, -math.inf)
    if case["groups"] > 1:
        by = c if case["bias"] or case["group_top"] == 1 else s.masked_fill(x == -math.inf, -math.inf)
        by = by.unflatten(1, (case["groups"], -1))
        best = by.sort(-1, descending=True).values[..., :case["group_top"]]
        size = torch.where(best == -math.inf, 0.0, best).sum(-1)
        size = size.masked_fill(best[..., 0] == -math.inf, -math.inf)
        order = size.sort(stable=True, dim=-1, descending=True).indices
        kept = torch.zeros_like(size, dtype=torch.bool).scatter_(
            1, order[:, :case["top_groups"]], True)
        c = c.masked_fill(~kept.repeat_interleave(by.shape[-1], 1), -math.inf)
    top = c.sort(stable=True, dim=-1, descending=True)
    there = top.values[:, :case["top_k"]] > -math.inf
    ids = top.indices[:, :case["top_k"]]
    w = torch.where(there, s.gather(1, ids), 0.0)
    if case["renormalize"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return (case["scale"] * w).float(), torch.where(there, ids, -1).int()


def _route_plain_backward(st, ids):
    case = st["case"]
    there = ids >= 0
    at = ids.clamp(min=0).long()
    g = torch.where(there, st["dweights"].double(), 0.0)
    s = _scores64(case, st["logits"])
    p = torch.where(there, s.gather(1, at), 0.0)
    if case["renormalize"]:
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
        d = p * (g - (p * g).sum(-1, keepdim=True))
        if case["scores"] == "sigmoid":
            d = d * (1.0 - s.gather(1, at))
        dense = torch.zeros_like(s).scatter_add_(1, at, d)
    elif case["scores"] == "sigmoid":
        dense = torch.zeros_like(s).scatter_add_(1, at, g * p * (1.0 - p))
    else:
        dense = torch.zeros_like(s).scatter_add_(1, at, g)
        dense = s * (dense - (p * g).sum(-1, keepdim=True))
    return (case["scale"] * dense).to(st["logits"].dtype)


def _experts_plain(st):
    case, x = st["case"], st["x"].float()
    e, k, most = case["experts"], case["top_k"], st["most"]
    ids = st["experts"].long().flatten()
    key = torch.where(ids >= 0, ids, e)
    order = key.sort(stable=True, dim=0).indices
    first = torch.zeros(e + 1, dtype=torch.int64, device=x.device).scatter_add_(
        0, key, torch.ones_like(key))
    first = first.cumsum(0) - first
    place = torch.empty_like(key)
    place[order] = torch.arange(len(key), device=x.device)
    slot = torch.where(ids >= 0, key * most + place - first[key], e * most)   # last: nobody's
    xs = torch.zeros(e * most + 1, case["hidden"], device=x.device)
    xs[slot] = x.repeat_interleave(k, 0)
    xs = xs[:-1].view(e, most, -1).transpose(1, 2).contiguous()
    h = torch.bmm(_values(st["gate_up"], case["fmt"], case["layout"]), xs)
    gate, up = h.split(case["inner"], 1)
    h = gate / (1.0 + torch.exp(-gate)) * up
    y = torch.bmm(_values(st["down"], case["fmt"], case["layout"]), h)
    y = y.transpose(1, 2).reshape(e * most, -1)
    y = torch.cat((y, torch.zeros_like(y[:1])))[slot].view(-1, k, case["hidden"])
    return (st["weights"][..., None] * y).sum(1).bfloat16()


def _norm_parts(st):
    case, b = st["case"], st["block"].float()
    gate = 1.0 if st["gate"] is None else st["gate"].float()
    rb = torch.rsqrt(b.square().mean(-1, keepdim=True) + EPS) if case["post"] else None
    hat = b * rb if case["post"] else b
    n = hat * st["block_weight"].float() if case["post"] else b
    y = case["scale"] * st["x"].float() + gate * n
    r = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    return gate, rb, hat, n, y, r


def _norm_plain(st):
    case = st["case"]
    gate, rb, hat, n, y, r = _norm_parts(st)
    w = st["weight"].float()
    out = y.bfloat16(), (y * r * w).bfloat16()
    if not case["train"]:
        return out
    dz = st["dz"].float()
    u, yh = w * dz, y * r
    dy = st["dy"].float() + r * (u - yh * (u * yh).mean(-1, keepdim=True))
    dgate = None
    if st["gate"] is not None:
        dgate = (dy * n).double().sum(0 if case["gate"] == "channel" else 1,
                                      keepdim=case["gate"] == "token").float()
    db, dbw = gate * dy, None
    if case["post"]:
        dbw = (db * hat).double().sum(0).float()
        dh = db * st["block_weight"].float()
        db = rb * (dh - hat * (dh * hat).mean(-1, keepdim=True))
    dw = (dz * yh).double().sum(0).float()
    return out + ((case["scale"] * dy).bfloat16(), db.bfloat16(), dbw, dw, dgate)


# ------------------------------------------------------------------ the framework's calls
def _handle(st, name):
    """The handle that a user's program keeps of its weights."""
    import block_scaled_fp4_reduce_amd as fp4
    if name + " handle" not in st:
        st[name + " handle"] = fp4.Fp4Weights(fmt=st["case"]["fmt"], **st[name])
    return st[name + " handle"]


def _own(st):
    import block_scaled_fp4_reduce_amd as fp4
    case = st["case"]
    if case["op"] == "linear":
        return fp4.fp4_linear(_handle(st, "w"), st["x"],
                              dtype=torch.float32 if case["f32"] else torch.bfloat16)
    if case["op"] == "route":
        how = dict(scores=case["scores"], renormalize=case["renormalize"], scale=case["scale"])
        w, ids = fp4.expert_route(st["logits"], case["top_k"], bias=st["bias"],
                                  groups=case["groups"], top_groups=case["top_groups"],
                                  group_top=case["group_top"], **how)
        if not case["train"]:
            return w, ids
        return w, ids, fp4.expert_route_backward(st["dweights"], st["logits"], ids, **how)
    if case["op"] == "experts":
        return fp4.fp4_experts(_handle(st, "gate_up"), _handle(st, "down"), st["x"],
                               st["weights"], st["experts"])
    a = (st["x"], st["block"], st["weight"])
    kw = dict(block_weight=st["block_weight"], gate=st["gate"], scale=case["scale"], eps=EPS)
    out = fp4.residual_norm(*a, **kw)
    if not case["train"]:
        return out
    return out + fp4.residual_norm_backward(st["dy"], st["dz"], *a, **kw)


def run(st):
    if own:
        return _own(st)
    op = st["case"]["op"]
    if op == "linear":
        return _linear_plain(st)
    if op == "route":
        w, ids = _route_plain(st)
        return (w, ids, _route_plain_backward(st, ids)) if st["case"]["train"] else (w, ids)
    if op == "experts":
        return _experts_plain(st)
    return _norm_plain(st)


# ------------------------------------------------------------------ work
def _held(fmt, layout):
    """Bytes of a weight."""
    return 0.5 + (1.0 / 256 if layout == "tiles" else 1.0 / _group(fmt))


def work(case):
    t = case["tokens"]
    if case["op"] == "linear":
        n, k = case["rows"], case["cols"]
        io = t * (2 * k + (4 if case["f32"] else 2) * n)
        return {"bytes": _held(case["fmt"], case["layout"]) * n * k + io, "flops": 2 * t * n * k}
    if case["op"] == "route":
        e, k, each = case["experts"], case["top_k"], 2 if case["bf16"] else 4
        both = 2 if case["train"] else 1               # scores in; then once more, gradients out
        size = t * (each * e * (3 if case["train"] else 1) + (16 if case["train"] else 8) * k)
        return {"bytes": size, "flops": 30 * both * t * e}
    if case["op"] == "experts":
        e, k, d, f = case["experts"], case["top_k"], case["hidden"], case["inner"]
        t = _real_tokens(case)
        awake = e * (1.0 - (1.0 - k / e) ** t)         # experts with a token, all being alike
        return {"bytes": awake * 3 * d * f * _held(case["fmt"], case["layout"])
                + t * 2 * d + case["tokens"] * (2 * d + 8 * k), "flops": 6 * t * k * d * f}
    x = t * case["dim"]
    if case["train"]:                                  # x, block, dy, dz in; y, z, dx, dblock out
        return {"bytes": 2 * 8 * x, "flops": 40 * x}
    return {"bytes": 2 * 4 * x, "flops": 12 * x}


# ------------------------------------------------------------------ 64 bits
def _exact_values(w, case):
    """Values in 64 bits of one matrix's codes [rows][cols/2], scales and alpha."""
    codes = w["codes"].int()
    c = torch.stack((codes % 16, codes // 16), -1).flatten(-2)
    e, f = (c % 8) // 2, (c % 2).double()
    mag = torch.where(e == 0, 0.5 * f, torch.ldexp(1 + 0.5 * f, e - 1))
    v = torch.where(c >= 8, -mag, mag)
    b = w["scales"].int()
    if case["fmt"] == MXFP4:
        s = torch.ldexp(torch.ones((), dtype=torch.float64, device=b.device), b - 127)
        return v * s.repeat_interleave(32, 1)
    m, e = (b % 8).double(), b // 8
    s = torch.where(e == 0, m / 512, torch.ldexp(1 + m / 8, e - 7))
    s = s.repeat_interleave(16, 1)
    if case["layout"] == "tiles":
        s = s.repeat_interleave(16, 0)
    return v * s * w["alpha"].double().reshape(-1, 1)


def _exact_route(st):
    case = st["case"]
    x = st["logits"].double()
    open_ = x > -math.inf
    x0 = torch.where(open_, x, -1e300).requires_grad_(case["train"])
    if case["scores"] == "sigmoid":
        s = torch.sigmoid(x0)
    else:
        s = torch.softmax(x0, 1)
    s = torch.where(open_, s, 0.0)
    with torch.no_grad():
        c = torch.where(open_, s + (st["bias"].double() if case["bias"] else 0.0), -math.inf)
        pick = c if case["bias"] else x                # scores alone are in their logits' order

        def rank(v):
            """Place of each value among its row's, ties by index."""
            out = torch.empty(v.shape, dtype=torch.int64, device=v.device)
            n = torch.arange(v.shape[1], device=v.device)
            for lo in range(0, len(v), 1024):
                a = v[lo:lo + 1024]
                ahead = (a[:, None, :] > a[:, :, None]) | (
                    (a[:, None, :] == a[:, :, None]) & (n[None, :] < n[:, None]))
                out[lo:lo + 1024] = ahead.sum(-1)
            return out

        if case["groups"] > 1:
            by = (c if case["group_top"] == 2 else pick).unflatten(1, (case["groups"], -1))
            size = by.amax(-1)
            if case["group_top"] == 2 and by.shape[-1] > 1:
                second = by.topk(2, -1).values[..., 1]
                size = size + torch.where(second > -math.inf, second, 0.0)
            kept = rank(size) < case["top_groups"]
            pick = torch.where(kept[..., None], pick.unflatten(1, (case["groups"], -1)),
                               -math.inf).flatten(1)
        place = rank(pick)
        mine = place[:, :, None] == torch.arange(case["top_k"], device=x.device)
        ids = mine.double().argmax(1)                  # the expert at each place
        there = pick.gather(1, ids) > -math.inf
    w = torch.where(there, s.gather(1, ids), 0.0)
    if case["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    w = case["scale"] * w
    out = w.detach(), torch.where(there, ids, -1).int()
    if not case["train"]:
        return out
    (w * st["dweights"].double()).sum().backward()
    return out + (x0.grad,)


def _exact_experts(st):
    case, f = st["case"], st["case"]["inner"]
    out = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda")

    def one(name, e):
        w = st[name]
        return _exact_values({n: v if v is None else v[e] for n, v in w.items()}, case)

    for e in range(case["experts"]):
        token, place = torch.nonzero(st["experts"] == e, as_tuple=True)
        if not len(token):
            continue
        h = one("gate_up", e) @ st["x"][token].double().T
        h = torch.nn.functional.silu(h[:f]) * h[f:]
        y = (one("down", e) @ h).T * st["weights"][token, place].double()[:, None]
        out.index_add_(0, token, y)
    return out


def _exact_norm(st):
    case = st["case"]
    leaves = {n: st[n].double() for n in ("x", "block", "block_weight", "weight", "gate")
              if st[n] is not None}
    for v in leaves.values():
        v.requires_grad_(case["train"])

    def normed(v, w):
        return v / torch.sqrt((v * v).sum(-1, keepdim=True) / case["dim"] + EPS) * w

    n = normed(leaves["block"], leaves["block_weight"]) if case["post"] else leaves["block"]
    y = case["scale"] * leaves["x"] + (leaves["gate"] * n if "gate" in leaves else n)
    z = normed(y, leaves["weight"])
    if not case["train"]:
        return y, z
    ((y * st["dy"].double()).sum() + (z * st["dz"].double()).sum()).backward()
    return (y.detach(), z.detach()) + tuple(
        leaves[n].grad if n in leaves else None
        for n in ("x", "block", "block_weight", "weight", "gate"))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linear":
        return st["x"].double() @ _exact_values(st["w"], case).T
    if case["op"] == "route":
        return _exact_route(st)
    if case["op"] == "experts":
        return _exact_experts(st)
    return _exact_norm(st)
