"""Cases of the attention operators over a block-scaled FP4 key/value cache.

The operators: the norm of queries and keys with the position rotation
(forward and backward), writing keys and values into a paged FP4 cache,
reading them back, and attention of new tokens over that cache.  ``run``
computes each in plain torch (``own`` false) or through
``block_scaled_fp4_reduce_amd`` (``own`` true) on the same state.

Cache layout, [page][kv head] outermost, P tokens per page, G values per
scale (16 for NVFP4, 32 for MXFP4), D values per head:
  k_codes  [P][D/2]   two codes per byte, the even value in the low nibble
  k_scales [P][D/G]
  v_codes  [D/2][P]   byte i of a token holds values 2i (low) and 2i+1
  v_scales [D/G][P]
"""
import math

import torch

own = False

NVFP4, MXFP4 = 0, 1
FOUR_OVER_SIX = 1
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def _norm(name, tokens, hq, hkv, dim, rot, interleaved, train):
    return dict(name=name, op="norm_rope", tokens=tokens, q_heads=hq, kv_heads=hkv, dim=dim,
                rot=rot, interleaved=interleaved, train=train)


def _write(name, tokens, hkv, dim, page, fmt, four_six, contiguous):
    return dict(name=name, op="write", tokens=tokens, kv_heads=hkv, dim=dim, page=page, fmt=fmt,
                four_six=four_six, contiguous=contiguous)


def _read(name, tokens, hkv, dim, page, fmt, four_six):
    return dict(name=name, op="read", tokens=tokens, kv_heads=hkv, dim=dim, page=page, fmt=fmt,
                four_six=four_six)


def _attend(name, seqs, new, kv, ragged, hq, hkv, dim, page, fmt, four_six=False, softcap=0.0,
            window=0):
    return dict(name=name, op="attend", seqs=seqs, new=new, kv=kv, ragged=ragged, q_heads=hq,
                kv_heads=hkv, dim=dim, page=page, fmt=fmt, four_six=four_six, softcap=softcap,
                window=window)


def listed():
    return [
        # one decoding step of a small batch: latency counts
        _norm("norm_rope_decode", 32, 32, 8, 128, 128, False, False),
        # odd token count, few heads, interleaved pairs on half of each head, training
        _norm("norm_rope_ragged", 1021, 7, 1, 64, 32, True, True),
        # a training step's activations of one layer: forward and backward
        _norm("norm_rope_train", 8192, 32, 8, 128, 128, False, True),
        # every sequence of a decoding batch stores one token (scattered pages), reads it back
        _write("write_decode", 256, 8, 128, 64, NVFP4, True, False),
        # a prompt's chunk stored page after page and read back
        _write("write_chunk", 8192, 8, 128, 64, NVFP4, True, True),
        # odd token count in small pages of the power-of-two format
        _read("read_ragged", 3001, 4, 64, 16, MXFP4, False),
        # a long context taken out of the cache in one call
        _read("read_long", 65536, 8, 128, 64, NVFP4, True),
        # one sequence decoding: latency counts
        _attend("decode_one", 1, 1, 2048, False, 32, 8, 128, 64, NVFP4, True),
        # a serving batch decoding over ragged contexts
        _attend("decode_batch", 64, 1, 8192, True, 32, 8, 128, 64, NVFP4, True),
        # few sequences over long contexts, power-of-two scales, small groups of heads
        _attend("decode_long", 2, 1, 131072, True, 16, 8, 128, 128, MXFP4),
        # chunks of new tokens of several sequences over what is already cached
        _attend("chunk", 4, 512, 6144, True, 32, 8, 128, 64, NVFP4, True),
        # a whole prompt, sliding window and capped scores
        _attend("prompt_window", 1, 8192, 8192, False, 32, 8, 128, 64, MXFP4, False, 30.0, 4096),
    ]


def _span(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _lengths(case):
    """Context lengths and numbers of new tokens of the sequences; the first has the full sizes."""
    lens, news = [], []
    for i in range(case["seqs"]):
        cut = 0.75 * (i * 0.6180339887 % 1.0) if case["ragged"] else 0.0
        lens.append(case["kv"] - int(cut * case["kv"]))
        cut = 0.75 * (i * 0.7548776662 % 1.0) if case["ragged"] else 0.0
        news.append(min(lens[-1], case["new"] - int(cut * case["new"])))
    return lens, news


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(["norm_rope", "write", "read", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.choice([NVFP4, MXFP4])
    four_six = fmt == NVFP4 and rng.random() < 0.6
    hkv = rng.randint(1, 8)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "norm_rope":
        hq = min(32, hkv * group)
        most = max(1, 8192 * 40 * 128 // ((hq + hkv) * dim))
        rot = dim if rng.random() < 0.6 else dim // 2
        return _norm("", _span(rng, 1, min(8192, most)), hq, hkv, dim, rot, rng.random() < 0.4,
                     rng.random() < 0.6)
    if op == "write":
        most = 8192 * 8 * 128 // (hkv * dim)
        return _write("", _span(rng, 1, min(8192, most)), hkv, dim, page, fmt, four_six,
                      rng.random() < 0.5)
    if op == "read":
        most = 65536 * 8 * 128 // (hkv * dim)
        return _read("", _span(rng, 1, min(65536, most)), hkv, dim, page, fmt, four_six)
    softcap = rng.choice([0.0, 0.0, 30.0])
    if rng.random() < 0.6:                        # decoding: one token for each sequence
        seqs = _span(rng, 1, 64)
        most = 64 * 8192 * 8 * 128 // (seqs * hkv * dim) // 2
        kv = _span(rng, 1, max(1, min(65536, most)))
        new = 1
    else:                                         # chunks of new tokens
        seqs = rng.randint(1, 4)
        new = _span(rng, 2, 1024)
        kv = _span(rng, new, 8192)
    window = rng.choice([0, 0, _span(rng, 1, 4096)])
    return _attend("", seqs, new, kv, rng.random() < 0.6, hkv * group, hkv, dim, page, fmt,
                   four_six, softcap, window)


# ------------------------------------------------------------------ formats, plain
def _group(fmt):
    return 16 if fmt == NVFP4 else 32


def _round_e2m1(t):
    """Magnitude index and sign bit of the nearest E2M1 value (ties to the even index)."""
    a = t.abs()
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
         + (a >= 3.5) + (a > 5.0))
    return m.to(torch.uint8) | (torch.signbit(t).to(torch.uint8) << 3)


def _grid(device):
    return torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=device)


def _quantize(x, fmt, four_six, amax):
    """Codes (one per byte) and scale bytes of x [..., heads, D] in float32; amax [heads]."""
    g = _group(fmt)
    y = x.float().unflatten(-1, (-1, g))
    m = y.abs().amax(-1, keepdim=True)
    if fmt == MXFP4:
        byte = (((m.view(torch.int32) >> 23) & 255) - 2).clamp(min=0)
        byte = torch.where(m > 0, byte, 0)
        t = y * ((254 - byte) << 23).view(torch.float32)
        return _round_e2m1(t).flatten(-2), byte.squeeze(-1).to(torch.uint8)
    c = 256.0 if four_six else 448.0
    am = amax.float().view(-1, 1, 1)
    alpha = am / (6.0 * c)
    grid = _grid(x.device)

    def candidate(k):
        delta = (m * torch.where(am > 0, k / am, 0.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        s = alpha * delta.float()
        q = _round_e2m1(y * torch.where(s > 0, 1.0 / s, 0.0))
        return q, delta.view(torch.uint8), s

    q6, d6, s6 = candidate(c)
    if four_six:
        q4, d4, s4 = candidate(1.5 * c)

        def off(q, s):
            return (grid[q.int()].double() * s.double() - y.double()).square().sum(-1, keepdim=True)

        four = off(q4, s4) < off(q6, s6)
        q6, d6 = torch.where(four, q4, q6), torch.where(four, d4, d6)
    return q6.flatten(-2), d6.squeeze(-1)


def _scale_of(byte, fmt, four_six, amax):
    """float32 decode scales of bytes [..., heads, D/G]."""
    if fmt == MXFP4:
        return (byte.int() << 23).view(torch.float32)
    alpha = amax.float() / (6.0 * (256.0 if four_six else 448.0))
    return alpha[:, None] * byte.view(torch.float8_e4m3fn).float()


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _values(packed, byte, fmt, four_six, amax):
    """float32 values [..., heads, D] of packed codes [..., heads, D/2] and their scale bytes."""
    grid = _grid(packed.device)
    q = torch.stack((grid[(packed & 15).int()], grid[(packed >> 4).int()]), -1).flatten(-2)
    s = _scale_of(byte, fmt, four_six, amax)
    return (q.unflatten(-1, (-1, _group(fmt))) * s[..., None]).flatten(-2)


# ------------------------------------------------------------------ inputs
def _heads(gen, tokens, heads, dim, spread):
    """Keys or values as a model makes them: channels of unequal size, a few large ones."""
    dev = "cuda"
    size = torch.exp(spread * torch.randn(heads, dim, generator=gen, device=dev))
    off = 0.5 * torch.randn(heads, dim, generator=gen, device=dev)
    x = torch.randn(tokens, heads, dim, generator=gen, device=dev)
    return x.add_(off).mul_(size).to(torch.bfloat16)


def _empty_cache(case, pages):
    h, p, d = case["kv_heads"], case["page"], case["dim"]
    g = _group(case["fmt"])
    u8 = dict(dtype=torch.uint8, device="cuda")
    return dict(k_codes=torch.zeros(pages, h, p, d // 2, **u8),
                k_scales=torch.zeros(pages, h, p, d // g, **u8),
                v_codes=torch.zeros(pages, h, d // 2, p, **u8),
                v_scales=torch.zeros(pages, h, d // g, p, **u8))


def _store(cache, case, slots, k, v, k_amax, v_amax):
    """Quantize k, v [tokens][heads][dim] and store them at their slots."""
    fmt, f46 = case["fmt"], case["four_six"]
    page, at = slots // case["page"], slots % case["page"]
    c, s = _quantize(k, fmt, f46, k_amax)
    cache["k_codes"][page, :, at] = _pack(c)
    cache["k_scales"][page, :, at] = s
    c, s = _quantize(v, fmt, f46, v_amax)
    cache["v_codes"][page, :, :, at] = _pack(c)
    cache["v_scales"][page, :, :, at] = s


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 2 + 1)
    d = case["dim"]
    st = {"case": case}
    if case["op"] == "norm_rope":
        t, hq, hkv = case["tokens"], case["q_heads"], case["kv_heads"]
        qkv = torch.randn(t, (hq + 2 * hkv) * d, generator=gen, device=dev)
        qkv *= torch.exp(0.5 * torch.randn(t, 1, generator=gen, device=dev))
        qkv = qkv.to(torch.bfloat16)               # the fused projection's rows
        st["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        st["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        w = 1.0 + 0.2 * torch.randn(2, d, generator=gen, device=dev)
        st["qw"], st["kw"] = w.to(torch.bfloat16).unbind(0)
        # positions of a packed batch: each stretch starts somewhere in its own context
        far = 32768
        start = torch.randint(0, far - t, (1,), generator=gen, device=dev)
        st["positions"] = start + torch.arange(t, device=dev)
        rot = case["rot"]
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        angle = torch.arange(far, dtype=torch.float64, device=dev)[:, None] * inv
        st["table"] = torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()
        if case["train"]:
            st["dq"] = torch.randn(t, hq, d, generator=gen, device=dev).to(torch.bfloat16)
            st["dk"] = torch.randn(t, hkv, d, generator=gen, device=dev).to(torch.bfloat16)
        return st

    h, p = case["kv_heads"], case["page"]
    tokens = case["tokens"] if case["op"] != "attend" else None
    if case["op"] == "attend":
        seqs, kv = case["seqs"], case["kv"]
        lens, news = (torch.tensor(x, device=dev) for x in _lengths(case))
        width = -(-kv // p)
        pages = seqs * width
        st["page_table"] = torch.randperm(pages, generator=gen, device=dev).view(seqs, width).int()
        st["kv_lens"] = lens.int()
        st["cu_q"] = torch.cat((torch.zeros(1, dtype=torch.int64, device=dev),
                                news.cumsum(0))).int()
        total = int(news.sum())
        st["max_q"] = int(news.max())
        tokens = pages * p
    else:
        pages = -(-tokens // p) + 3
    k = _heads(gen, tokens, h, d, 0.4)
    v = _heads(gen, tokens, h, d, 0.2)
    # the per-head maxima come from calibration on other data, so some values lie past them
    other = 0.9 + 0.08 * torch.rand(2, h, generator=gen, device=dev)
    st["k_amax"] = other[0] * k.abs().amax((0, 2)).float()
    st["v_amax"] = other[1] * v.abs().amax((0, 2)).float()
    cache = _empty_cache(case, pages)
    if case["op"] == "write":
        st["k"], st["v"] = k, v
        if case["contiguous"]:
            order = torch.randperm(pages, generator=gen, device=dev)
            at = torch.arange(tokens, device=dev)
            st["slots"] = order[at // p] * p + at % p
        else:
            st["slots"] = torch.randperm(pages * p, generator=gen, device=dev)[:tokens].contiguous()
    elif case["op"] == "read":
        st["slots"] = torch.randperm(pages, generator=gen, device=dev)[:-(-tokens // p)]
        st["slots"] = (st["slots"][:, None] * p + torch.arange(p, device=dev)).flatten()[:tokens]
        st["slots"] = st["slots"].contiguous()
        _store(cache, case, st["slots"], k, v, st["k_amax"], st["v_amax"])
    else:
        _store(cache, case, torch.arange(tokens, device=dev), k, v, st["k_amax"], st["v_amax"])
        # queries look for some key of their own context, at usual score sizes
        hq = case["q_heads"]
        seq = torch.repeat_interleave(torch.arange(seqs, device=dev), news)
        pick = (torch.rand(total, hq, generator=gen, device=dev) * lens[seq][:, None]).long()
        slot = st["page_table"].long()[seq[:, None], pick // p] * p + pick % p
        head = torch.arange(hq, device=dev) // (hq // h)
        near = k[slot, head].float()
        near = near / near.square().mean(-1, keepdim=True).sqrt()
        q = torch.randn(total, hq, d, generator=gen, device=dev) + 0.6 * near
        st["q"] = q.to(torch.bfloat16)
    st["cache"] = cache
    return st


# ------------------------------------------------------------------ plain forms
def _rotate(x, c, s, rot, interleaved, back):
    """Rotate the first `rot` values of x [T][H][D] by the angles' cosines and sines [T][1][rot/2]."""
    if back:
        s = -s
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _norm_rope_plain(st, x, w):
    case = st["case"]
    cs = st["table"][st["positions"]][:, None]
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    return _rotate(y, cs[..., 0], cs[..., 1], case["rot"], case["interleaved"], False).bfloat16()


def _norm_rope_plain_backward(st, dy, x, w):
    case = st["case"]
    cs = st["table"][st["positions"]][:, None]
    g = _rotate(dy.float(), cs[..., 0], cs[..., 1], case["rot"], case["interleaved"], True)
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    n = x * r
    gw = g * w.float()
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    return dx.bfloat16(), (g * n).double().sum((0, 1)).float()


def _read_plain(st):
    case, cache = st["case"], st["cache"]
    page, at = st["slots"] // case["page"], st["slots"] % case["page"]
    fmt, f46 = case["fmt"], case["four_six"]
    k = _values(cache["k_codes"][page, :, at], cache["k_scales"][page, :, at], fmt, f46,
                st["k_amax"])
    v = _values(cache["v_codes"][page, :, :, at], cache["v_scales"][page, :, :, at], fmt, f46,
                st["v_amax"])
    return k.bfloat16(), v.bfloat16()


def _attend_plain(st):
    case, cache = st["case"], st["cache"]
    fmt, f46, d, h = case["fmt"], case["four_six"], case["dim"], case["kv_heads"]
    group = case["q_heads"] // h
    pt = st["page_table"].long()

    def gathered(codes, scales, amax, token_last):
        c, s = cache[codes][pt], cache[scales][pt]     # [B][W][H][...]
        if token_last:
            c, s = c.transpose(-1, -2), s.transpose(-1, -2)
        x = _values(c.permute(0, 1, 3, 2, 4), s.permute(0, 1, 3, 2, 4), fmt, f46, amax)
        return x.flatten(1, 2).permute(0, 2, 1, 3)     # [B][H][W*P][D]

    k = gathered("k_codes", "k_scales", st["k_amax"], False)
    v = gathered("v_codes", "v_scales", st["v_amax"], True)
    lens, cu = st["kv_lens"].long(), st["cu_q"].long()
    news = cu[1:] - cu[:-1]
    most = st["max_q"]
    b, kv = k.shape[0], k.shape[2]
    i = torch.arange(most, device=k.device)
    there = i[None] < news[:, None]                    # [B][most]
    row = torch.where(there, cu[:-1, None] + i[None], 0)
    q = st["q"].float()[row].unflatten(2, (h, group))  # [B][most][H][group][D]
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3).contiguous()
    s = torch.matmul(q, k.transpose(-1, -2).contiguous()) * (1.0 / math.sqrt(d))
    if case["softcap"]:
        s = case["softcap"] * torch.tanh(s / case["softcap"])
    pos = (lens - news)[:, None] + i[None]             # [B][most]
    j = torch.arange(kv, device=k.device)
    seen = j[None, None] <= pos[..., None]
    if case["window"]:
        seen = seen & (j[None, None] > pos[..., None] - case["window"])
    seen = seen.repeat_interleave(group, 1)[:, None]   # [B][1][most*group][kv]
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(s - m)
    del s, seen
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v.contiguous()) / torch.where(l > 0, l, 1.0)
    lse = (m + torch.log(l)).squeeze(-1)
    o = o.unflatten(2, (most, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)[there]
    lse = lse.unflatten(2, (most, group)).permute(0, 2, 1, 3).flatten(2, 3)[there]
    return o.bfloat16(), lse


# ------------------------------------------------------------------ the framework's calls
def _handle(st):
    """The cache handle that a user's program keeps beside its buffers."""
    import block_scaled_fp4_reduce_amd as fp4
    if "handle" not in st:
        case = st["case"]
        flags = fp4.FOUR_OVER_SIX if case["four_six"] else 0
        st["handle"] = fp4.KvCache(fmt=case["fmt"], flags=flags, k_amax=st["k_amax"],
                                   v_amax=st["v_amax"], **st["cache"])
    return fp4, st["handle"]


def _own(st):
    case = st["case"]
    if case["op"] == "norm_rope":
        import block_scaled_fp4_reduce_amd as fp4
        a = (st["qw"], st["kw"], st["positions"], st["table"])
        kw = dict(eps=1e-6, interleaved=case["interleaved"])
        yq, yk = fp4.qk_norm_rope(st["q"], st["k"], *a, **kw)
        if not case["train"]:
            return yq, yk
        return (yq, yk) + fp4.qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], *a, **kw)
    fp4, handle = _handle(st)
    if case["op"] == "write":
        fp4.fp4_kv_write(handle, st["k"], st["v"], st["slots"])
        return fp4.fp4_kv_read(handle, st["slots"])
    if case["op"] == "read":
        return fp4.fp4_kv_read(handle, st["slots"])
    return fp4.fp4_kv_attention(handle, st["q"], st["page_table"], st["kv_lens"], st["cu_q"],
                                max_q=st["max_q"], softcap=case["softcap"],
                                window=case["window"], want_lse=True)


def run(st):
    if own:
        return _own(st)
    case = st["case"]
    if case["op"] == "norm_rope":
        yq, yk = _norm_rope_plain(st, st["q"], st["qw"]), _norm_rope_plain(st, st["k"], st["kw"])
        if not case["train"]:
            return yq, yk
        dq, dqw = _norm_rope_plain_backward(st, st["dq"], st["q"], st["qw"])
        dk, dkw = _norm_rope_plain_backward(st, st["dk"], st["k"], st["kw"])
        return yq, yk, dq, dk, dqw, dkw
    if case["op"] == "write":
        _store(st["cache"], case, st["slots"], st["k"], st["v"], st["k_amax"], st["v_amax"])
        return _read_plain(st)
    if case["op"] == "read":
        return _read_plain(st)
    return _attend_plain(st)


# ------------------------------------------------------------------ work
def _causal(n, kv, w):
    """Query-key pairs of the last n of kv tokens, each seeing at most its last w."""
    lo, hi = kv - n + 1, kv                            # keys in reach of the first, the last
    if not w or hi <= w:
        return n * (lo + hi) / 2
    if lo >= w:
        return n * w
    ramp = w - lo
    return ramp * (lo + w) / 2 + (n - ramp) * w


def work(case):
    d = case["dim"]
    if case["op"] == "norm_rope":
        x = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * d
        cs = case["tokens"] * case["rot"] * 4
        if case["train"]:                              # x and dy in, y and dx out
            return {"bytes": 8 * x + cs, "flops": 22 * x}
        return {"bytes": 4 * x + cs, "flops": 8 * x}
    held = 0.5 + 1.0 / _group(case["fmt"])             # bytes of a value in the cache
    if case["op"] == "write":
        x = 2 * case["tokens"] * case["kv_heads"] * d
        return {"bytes": (2 + held + 2) * x, "flops": (40 if case["four_six"] else 16) * x}
    if case["op"] == "read":
        x = 2 * case["tokens"] * case["kv_heads"] * d
        return {"bytes": (held + 2) * x, "flops": 2 * x}
    w, reach, rows, pairs = case["window"], 0, 0, 0
    for kv, n in zip(*_lengths(case)):
        reach += min(kv, w + n - 1) if w else kv
        rows += n
        pairs += _causal(n, kv, w)
    read = 2 * held * reach * case["kv_heads"] * d
    return {"bytes": read + (4 * d + 4) * rows * case["q_heads"],
            "flops": 4 * d * case["q_heads"] * pairs}


# ------------------------------------------------------------------ 64 bits
def _exact_values(packed, byte, case, amax):
    """Values in 64 bits of codes [...][D/2] and scales [...][D/G]; amax a number."""
    c = torch.stack((packed % 16, packed // 16), -1).flatten(-2).double()
    sign = torch.where(c >= 8, -1.0, 1.0)
    m = torch.where(c >= 8, c - 8, c)
    e = (m / 2).floor()
    f = m - 2 * e
    mag = torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * 2.0 ** (e - 1))
    b = byte.double()
    if case["fmt"] == MXFP4:
        s = 2.0 ** (b - 127)
    else:
        e = (b / 8).floor()
        f = b - 8 * e
        s = torch.where(e == 0, f / 512, (1 + f / 8) * 2.0 ** (e - 7))
        s = s * (amax.double() / (6 * (256 if case["four_six"] else 448)))
    g = _group(case["fmt"])
    return sign * mag * s.repeat_interleave(g, -1)


def _exact_cached(st, which, slots, head):
    """Values [slots][D] of one head in 64 bits."""
    case, cache = st["case"], st["cache"]
    page, at = slots // case["page"], slots % case["page"]
    if which == "k":
        c, s = cache["k_codes"][page, head, at], cache["k_scales"][page, head, at]
    else:
        c, s = cache["v_codes"][page, head, :, at], cache["v_scales"][page, head, :, at]
    return _exact_values(c, s, case, st[which + "_amax"][head])


def _exact_quantized(x, case, amax):
    """What x [tokens][D] of one head reads back as: its nearest values, in 64 bits."""
    g = _group(case["fmt"])
    y = x.double().unflatten(-1, (-1, g))
    m = y.abs().amax(-1, keepdim=True)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)

    def nearest(t):
        a = t.abs().clamp(max=6.0).contiguous()
        hi = torch.searchsorted(grid, a).clamp(1, 7)
        lo = hi - 1
        mid = (grid[lo] + grid[hi]) / 2
        up = (a > mid) | ((a == mid) & (hi % 2 == 0))
        return torch.where(up, grid[hi], grid[lo]) * torch.sign(t)

    if case["fmt"] == MXFP4:
        s = 2.0 ** (torch.frexp(m).exponent.double() - 3)
        return torch.where(m > 0, nearest(y / s) * s, 0.0).flatten(-2)
    c = 256.0 if case["four_six"] else 448.0
    alpha = amax.double() / (6 * c)
    found, err = None, None
    for top in (6.0, 4.0) if case["four_six"] else (6.0,):
        z = (m / (top * alpha)).clamp(max=448.0)
        step = 2.0 ** (torch.frexp(z).exponent.clamp(min=-5).double() - 4)
        s = alpha * torch.round(z / step) * step
        v = torch.where(s > 0, nearest(y / torch.where(s > 0, s, 1.0)) * s, 0.0)
        off = (v - y).square().sum(-1, keepdim=True)
        if found is None:
            found, err = v, off
        else:
            found = torch.where(off < err, v, found)
    return found.flatten(-2)


def _exact_norm_rope(st, x, w, dy):
    case = st["case"]
    rot, d = case["rot"], case["dim"]
    cs = st["table"].double()[st["positions"]]
    turn = torch.complex(cs[..., 0], cs[..., 1])[:, None]

    def rotated(y, t):
        head, tail = y[..., :rot], y[..., rot:]
        pairs = head.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else head.unflatten(
            -1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * t)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat((z.flatten(-2), tail), -1)

    x, w = x.double(), w.double()
    size = (x.square().sum(-1, keepdim=True) / d + 1e-6).sqrt()
    y = rotated(x / size * w, turn)
    if dy is None:
        return y, None, None
    g = rotated(dy.double(), turn.conj())
    dn = g * w
    dx = dn / size - x * (dn * x).sum(-1, keepdim=True) / (d * size ** 3)
    return y, dx, (g * x / size).sum((0, 1))


def _exact_attend(st):
    case = st["case"]
    p, group = case["page"], case["q_heads"] // case["kv_heads"]
    lens, cu = st["kv_lens"].tolist(), st["cu_q"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, kv in enumerate(lens):
        n = cu[b + 1] - cu[b]
        at = torch.arange(kv, device="cuda")
        slots = st["page_table"][b].long()[at // p] * p + at % p
        for h in range(case["kv_heads"]):
            k, v = _exact_cached(st, "k", slots, h), _exact_cached(st, "v", slots, h)
            for lo in range(0, n, 1024):
                rows = torch.arange(lo, min(n, lo + 1024), device="cuda")
                q = st["q"][cu[b] + rows, h * group:(h + 1) * group].double()
                s = (q.flatten(0, 1) @ k.T).unflatten(0, (-1, group)) / math.sqrt(case["dim"])
                if case["softcap"]:
                    s = case["softcap"] * torch.tanh(s / case["softcap"])
                pos = kv - n + rows[:, None, None]
                hide = at > pos
                if case["window"]:
                    hide = hide | (at <= pos - case["window"])
                s = s.masked_fill(hide, -math.inf)
                z = torch.logsumexp(s, -1, keepdim=True)
                a = torch.where(z > -math.inf, torch.exp(s - z), 0.0)
                out[cu[b] + rows, h * group:(h + 1) * group] = (a.flatten(0, 1) @ v).unflatten(
                    0, (-1, group))
                lse[cu[b] + rows, h * group:(h + 1) * group] = z.squeeze(-1)
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rope":
        q, dq, dqw = _exact_norm_rope(st, st["q"], st["qw"], st.get("dq"))
        k, dk, dkw = _exact_norm_rope(st, st["k"], st["kw"], st.get("dk"))
        return (q, k, dq, dk, dqw, dkw) if case["train"] else (q, k)
    h = case["kv_heads"]
    if case["op"] == "write":
        return tuple(torch.stack([_exact_quantized(st[n][:, i], case, st[n + "_amax"][i])
                                  for i in range(h)], 1) for n in ("k", "v"))
    if case["op"] == "read":
        return tuple(torch.stack([_exact_cached(st, n, st["slots"], i) for i in range(h)], 1)
                     for n in ("k", "v"))
    return _exact_attend(st)
