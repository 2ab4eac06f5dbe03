"""Plain 64-bit references of the operators around the paged FP4 cache:
attention, norm with rotation and its gradient; and the cache's bytes from
the CPU oracle's quantizers."""
import numpy as np

import oracle as O

RTN6, FOUR_OVER_SIX = 0, 1
NVFP4, MXFP4 = 0, 1


def bf16_bits(x):
    """Nearest-even bf16 bit patterns of float64/float32 values."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_values(bits):
    return (np.ascontiguousarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def group(fmt):
    return 16 if fmt == NVFP4 else 32


def empty_cache(pages, heads, page, dim, fmt, fill=0):
    g = group(fmt)
    new = lambda *s: np.full((pages, heads) + s, fill, np.uint8)
    return dict(k_codes=new(page, dim // 2), k_scales=new(page, dim // g),
                v_codes=new(dim // 2, page), v_scales=new(dim // g, page))


def quantize(bits, fmt, flags, amax):
    """Codes [tokens][heads][D/2], scales [tokens][heads][D/G] of bf16 bits [tokens][heads][D]."""
    t, h, d = bits.shape
    codes = np.zeros((t, h, d // 2), np.uint8)
    scales = np.zeros((t, h, d // group(fmt)), np.uint8)
    for i in range(h if t else 0):
        x = np.ascontiguousarray(bits[:, i])
        if fmt == NVFP4:
            r = O.nvfp4_quantize(x, flags, amax=np.float32(amax[i]))
            codes[:, i], scales[:, i] = r["codes"], r["scales"]
        else:
            r = O.mxfp4_quantize(x, O.ROWWISE)
            codes[:, i], scales[:, i] = r["codes_r"], r["scales_r"]
    return codes, scales


def write(cache, fmt, flags, k_bits, v_bits, slots, k_amax, v_amax):
    """Store tokens at their slots; slots outside the cache are skipped."""
    pages, _, page, _ = cache["k_codes"].shape
    kc, ks = quantize(k_bits, fmt, flags, k_amax)
    vc, vs = quantize(v_bits, fmt, flags, v_amax)
    for t, s in enumerate(slots):
        if not 0 <= s < pages * page:
            continue
        p, at = s // page, s % page
        cache["k_codes"][p, :, at], cache["k_scales"][p, :, at] = kc[t], ks[t]
        cache["v_codes"][p, :, :, at], cache["v_scales"][p, :, :, at] = vc[t], vs[t]


def decode(codes, scales, fmt, flags, amax, f32=True):
    """Values [tokens][heads][D] (float64) of codes and scales; with f32 each
    scale and product rounded to fp32, as the decode is defined."""
    t, h, half = codes.shape
    q = np.empty((t, h, 2 * half))
    q[..., 0::2] = O.e2m1_decode(codes & 15)
    q[..., 1::2] = O.e2m1_decode(codes >> 4)
    if fmt == NVFP4:
        c = np.float32(6.0 * (256.0 if flags & FOUR_OVER_SIX else 448.0))
        alpha = (np.asarray(amax, np.float32) / c)
        delta = O.e4m3_decode(scales & 0x7F)
        s = (alpha[None, :, None] * delta.astype(np.float32)) if f32 else (
            alpha.astype(np.float64)[None, :, None] * delta)
    else:
        s = np.ldexp(1.0, scales.astype(np.int64) - 127)
    s = np.repeat(s.astype(np.float64), group(fmt), axis=-1)
    return (q * s).astype(np.float32).astype(np.float64) if f32 else q * s


def at_slots(cache, slots):
    """(k codes, k scales, v codes, v scales) of slots, token first."""
    page = cache["k_codes"].shape[2]
    p, at = np.asarray(slots) // page, np.asarray(slots) % page
    return (cache["k_codes"][p, :, at], cache["k_scales"][p, :, at],
            cache["v_codes"][p, :, :, at], cache["v_scales"][p, :, :, at])


def attention(cache, fmt, flags, k_amax, v_amax, q, page_table, lens, cu, scale, cap, window):
    """64-bit attention.  Returns out, lse, the mean of |v| under the weights
    and the largest sum of |q k| scale of each row (for error bounds)."""
    pages, h, page, half = cache["k_codes"].shape
    tokens, hq, d = q.shape
    grp = hq // h
    out, size = np.zeros((tokens, hq, d)), np.zeros((tokens, hq, d))
    lse, mag = np.full((tokens, hq), -np.inf), np.zeros((tokens, hq))
    width = page_table.shape[1]
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        kv = min(int(lens[b]), width * page)
        j = np.arange(max(kv, 0))
        pg = page_table[b][j // page] if kv > 0 else np.zeros(0, np.int64)
        ok = (pg >= 0) & (pg < pages)
        slots = np.where(ok, pg, 0).astype(np.int64) * page + j % page
        if not n or not len(j):
            continue
        kc, ks, vc, vs = at_slots(cache, slots)
        k = decode(kc, ks, fmt, flags, k_amax, False)
        v = decode(vc, vs, fmt, flags, v_amax, False)
        for i in range(n):
            pos = kv - n + i
            see = ok & (j <= pos)
            if window:
                see &= j > pos - window
            if not see.any():
                continue
            for hh in range(hq):
                x = q[cu[b] + i, hh]
                s = k[see, hh // grp] @ x * scale
                mag[cu[b] + i, hh] = (np.abs(k[see, hh // grp]) @ np.abs(x)).max() * scale
                if cap:
                    s = cap * np.tanh(s / cap)
                m = s.max()
                e = np.exp(s - m)
                p = e / e.sum()
                out[cu[b] + i, hh] = p @ v[see, hh // grp]
                size[cu[b] + i, hh] = p @ np.abs(v[see, hh // grp])
                lse[cu[b] + i, hh] = m + np.log(e.sum())
    return out, lse, size, mag


# ------------------------------------------------------------------ norm + rotation
def rotate(y, cs, rot, interleaved, back=False):
    """R y (R^T y with back) for y [tokens][heads][D] and cs [tokens][rot/2][2]."""
    c, s = cs[:, None, :, 0], cs[:, None, :, 1] * (-1.0 if back else 1.0)
    out = y.copy()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return out


def norm_rope(x, w, cs, rot, interleaved, eps):
    y = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return rotate(y, cs, rot, interleaved)


def norm_rope_backward(dy, x, w, cs, rot, interleaved, eps):
    g = rotate(dy, cs, rot, interleaved, back=True)
    if w is None:
        return g, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dn = g * w
    return r * (dn - n * (dn * n).mean(-1, keepdims=True)), (g * n).sum((0, 1))
