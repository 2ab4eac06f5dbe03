"""GPU parity of the paged FP4 cache: bytes written and values read back
against the CPU oracle's quantizers, bit for bit."""
import numpy as np
import pytest

import kv_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402

MODES = {"nvfp4": (0, 0), "nvfp4_46": (0, 1), "mxfp4": (1, 0)}


def bits(rng, t, h, d, spread=0.5):
    x = rng.standard_normal((t, h, d)) * np.exp(spread * rng.standard_normal((1, h, d)))
    return R.bf16_bits(x)


def tensor(b):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).cuda().view(torch.bfloat16)


def amaxes(rng, b, h):
    m = np.abs(R.bf16_values(b)).max((0, 2)) if b.shape[0] else np.ones(h)
    return (m * (0.7 + 0.3 * rng.random(h))).astype(np.float32)     # some values lie past it


def handle(ref, fmt, flags, k_amax, v_amax):
    dev = {k: torch.from_numpy(v.copy()).cuda() for k, v in ref.items()}
    nv = fmt == 0
    return fp4.KvCache(fmt=fmt, flags=flags,
                       k_amax=torch.from_numpy(k_amax).cuda() if nv else None,
                       v_amax=torch.from_numpy(v_amax).cuda() if nv else None, **dev)


def check_bytes(cache, ref):
    for n in ref:
        got = getattr(cache, n).cpu().numpy()
        bad = np.argwhere(got != ref[n])
        assert not len(bad), "%s differs at %d places, first %s" % (n, len(bad), bad[0].tolist())


CASES = [  # tokens, heads, dim, page, pages
    (1, 1, 64, 16, 1), (5, 3, 128, 16, 2), (33, 2, 64, 32, 3), (130, 8, 128, 64, 4),
    (257, 1, 256, 128, 4), (64, 5, 256, 16, 6), (1000, 4, 128, 64, 20), (48, 2, 64, 4096, 1),
    (0, 2, 128, 16, 1),
]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("order", ["run", "unaligned", "scattered"])
@pytest.mark.parametrize("t,h,d,page,pages", CASES)
def test_write_then_read(mode, order, t, h, d, page, pages):
    print("kv write/read", mode, order, t, h, d, page, pages, flush=True)
    fmt, flags = MODES[mode]
    rng = np.random.default_rng(t * 7 + d)
    kb, vb = bits(rng, t, h, d), bits(rng, t, h, d, 0.2)
    ka, va = amaxes(rng, kb, h), amaxes(rng, vb, h)
    total = pages * page
    if order == "scattered":
        slots = rng.permutation(total)[:t].astype(np.int64)
    else:                                  # page after page, from the start or inside a page
        first = min(3, total - t) if order == "unaligned" else 0
        pg = rng.permutation(pages)
        at = first + np.arange(t)
        slots = (pg[at // page] * page + at % page).astype(np.int64)
    ref = R.empty_cache(pages, h, page, d, fmt, fill=0xA5)
    cache = handle(ref, fmt, flags, ka, va)
    R.write(ref, fmt, flags, kb, vb, slots, ka, va)
    st = torch.from_numpy(slots).cuda()
    fp4.fp4_kv_write(cache, tensor(kb), tensor(vb), st)
    k, v = fp4.fp4_kv_read(cache, st)
    torch.cuda.synchronize()
    check_bytes(cache, ref)
    kc, ks, vc, vs = R.at_slots(ref, slots)
    for got, c, s, a in ((k, kc, ks, ka), (v, vc, vs, va)):
        want = R.bf16_bits(R.decode(c, s, fmt, flags, a))
        assert np.array_equal(got.cpu().view(torch.int16).numpy().view(np.uint16), want)


@pytest.mark.parametrize("mode", MODES)
def test_strided_rows_and_slots_outside(mode):
    """Keys and values as slices of a fused projection; slots outside the cache
    are skipped by the write, read as zeros, and touch nothing else."""
    fmt, flags = MODES[mode]
    rng = np.random.default_rng(5)
    t, h, d, page, pages = 37, 3, 128, 16, 4
    both = bits(rng, t, 2 * h + 1, d)
    x = tensor(both)
    kb, vb = both[:, :h], both[:, h + 1:]
    ka, va = amaxes(rng, kb, h), amaxes(rng, vb, h)
    slots = rng.permutation(pages * page)[:t].astype(np.int64)
    slots[[0, 4, 17, 36]] = [-1, pages * page, -(1 << 40), 1 << 40]
    ref = R.empty_cache(pages, h, page, d, fmt, fill=0x5A)
    cache = handle(ref, fmt, flags, ka, va)
    R.write(ref, fmt, flags, kb, vb, slots, ka, va)
    st = torch.from_numpy(slots).cuda()
    fp4.fp4_kv_write(cache, x[:, :h], x[:, h + 1:], st)
    check_bytes(cache, ref)
    out = torch.full((t, 2 * h + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = fp4.fp4_kv_read(cache, st, out=(out[:, :h], out[:, h + 1:]))
    torch.cuda.synchronize()
    inside = (slots >= 0) & (slots < pages * page)
    kc, ks, vc, vs = R.at_slots(ref, np.where(inside, slots, 0))
    for got, c, s, a in ((k, kc, ks, ka), (v, vc, vs, va)):
        want = R.decode(c, s, fmt, flags, a)
        want[~inside] = 0.0
        assert np.array_equal(got.float().cpu().numpy(), R.bf16_values(R.bf16_bits(want)))
    assert (out[:, h].float() == 7.0).all()


@pytest.mark.parametrize("mode", MODES)
def test_special_values(mode):
    """Zeros of both signs, subnormals, equal values, lone outliers, a zero
    amax and an amax far below the values; infinities and NaN must not fault
    and leave other tokens alone."""
    fmt, flags = MODES[mode]
    rng = np.random.default_rng(11)
    t, h, d, page, pages = 40, 4, 64, 16, 3
    kb = bits(rng, t, h, d)
    kb[0], kb[1] = 0, 0x8000
    kb[2] = rng.integers(1, 0x80, (h, d))
    kb[3] = R.bf16_bits(np.full((h, d), 1.5))
    kb[4] = 0
    kb[4, :, 7] = R.bf16_bits(np.array([3.0]))
    ka = np.array([4.0, 0.0, 1e-3, 7.25], np.float32)
    slots = np.arange(t, dtype=np.int64)
    ref = R.empty_cache(pages, h, page, d, fmt)
    cache = handle(ref, fmt, flags, ka, ka)
    R.write(ref, fmt, flags, kb, kb, slots, ka, ka)
    x = kb.copy()
    x[9, 1, 5], x[9, 2, 6], x[9, 3, 7] = 0x7F80, 0xFF80, 0x7FC0
    st = torch.from_numpy(slots).cuda()
    fp4.fp4_kv_write(cache, tensor(x), tensor(x), st)
    torch.cuda.synchronize()
    for n in ref:                            # every token but the one with Inf and NaN
        got, want = getattr(cache, n).cpu().numpy().copy(), ref[n].copy()
        for a in (got, want):
            (a[0, :, 9] if n[0] == "k" else a[0, :, :, 9])[...] = 0
        assert np.array_equal(got, want), n
    if fmt == 0:
        assert (cache.k_scales.cpu().numpy() != 0x7F).all()


@pytest.mark.parametrize("mode", ["nvfp4_46", "mxfp4"])
def test_cache_past_4_gib(mode):
    """Pages whose byte offsets pass 32 bits."""
    fmt, flags = MODES[mode]
    rng = np.random.default_rng(3)
    h, d, page = 8, 256, 64
    pages = (1 << 32) // (h * page * d // 2) + 70
    ka = np.full(h, 3.0, np.float32)
    nv = fmt == 0
    am = torch.from_numpy(ka).cuda() if nv else None
    cache = fp4.KvCache.alloc(pages, page, h, d, fmt=fmt, flags=flags, k_amax=am, v_amax=am)
    t = 50
    kb, vb = bits(rng, t, h, d), bits(rng, t, h, d)
    last = pages * page
    slots = np.concatenate((np.arange(20), last - 1 - np.arange(30) * 7)).astype(np.int64)
    st = torch.from_numpy(slots).cuda()
    fp4.fp4_kv_write(cache, tensor(kb), tensor(vb), st)
    k, v = fp4.fp4_kv_read(cache, st)
    torch.cuda.synchronize()
    for got, b in ((k, kb), (v, vb)):
        c, s = R.quantize(b, fmt, flags, ka)
        want = R.decode(c, s, fmt, flags, ka)
        assert np.array_equal(got.float().cpu().numpy(), R.bf16_values(R.bf16_bits(want)))


def test_side_stream_and_graph():
    """The calls work on another stream and in a captured graph replayed on
    new contents, with eager work between the replays."""
    rng = np.random.default_rng(8)
    t, h, d, page, pages = 96, 2, 128, 32, 4
    ka = np.full(h, 3.0, np.float32)
    ref = R.empty_cache(pages, h, page, d, 0)
    cache = handle(ref, 0, 1, ka, ka)
    st = torch.from_numpy(rng.permutation(pages * page)[:t].astype(np.int64)).cuda()
    k = torch.zeros(t, h, d, dtype=torch.bfloat16, device="cuda")
    out = (torch.empty_like(k), torch.empty_like(k))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp4.fp4_kv_write(cache, k, k, st)
        fp4.fp4_kv_read(cache, st, out=out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert (out[0] == 0).all() and (out[1] == 0).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp4.fp4_kv_write(cache, k, k, st)
        fp4.fp4_kv_read(cache, st, out=out)
    for i in range(3):
        b = bits(np.random.default_rng(i), t, h, d)
        k.copy_(tensor(b))
        g.replay()
        torch.cuda.synchronize()
        c, s = R.quantize(b, 0, 1, ka)
        want = R.bf16_values(R.bf16_bits(R.decode(c, s, 0, 1, ka)))
        assert np.array_equal(out[0].float().cpu().numpy(), want), i
        assert np.array_equal(out[1].float().cpu().numpy(), want), i
        (k.float() * 2).sum().item()
