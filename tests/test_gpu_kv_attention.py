"""Attention over the paged FP4 cache against 64-bit attention on the same
bytes.

Bounds, in units u = 2^-24 (fp32) with A = sum p |v|: the output's rounding is
2^-8 |out| (bf16); the weights of the value product are rounded to the value
operand's type, 2^-11 A (fp16, NVFP4) or 2^-8 A (bf16, MXFP4); a score is a
fp32 sum of D exact products, off by at most D u sum |q k| scale, which shifts
a weight by twice that; the exponentials and the fp32 sums over n keys add
(n + 16) u A."""
import numpy as np
import pytest

import kv_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402

MODES = {"nvfp4": (0, 0), "nvfp4_46": (0, 1), "mxfp4": (1, 0)}
U = 2.0 ** -24


def tensor(b):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).cuda().view(torch.bfloat16)


def build(rng, mode, lens, news, h, grp, d, page, spare=2, fill=0xFF, qscale=1.0, peak=0.6):
    """Cache bytes, page table and queries of sequences; every byte that no
    sequence holds is `fill` (0xFF: NaN scales)."""
    fmt, flags = MODES[mode]
    width = max(1, max(-(-n // page) for n in lens))
    pages = len(lens) * width + spare
    pt = rng.permutation(pages)[:len(lens) * width].reshape(len(lens), width).astype(np.int32)
    ref = R.empty_cache(pages, h, page, d, fmt, fill=fill)
    size = np.exp(0.4 * rng.standard_normal((1, h, d)))
    ka = (3.0 * size.max((0, 2)) * (0.9 + 0.2 * rng.random(h))).astype(np.float32)
    cu = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    q = rng.standard_normal((cu[-1], h * grp, d))
    for b, n in enumerate(lens):
        if not n:
            continue
        j = np.arange(n)
        x = (rng.standard_normal((n, h, d)) + 0.3) * size
        kb, vb = R.bf16_bits(x), R.bf16_bits(rng.standard_normal((n, h, d)) + 0.2)
        R.write(ref, fmt, flags, kb, vb, pt[b][j // page].astype(np.int64) * page + j % page, ka, ka)
        for i in range(cu[b], cu[b + 1]):       # look for some key
            near = x[rng.integers(n)]
            q[i] += peak * np.repeat(near / np.sqrt((near ** 2).mean(-1, keepdims=True)), grp, 0)
    return ref, ka, pt, cu, R.bf16_bits(q * qscale)


def run(mode, ref, ka, pt, lens, cu, qb, use_cu=True, max_q=0, softcap=0.0, window=0, scale=None,
        out=None, q=None, ws=None):
    fmt, flags = MODES[mode]
    dev = {k: torch.from_numpy(v).cuda() for k, v in ref.items()}
    am = torch.from_numpy(ka).cuda() if fmt == 0 else None
    cache = fp4.KvCache(fmt=fmt, flags=flags, k_amax=am, v_amax=am, **dev)
    q = tensor(qb) if q is None else q
    got = fp4.fp4_kv_attention(cache, q, torch.from_numpy(pt).cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"),
                               torch.from_numpy(cu).cuda() if use_cu else None, max_q=max_q,
                               scale=scale, softcap=softcap, window=window, want_lse=True, out=out,
                               ws=ws)
    torch.cuda.synchronize()
    return got


def check(mode, got, ref, ka, pt, lens, cu, qb, softcap=0.0, window=0, scale=None):
    fmt, flags = MODES[mode]
    d = qb.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    out, lse, size, mag = R.attention(ref, fmt, flags, ka, ka, R.bf16_values(qb), pt, lens, cu,
                                      scale, softcap, window)
    n = max(max(lens), 1)
    score = d * U * mag
    if softcap:                                  # tanh's own error, a few ulp of the cap
        score = score + 8 * U * softcap
    weight = 2.0 ** -11 if fmt == 0 else 2.0 ** -8
    o, l = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(out) + (weight + 2 * score[..., None] + (n + 16) * U) * size + 1e-30
    bad = np.argwhere(~(np.abs(o - out) <= tol))
    assert not len(bad), "out off at %d of %d, first %s: %r for %r (bound %r)" % (
        len(bad), o.size, bad[0], o[tuple(bad[0])], out[tuple(bad[0])], tol[tuple(bad[0])])
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(l), empty)
    assert not o[empty].any()
    lt = score + (n + 16) * U + 4 * U * np.abs(np.where(empty, 0, lse))
    bad = np.argwhere(~empty & ~(np.abs(np.where(empty, 0, l - np.where(empty, 0, lse))) <= lt))
    assert not len(bad), "lse off at %s: %r for %r" % (
        bad[0], l[tuple(bad[0])], lse[tuple(bad[0])])


DECODE = [  # lens, kv heads, group, dim, page
    ([1], 1, 1, 64, 16), ([15], 1, 3, 64, 16), ([64], 2, 4, 128, 64), ([65, 1, 63, 130], 2, 8, 128, 32),
    ([257, 300, 2], 3, 5, 128, 16), ([511], 1, 16, 64, 128), ([129, 700], 2, 7, 256, 64),
    ([1025, 33], 1, 17, 128, 64), ([90], 1, 40, 256, 16), ([5000], 2, 4, 128, 64),
    ([2100, 0, 1], 1, 2, 64, 4096),
]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("use_cu", [True, False])
@pytest.mark.parametrize("lens,h,grp,d,page", DECODE)
def test_decode(mode, use_cu, lens, h, grp, d, page):
    print("decode", mode, use_cu, lens, h, grp, d, page, flush=True)
    rng = np.random.default_rng(sum(lens) + d)
    ref, ka, pt, cu, qb = build(rng, mode, lens, [1] * len(lens), h, grp, d, page)
    got = run(mode, ref, ka, pt, lens, cu, qb, use_cu, max_q=1 if use_cu else 0)
    check(mode, got, ref, ka, pt, lens, cu, qb)


CHUNKS = [  # lens, new tokens, kv heads, group, dim, page, softcap, window
    ([40], [40], 1, 1, 64, 16, 0.0, 0), ([100, 31, 64], [17, 31, 1], 2, 4, 128, 32, 0.0, 0),
    ([300, 5], [65, 5], 1, 8, 128, 64, 0.0, 0), ([200], [130], 2, 3, 64, 16, 30.0, 0),
    ([260, 90], [70, 80], 1, 2, 256, 64, 0.0, 37), ([150, 400, 3], [150, 20, 3], 2, 5, 128, 16, 20.0, 1),
    ([513], [129], 1, 7, 128, 128, 0.0, 128), ([64, 64, 64], [0, 64, 0], 1, 4, 64, 64, 0.0, 0),
    ([700], [300], 1, 4, 128, 64, 5.0, 500), ([33], [20], 1, 33, 64, 16, 0.0, 0),
]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("known", [True, False])
@pytest.mark.parametrize("lens,news,h,grp,d,page,cap,window", CHUNKS)
def test_chunks(mode, known, lens, news, h, grp, d, page, cap, window):
    print("chunk", mode, known, lens, news, h, grp, d, page, cap, window, flush=True)
    rng = np.random.default_rng(sum(lens) * 3 + d)
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, h, grp, d, page)
    got = run(mode, ref, ka, pt, lens, cu, qb, max_q=max(news) if known else 0, softcap=cap,
              window=window)
    check(mode, got, ref, ka, pt, lens, cu, qb, cap, window)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("new", [1, 9, 200])
def test_rows_that_see_nothing(mode, new):
    """No cached token, fewer cached tokens than new ones, a negative length."""
    rng = np.random.default_rng(new)
    lens, news = [0, new // 2, new + 3], [new, new, new]
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, 2, 2, 128, 16)
    got = run(mode, ref, ka, pt, lens, cu, qb, max_q=new)
    check(mode, got, ref, ka, pt, lens, cu, qb)
    got = run(mode, ref, ka, pt, [-5, lens[1], lens[2]], cu, qb, max_q=new)
    check(mode, got, ref, ka, pt, lens, cu, qb)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("new", [1, 70])
def test_bad_pages_and_lengths(mode, new):
    """Page ids outside the cache contribute nothing; a length past the table
    is cut to it."""
    rng = np.random.default_rng(21 + new)
    lens, news = [400, 400], [new, new]       # every slot of both tables is written
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, 2, 4, 128, 16)
    pt[0, [0, 5, 11]] = [-1, ref["k_codes"].shape[0], 2 ** 31 - 1]
    pt[1, 2] = -2 ** 31
    got = run(mode, ref, ka, pt, lens, cu, qb, max_q=new)
    check(mode, got, ref, ka, pt, lens, cu, qb)
    lens = [pt.shape[1] * 16, 2 ** 31 - 1]       # the second is cut to the first's length
    got = run(mode, ref, ka, pt, lens, cu, qb, max_q=new)
    check(mode, got, ref, ka, pt, [lens[0]] * 2, cu, qb)
    none = np.full_like(pt, -1)
    out, lse = run(mode, ref, ka, none, lens, cu, qb, max_q=new)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("size", [2.0 ** -40, 2.0 ** 30, 60.0])
def test_query_sizes(mode, size):
    """Queries far from 1: the scale makes up for them, but for the last,
    where one key takes all the weight."""
    rng = np.random.default_rng(4)
    lens, news = [333], [3]
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, 2, 4, 128, 16, qscale=size)
    scale = 128 ** -0.5 / size if size != 60.0 else None
    got = run(mode, ref, ka, pt, lens, cu, qb, max_q=3, scale=scale)
    check(mode, got, ref, ka, pt, lens, cu, qb, scale=scale)


@pytest.mark.parametrize("new", [1, 100])
def test_rising_scores(new):
    """Scores that grow along the context, so the running maximum moves on
    every block, and far apart ones that leave early weights at zero."""
    rng = np.random.default_rng(2)
    lens, news = [1500], [new]
    ref, ka, pt, cu, qb = build(rng, "nvfp4", lens, news, 1, 4, 64, 16, peak=0.0)
    j = np.arange(1500)
    ramp = np.linspace(-1, 1, 1500)[:, None, None] * np.ones((1, 1, 64))
    kb = R.bf16_bits(ramp * 3 + 0.05 * rng.standard_normal((1500, 1, 64)))
    ka = np.array([3.3], np.float32)
    vb = R.bf16_bits(rng.standard_normal((1500, 1, 64)))
    R.write(ref, 0, 0, kb, vb, pt[0][j // 16].astype(np.int64) * 16 + j % 16, ka, ka)
    for size in (0.2, 3.0, -3.0):
        qb = R.bf16_bits(np.full((new, 4, 64), size) + 0.05 * rng.standard_normal((new, 4, 64)))
        got = run("nvfp4", ref, ka, pt, lens, cu, qb, max_q=new)
        check("nvfp4", got, ref, ka, pt, lens, cu, qb)


@pytest.mark.parametrize("new", [1, 40])
def test_strided_queries_and_outputs(new):
    rng = np.random.default_rng(9)
    lens, news = [120, 77], [new, new]
    ref, ka, pt, cu, qb = build(rng, "nvfp4_46", lens, news, 2, 2, 128, 32)
    wide = torch.zeros(qb.shape[0], 9, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:7] = tensor(qb)
    out = torch.full((qb.shape[0], 6, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    got = run("nvfp4_46", ref, ka, pt, lens, cu, qb, max_q=new, q=wide[:, 3:7], out=out[:, 1:5])
    check("nvfp4_46", got, ref, ka, pt, lens, cu, qb)
    assert (out[:, 0] == 3).all() and (out[:, 5] == 3).all()


@pytest.mark.parametrize("lens,news", [([4000, 100], [1, 1]), ([900, 600], [130, 5])])
def test_same_bits_again_on_another_stream_and_in_a_graph(lens, news):
    """Equal calls give equal bits, on any stream, with a workspace full of
    NaN, and in a graph replayed after the queries change."""
    rng = np.random.default_rng(6)
    ref, ka, pt, cu, qb = build(rng, "nvfp4_46", lens, news, 2, 4, 128, 64)
    first = run("nvfp4_46", ref, ka, pt, lens, cu, qb, max_q=max(news))
    dev = {k: torch.from_numpy(v).cuda() for k, v in ref.items()}
    am = torch.from_numpy(ka).cuda()
    cache = fp4.KvCache(fmt=0, flags=1, k_amax=am, v_amax=am, **dev)
    q, table = tensor(qb), torch.from_numpy(pt).cuda()
    ln, cut = torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.from_numpy(cu).cuda()
    need = fp4.fp4_kv_attention_workspace_bytes(cache, q, table, ln, cut, max_q=max(news))
    ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")

    def call():
        fp4.fp4_kv_attention(cache, q, table, ln, cut, max_q=max(news), out=out, lse=lse, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), first[0].view(torch.int16))
    assert torch.equal(lse, first[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(3):
        q.copy_(tensor(qb) * (1.0 + i))
        call()
        torch.cuda.synchronize()
        want = out.clone(), lse.clone()
        out.fill_(9)
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want[0].view(torch.int16)), i
        assert torch.equal(lse, want[1]), i


def test_no_tokens_and_no_table():
    rng = np.random.default_rng(1)
    ref, ka, pt, cu, qb = build(rng, "nvfp4", [8], [1], 1, 2, 64, 16)
    out, lse = run("nvfp4", ref, ka, pt[:, :0].copy(), [8], cu, qb)
    assert not out.any() and torch.isneginf(lse).all()
    out, lse = run("nvfp4", ref, ka, pt[:0].copy(), [], cu[:1], qb[:0])
    assert out.shape == (0, 2, 64)


def test_long_context_past_32_bits():
    """A context at the end of a cache whose byte offsets pass 32 bits."""
    rng = np.random.default_rng(13)
    h, d, page = 8, 256, 64
    pages = (1 << 32) // (h * page * d // 2) + 40
    ka = np.full(h, 3.0, np.float32)
    am = torch.from_numpy(ka).cuda()
    cache = fp4.KvCache.alloc(pages, page, h, d, k_amax=am, v_amax=am)
    n = 500
    kb, vb = (R.bf16_bits(rng.standard_normal((n, h, d))) for _ in range(2))
    pt = (pages - 1 - np.arange(8)).astype(np.int32)[None]
    j = np.arange(n)
    slots = pt[0][j // page].astype(np.int64) * page + j % page
    fp4.fp4_kv_write(cache, tensor(kb), tensor(vb), torch.from_numpy(slots).cuda())
    small = R.empty_cache(8, h, page, d, 0)
    R.write(small, 0, 0, kb, vb, j, ka, ka)
    for new in (1, 33):
        cu = np.array([0, new], np.int32)
        qb = R.bf16_bits(rng.standard_normal((new, 2 * h, d)))
        got = fp4.fp4_kv_attention(cache, tensor(qb), torch.from_numpy(pt).cuda(),
                                   torch.tensor([n], dtype=torch.int32, device="cuda"),
                                   torch.from_numpy(cu).cuda(), max_q=new, want_lse=True)
        torch.cuda.synchronize()
        check("nvfp4", got, small, ka, np.arange(8, dtype=np.int32)[None], [n], cu, qb)
