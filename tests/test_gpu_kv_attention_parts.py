"""Attention over the paged FP4 cache where its work is cut up: many
sequences, contexts in parts joined afterwards, tiles of many rows at every
head size and page size, scales and queries out of the ordinary.  Bounds as in
test_gpu_kv_attention."""
import numpy as np
import pytest

import kv_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_kv_attention import MODES, build, check, run, tensor  # noqa: E402

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402


@pytest.mark.parametrize("use_cu", [True, False])
def test_more_sequences_than_lanes(use_cu):
    """Sequences are searched 64 at a time."""
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(0, 90, 150)]
    lens[70], lens[149] = 900, 700
    print("sequences", len(lens), use_cu, flush=True)
    ref, ka, pt, cu, qb = build(rng, "nvfp4", lens, [1] * 150, 1, 2, 64, 16)
    got = run("nvfp4", ref, ka, pt, lens, cu, qb, use_cu, max_q=1 if use_cu else 0)
    check("nvfp4", got, ref, ka, pt, lens, cu, qb)


def test_many_sequences_most_without_new_tokens():
    rng = np.random.default_rng(6)
    lens = [40] * 140
    news = [0] * 140
    news[3], news[64], news[65], news[139] = 9, 1, 40, 17
    ref, ka, pt, cu, qb = build(rng, "mxfp4", lens, news, 1, 4, 64, 16)
    got = run("mxfp4", ref, ka, pt, lens, cu, qb, max_q=40)
    check("mxfp4", got, ref, ka, pt, lens, cu, qb)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,grp", [(1, 4), (5, 5), (11, 4)])
def test_long_contexts_in_parts(mode, page, d, new, grp):
    """Few rows over long contexts: parts of every sequence, of unequal
    lengths, joined; one column tile, two, and the tiled kernel."""
    print("parts", mode, page, d, new, grp, flush=True)
    rng = np.random.default_rng(page + d + new)
    lens, news = [1900, 333, 61], [new, new, min(new, 61)]
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, 1, grp, d, page)
    got = run(mode, ref, ka, pt, lens, cu, qb, max_q=new)
    check(mode, got, ref, ka, pt, lens, cu, qb)


@pytest.mark.parametrize("mode", ["nvfp4_46", "mxfp4"])
@pytest.mark.parametrize("d,page", [(64, 128), (128, 16), (256, 32), (256, 16)])
def test_tiles_of_many_rows(mode, d, page):
    """More rows than one tile, a window and a cap, rows of the last tile missing."""
    print("tiles", mode, d, page, flush=True)
    rng = np.random.default_rng(d + page)
    lens, news = [410, 90], [75, 90]
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, 1, 3, d, page)
    for cap, window in ((0.0, 0), (12.0, 0), (0.0, 50), (12.0, 33)):
        got = run(mode, ref, ka, pt, lens, cu, qb, max_q=90, softcap=cap, window=window)
        check(mode, got, ref, ka, pt, lens, cu, qb, cap, window)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("window", [1, 63, 64, 65, 700])
def test_windows_over_long_contexts(new, window):
    """The window starts inside a block, on its border and before the context."""
    rng = np.random.default_rng(window)
    lens, news = [1300, 640], [new, new]
    ref, ka, pt, cu, qb = build(rng, "nvfp4", lens, news, 1, 4, 64, 64)
    got = run("nvfp4", ref, ka, pt, lens, cu, qb, max_q=new, window=window)
    check("nvfp4", got, ref, ka, pt, lens, cu, qb, 0.0, window)


@pytest.mark.parametrize("mode", ["nvfp4_46", "mxfp4"])
@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("scale,cap", [(0.0, 0.0), (-0.2, 0.0), (-0.2, 10.0), (0.0, 10.0)])
def test_zero_and_negative_scales(mode, new, scale, cap):
    rng = np.random.default_rng(17)
    lens, news = [190], [new]
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, 2, 2, 64, 16)
    fmt, flags = MODES[mode]
    got = run(mode, ref, ka, pt, lens, cu, qb, max_q=new, softcap=cap, scale=scale)
    out, lse, size, mag = R.attention(ref, fmt, flags, ka, ka, R.bf16_values(qb), pt, lens, cu,
                                      scale, cap, 0)
    u = 2.0 ** -24
    score = 64 * u * np.abs(mag) + (8 * u * cap if cap else 0.0)
    weight = 2.0 ** -11 if fmt == 0 else 2.0 ** -8
    tol = 2.0 ** -8 * np.abs(out) + (weight + 2 * score[..., None] + 206 * u) * size + 1e-30
    assert (np.abs(got[0].double().cpu().numpy() - out) <= tol).all()
    assert (np.abs(got[1].double().cpu().numpy() - lse) <= score + 206 * u + 4 * u * np.abs(lse)).all()


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("new", [2, 40])
def test_nan_and_infinite_queries_stay_in_their_rows(mode, new):
    rng = np.random.default_rng(18)
    lens, news = [700], [new]
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, 1, 4, 128, 16)
    clean = run(mode, ref, ka, pt, lens, cu, qb, max_q=new)
    bad = qb.copy()
    bad[1, 2, 5], bad[new - 1, 0, 77] = 0x7FC0, 0x7F80
    out, lse = run(mode, ref, ka, pt, lens, cu, bad, max_q=new)
    assert out[1, 2].isnan().all() and lse[1, 2].isnan()
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    keep[1, 2] = keep[new - 1, 0] = False
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


@pytest.mark.parametrize("new", [1, 60])
def test_lse_is_optional_and_workspace_is_checked(new):
    rng = np.random.default_rng(19)
    lens, news = [3000, 50], [new, new]
    ref, ka, pt, cu, qb = build(rng, "nvfp4", lens, [new, min(new, 50)], 1, 4, 128, 64)
    news = [new, min(new, 50)]
    dev = {k: torch.from_numpy(v).cuda() for k, v in ref.items()}
    am = torch.from_numpy(ka).cuda()
    cache = fp4.KvCache(k_amax=am, v_amax=am, **dev)
    args = (cache, tensor(qb), torch.from_numpy(pt).cuda(),
            torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.from_numpy(cu).cuda())
    out, lse = fp4.fp4_kv_attention(*args, max_q=max(news), want_lse=True)
    only = fp4.fp4_kv_attention(*args, max_q=max(news))
    assert torch.equal(only, out)
    need = fp4.fp4_kv_attention_workspace_bytes(*args, max_q=max(news))
    assert need > 0
    with pytest.raises(fp4.Fp4Error):
        fp4.fp4_kv_attention(*args, max_q=max(news),
                             ws=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    side = torch.cuda.Stream()                     # an explicit stream, its own workspace
    side.wait_stream(torch.cuda.current_stream())
    again = fp4.fp4_kv_attention(*args, max_q=max(news), stream=side)
    side.synchronize()
    assert torch.equal(again, out)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("page", [32, 64, 128])
def test_bad_pages_of_whole_blocks(mode, new, page):
    """Pages outside the cache where a block lies in one page: first, middle and
    last ones contribute nothing, their neighbours everything."""
    rng = np.random.default_rng(page + new)
    lens, news = [9 * page, 9 * page - 5], [new, new]
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, 1, 4, 64, page)
    pt[0, [0, 4, 8]] = [-1, ref["k_codes"].shape[0], 2 ** 31 - 1]
    pt[1, [3, 5]] = -2 ** 31
    got = run(mode, ref, ka, pt, lens, cu, qb, max_q=new)
    check(mode, got, ref, ka, pt, lens, cu, qb)
