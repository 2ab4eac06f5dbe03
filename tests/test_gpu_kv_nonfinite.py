"""Infinities and NaN among written keys and values reach only the tokens that
see them: rows before them, and other sequences, get what they get without.
Bounds as in test_gpu_kv_attention."""
import numpy as np
import pytest

import kv_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_kv_attention import MODES, U, tensor  # noqa: E402


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("what", ["value", "key", "both"])
@pytest.mark.parametrize("bad", [0x7F80, 0xFF80, 0x7FC0])
@pytest.mark.parametrize("n,new,at", [(70, 3, 69), (70, 3, 68), (130, 40, 120), (64, 64, 9)])
def test_rows_before_a_non_finite_token(mode, what, bad, n, new, at):
    """Token `at` of the first sequence is not finite; the rows before it are checked."""
    print("non-finite", mode, what, hex(bad), n, new, at, flush=True)
    fmt, flags = MODES[mode]
    rng = np.random.default_rng(n + at)
    h, grp, d, page = 2, 2, 128, 16
    lens, news = [n, 33], [new, 2]
    cu = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    width = -(-n // page)
    pt = rng.permutation(2 * width).reshape(2, width).astype(np.int32)
    kb, vb = (R.bf16_bits(rng.standard_normal((n + 33, h, d)) + 0.2) for _ in range(2))
    qb = R.bf16_bits(rng.standard_normal((cu[-1], h * grp, d)))
    slots = np.concatenate([pt[b][np.arange(m) // page].astype(np.int64) * page +
                            np.arange(m) % page for b, m in enumerate(lens)])
    ka = np.full(h, 4.0, np.float32)
    ref = R.empty_cache(2 * width, h, page, d, fmt)
    R.write(ref, fmt, flags, kb, vb, slots, ka, ka)
    out, lse, size, mag = R.attention(ref, fmt, flags, ka, ka, R.bf16_values(qb), pt, lens, cu,
                                      d ** -0.5, 0.0, 0)
    k2, v2 = kb.copy(), vb.copy()
    if what != "key":
        v2[at, 0, 5], v2[at, 1, 120] = bad, bad
    if what != "value":
        k2[at, 0, 7], k2[at, 1, 99] = bad, bad
    am = torch.from_numpy(ka).cuda() if fmt == 0 else None
    cache = fp4.KvCache.alloc(2 * width, page, h, d, fmt, flags, am, am)
    fp4.fp4_kv_write(cache, tensor(k2), tensor(v2), torch.from_numpy(slots).cuda())
    o, l = fp4.fp4_kv_attention(cache, tensor(qb), torch.from_numpy(pt).cuda(),
                                torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                torch.from_numpy(cu).cuda(), max_q=max(news), want_lse=True)
    torch.cuda.synchronize()
    o, l = o.double().cpu().numpy(), l.double().cpu().numpy()
    clean = np.ones(cu[-1], bool)
    clean[max(0, at - (n - new)):new] = False
    score = d * U * mag
    weight = 2.0 ** -11 if fmt == 0 else 2.0 ** -8
    tol = 2.0 ** -8 * np.abs(out) + (weight + 2 * score[..., None] + (n + 16) * U) * size + 1e-30
    assert (np.abs(o - out) <= tol)[clean].all()
    assert (np.abs(l - lse) <= score + (n + 16) * U + 4 * U * np.abs(lse))[clean].all()
