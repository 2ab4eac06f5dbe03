"""Tokens that belong to no sequence (a batch padded to the size of a captured
graph): cu_q starts past 0 or ends before the last token.  They get out = 0 and
lse = -inf, the others what they get without them; with and without parts,
whatever the workspace held.  Bounds as in test_gpu_kv_attention."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_kv_attention import MODES, build, check, tensor  # noqa: E402

CASES = [  # lens, news, tokens before, tokens after, group, page
    ([40], [1], 0, 7, 4, 16), ([40, 33, 9], [1, 1, 1], 3, 60, 4, 16), ([100, 77], [5, 9], 50, 0, 5, 64),
    ([100, 77], [40, 60], 33, 70, 4, 64), ([64, 0, 0], [30, 0, 0], 1, 129, 4, 16),
    ([0, 0, 90], [0, 0, 20], 130, 1, 8, 32), ([3000, 500], [1, 1], 0, 30, 4, 64),
    ([3000, 500], [1, 1], 9, 1200, 4, 64), ([2500], [7], 2, 600, 8, 32), ([2500, 800], [90, 20], 40, 1000, 4, 16),
    ([0], [0], 5, 5, 4, 16),
]


@pytest.mark.parametrize("mode", ["nvfp4_46", "mxfp4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("known", [True, False])
@pytest.mark.parametrize("fill", [0, 0xFF, 0x7F])
@pytest.mark.parametrize("lens,news,before,after,grp,page", CASES)
def test_tokens_of_no_sequence(mode, d, known, fill, lens, news, before, after, grp, page):
    print("padded", mode, d, known, fill, lens, news, before, after, grp, page, flush=True)
    fmt, flags = MODES[mode]
    rng = np.random.default_rng(before + after)
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, 2, grp, d, page)
    pad = lambda n: rng.integers(0, 1 << 15, (n,) + qb.shape[1:]).astype(np.uint16)
    qb = np.concatenate((pad(before), qb, pad(after)))
    cu = cu + before
    dev = {k: torch.from_numpy(v).cuda() for k, v in ref.items()}
    am = torch.from_numpy(ka).cuda() if fmt == 0 else None
    cache = fp4.KvCache(fmt=fmt, flags=flags, k_amax=am, v_amax=am, **dev)
    args = (cache, tensor(qb), torch.from_numpy(pt).cuda(),
            torch.tensor(lens, dtype=torch.int32, device="cuda"),
            torch.from_numpy(cu.astype(np.int32)).cuda())
    most = max(news) if known else 0
    need = fp4.fp4_kv_attention_workspace_bytes(*args, max_q=most)
    ws = torch.full((max(need, 16),), fill, dtype=torch.uint8, device="cuda")
    out = torch.full(qb.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(qb.shape[:2], 7.0, device="cuda")
    fp4.fp4_kv_attention(*args, max_q=most, out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    for part in (slice(0, before), slice(before + sum(news), None)):
        assert not out[part].any() and torch.isneginf(lse[part]).all()
    qb = np.where((np.arange(len(qb)) >= before)[:, None, None] &
                  (np.arange(len(qb)) < before + sum(news))[:, None, None], qb, 0).astype(np.uint16)
    check(mode, (out, lse), ref, ka, pt, lens, cu, qb)
