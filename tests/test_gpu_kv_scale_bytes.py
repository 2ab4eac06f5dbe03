"""The sign bit of an E4M3 scale byte is ignored by every operator on the
cache's bytes: attention and the read give the same bits with it set and clear."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_kv_attention import MODES, build, check, run  # noqa: E402


@pytest.mark.parametrize("mode", ["nvfp4", "nvfp4_46"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("new", [1, 6, 50])
def test_sign_bits_of_scales(mode, d, page, new):
    print("scale signs", mode, d, page, new, flush=True)
    rng = np.random.default_rng(new + d)
    lens, news = [300, 77], [new, new]
    ref, ka, pt, cu, qb = build(rng, mode, lens, news, 2, 4, d, page)
    plain = run(mode, ref, ka, pt, lens, cu, qb, max_q=new)
    check(mode, plain, ref, ka, pt, lens, cu, qb)
    signed = dict(ref)
    for n in ("k_scales", "v_scales"):
        signed[n] = ref[n] | (rng.integers(0, 2, ref[n].shape) << 7).astype(np.uint8)
    got = run(mode, signed, ka, pt, lens, cu, qb, max_q=new)
    assert torch.equal(got[0].view(torch.int16), plain[0].view(torch.int16))
    assert torch.equal(got[1], plain[1])
    fmt, flags = MODES[mode]
    am = torch.from_numpy(ka).cuda()
    slots = torch.from_numpy(np.concatenate([pt[b][np.arange(n) // page].astype(np.int64) * page +
                                             np.arange(n) % page for b, n in enumerate(lens)])).cuda()
    reads = []
    for r in (ref, signed):
        dev = {k: torch.from_numpy(v).cuda() for k, v in r.items()}
        cache = fp4.KvCache(fmt=fmt, flags=flags, k_amax=am, v_amax=am, **dev)
        reads.append(fp4.fp4_kv_read(cache, slots))
    for a, b in zip(*reads):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
