"""Bytes written and values read back by the cache's larger tiles (32 and 64
tokens a workgroup, taken with many tiles), against the CPU oracle's
quantizers, bit for bit: odd token counts, strided rows, slots in order, inside
a page, scattered and partly outside the cache."""
import numpy as np
import pytest

import kv_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_kv_cache import MODES, amaxes, bits, check_bytes, handle, tensor  # noqa: E402


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("order", ["run", "unaligned", "mixed"])
@pytest.mark.parametrize("t,h,d,page", [(1030, 17, 64, 16), (1030, 17, 128, 64), (1029, 17, 256, 32),
                                        (4131, 65, 64, 64)])
def test_larger_tiles(mode, order, t, h, d, page):
    print("kv tiles", mode, order, t, h, d, page, flush=True)
    fmt, flags = MODES[mode]
    rng = np.random.default_rng(t + d)
    both = bits(rng, t, 2 * h, d, 0.2)
    kb, vb = both[:, :h], both[:, h:]
    ka, va = amaxes(rng, kb, h), amaxes(rng, vb, h)
    pages = -(-t // page) + 2
    pg = rng.permutation(pages)
    at = (3 if order == "unaligned" else 0) + np.arange(t)
    slots = (pg[at // page] * page + at % page).astype(np.int64)
    if order == "mixed":                   # runs, a shuffled stretch, slots outside
        slots[200:500] = rng.permutation(slots[200:500])
        slots[[0, 77, t - 1]] = [-1, pages * page, -(1 << 40)]
    ref = R.empty_cache(pages, h, page, d, fmt, fill=0x3C)
    cache = handle(ref, fmt, flags, ka, va)
    R.write(ref, fmt, flags, kb, vb, slots, ka, va)
    x, st = tensor(both), torch.from_numpy(slots).cuda()
    fp4.fp4_kv_write(cache, x[:, :h], x[:, h:], st)
    out = torch.full((t, 2 * h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = fp4.fp4_kv_read(cache, st, out=(out[:, :h], out[:, h:]))
    torch.cuda.synchronize()
    check_bytes(cache, ref)
    inside = (slots >= 0) & (slots < pages * page)
    kc, ks, vc, vs = R.at_slots(ref, np.where(inside, slots, 0))
    for got, c, s, a in ((k, kc, ks, ka), (v, vc, vs, va)):
        want = R.decode(c, s, fmt, flags, a)
        want[~inside] = 0.0
        assert np.array_equal(got.float().cpu().numpy(), R.bf16_values(R.bf16_bits(want)))
