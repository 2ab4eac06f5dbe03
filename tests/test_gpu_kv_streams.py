"""Calls on a stream of the caller's own while the current stream is busy: new
outputs and workspaces are not memory that pending work still uses."""
import numpy as np
import pytest

import kv_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_kv_attention import build, tensor  # noqa: E402
from test_gpu_qk_norm_rope import make  # noqa: E402


def busy_then(call):
    """call(stream) twice alike: on an idle device, and while the current stream
    still has writes to come into memory of every size that the call may need,
    freed on the host."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    first = call(side)
    side.synchronize()
    want = [None if t is None else t.clone() for t in first]
    torch.cuda.synchronize()
    x = torch.zeros(1 << 24, device="cuda")
    for _ in range(300):                        # some milliseconds of work ahead
        x.add_(1.0)
    held = [torch.empty(n, dtype=torch.uint8, device="cuda")
            for n in [1 << k for k in range(9, 25)] for _ in range(6)]
    for t in held:
        t.fill_(0x55)
    del held, t
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert (g is None) == (w is None)
        if w is not None:
            assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("new", [1, 60])
def test_attention(new):
    rng = np.random.default_rng(new)
    lens, news = [3000, 200], [new, new]
    ref, ka, pt, cu, qb = build(rng, "nvfp4", lens, news, 1, 4, 128, 64)
    am = torch.from_numpy(ka).cuda()
    cache = fp4.KvCache(k_amax=am, v_amax=am, **{k: torch.from_numpy(v).cuda() for k, v in ref.items()})
    args = (cache, tensor(qb), torch.from_numpy(pt).cuda(),
            torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.from_numpy(cu).cuda())
    busy_then(lambda s: fp4.fp4_kv_attention(*args, max_q=new, want_lse=True, stream=s))


def test_read():
    rng = np.random.default_rng(3)
    am = torch.full((2,), 3.0, device="cuda")
    cache = fp4.KvCache.alloc(8, 16, 2, 128, k_amax=am, v_amax=am)
    kb = tensor(R.bf16_bits(rng.standard_normal((128, 2, 128))))
    slots = torch.from_numpy(rng.permutation(128)).cuda()
    fp4.fp4_kv_write(cache, kb, kb, slots)
    busy_then(lambda s: fp4.fp4_kv_read(cache, slots, stream=s))


@pytest.mark.parametrize("t", [3, 500])
def test_norm_and_its_gradient(t):
    q, k, qw, kw, dq, dk, table, pos = make(np.random.default_rng(t), t, 4, 2, 128, 128)
    x = [tensor(v) for v in (q, k, qw, kw)] + [torch.from_numpy(pos).cuda(), table]
    dy = [tensor(v) for v in (dq, dk)]
    busy_then(lambda s: fp4.qk_norm_rope(*x, stream=s))
    busy_then(lambda s: fp4.qk_norm_rope_backward(*dy, *x, stream=s))


def test_stream_forms():
    """A torch stream, its address and the current stream itself."""
    q, k, qw, kw, _, _, table, pos = make(np.random.default_rng(5), 7, 4, 2, 64, 64)
    x = [tensor(v) for v in (q, k, qw, kw)] + [torch.from_numpy(pos).cuda(), table]
    want = fp4.qk_norm_rope(*x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream, torch.cuda.current_stream(), 0):
        got = fp4.qk_norm_rope(*x, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
