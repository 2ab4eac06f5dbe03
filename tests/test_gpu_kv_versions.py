"""Tensors that a call writes at the caller's request count as modified, as by
torch's own operators, so that a backward pass that saved one refuses to use it."""
import numpy as np
import pytest

import kv_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_reduce_amd as fp4  # noqa: E402
from test_gpu_kv_attention import tensor  # noqa: E402
from test_gpu_qk_norm_rope import make  # noqa: E402


def counted(call, *tensors):
    before = [t._version for t in tensors]
    call()
    assert all(t._version > b for t, b in zip(tensors, before))


def setup():
    q, k, qw, kw, dq, dk, table, pos = make(np.random.default_rng(1), 5, 4, 2, 64, 32)
    return ([tensor(v) for v in (q, k, qw, kw)] + [torch.from_numpy(pos).cuda(), table],
            [tensor(v) for v in (dq, dk)])


def test_norm():
    x, dy = setup()
    out = [torch.empty_like(v) for v in x[:2]]
    counted(lambda: fp4.qk_norm_rope(*x, out=out), *out)
    counted(lambda: fp4.qk_norm_rope_backward(*dy, *x, out=out), *out)
    with torch.inference_mode():                # these have no version
        y = [torch.empty_like(v) for v in x[:2]]
        fp4.qk_norm_rope(*x, out=y)
    assert torch.equal(y[0], fp4.qk_norm_rope(*x)[0])


def test_read_and_attention():
    am = torch.full((2,), 3.0, device="cuda")
    cache = fp4.KvCache.alloc(4, 16, 2, 64, k_amax=am, v_amax=am)
    kv = tensor(R.bf16_bits(np.random.default_rng(2).standard_normal((40, 2, 64))))
    slots = torch.arange(40, device="cuda")
    fp4.fp4_kv_write(cache, kv, kv, slots)
    out = torch.empty_like(kv), torch.empty_like(kv)
    counted(lambda: fp4.fp4_kv_read(cache, slots, out=out), *out)
    q = kv[:3, :].contiguous()
    o, lse = torch.empty_like(q), torch.empty(3, 2, device="cuda")
    args = (cache, q, torch.arange(4, dtype=torch.int32, device="cuda")[None],
            torch.tensor([40], dtype=torch.int32, device="cuda"),
            torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    counted(lambda: fp4.fp4_kv_attention(*args, out=o, lse=lse), o, lse)


def test_a_saved_tensor_is_missed():
    x, _ = setup()
    leaf = x[0].float().requires_grad_()
    saved = leaf.bfloat16()
    loss = (saved * saved).sum()
    with torch.no_grad():
        fp4.qk_norm_rope(saved, *x[1:], out=(saved, torch.empty_like(x[1])))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
