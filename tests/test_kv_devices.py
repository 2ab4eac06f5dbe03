"""Tensors of one call on different GPUs are refused before any of their memory
is looked at.  Tensors without memory stand in for those of two GPUs, so that
none is needed."""
import os

import pytest

import block_scaled_fp4_reduce_amd as fp4
from test_kv_handle import buffers

torch = pytest.importorskip("torch")
from torch._subclasses.fake_tensor import FakeTensorMode  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(fp4.LIB_PATH):
        from block_scaled_fp4_reduce_amd import build
        build.build()


def fake(device, dtype, *shape):
    """A tensor of a GPU that holds nothing: only its description is read."""
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device=device)


BF, I64, I32, F32 = torch.bfloat16, torch.int64, torch.int32, torch.float32

CALLS = {  # name: (call, its tensors)
    "write": (lambda c, *t: fp4.fp4_kv_write(c, *t), [(BF, 3, 2, 64), (BF, 3, 2, 64), (I64, 3)]),
    "read": (lambda c, s, k, v: fp4.fp4_kv_read(c, s, out=(k, v)),
             [(I64, 3), (BF, 3, 2, 64), (BF, 3, 2, 64)]),
    "attention": (lambda c, q, t, n, cu, o, l, ws: fp4.fp4_kv_attention(c, q, t, n, cu, out=o, lse=l, ws=ws),
                  [(BF, 3, 4, 64), (I32, 1, 2), (I32, 1), (I32, 2), (BF, 3, 4, 64), (F32, 3, 4),
                   (torch.uint8, 999)]),
    "workspace": (lambda c, *t: fp4.fp4_kv_attention_workspace_bytes(c, *t),
                  [(BF, 3, 4, 64), (I32, 1, 2), (I32, 1), (I32, 2)]),
    "norm": (lambda c, q, k, qw, kw, p, t, a, b: fp4.qk_norm_rope(q, k, qw, kw, p, t, out=(a, b)),
             [(BF, 3, 2, 64), (BF, 3, 1, 64), (BF, 64), (BF, 64), (I64, 3), (F32, 9, 32, 2),
              (BF, 3, 2, 64), (BF, 3, 1, 64)]),
    "backward": (lambda c, *t: fp4.qk_norm_rope_backward(*t[:8], out=t[8:10], ws=t[10]),
                 [(BF, 3, 2, 64), (BF, 3, 1, 64), (BF, 3, 2, 64), (BF, 3, 1, 64), (BF, 64), (BF, 64),
                  (I64, 3), (F32, 9, 32, 2), (BF, 3, 2, 64), (BF, 3, 1, 64), (torch.uint8, 999)]),
}


@pytest.mark.parametrize("name,other", [(n, i) for n, (_, t) in CALLS.items() for i in range(len(t))])
def test_one_tensor_elsewhere(name, other):
    call, tensors = CALLS[name]
    cache = fp4.KvCache(**buffers("cuda:0"))
    made = [fake("cuda:1" if i == other else "cuda:0", *t) for i, t in enumerate(tensors)]
    with pytest.raises(ValueError, match="device"):
        call(cache, *made)


@pytest.mark.parametrize("name", ["write", "read", "attention", "workspace"])
def test_cache_elsewhere(name):
    call, tensors = CALLS[name]
    cache = fp4.KvCache(**buffers("cuda:1"))
    with pytest.raises(ValueError, match="device"):
        call(cache, *[fake("cuda:0", *t) for t in tensors])


@pytest.mark.parametrize("name", ["k_scales", "v_codes", "v_scales", "k_amax", "v_amax"])
def test_cache_on_two_devices(name):
    b = buffers("cuda:0")
    b[name] = buffers("cuda:1")[name]
    with pytest.raises(ValueError, match="device"):
        fp4.KvCache(**b)
