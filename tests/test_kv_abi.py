"""Refusals of the FP4 cache, attention and norm-with-rotation entry points:
every check runs on the host before any HIP call, so fake pointers are never
dereferenced and no GPU is needed."""
import math
import os

import pytest

import block_scaled_fp4_reduce_amd as fp4

OK, E_NULL, E_SHAPE, E_ALIGN, E_FLAGS, E_WS = 0, -1, -2, -3, -4, -5
P = 0x10000          # a 16-byte-aligned fake device address: never used
F4 = 0x20004         # 4-byte aligned only


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fp4.LIB_PATH):
        from block_scaled_fp4_reduce_amd import build
        build.build()
    return fp4.lib()


def cache(**kw):
    c = fp4._CCache(P, P, P, P, F4, F4, 10, 64, 2, 128, fp4.FORMAT_NVFP4, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


CACHE_BAD = [
    (dict(k_codes=None), E_NULL), (dict(v_scales=None), E_NULL), (dict(k_amax=None), E_NULL),
    (dict(v_amax=None), E_NULL), (dict(pages=-1), E_SHAPE), (dict(page_size=48), E_SHAPE),
    (dict(page_size=8), E_SHAPE), (dict(page_size=8192), E_SHAPE), (dict(heads=0), E_SHAPE),
    (dict(head_dim=96), E_SHAPE), (dict(head_dim=0), E_SHAPE), (dict(format=2), E_FLAGS),
    (dict(flags=fp4.SR), E_FLAGS), (dict(format=fp4.FORMAT_MXFP4, flags=1), E_FLAGS),
    (dict(k_codes=P + 8), E_ALIGN), (dict(v_scales=P + 4), E_ALIGN), (dict(k_amax=F4 + 2), E_ALIGN),
    (dict(pages=1 << 31), E_SHAPE), (dict(pages=1 << 30, heads=65536), E_SHAPE),
]


@pytest.mark.parametrize("kw,want", CACHE_BAD)
def test_bad_cache(L, kw, want):
    c = cache(**kw)
    assert L.fp4_kv_write(c, P, 256, P, 256, P, 4, None) == want
    assert L.fp4_kv_read(c, P, 4, P, 256, P, 256, None) == want
    assert L.fp4_kv_attention(c, queries(), P, 512, None, P, 1 << 40, None) == want
    assert L.fp4_kv_attention_workspace_bytes(c, queries()) == 0


def test_write_and_read_reject(L):
    c = cache()

    def wr(k=P, ks=256, v=P, vs=256, slots=P, n=4):
        return (L.fp4_kv_write(c, k, ks, v, vs, slots, n, None),
                L.fp4_kv_read(c, slots, n, k, ks, v, vs, None))
    assert wr(k=None) == (E_NULL, E_NULL)
    assert wr(v=None) == (E_NULL, E_NULL)
    assert wr(slots=None) == (E_NULL, E_NULL)
    assert wr(n=-1) == (E_SHAPE, E_SHAPE)
    assert wr(n=1 << 40) == (E_SHAPE, E_SHAPE)
    assert wr(ks=248) == (E_SHAPE, E_SHAPE)          # less than heads * head_dim
    assert wr(vs=260) == (E_SHAPE, E_SHAPE)          # not a multiple of 8
    assert wr(ks=1 << 39) == (E_SHAPE, E_SHAPE)
    assert wr(k=P + 8) == (E_ALIGN, E_ALIGN)
    assert wr(slots=F4) == (E_ALIGN, E_ALIGN)
    assert wr(k=None, v=None, slots=None, n=0) == (OK, OK)
    assert L.fp4_kv_write(None, P, 256, P, 256, P, 4, None) == E_NULL
    # a cache without pages takes nothing
    e = cache(pages=0, k_codes=None, k_scales=None, v_codes=None, v_scales=None)
    assert L.fp4_kv_write(e, P, 256, P, 256, P, 4, None) == OK


def queries(**kw):
    x = fp4._CQueries(P, 512, 6, 3, F4, 0, F4, F4, 5, 4, 0, 0.1, 0.0)
    for k, v in kw.items():
        setattr(x, k, v)
    return x


QUERIES_BAD = [
    (dict(q=None), E_NULL), (dict(kv_lens=None), E_NULL), (dict(page_table=None), E_NULL),
    (dict(tokens=-1), E_SHAPE), (dict(seqs=-1), E_SHAPE), (dict(seqs=0), E_SHAPE),
    (dict(max_q=-1), E_SHAPE), (dict(cu_q=None), E_SHAPE),          # 6 tokens, 3 sequences
    (dict(q_heads=3), E_SHAPE), (dict(q_heads=0), E_SHAPE), (dict(q_stride=504), E_SHAPE),
    (dict(q_stride=516), E_SHAPE), (dict(window=-1), E_SHAPE), (dict(softcap=-1.0), E_SHAPE),
    (dict(softcap=math.nan), E_SHAPE), (dict(softcap=math.inf), E_SHAPE),
    (dict(scale=math.nan), E_SHAPE), (dict(scale=math.inf), E_SHAPE),
    (dict(table_width=-1), E_SHAPE), (dict(table_width=1 << 31), E_SHAPE),
    (dict(tokens=1 << 31), E_SHAPE), (dict(q=P + 8), E_ALIGN), (dict(cu_q=F4 + 1), E_ALIGN),
    (dict(kv_lens=F4 + 2), E_ALIGN),
]


@pytest.mark.parametrize("kw,want", QUERIES_BAD)
def test_bad_queries(L, kw, want):
    assert L.fp4_kv_attention(cache(), queries(**kw), P, 512, None, P, 1 << 40, None) == want


def test_attention_rejects(L):
    c, x = cache(), queries()
    assert L.fp4_kv_attention(c, None, P, 512, None, P, 1 << 40, None) == E_NULL
    assert L.fp4_kv_attention(None, x, P, 512, None, P, 1 << 40, None) == E_NULL
    assert L.fp4_kv_attention(c, x, None, 512, None, P, 1 << 40, None) == E_NULL
    assert L.fp4_kv_attention(c, x, P, 504, None, P, 1 << 40, None) == E_SHAPE
    assert L.fp4_kv_attention(c, x, P + 4, 512, None, P, 1 << 40, None) == E_ALIGN
    assert L.fp4_kv_attention(c, x, P, 512, F4 + 2, P, 1 << 40, None) == E_ALIGN
    assert L.fp4_kv_attention(c, x, P, 512, None, P + 4, 1 << 40, None) == E_ALIGN
    assert L.fp4_kv_attention(c, queries(tokens=0, seqs=0, q=None, cu_q=None), None, 512, None,
                              None, 0, None) == OK
    need = L.fp4_kv_attention_workspace_bytes(c, x)
    if need:
        assert L.fp4_kv_attention(c, x, P, 512, None, P, need - 1, None) == E_WS
        assert L.fp4_kv_attention(c, x, P, 512, None, None, need, None) == E_NULL


def rope(**kw):
    a = fp4._CRope(P, P, 512, 256, 6, P, P, P, P, 100, 4, 2, 128, 128, 1e-6, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


ROPE_BAD = [
    (dict(q=None), E_NULL), (dict(k=None), E_NULL), (dict(positions=None), E_NULL),
    (dict(table=None), E_NULL), (dict(tokens=-1), E_SHAPE), (dict(q_heads=-1), E_SHAPE),
    (dict(head_dim=130), E_SHAPE), (dict(head_dim=264), E_SHAPE), (dict(head_dim=8), E_SHAPE),
    (dict(rot_dim=24), E_SHAPE), (dict(rot_dim=144), E_SHAPE), (dict(table_rows=0), E_SHAPE),
    (dict(q_stride=504), E_SHAPE), (dict(k_stride=260), E_SHAPE), (dict(eps=-1.0), E_SHAPE),
    (dict(eps=math.nan), E_SHAPE), (dict(flags=2), E_FLAGS), (dict(q=P + 8), E_ALIGN),
    (dict(q_weight=P + 2), E_ALIGN), (dict(table=F4), E_ALIGN), (dict(positions=F4), E_ALIGN),
]


@pytest.mark.parametrize("kw,want", ROPE_BAD)
def test_bad_rope(L, kw, want):
    a = rope(**kw)
    assert L.qk_norm_rope(a, P, 512, P, 256, None) == want
    assert L.qk_norm_rope_backward(a, P, 512, P, 256, P, 512, P, 256, F4, F4, P, 1 << 30,
                                   None) == want


def test_rope_rejects(L):
    a = rope()
    assert L.qk_norm_rope(None, P, 512, P, 256, None) == E_NULL
    assert L.qk_norm_rope(a, None, 512, P, 256, None) == E_NULL
    assert L.qk_norm_rope(a, P, 504, P, 256, None) == E_SHAPE
    assert L.qk_norm_rope(a, P, 512, P + 8, 256, None) == E_ALIGN
    assert L.qk_norm_rope(rope(tokens=0, q=None, k=None), None, 512, None, 256, None) == OK
    need = L.qk_norm_rope_workspace_bytes(128)
    assert need > 0 and L.qk_norm_rope_workspace_bytes(0) == 0

    def bwd(dqo=P, dko=P, dq=P, dk=P, wq=F4, wk=F4, ws=P, n=need, a=a):
        return L.qk_norm_rope_backward(a, dqo, 512, dko, 256, dq, 512, dk, 256, wq, wk, ws, n, None)
    assert bwd(dqo=None) == E_NULL
    assert bwd(dk=None) == E_NULL
    assert bwd(ws=None) == E_NULL
    assert bwd(n=need - 1) == E_WS
    assert bwd(wq=F4 + 2) == E_ALIGN
    assert bwd(dq=P + 4) == E_ALIGN
    assert bwd(a=rope(q_weight=None)) == E_NULL       # a gradient of no weight


def test_tensor_layer_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fp4.KvCache(u8(2, 1, 16, 32), u8(2, 1, 16, 4), u8(2, 1, 32, 16), u8(2, 1, 4, 16),
                    torch.ones(1), torch.ones(1))
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fp4.qk_norm_rope(q, q, None, None, torch.zeros(3, dtype=torch.int64), torch.zeros(9, 32, 2))
    with pytest.raises(TypeError):
        fp4.qk_norm_rope(q.float(), q, None, None, torch.zeros(3, dtype=torch.int64),
                         torch.zeros(9, 32, 2))
