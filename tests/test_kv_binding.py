"""Refusals of the compiled binding (wrong types, shapes, devices, argument
counts): all of them come before any GPU call, so no GPU is needed."""
import os

import pytest

import block_scaled_fp4_reduce_amd as fp4

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(fp4.LIB_PATH):
        from block_scaled_fp4_reduce_amd import build
        build.build()


class Handle:
    """A cache handle that was never allocated: only its numbers are read."""

    def __init__(self):
        p = 0x10000
        self._c = fp4._CCache(p, p, p, p, p, p, 4, 16, 2, 64, fp4.FORMAT_NVFP4, 0)
        self._at = fp4.C.addressof(self._c)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_host_tensors_and_types():
    c = Handle()
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        fp4.fp4_kv_write(c, bf(3, 2, 64), bf(3, 2, 64), slots)
    with pytest.raises(TypeError):
        fp4.fp4_kv_write(c, bf(3, 2, 64).float(), bf(3, 2, 64), slots)
    with pytest.raises(TypeError):
        fp4.fp4_kv_write(c, [1.0], bf(3, 2, 64), slots)
    with pytest.raises(ValueError):
        fp4.fp4_kv_read(c, slots)
    with pytest.raises(TypeError):
        fp4.fp4_kv_read(c, slots.int())
    lens = torch.ones(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        fp4.fp4_kv_attention(c, bf(3, 4, 64), torch.zeros(3, 1, dtype=torch.int32), lens)
    with pytest.raises(TypeError):
        fp4.fp4_kv_attention(c, bf(3, 4, 64).half(), torch.zeros(3, 1, dtype=torch.int32), lens)
    with pytest.raises(TypeError):
        fp4.fp4_kv_attention(c, None, torch.zeros(3, 1, dtype=torch.int32), lens)
    pos, table = torch.zeros(3, dtype=torch.int64), torch.zeros(9, 32, 2)
    with pytest.raises(ValueError):
        fp4.qk_norm_rope_backward(bf(3, 2, 64), bf(3, 1, 64), bf(3, 2, 64), bf(3, 1, 64), None, None,
                                  pos, table)
    with pytest.raises(TypeError):
        fp4.qk_norm_rope(None, bf(3, 2, 64), None, None, pos, table)


def test_argument_counts():
    native = fp4._binding()
    for name in ("kv_write", "kv_read", "kv_attention", "kv_attention_ws", "norm_rope",
                 "norm_rope_backward"):
        with pytest.raises(TypeError):
            getattr(native, name)()


def test_rows_are_counted_in_32_bits():
    c = Handle()._c
    p = 0x10000
    x = fp4._CQueries(p, 65536 * 64, 1 << 20, 1 << 20, None, 0, p, p, 5, 65536, 0, 0.1, 0.0)
    assert fp4.lib().fp4_kv_attention(c, x, p, 65536 * 64, None, p, 1 << 40, None) == -2
    assert fp4.lib().fp4_kv_attention_workspace_bytes(c, x) == 0


def test_any_hint_of_new_tokens_plans_the_call():
    c, p = Handle()._c, 0x10000
    for hint in (0, 1, 6, 7, 1 << 62):
        x = fp4._CQueries(p, 256, 6, 3, p, hint, p, p, 40, 4, 0, 0.1, 0.0)
        assert 0 <= fp4.lib().fp4_kv_attention_workspace_bytes(c, x) < 1 << 24
