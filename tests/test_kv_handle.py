"""The cache handle: its fields are fixed once its addresses are taken.  Stand-ins
for GPU tensors, so that no GPU is needed."""
import copy

import pytest

import block_scaled_fp4_reduce_amd as fp4

torch = pytest.importorskip("torch")


class Stand:
    """What the handle reads of a tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, at, device="cuda:0"):
        self.shape, self.dtype, self.at, self.device = torch.Size(shape), dtype, at, torch.device(device)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


def buffers(device="cuda:0"):
    u8 = lambda at, *s: Stand((4, 2) + s, torch.uint8, at, device)
    am = lambda at: Stand((2,), torch.float32, at, device)
    return dict(k_codes=u8(0x100, 16, 32), k_scales=u8(0x200, 16, 4), v_codes=u8(0x300, 32, 16),
                v_scales=u8(0x400, 4, 16), k_amax=am(0x500), v_amax=am(0x600))


FIELDS = ["k_codes", "k_scales", "v_codes", "v_scales", "k_amax", "v_amax", "fmt", "flags", "pages",
          "heads", "page_size", "head_dim", "_at", "_c"]


@pytest.mark.parametrize("name", FIELDS)
def test_fields_are_fixed(name):
    """A field that could be set would leave the calls with the old address."""
    b = buffers()
    cache = fp4.KvCache(flags=fp4.FOUR_OVER_SIX, **b)
    before = getattr(cache, name)
    with pytest.raises(AttributeError):
        setattr(cache, name, buffers().get(name, 1))
    with pytest.raises(AttributeError):
        delattr(cache, name)
    assert getattr(cache, name) is before


def test_struct_holds_what_the_fields_say():
    b = buffers()
    cache = fp4.KvCache(flags=fp4.FOUR_OVER_SIX, **b)
    for n in FIELDS[:6]:
        assert getattr(cache, n) is b[n] and getattr(cache._c, n) == b[n].at
    assert (cache.pages, cache.heads, cache.page_size, cache.head_dim) == (4, 2, 16, 64)
    c = cache._c
    assert (c.pages, c.heads, c.page_size, c.head_dim, c.format, c.flags) == (4, 2, 16, 64, 0, 1)
    assert cache._at == fp4.C.addressof(c)


def test_no_unknown_fields():
    with pytest.raises(AttributeError):
        fp4.KvCache(**buffers()).k_max = 1.0


def test_a_copy_shares_the_buffers():
    cache = fp4.KvCache(**buffers())
    again = copy.copy(cache)
    assert again.k_codes is cache.k_codes and again._at == fp4.C.addressof(again._c)
