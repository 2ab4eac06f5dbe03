"""Refusals of the feed-forward calls and of the weights handle (types, shapes,
devices, argument counts): all of them come before any GPU call.  Tensors
without memory stand in for those of GPUs."""
import copy
import os

import pytest

import block_scaled_fp4_reduce_amd as fp4

torch = pytest.importorskip("torch")
from torch._subclasses.fake_tensor import FakeTensorMode  # noqa: E402

BF, I32, F32, U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(fp4.LIB_PATH):
        from block_scaled_fp4_reduce_amd import build
        build.build()


def fake(device, dtype, *shape):
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device=device)


def weights(device="cuda:0", lead=(), rows=64, cols=96):
    """A handle of weights that are nowhere."""
    class Handle:
        pass
    h = Handle()
    h._c = fp4._CWeights(0x10000, 0x10000, 0x10000, lead[0] if lead else 1, rows, cols, 0, 0)
    h._at = fp4._Address(h._c, torch.device(device).index)
    return h


def linear(w, x, out, ws):
    return fp4.fp4_linear(w[0], x, out=out, ws=ws)


def experts(w, x, wt, ids, out, ws):
    return fp4.fp4_experts(w[1], w[2], x, wt, ids, out=out, ws=ws)


CALLS = {
    "linear": (linear, [(BF, 5, 96), (BF, 5, 64), (U8, 99)]),
    "experts": (experts, [(BF, 5, 96), (F32, 5, 2), (I32, 5, 2), (BF, 5, 96), (U8, 99)]),
    "route": (lambda w, x, b, o, e: fp4.expert_route(x, 3, bias=b, out=(o, e)),
              [(F32, 5, 60), (F32, 60), (F32, 5, 3), (I32, 5, 3)]),
    "route_backward": (lambda w, g, x, e, o: fp4.expert_route_backward(g, x, e, out=o),
                       [(F32, 5, 3), (F32, 5, 60), (I32, 5, 3), (F32, 5, 60)]),
    "residual": (lambda w, x, b, wt, bw, g, y, z: fp4.residual_norm(x, b, wt, bw, g, out=(y, z)),
                 [(BF, 5, 64), (BF, 5, 64), (BF, 64), (BF, 64), (BF, 64), (BF, 5, 64), (BF, 5, 64)]),
    "residual_backward": (
        lambda w, *t: fp4.residual_norm_backward(*t[:7], out=t[7:9], ws=t[9]),
        [(BF, 5, 64)] * 4 + [(BF, 64), (BF, 64), (BF, 5, 1), (BF, 5, 64), (BF, 5, 64), (U8, 99)]),
}


def handles(device="cuda:0"):
    return weights(device), weights(device, (4,), 128, 96), weights(device, (4,), 96, 64)


@pytest.mark.parametrize("name,other", [(n, i) for n, (_, t) in CALLS.items() for i in range(len(t))])
def test_one_tensor_elsewhere(name, other):
    call, tensors = CALLS[name]
    made = [fake("cuda:1" if i == other else "cuda:0", *t) for i, t in enumerate(tensors)]
    with pytest.raises(ValueError, match="device"):
        call(handles(), *made)


@pytest.mark.parametrize("name", ["linear", "experts"])
def test_weights_elsewhere(name):
    call, tensors = CALLS[name]
    with pytest.raises(ValueError, match="device"):
        call(handles("cuda:1"), *[fake("cuda:0", *t) for t in tensors])


@pytest.mark.parametrize("name,which", [(n, i) for n, (_, t) in CALLS.items()
                                        for i in range(len(t)) if t[i][0] is not U8])
def test_host_tensors_types_and_shapes(name, which):
    call, tensors = CALLS[name]

    def at(i, make):
        return [make(*t) if j == i else fake("cuda:0", *t) for j, t in enumerate(tensors)]
    with pytest.raises(ValueError):
        call(handles(), *[torch.empty(t[1:], dtype=t[0]) for t in tensors])
    with pytest.raises(TypeError):
        call(handles(), *at(which, lambda d, *s: fake("cuda:0", torch.float16, *s)))
    with pytest.raises((ValueError, fp4.Fp4Error)):
        call(handles(), *at(which, lambda d, *s: fake("cuda:0", d, *s[:-1], s[-1] + 1)))
    with pytest.raises(TypeError):
        call(handles(), *at(which, lambda d, *s: 1.5))


def test_argument_counts():
    native = fp4._binding()
    for name in ("linear", "experts", "experts_ws", "route", "route_backward", "residual",
                 "residual_backward"):
        with pytest.raises(TypeError):
            getattr(native, name)()


def test_choices():
    x = fake("cuda:0", F32, 5, 60)
    with pytest.raises(ValueError, match="scores"):
        fp4.expert_route(x, 3, scores="relu")
    with pytest.raises(TypeError, match="scores"):
        fp4.expert_route(x, 3, scores=1)
    with pytest.raises(TypeError, match="dtype"):
        fp4.fp4_linear(weights(), fake("cuda:0", BF, 5, 96), dtype=torch.float16)
    with pytest.raises(ValueError):
        fp4.expert_route(x, 1 << 40)


HANDLES = {
    "plain": ((U8, 64, 48), (U8, 64, 6), (F32, 1), 0, 0),
    "rows": ((U8, 64, 48), (U8, 64, 6), (F32, 64), 0, fp4.ROW_ALPHA),
    "tiles": ((U8, 64, 48), (U8, 4, 6), (F32, 1), 0, fp4.BLOCK2D),
    "experts": ((U8, 3, 64, 48), (U8, 3, 64, 6), (F32, 3), 0, 0),
    "expert rows": ((U8, 3, 64, 48), (U8, 3, 64, 6), (F32, 3, 64), 0, fp4.ROW_ALPHA),
    "expert tiles": ((U8, 3, 64, 48), (U8, 3, 4, 6), (F32, 3), 0, fp4.BLOCK2D),
    "mx": ((U8, 64, 48), (U8, 64, 3), None, 1, 0),
    "one row": ((U8, 1, 48), (U8, 1, 6), (F32, 1), 0, 0),
}


@pytest.mark.parametrize("name", HANDLES)
def test_handles(name):
    codes, scales, alpha, fmt, flags = HANDLES[name]
    new = lambda t, d="cuda:0": None if t is None else fake(d, *t)
    with FakeTensorMode(allow_non_fake_inputs=True):
        w = fp4.Fp4Weights(new(codes), new(scales), new(alpha), fmt)
        assert (w.flags, w.rows, w.cols) == (flags, codes[-2], 96)
        assert w.experts == (codes[1] if len(codes) == 4 else 1)
        for field in ("codes", "alpha", "rows", "_at"):
            with pytest.raises(AttributeError):
                setattr(w, field, None)
        with pytest.raises(AttributeError):
            del w.codes
        assert copy.copy(w) is w
        with pytest.raises(ValueError):
            fp4.Fp4Weights(new(codes), fake("cuda:0", U8, *scales[1:-1], scales[-1] + 1), new(alpha), fmt)
        with pytest.raises(ValueError):
            fp4.Fp4Weights(new(codes), new(scales, "cuda:1"), new(alpha), fmt)
        with pytest.raises(TypeError):
            fp4.Fp4Weights(fake("cuda:0", torch.int8, *codes[1:]), new(scales), new(alpha), fmt)
        with pytest.raises(ValueError):
            fp4.Fp4Weights(new(codes, "cpu"), new(scales, "cpu"), new(alpha, "cpu"), fmt)
        with pytest.raises(ValueError):
            fp4.Fp4Weights(new(codes), new(scales), fake("cuda:0", F32, 2) if fmt else None, fmt)
        with pytest.raises(ValueError):
            fp4.Fp4Weights(fake("cuda:0", U8, 48), new(scales), new(alpha), fmt)
