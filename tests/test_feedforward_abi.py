"""Refusals of the feed-forward entry points: every check runs on the host
before any HIP call, so fake pointers are never dereferenced and no GPU is needed."""
import math
import os

import pytest

import block_scaled_fp4_reduce_amd as fp4

OK, E_NULL, E_SHAPE, E_ALIGN, E_FLAGS, E_WS = 0, -1, -2, -3, -4, -5
P = 0x10000          # a 16-byte-aligned fake device address: never used
F4 = 0x20004         # 4-byte aligned only
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fp4.LIB_PATH):
        from block_scaled_fp4_reduce_amd import build
        build.build()
    return fp4.lib()


def weights(**kw):
    w = fp4._CWeights(P, P, F4, 1, 64, 96, fp4.FORMAT_NVFP4, 0)
    for k, v in kw.items():
        setattr(w, k, v)
    return w


WEIGHTS_BAD = [
    (dict(codes=None), E_NULL), (dict(scales=None), E_NULL), (dict(alpha=None), E_NULL),
    (dict(codes=P + 8), E_ALIGN), (dict(scales=P + 1), E_ALIGN), (dict(alpha=F4 + 2), E_ALIGN),
    (dict(rows=-1), E_SHAPE), (dict(cols=-32), E_SHAPE), (dict(cols=80), E_SHAPE),
    (dict(experts=-1), E_SHAPE), (dict(rows=1 << 24), E_SHAPE), (dict(cols=1 << 22), E_SHAPE),
    (dict(format=2), E_FLAGS), (dict(format=-1), E_FLAGS), (dict(flags=fp4.RHT16), E_FLAGS),
    (dict(flags=fp4.HAD32), E_FLAGS), (dict(format=fp4.FORMAT_MXFP4, flags=fp4.ROW_ALPHA), E_FLAGS),
    (dict(format=fp4.FORMAT_MXFP4, flags=fp4.BLOCK2D), E_FLAGS),
    (dict(flags=fp4.BLOCK2D, rows=72), E_SHAPE),
    (dict(experts=1 << 20, rows=1 << 20, cols=1 << 20), E_SHAPE),
]


def linear(L, w, x=P, xs=96, tokens=5, out=P, os_=64, f32=0):
    return L.fp4_linear(w, x, xs, tokens, out, os_, f32, None, 0, None)


@pytest.mark.parametrize("kw,want", WEIGHTS_BAD)
def test_bad_weights(L, kw, want):
    w = weights(**kw)
    assert linear(L, w) == want
    assert L.fp4_linear_workspace_bytes(w, 5) == 0


def test_linear_rejects(L):
    w = weights()
    assert linear(L, None) == E_NULL
    assert linear(L, w, x=None) == E_NULL
    assert linear(L, w, out=None) == E_NULL
    assert linear(L, weights(experts=2)) == E_SHAPE
    assert linear(L, w, tokens=-1) == E_SHAPE
    assert linear(L, w, tokens=1 << 31) == E_SHAPE
    assert linear(L, w, xs=88) == E_SHAPE            # less than a row
    assert linear(L, w, xs=100) == E_SHAPE           # not a multiple of 8
    assert linear(L, w, os_=63) == E_SHAPE
    assert linear(L, w, xs=1 << 39) == E_SHAPE
    assert linear(L, w, xs=1 << 23) == E_SHAPE
    assert linear(L, w, x=P + 8) == E_ALIGN
    assert linear(L, w, out=P + 1) == E_ALIGN
    assert linear(L, w, out=P + 2, f32=1) == E_ALIGN
    assert linear(L, w, tokens=0, x=None, out=None) == OK
    assert linear(L, weights(rows=0, codes=None, scales=None), out=None) == OK


def experts(L, gu, dn, x=P, xs=96, tokens=5, w=F4, ids=F4, k=2, out=P, os_=96, ws=P, wsb=BIG):
    return L.fp4_experts(gu, dn, x, xs, tokens, w, ids, k, out, os_, ws, wsb, None)


def pair(**kw):
    return weights(experts=4, rows=128, cols=96, **kw), weights(experts=4, rows=96, cols=64, **kw)


@pytest.mark.parametrize("kw,want", WEIGHTS_BAD)
def test_bad_experts(L, kw, want):
    gu, dn = pair()
    for k, v in kw.items():
        setattr(gu, k, v)
    assert experts(L, gu, dn) != OK
    if want in (E_NULL, E_ALIGN, E_FLAGS):
        assert experts(L, gu, dn) == want
    gu, dn = pair()
    for k, v in kw.items():
        setattr(dn, k, v)
    assert experts(L, gu, dn) != OK
    assert L.fp4_experts_workspace_bytes(gu, dn, 5, 2) == 0


def test_experts_reject(L):
    gu, dn = pair()
    assert experts(L, None, dn) == E_NULL and experts(L, gu, None) == E_NULL
    for name in ("x", "w", "ids", "out", "ws"):
        assert experts(L, gu, dn, **{name: None}) == E_NULL
    assert experts(L, gu, weights(experts=3, rows=96, cols=64)) == E_SHAPE
    assert experts(L, gu, weights(experts=4, rows=96, cols=96)) == E_SHAPE
    assert experts(L, gu, weights(experts=4, rows=64, cols=64)) == E_SHAPE
    many = [weights(experts=1025, rows=r, cols=c) for r, c in ((128, 96), (96, 64))]
    assert experts(L, *many) == E_SHAPE
    assert experts(L, gu, dn, tokens=-1) == E_SHAPE
    assert experts(L, gu, dn, k=0) == E_SHAPE
    assert experts(L, gu, dn, k=65) == E_SHAPE
    assert experts(L, gu, dn, tokens=1 << 31) == E_SHAPE
    assert experts(L, gu, dn, xs=88) == E_SHAPE
    assert experts(L, gu, dn, os_=100) == E_SHAPE
    assert experts(L, gu, dn, xs=1 << 23) == E_SHAPE
    assert experts(L, gu, dn, x=P + 8) == E_ALIGN
    assert experts(L, gu, dn, out=P + 8) == E_ALIGN
    assert experts(L, gu, dn, ids=F4 + 2) == E_ALIGN
    assert experts(L, gu, dn, ws=P + 8) == E_ALIGN
    need = L.fp4_experts_workspace_bytes(gu, dn, 5, 2)
    assert need > 0 and experts(L, gu, dn, wsb=need - 1) == E_WS
    assert experts(L, gu, dn, tokens=0, x=None, w=None, ids=None, out=None, ws=None, wsb=0) == OK


def routing(**kw):
    r = fp4._CRouting(P, 60, 7, None, 60, 4, 1, 1, 1, 0, 1, 0, 1.0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


ROUTING_BAD = [
    (dict(logits=None), E_NULL), (dict(tokens=-1), E_SHAPE), (dict(tokens=1 << 31), E_SHAPE),
    (dict(experts=0), E_SHAPE), (dict(experts=1025, stride=1025), E_SHAPE), (dict(top_k=0), E_SHAPE),
    (dict(top_k=65, experts=128, stride=128), E_SHAPE), (dict(top_k=61), E_SHAPE),
    (dict(stride=59), E_SHAPE), (dict(scale=math.nan), E_SHAPE), (dict(scale=math.inf), E_SHAPE),
    (dict(logits=P + 2), E_ALIGN), (dict(logits=P + 1, logits_bf16=1), E_ALIGN),
]
CHOICE_BAD = [
    (dict(groups=0), E_SHAPE), (dict(groups=7), E_SHAPE), (dict(groups=60, top_groups=61), E_SHAPE),
    (dict(groups=4, top_groups=0), E_SHAPE), (dict(groups=30, top_groups=1), E_SHAPE),
    (dict(group_top=0), E_SHAPE), (dict(group_top=3), E_SHAPE), (dict(bias=F4 + 1), E_ALIGN),
    (dict(groups=65, experts=65, stride=65, top_groups=65), E_SHAPE),
]


@pytest.mark.parametrize("kw,want", ROUTING_BAD + CHOICE_BAD)
def test_bad_routing(L, kw, want):
    assert L.expert_route(routing(**kw), F4, F4, None) == want


@pytest.mark.parametrize("kw,want", ROUTING_BAD)
def test_bad_routing_backward(L, kw, want):
    stride = kw.get("stride", 60)
    assert L.expert_route_backward(routing(**kw), F4, F4, P, stride, None) == want


def test_routing_rejects(L):
    r = routing()
    assert L.expert_route(None, F4, F4, None) == E_NULL
    assert L.expert_route(r, None, F4, None) == E_NULL
    assert L.expert_route(r, F4, None, None) == E_NULL
    assert L.expert_route(r, F4 + 2, F4, None) == E_ALIGN
    assert L.expert_route(routing(tokens=0, logits=None), None, None, None) == OK
    assert L.expert_route_backward(None, F4, F4, P, 60, None) == E_NULL
    assert L.expert_route_backward(r, None, F4, P, 60, None) == E_NULL
    assert L.expert_route_backward(r, F4, F4, None, 60, None) == E_NULL
    assert L.expert_route_backward(r, F4, F4, P, 59, None) == E_SHAPE
    assert L.expert_route_backward(r, F4, F4, P + 2, 60, None) == E_ALIGN
    assert L.expert_route_backward(routing(tokens=0, logits=None), None, None, None, 60, None) == OK


def residual(**kw):
    a = fp4._CResidual(P, P, 64, 64, 6, P, P, P, 0, 64, 1.0, 1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


RESIDUAL_BAD = [
    (dict(x=None), E_NULL), (dict(block=None), E_NULL), (dict(weight=None), E_NULL),
    (dict(tokens=-1), E_SHAPE), (dict(tokens=1 << 31), E_SHAPE), (dict(dim=0), E_SHAPE),
    (dict(dim=60), E_SHAPE), (dict(dim=16392, x_stride=16392, block_stride=16392), E_SHAPE),
    (dict(x_stride=56), E_SHAPE), (dict(block_stride=68), E_SHAPE), (dict(eps=-1.0), E_SHAPE),
    (dict(eps=math.nan), E_SHAPE), (dict(eps=math.inf), E_SHAPE), (dict(scale=math.nan), E_SHAPE),
    (dict(scale=math.inf), E_SHAPE), (dict(x=P + 8), E_ALIGN), (dict(weight=P + 2), E_ALIGN),
    (dict(block_weight=P + 2), E_ALIGN), (dict(gate=P + 2), E_ALIGN),
    (dict(gate=P + 1, token_gate=1), E_ALIGN),
]


@pytest.mark.parametrize("kw,want", RESIDUAL_BAD)
def test_bad_residual(L, kw, want):
    a = residual(**kw)
    s = max(64, a.dim)
    assert L.residual_norm(a, P, s, P, s, None) == want
    assert L.residual_norm_backward(a, P, s, P, s, P, s, P, s, None, None, None, P, BIG, None) == want


def test_residual_rejects(L):
    a = residual()

    def back(a=a, dy=P, dz=P, dx=P, db=P, s=64, dbw=F4, dw=F4, dg=F4, ws=P, wsb=BIG):
        return L.residual_norm_backward(a, dy, s, dz, s, dx, s, db, s, dbw, dw, dg, ws, wsb, None)
    assert L.residual_norm(None, P, 64, P, 64, None) == E_NULL
    assert L.residual_norm(a, None, 64, P, 64, None) == E_NULL
    assert L.residual_norm(a, P, 64, None, 64, None) == E_NULL
    assert L.residual_norm(a, P, 56, P, 64, None) == E_SHAPE
    assert L.residual_norm(a, P, 64, P + 8, 64, None) == E_ALIGN
    assert L.residual_norm(residual(tokens=0, x=None, block=None), None, 64, None, 64, None) == OK
    assert back(a=None) == E_NULL
    for name in ("dy", "dz", "dx", "db", "ws"):
        assert back(**{name: None}) == E_NULL
    assert back(s=60) == E_SHAPE
    assert back(a=residual(block_weight=None)) == E_NULL      # a gradient of nothing
    assert back(a=residual(gate=None)) == E_NULL
    assert back(dw=F4 + 2) == E_ALIGN
    assert back(wsb=L.residual_norm_workspace_bytes(6, 64) - 1) == E_WS
    assert L.residual_norm_workspace_bytes(-1, 64) == 0 and L.residual_norm_workspace_bytes(6, 4) == 0
    none = dict(dbw=None, dw=None, dg=None, ws=None, wsb=0, dy=None, dz=None, dx=None, db=None)
    assert back(a=residual(tokens=0, x=None, block=None), **none) == OK
