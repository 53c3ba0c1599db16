"""The block operators reject bad arguments before touching the GPU (CPU only:
every call here fails validation or has nothing to do)."""
import ctypes as C

import pytest
import torch

import mxfp4_routed_expert_e2m1_amd as m
from mxfp4_routed_expert_e2m1_amd import block as b

OK, INVALID, SHAPE, STRIDE, WORKSPACE, ALIGN = 0, -1, -2, -3, -4, -5
A = C.c_void_p(0x100000)     # fake device address, never dereferenced
MIS4 = C.c_void_p(0x100002)  # not 4-byte aligned
MIS = C.c_void_p(0x100004)   # 4-byte aligned only


def norm(d=64, post=1, eps=1e-6, rs=1.0, pre_w=0, post_w=0):
    return C.byref(b.moe_norm_t(d, post, eps, rs, pre_w, post_w))


def test_norm_pre_validation():
    f = m.lib().moe_norm_pre

    def call(N=None, x=A, xt=0, ldx=64, rows=4, h=A, ht=0, ldh=64, quant=0, q=A, ldq=64, qs=A,
             ldqs=2):
        return f(N or norm(), x, xt, ldx, rows, h, ht, ldh, quant, q, ldq, qs, ldqs, None)
    assert f(None, A, 0, 64, 4, A, 0, 64, 0, A, 64, A, 2, None) == INVALID
    assert call(rows=0, x=None, h=None) == OK
    assert call(N=norm(d=0)) == SHAPE
    assert call(N=norm(d=16385)) == SHAPE
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert call(N=norm(eps=bad)) == INVALID
    assert call(N=norm(rs=float("nan"))) == INVALID
    assert call(N=norm(post=2)) == INVALID
    assert call(N=norm(pre_w=0x100002)) == ALIGN
    assert call(rows=-1) == INVALID
    assert call(xt=2) == INVALID
    assert call(x=None) == INVALID
    assert call(ldx=63) == STRIDE
    assert call(x=MIS4) == ALIGN
    assert call(h=None) == INVALID              # neither rows nor codes asked for
    assert call(ht=5) == INVALID
    assert call(ldh=63) == STRIDE
    assert call(h=MIS4) == ALIGN
    assert call(quant=3) == INVALID
    assert call(quant=1, q=None) == INVALID
    assert call(quant=2, qs=None) == INVALID
    assert call(N=norm(d=48), quant=1) == SHAPE
    assert call(quant=1, ldq=56) == STRIDE
    assert call(quant=1, ldqs=1) == STRIDE
    assert call(quant=2, ldqs=0) == STRIDE
    assert call(quant=1, q=MIS) == ALIGN
    assert call(quant=1, ldq=68) == ALIGN
    assert call(quant=2, qs=MIS4) == ALIGN


def test_norm_post_validation():
    f = m.lib().moe_norm_post

    def call(N=None, y=A, yt=0, ldy=64, res=A, rt=0, ldr=64, gate=None, gt=0, gr=0, gc=0, rows=4,
             out=A, ldo=64, nx=None, h=A, ht=0, ldh=64, quant=0, q=A, ldq=64, qs=A, ldqs=2):
        return f(N or norm(), y, yt, ldy, res, rt, ldr, gate, gt, gr, gc, rows, out, ldo, nx, h,
                 ht, ldh, quant, q, ldq, qs, ldqs, None)
    assert call(rows=0, y=None, res=None, out=None) == OK
    assert call(N=norm(d=0)) == SHAPE
    assert call(rows=-1) == INVALID
    assert call(yt=9) == INVALID
    assert call(rt=-1) == INVALID
    for k in ("y", "res", "out"):
        assert call(**{k: None}) == INVALID
        assert call(**{k: MIS4}) == ALIGN
    for k in ("ldy", "ldr", "ldo"):
        assert call(**{k: 63}) == STRIDE
    assert call(gate=A, gt=7) == INVALID
    assert call(gate=A, gr=-1) == INVALID
    assert call(gate=A, gc=2) == INVALID
    assert call(gate=MIS4) == ALIGN
    assert call(nx=norm(d=65)) == SHAPE
    assert call(nx=norm(eps=0.0)) == INVALID
    assert call(nx=norm(), h=None) == INVALID
    assert call(nx=norm(), ldh=1) == STRIDE
    assert call(nx=norm(), quant=1, ldq=60) == STRIDE
    assert call(nx=norm(), quant=2, ldq=68) == ALIGN


def test_quant_row_validation():
    f = m.lib().moe_quant_row_q8

    def call(x=A, xt=0, ldx=64, rows=4, cols=64, q=A, ldq=64, s=A):
        return f(x, xt, ldx, rows, cols, q, ldq, s, None)
    assert call(rows=0, x=None, q=None, s=None) == OK
    assert call(rows=-1) == INVALID
    assert call(xt=2) == INVALID
    assert call(cols=0) == SHAPE
    for k in ("x", "q", "s"):
        assert call(**{k: None}) == INVALID
    assert call(ldx=63) == STRIDE
    assert call(ldq=56) == STRIDE
    assert call(x=MIS4) == ALIGN
    assert call(q=MIS) == ALIGN
    assert call(ldq=68) == ALIGN
    assert call(s=MIS4) == ALIGN


def rule(E=256, k=6, G=8, top=4, score=1, gs=1, renorm=1, scale=1.0, bias=0):
    return C.byref(b.moe_router_rule_t(E, k, G, top, score, gs, renorm, scale, bias))


def test_route_scored_validation():
    L = m.lib()

    def call(R=None, lg=A, lt=0, ldl=256, rows=4, ids=A, w=A, counts=A, offsets=A, srt=A, ws=A,
             wsb=1 << 30):
        return L.moe_route_scored(R or rule(), lg, lt, ldl, rows, ids, w, counts, offsets, srt,
                                  ws, wsb, None)
    assert L.moe_route_scored(None, A, 0, 256, 4, A, A, A, A, A, A, 1 << 30, None) == INVALID
    for kw in (dict(E=0), dict(E=520), dict(E=255), dict(G=0), dict(G=128), dict(top=0),
               dict(top=9), dict(k=0), dict(k=17), dict(E=16, k=9, G=8, top=4)):
        assert call(R=rule(**kw), ldl=1024) == SHAPE, kw
    for kw in (dict(score=2), dict(gs=-1), dict(renorm=2), dict(scale=float("inf"))):
        assert call(R=rule(**kw)) == INVALID, kw
    assert call(R=rule(bias=0x100001)) == ALIGN
    assert call(rows=-1) == INVALID
    assert call(lt=4) == INVALID
    for k in ("lg", "ids", "w", "counts", "offsets", "srt"):
        assert call(**{k: None}) == INVALID
        assert call(**{k: C.c_void_p(0x100001)}) == ALIGN
    assert call(ldl=255) == STRIDE
    assert call(rows=1 << 22) == SHAPE
    assert call(rows=100, ws=None) == INVALID
    assert call(rows=100, wsb=16) == WORKSPACE
    assert call(rows=100, ws=C.c_void_p(0x100008)) == ALIGN
    assert L.moe_route_scored_workspace_bytes(rule(), 16) == 0
    assert L.moe_route_scored_workspace_bytes(rule(k=99), 1000) == 0
    assert 0 < L.moe_route_scored_workspace_bytes(rule(), 1 << 21) <= 512 * 256 * 2


def lin(N=64, K=64, w=0x100000, ldw=64, ws=0x100000, bias=0):
    return C.byref(b.moe_linear_t(N, K, w, ldw, ws, bias))


def test_linear_validation():
    L = m.lib()

    def call(lay=None, q=A, ldq=64, qs=A, rows=4, y=A, yt=0, ldy=64, ws=A, wsb=1 << 30):
        return L.moe_linear_q8(lay or lin(), q, ldq, qs, rows, y, yt, ldy, ws, wsb, None)
    assert L.moe_linear_q8(None, A, 64, A, 4, A, 0, 64, A, 1 << 30, None) == INVALID
    assert call(rows=0, q=None, qs=None, y=None, ws=None) == OK
    assert call(lay=lin(w=0)) == INVALID
    assert call(lay=lin(ws=0)) == INVALID
    assert call(lay=lin(N=0)) == SHAPE
    assert call(lay=lin(K=0)) == SHAPE
    assert call(lay=lin(K=65537, ldw=65552)) == SHAPE
    assert call(lay=lin(ldw=48)) == STRIDE
    assert call(lay=lin(ldw=72)) == ALIGN
    assert call(lay=lin(w=0x100008)) == ALIGN
    assert call(lay=lin(ws=0x100002)) == ALIGN
    assert call(lay=lin(bias=0x100002)) == ALIGN
    assert call(rows=-1) == INVALID
    assert call(yt=2) == INVALID
    for k in ("q", "qs", "y"):
        assert call(**{k: None}) == INVALID
    assert call(ldq=48) == STRIDE
    assert call(ldy=63) == STRIDE
    assert call(q=C.c_void_p(0x100008)) == ALIGN
    assert call(ldq=72) == ALIGN
    assert call(qs=MIS4) == ALIGN
    assert call(y=MIS4) == ALIGN


def test_python_argument_checks():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        m.moe_norm_pre(m.Norm(64), x)                       # not on the GPU
    with pytest.raises(TypeError):
        m.moe_norm_pre(m.Norm(64), x.half())
    with pytest.raises(TypeError):
        m.Norm(64, pre_w=torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        m.Norm(64, pre_w=torch.zeros(64))
    with pytest.raises(ValueError):
        m.RouterRule(8, 2, score="tanh")
    with pytest.raises(TypeError):
        m.Linear(x, torch.zeros(4))
    with pytest.raises(TypeError):
        m.moe_route_scored(m.RouterRule(8, 2), x.double())
    with pytest.raises(TypeError):
        m.moe_quant_row_q8(x.double())
    with pytest.raises(ValueError):
        m.route_outputs(4, 8, 2, device="cpu")


def test_linear_refuses_more_tiles_than_a_launch():
    L = m.lib()
    lay = lin(N=1 << 22, K=64)
    assert L.moe_linear_q8(lay, A, 64, A, 2**31 - 1, A, 0, 1 << 22, A, 1 << 30, None) == SHAPE
