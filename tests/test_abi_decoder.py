"""Argument checks of the norm, routing, expert and adapter entry points, on the CPU: every check runs before any HIP
call, so none of these calls launches anything."""
import ctypes
import math

import pytest

import bit_quantized_linear_int8_amd as qa

OK, NULL, SHAPE, ALIGN, VALUE, WORKSPACE = 0, 1, 2, 3, 4, 5

A = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10001)


def call(fn, base, **kw):
    a = dict(base)
    a.update(kw)
    s = getattr(qa.lib(), fn)(*a.values())
    assert (qa.last_error() == "") == (s == OK)
    return s


NORM = dict(X=A, ldx=256, res=A, ldr=256, g=A, dt=1, rows=4, K=256, eps=1e-6, Xq=A, s=A, sum=A, lds=256, y=A, st=None)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), NULL), (dict(g=None), NULL), (dict(Xq=None), NULL), (dict(s=None), NULL),
    (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(K=0), SHAPE), (dict(K=(1 << 26) + 1), SHAPE),
    (dict(ldx=255), SHAPE), (dict(ldr=255), SHAPE), (dict(lds=255), SHAPE),
    (dict(dt=3), VALUE), (dict(eps=0.0), VALUE), (dict(eps=-1e-6), VALUE), (dict(eps=math.nan), VALUE),
    (dict(eps=math.inf), VALUE),
    (dict(X=MIS), ALIGN), (dict(res=MIS), ALIGN), (dict(g=MIS), ALIGN), (dict(sum=MIS), ALIGN), (dict(y=MIS), ALIGN),
    (dict(s=MIS), ALIGN), (dict(dt=0, X=ctypes.c_void_p(0x10002)), ALIGN),
    (dict(rows=0), OK), (dict(rows=0, X=None, Xq=None, s=None, res=None, ldr=0, sum=None, lds=0), OK),
])
def test_norm(kw, status):
    assert call("qa_rmsnorm_int8", NORM, **kw) == status


ROUTE = dict(x=A, dt=0, T=10, E=64, ld=64, bias=A, score=0, groups=1, top=1, gtop=1, k=4, renorm=1, scale=1.0, ids=A, w=A,
             order=A, offsets=A, ws=A, wsb=1 << 20, st=None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), NULL), (dict(ids=None), NULL), (dict(w=None), NULL), (dict(order=None), NULL),
    (dict(offsets=None), NULL), (dict(ws=None), NULL), (dict(T=0, offsets=None), NULL),
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(T=(1 << 23) + 1), SHAPE), (dict(E=0), SHAPE),
    (dict(E=1025, ld=1025), SHAPE), (dict(ld=63), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE),
    (dict(E=3, k=4), SHAPE), (dict(groups=0), SHAPE), (dict(groups=64, top=64), SHAPE), (dict(groups=5, top=5), SHAPE),
    (dict(groups=4, top=0), SHAPE), (dict(groups=4, top=5), SHAPE), (dict(groups=32, top=1), SHAPE),
    (dict(dt=5), VALUE), (dict(score=2), VALUE), (dict(gtop=0), VALUE), (dict(gtop=3), VALUE),
    (dict(scale=math.nan), VALUE), (dict(scale=math.inf), VALUE),
    (dict(x=MIS), ALIGN), (dict(bias=MIS), ALIGN), (dict(ids=MIS), ALIGN), (dict(w=MIS), ALIGN), (dict(order=MIS), ALIGN),
    (dict(offsets=MIS), ALIGN), (dict(wsb=16), WORKSPACE),
])
def test_route(kw, status):
    assert call("qa_route_experts", ROUTE, **kw) == status


EXPERTS = dict(Xq=A, sx=A, T=6, K=64, w=A, order=A, offsets=A, E=4, k=2, W13=A, s13=A, F=32, W2=A, s2=A, out=A, dt=1,
               ws=A, wsb=1 << 24, st=None)


@pytest.mark.parametrize("kw,status", [(dict([(n, None)]), NULL) for n in ("Xq", "sx", "w", "order", "offsets", "W13",
                                                                         "s13", "W2", "s2", "out", "ws")] + [
    (dict(T=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=56), SHAPE), (dict(K=131088), SHAPE), (dict(F=8), SHAPE),
    (dict(F=0), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE),
    (dict(T=1 << 26, K=32), SHAPE),                         # T K
    (dict(K=65536, F=16384), SHAPE),                        # 2 F K
    (dict(T=1 << 22, K=16, k=3), SHAPE),                    # T k
    (dict(T=1 << 22, K=64, F=131072, k=2), SHAPE),          # tiles
    (dict(dt=3), VALUE),
    (dict(Xq=MIS), ALIGN), (dict(W13=ctypes.c_void_p(0x10008)), ALIGN), (dict(s2=ctypes.c_void_p(0x10004)), ALIGN),
    (dict(out=ctypes.c_void_p(0x10008)), ALIGN), (dict(ws=ctypes.c_void_p(0x10010)), ALIGN), (dict(sx=MIS), ALIGN),
    (dict(wsb=64), WORKSPACE), (dict(T=0), OK), (dict(T=0, Xq=None, out=None), OK),
])
def test_experts(kw, status):
    assert call("qa_experts_int8", EXPERTS, **kw) == status


LORA = dict(Xq=A, sx=A, X=A, dt=1, M=6, K=64, Wq=A, sw=A, N=48, A=A, B=A, alpha=A, r=16, L=2, seg=A, which=A, R=3, out=A,
            odt=1, ws=A, wsb=1 << 20, st=None)


@pytest.mark.parametrize("kw,status", [(dict([(n, None)]), NULL) for n in ("Xq", "sx", "X", "Wq", "sw", "A", "B", "alpha",
                                                                         "seg", "which", "out", "ws")] + [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=72), SHAPE), (dict(K=131088), SHAPE),
    (dict(r=0), SHAPE), (dict(r=12), SHAPE), (dict(r=264), SHAPE), (dict(L=-1), SHAPE), (dict(R=-1), SHAPE),
    (dict(R=(1 << 31) - 1), SHAPE), (dict(M=(1 << 23) + 1), SHAPE), (dict(M=1 << 23, N=1 << 13), SHAPE),
    (dict(dt=0), VALUE), (dict(dt=7), VALUE), (dict(odt=3), VALUE),
    (dict(Xq=MIS), ALIGN), (dict(B=ctypes.c_void_p(0x10008)), ALIGN), (dict(seg=MIS), ALIGN), (dict(out=MIS), ALIGN),
    (dict(ws=ctypes.c_void_p(0x10020)), ALIGN), (dict(wsb=64), WORKSPACE),
    (dict(M=0), OK), (dict(N=0), OK),
])
def test_lora(kw, status):
    assert call("qa_qlinear_int8_lora", LORA, **kw) == status


def test_workspaces():
    L = qa.lib()
    assert L.qa_route_experts_workspace(-1, 8, 2) == 0 and L.qa_route_experts_workspace(5, 2000, 2) == 0
    assert L.qa_route_experts_workspace(1000, 256, 8) >= 4 * 256 * 16
    assert L.qa_experts_int8_workspace(4, 60, 2, 4, 32) == 0
    assert L.qa_experts_int8_workspace(100, 64, 2, 4, 128) >= 200 * (128 * 4 + 128 + 8)
    assert L.qa_qlinear_int8_lora_workspace(10, 64, 7) == 0
    for M in (1, 64, 65, 4096):
        assert L.qa_qlinear_int8_lora_workspace(M, 64, 40) >= M * 40 * 4
