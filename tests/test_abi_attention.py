"""Argument checks of the quantized cache, the attention over it and the linear with an epilogue, on the CPU: every
check runs before any HIP call, so none of these calls launches anything."""
import ctypes
import math

import pytest

import bit_quantized_linear_int8_amd as qa

OK, NULL, SHAPE, ALIGN, VALUE, WORKSPACE = 0, 1, 2, 3, 4, 5

A = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10001)
MIS8 = ctypes.c_void_p(0x10008)


def call(fn, base, **kw):
    a = dict(base)
    assert set(kw) <= set(a)
    a.update(kw)
    s = getattr(qa.lib(), fn)(*a.values())
    assert (qa.last_error() == "") == (s == OK)
    return s


CACHE = [(dict(heads=0), SHAPE), (dict(heads=65536), SHAPE), (dict(page=8), SHAPE), (dict(page=48), SHAPE),
         (dict(page=2048), SHAPE), (dict(D=0), SHAPE), (dict(D=72), SHAPE), (dict(D=272), SHAPE), (dict(pages=-1), SHAPE),
         (dict(pages=1 << 31), SHAPE), (dict(bits=2), VALUE), (dict(bits=16), VALUE)] + \
    [(dict([(n, None)]), NULL) for n in ("kc", "ks", "vc", "vs")] + \
    [(dict([(n, MIS8)]), ALIGN) for n in ("kc", "ks", "vc", "vs")]

WRITE = dict(K=A, ldk=512, V=A, ldv=512, dt=1, T=5, slots=A, bits=8, pages=9, heads=4, page=16, D=128, kc=A, ks=A, vc=A,
             vs=A, st=None)


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(K=None), NULL), (dict(V=None), NULL), (dict(slots=None), NULL),
    (dict(T=-1), SHAPE), (dict(T=(1 << 23) + 1), SHAPE), (dict(ldk=511), SHAPE), (dict(ldk=516), SHAPE),
    (dict(ldv=508), SHAPE), (dict(dt=0, ldk=514), SHAPE), (dict(dt=3), VALUE), (dict(dt=-1), VALUE),
    (dict(K=MIS8), ALIGN), (dict(V=MIS8), ALIGN), (dict(slots=MIS), ALIGN), (dict(slots=ctypes.c_void_p(0x10004)), ALIGN),
    (dict(T=0), OK), (dict(T=0, K=None, V=None, slots=None), OK),
])
def test_write(kw, status):
    assert call("qa_kv_write", WRITE, **kw) == status


READ = dict(slots=A, T=5, bits=8, pages=9, heads=4, page=16, D=128, kc=A, ks=A, vc=A, vs=A, K=A, V=A, dt=1, st=None)


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(K=None), NULL), (dict(V=None), NULL), (dict(slots=None), NULL), (dict(T=-1), SHAPE),
    (dict(T=(1 << 23) + 1), SHAPE), (dict(dt=3), VALUE), (dict(K=MIS8), ALIGN), (dict(V=MIS), ALIGN),
    (dict(slots=MIS), ALIGN), (dict(T=0), OK), (dict(T=0, K=None), OK),
])
def test_read(kw, status):
    assert call("qa_kv_read", READ, **kw) == status


ATTN = dict(q=A, ldq=1024, qdt=1, B=3, H=8, bits=8, pages=99, heads=4, page=16, D=128, kc=A, ks=A, vc=A, vs=A, table=A,
            ldt=10, width=10, lengths=A, max_len=160, window=0, scale=0.1, out=A, odt=1, lse=A, ws=A, wsb=1 << 24, st=None)


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(q=None), NULL), (dict(table=None), NULL), (dict(lengths=None), NULL), (dict(out=None), NULL),
    (dict(max_len=4096, width=256, ldt=256, ws=None), NULL),
    (dict(B=-1), SHAPE), (dict(B=(1 << 20) + 1), SHAPE), (dict(H=0), SHAPE), (dict(H=9), SHAPE), (dict(H=2), SHAPE),
    (dict(H=65540, ldq=1 << 24), SHAPE), (dict(B=1 << 20, H=16, ldq=2048), SHAPE), (dict(ldq=1023), SHAPE),
    (dict(ldq=1028), SHAPE), (dict(qdt=0, ldq=1026), SHAPE), (dict(width=-1, max_len=0), SHAPE), (dict(ldt=9), SHAPE),
    (dict(max_len=161), SHAPE), (dict(max_len=-1), SHAPE), (dict(window=-1), SHAPE),
    (dict(width=1 << 27, ldt=1 << 27), SHAPE),
    (dict(qdt=3), VALUE), (dict(odt=3), VALUE), (dict(scale=math.nan), VALUE), (dict(scale=math.inf), VALUE),
    (dict(q=MIS8), ALIGN), (dict(out=MIS8), ALIGN), (dict(table=MIS), ALIGN), (dict(lengths=MIS), ALIGN),
    (dict(lse=MIS), ALIGN), (dict(max_len=4096, width=256, ldt=256, ws=ctypes.c_void_p(0x10010)), ALIGN),
    (dict(max_len=4096, width=256, ldt=256, wsb=256), WORKSPACE),
    (dict(B=0), OK), (dict(B=0, q=None, table=None, lengths=None, out=None, ws=None, wsb=0), OK),
])
def test_attn(kw, status):
    assert call("qa_attn_decode", ATTN, **kw) == status


def test_attn_workspace():
    L = qa.lib()
    assert L.qa_attn_decode_workspace(0, 8, 4, 128, 1000, 0) == 0
    assert L.qa_attn_decode_workspace(1, 8, 3, 128, 1000, 0) == 0           # not a multiple
    assert L.qa_attn_decode_workspace(1, 8, 4, 100, 1000, 0) == 0
    assert L.qa_attn_decode_workspace(1, 32, 8, 128, 128, 0) == 0           # a single chunk
    assert L.qa_attn_decode_workspace(2000, 32, 8, 128, 1 << 20, 0) == 0    # enough sequences for the card
    n = L.qa_attn_decode_workspace(1, 32, 8, 128, 4096, 0)
    assert n >= 2 * 32 * 129 * 4 and n % 256 == 0
    assert L.qa_attn_decode_workspace(1, 32, 8, 128, 1 << 30, 90) == 0       # the window bounds the work


LINEAR = dict(Xq=A, sx=A, M=6, K=64, Wq=A, sw=A, N=48, bias=A, act=0, res=A, ldr=48, out=A, ldo=48, dt=1, st=None)


@pytest.mark.parametrize("kw,status", [(dict([(n, None)]), NULL) for n in ("Xq", "sx", "Wq", "sw", "out")] + [
    (dict(M=-1), SHAPE), (dict(M=(1 << 23) + 1), SHAPE), (dict(N=-1), SHAPE), (dict(N=1 << 31, ldo=1 << 31, ldr=1 << 31), SHAPE),
    (dict(M=1 << 23, N=1 << 13, ldo=1 << 13, ldr=1 << 13), SHAPE), (dict(K=0), SHAPE), (dict(K=72), SHAPE),
    (dict(K=131088), SHAPE), (dict(ldo=47), SHAPE), (dict(ldr=47), SHAPE), (dict(res=None, ldr=0, M=0), OK),
    (dict(dt=3), VALUE), (dict(act=-1), VALUE), (dict(act=5), VALUE),
    (dict(Xq=MIS8), ALIGN), (dict(Wq=MIS8), ALIGN), (dict(sx=MIS), ALIGN), (dict(sw=MIS), ALIGN), (dict(bias=MIS), ALIGN),
    (dict(res=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(dt=0, out=ctypes.c_void_p(0x10002)), ALIGN),
    (dict(M=0), OK), (dict(N=0, ldo=0, ldr=0), OK), (dict(M=0, Xq=None, out=None), OK),
])
def test_linear(kw, status):
    assert call("qa_qlinear_int8_act", LINEAR, **kw) == status


def test_binding_refuses_host_tensors():
    import torch
    t = torch.zeros(4, 8, 16)
    with pytest.raises(TypeError):
        qa.qa_kv_write(t, t, torch.zeros(4, dtype=torch.int64), (torch.zeros(2, 8, 16, 16), t, t, t))
    with pytest.raises(TypeError):
        qa.qa_kv_read(torch.zeros(4, dtype=torch.int64), (torch.zeros(2, 8, 16, 16, dtype=torch.int8), t, t, t))
    with pytest.raises(TypeError):
        qa.qa_qlinear_int8_act(torch.zeros(4, 16, dtype=torch.int8), t, t, t)
