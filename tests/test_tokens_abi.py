"""Refusals of the token operators: every invalid argument returns its status
before any HIP call (so without a GPU), and the tensor functions raise."""

import ctypes
import os

import pytest
import torch

from gaussian_splatting_differentiable_ewa_amd import _lib as L
from gaussian_splatting_differentiable_ewa_amd import tokens as T

INV, UNS, OK = L.GS_ERR_INVALID_ARGUMENT, L.GS_ERR_UNSUPPORTED, L.GS_OK
FAKE = ctypes.c_void_p(4096)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from gaussian_splatting_differentiable_ewa_amd import build
        build.build()
    return L.lib()


def tok(data=4096, sb=1 << 20, st=1024, sh=64):
    return ctypes.byref(L.GsTokens(data, sb, st, sh))


def call(f, defaults, **kw):
    assert not set(kw) - set(defaults), kw
    return f(*{**defaults, **kw}.values())


def test_rope_refusals(lib):
    ok = dict(q=tok(), k=tok(), qo=tok(), ko=tok(), b=1, n=10, hq=2, hk=1, d=64, t=L.GS_BF16, pos=FAKE, sp=0, freq=FAKE,
              pairs=(ctypes.c_int32 * 3)(8, 12, 12), il=0, inv=0, s=None)

    def f(**kw):
        return call(lib.gs_rope_axes, ok, **kw)

    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(b=-1), dict(n=-1), dict(hq=-1), dict(hk=-1),
                dict(d=0), dict(d=63), dict(d=514), dict(t=3), dict(t=-1), dict(pos=None), dict(freq=None),
                dict(pairs=None), dict(pairs=(ctypes.c_int32 * 3)(-1, 0, 0)), dict(pairs=(ctypes.c_int32 * 3)(16, 16, 1)),
                dict(pairs=(ctypes.c_int32 * 3)(2 ** 31 - 1, 2 ** 31 - 1, 2)), dict(q=tok(0)), dict(ko=tok(0)),
                dict(n=1 << 41), dict(b=1 << 30, n=1 << 30)):
        assert f(**bad) == INV, bad
    assert f(b=1 << 16, n=1 << 16, t=L.GS_F32) == UNS
    assert f(n=0) == OK and f(b=0) == OK and f(hq=0, hk=0) == OK


def test_norm_refusals(lib):
    ok = dict(x=FAKE, f=FAKE, g=FAKE, w2=FAKE, w1=FAKE, y=FAKE, h=FAKE, st=FAKE, rows=10, c=64, per=5, a=1.0, eps=1e-6,
              t=L.GS_F32, s=None)

    def f(**kw):
        return call(lib.gs_norm_gate_fwd, ok, **kw)

    for bad in (dict(x=None), dict(y=None), dict(h=None), dict(st=None), dict(rows=-1), dict(c=0), dict(c=16385),
                dict(per=0), dict(eps=-1.0), dict(eps=float("nan")), dict(t=7)):
        assert f(**bad) == INV, bad
    assert f(rows=0) == OK
    need = L.norm_gate_bwd_workspace_bytes(10, 64, 5)
    assert need > 0 and L.norm_gate_bwd_workspace_bytes(-1, 64, 5) == 0 and L.norm_gate_bwd_workspace_bytes(1, 0, 5) == 0
    ok2 = dict(gy=FAKE, gh=FAKE, x=FAKE, f=FAKE, g=FAKE, w2=FAKE, w1=FAKE, st=FAKE, gx=FAKE, gf=FAKE, gg=FAKE, gw2=FAKE,
               gw1=FAKE, rows=10, c=64, per=5, a=1.0, t=L.GS_F32, ws=FAKE, wsb=need, s=None)

    def b(**kw):
        return call(lib.gs_norm_gate_bwd, ok2, **kw)

    for bad in (dict(gh=None), dict(x=None), dict(st=None), dict(gx=None), dict(gf=None), dict(ws=None), dict(wsb=need - 1),
                dict(ws=ctypes.c_void_p(4100)), dict(rows=-1), dict(c=0), dict(per=0), dict(t=9)):
        assert b(**bad) == INV, bad
    assert b(rows=1 << 22, per=1, wsb=1 << 60) == UNS


def test_select_refusals(lib):
    ok = dict(k=tok(), b=1, n=100, h=2, d=64, t=L.GS_BF16, kl=None, b0=0, nb=2, s8=tok(), sc=tok(), s=None)

    def f(**kw):
        return call(lib.gs_block_summary, ok, **kw)

    for bad in (dict(k=None), dict(s8=None), dict(sc=None), dict(b=-1), dict(n=-1), dict(h=-1), dict(d=4), dict(d=60),
                dict(d=264), dict(t=5), dict(b0=-1), dict(nb=-1), dict(b0=1), dict(b0=3, nb=0), dict(k=tok(0)),
                dict(s8=tok(0)), dict(sc=tok(0))):
        assert f(**bad) == INV, bad
    assert f(k=tok(4098)) == UNS and f(k=tok(st=65)) == UNS and f(k=tok(sh=4)) == UNS and f(b=1 << 23) == UNS
    assert f(nb=0) == OK and f(b=0) == OK
    ok2 = dict(q=tok(), s8=tok(), sc=tok(), b=1, nq=100, nk=1000, hq=4, hk=2, d=64, t=L.GS_BF16, kl=None, ca=0, top=4,
               li=FAKE, s=None)

    def g(**kw):
        return call(lib.gs_block_select, ok2, **kw)

    for bad in (dict(q=None), dict(s8=None), dict(sc=None), dict(b=-1), dict(nq=-1), dict(nk=-1),
                dict(nk=L.GS_MAX_SELECT_TOKENS + 1), dict(hq=0), dict(hk=0), dict(hk=3), dict(d=12), dict(t=4), dict(top=0),
                dict(top=32769), dict(li=None), dict(q=tok(0)), dict(s8=tok(0))):
        assert g(**bad) == INV, bad
    assert g(q=tok(4104)) == UNS and g(s8=tok(4100)) == UNS and g(s8=tok(st=60)) == UNS and g(b=1 << 22) == UNS
    assert g(nq=0) == OK and g(b=0) == OK


def test_attention_refusals(lib):
    fwd = dict(q=tok(), k=tok(), v=tok(), li=FAKE, b=1, nq=100, nk=1000, hq=4, hk=2, d=64, t=L.GS_BF16, kl=None, ca=0,
               top=4, sm=0.1, o=tok(), lse=FAKE, ws=FAKE, wsb=1 << 40, s=None)
    need = L.block_attn_bwd_workspace_bytes(1, 100, 1000, 4, 2, 64)
    assert need > 0 and L.block_attn_bwd_workspace_bytes(1, 100, 1000, 4, 2, 96) == 0
    bwd = dict(go=tok(), q=tok(), k=tok(), v=tok(), o=tok(), lse=FAKE, li=FAKE, b=1, nq=100, nk=1000, hq=4, hk=2, d=64,
               t=L.GS_BF16, kl=None, ca=0, top=4, sm=0.1, gq=tok(), gk=tok(), gv=tok(), ws=FAKE, wsb=need, s=None)
    both = (dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(li=None), dict(lse=None), dict(b=-1), dict(nq=-1),
            dict(nk=-1), dict(nk=1 << 37), dict(hq=0), dict(hk=0), dict(hk=3), dict(d=0), dict(t=3), dict(top=0),
            dict(sm=0.0), dict(sm=-1.0), dict(sm=float("nan")), dict(sm=float("inf")), dict(q=tok(0)), dict(k=tok(0)),
            dict(v=tok(0)), dict(o=tok(0)))
    odd = (dict(t=L.GS_F32), dict(d=32), dict(d=96), dict(d=256), dict(q=tok(4104)), dict(k=tok(st=1028)), dict(v=tok(sh=60)),
           dict(o=tok(4098)), dict(b=1 << 23, wsb=1 << 62))
    for f, ok in ((lib.gs_block_attn_fwd, fwd), (lib.gs_block_attn_bwd, bwd)):
        for bad in both:
            assert call(f, ok, **bad) == INV, bad
        for bad in odd:
            assert call(f, ok, **bad) == UNS, bad
        assert call(f, ok, b=0) == OK
    for bad in (dict(go=None), dict(gq=None), dict(gk=None), dict(gv=None), dict(ws=None), dict(wsb=need - 1),
                dict(ws=ctypes.c_void_p(4100)), dict(go=tok(0)), dict(gv=tok(0))):
        assert call(lib.gs_block_attn_bwd, bwd, **bad) == INV, bad
    assert call(lib.gs_block_attn_fwd, fwd, nq=0) == OK
    # one token over a long list needs a workspace
    n = L.block_attn_fwd_workspace_bytes(1, 1, 4, 64, 64)
    assert n > 0
    assert call(lib.gs_block_attn_fwd, fwd, nq=1, top=64, wsb=n - 1) == INV
    assert call(lib.gs_block_attn_fwd, fwd, nq=1, top=64, ws=None) == INV


def test_tensor_functions_refuse(lib):
    """Shapes, types and devices, before the library is called."""
    cpu = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError):
        T.rope_axes(cpu, None, torch.zeros(1, 4, 3, dtype=torch.int32), torch.zeros(32), (1, 1, 1))
    with pytest.raises(ValueError):
        T.rope_axes(torch.zeros(4, 64), None, torch.zeros(1, 4, 3, dtype=torch.int32), torch.zeros(32), (1, 1, 1))
    with pytest.raises(ValueError):
        T.norm_gate(torch.zeros(4, 8), None)
    with pytest.raises(ValueError):
        T.norm_gate(torch.zeros(4), None)
    with pytest.raises(ValueError):
        T.block_summary(cpu)
    with pytest.raises(ValueError):
        T.select_blocks(cpu, (torch.zeros(1, 1, 1, 64, dtype=torch.int8), torch.zeros(1, 1, 1)), 4, 1)
    with pytest.raises(ValueError):
        T.block_attention(cpu, cpu, cpu, torch.zeros(1, 2, 1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        T.block_attention_backward(cpu, cpu, cpu, cpu, cpu, torch.zeros(1, 2, 4), torch.zeros(1, 2, 1, 1, dtype=torch.int32))
    with pytest.raises(L.GsError):
        L.dtype_of(torch.zeros(1, dtype=torch.float64))
