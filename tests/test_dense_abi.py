"""Refusals of layer norm, the gated feed-forward block and 4-bit linear layers:
every invalid argument returns its status before any HIP call (so without a
GPU), and the tensor functions raise."""

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


def mat(data=4096, stride=1024):
    return ctypes.byref(L.GsMatrix(data, stride))


def call(f, defaults, **kw):
    assert not set(kw) - set(defaults), kw
    return f(*{**defaults, **kw}.values())


def test_layer_norm_refusals(lib):
    fwd = dict(x=mat(), w=FAKE, b=FAKE, y=FAKE, st=FAKE, rows=10, c=64, eps=1e-5, t=L.GS_BF16, s=None)
    for bad in (dict(x=None), dict(x=mat(0)), dict(x=mat(4097)), dict(x=mat(stride=-1)), dict(x=mat(stride=1 << 20)),
                dict(y=None), dict(st=None), dict(rows=-1), dict(rows=1 << 41), dict(c=0), dict(c=16385), dict(eps=-1.0),
                dict(eps=float("nan")), dict(t=3), dict(t=-1)):
        assert call(lib.gs_layer_norm_fwd, fwd, **bad) == INV, bad
    assert call(lib.gs_layer_norm_fwd, fwd, rows=0, x=None) == OK
    need = L.layer_norm_bwd_workspace_bytes(10, 64)
    assert need > 0 and L.layer_norm_bwd_workspace_bytes(-1, 64) == 0 and L.layer_norm_bwd_workspace_bytes(1, 0) == 0
    bwd = dict(gy=mat(), x=mat(), w=FAKE, st=FAKE, gx=FAKE, gw=FAKE, gb=FAKE, rows=10, c=64, t=L.GS_F32, ws=FAKE, wsb=need,
               s=None)
    for bad in (dict(gy=None), dict(x=None), dict(gy=mat(0)), dict(gy=mat(4098)), dict(x=mat(stride=1 << 20)), dict(st=None),
                dict(gx=None), dict(ws=None), dict(ws=ctypes.c_void_p(4100)), dict(wsb=need - 1), dict(rows=-1), dict(c=0),
                dict(t=9)):
        assert call(lib.gs_layer_norm_bwd, bwd, **bad) == INV, bad


def test_gated_ff_refusals(lib):
    fwd = dict(x=mat(), wg=mat(), wu=mat(), wd=mat(), rows=10, c=64, hid=128, co=64, act=L.GS_SILU, t=L.GS_BF16, h=FAKE,
               kept=FAKE, y=FAKE, ws=FAKE, wsb=1 << 40, s=None)
    need = L.gated_ff_bwd_workspace_bytes(10, 64, 128, 64)
    assert need > 0 and L.gated_ff_bwd_workspace_bytes(10, 64, 12, 64) == 0
    assert L.gated_ff_kept_bytes(10, 128, L.GS_BF16) == 6400 and L.gated_ff_kept_bytes(10, 128, L.GS_F16) == 7680
    assert L.gated_ff_kept_bytes(10, 128, L.GS_F32) == 0 and L.gated_ff_kept_bytes(10, 12, L.GS_F16) == 0
    assert L.gated_ff_fwd_workspace_bytes(-1, 64, 128, 64) == 0
    bwd = dict(gy=mat(), x=mat(), wg=mat(), wu=mat(), wd=mat(), h=FAKE, kept=FAKE, rows=10, c=64, hid=128, co=64, act=L.GS_SILU,
               t=L.GS_BF16, gx=FAKE, gwg=FAKE, gwu=FAKE, gwd=FAKE, ws=FAKE, wsb=need, s=None)
    both = (dict(x=None), dict(wg=None), dict(wu=None), dict(wd=None), dict(x=mat(0)), dict(wd=mat(0)), dict(h=None),
            dict(rows=-1), dict(rows=(1 << 24) + 1), dict(c=0), dict(c=60), dict(hid=4), dict(hid=-8), dict(co=12),
            dict(c=(1 << 17) + 8), dict(hid=1 << 18), dict(act=2), dict(act=-1), dict(t=3))
    odd = (dict(t=L.GS_F32), dict(x=mat(4104)), dict(wg=mat(stride=1028)), dict(wu=mat(stride=-8)), dict(wd=mat(stride=1 << 21)), dict(x=mat(stride=56)),
           dict(h=ctypes.c_void_p(4104)), dict(kept=ctypes.c_void_p(4104)), dict(rows=1 << 24, hid=1 << 17))
    for f, ok in ((lib.gs_gated_ff_fwd, fwd), (lib.gs_gated_ff_bwd, bwd)):
        big = {"wsb": 1 << 60} if ok is bwd else {}
        for bad in both:
            assert call(f, ok, **bad, **big) == INV, bad
        for bad in odd:
            assert call(f, ok, **bad, **big) == UNS, bad
    for bad in (dict(y=None), dict(rows=1, hid=4096, ws=None), dict(rows=1, hid=4096, ws=ctypes.c_void_p(4100)),
                dict(rows=1, hid=4096, wsb=0)):
        if "hid" in bad and not L.gated_ff_fwd_workspace_bytes(1, 64, 4096, 64):
            continue
        assert call(lib.gs_gated_ff_fwd, fwd, **bad) == INV, bad
    assert call(lib.gs_gated_ff_fwd, fwd, y=ctypes.c_void_p(4104)) == UNS
    assert call(lib.gs_gated_ff_fwd, fwd, rows=0, x=None) == OK
    for bad in (dict(gy=None), dict(kept=None), dict(gwg=None), dict(gwu=None), dict(ws=None), dict(wsb=need - 1),
                dict(ws=ctypes.c_void_p(4100))):
        assert call(lib.gs_gated_ff_bwd, bwd, **bad) == INV, bad
    assert call(lib.gs_gated_ff_bwd, bwd, gx=ctypes.c_void_p(4104)) == UNS
    assert call(lib.gs_gated_ff_bwd, bwd, rows=0, gwg=None, gwu=None, gwd=None) == OK


def test_fp4_refusals(lib):
    quant = dict(x=mat(), rows=10, c=64, t=L.GS_BF16, codes=FAKE, scales=FAKE, s=None)
    back = dict(codes=mat(), scales=mat(), rows=10, c=64, t=L.GS_F32, out=FAKE, s=None)
    need = L.linear_fp4_workspace_bytes(100, 64, 40)
    assert need > 0 and L.linear_fp4_workspace_bytes(100, 48, 40) == 0 and L.linear_fp4_workspace_bytes(100, 64, 0) == 0
    linear = dict(x=mat(), codes=mat(), scales=mat(), rows=100, c=64, n=40, t=L.GS_BF16, y=FAKE, ws=FAKE, wsb=need, s=None)
    sizes = (dict(rows=-1), dict(rows=(1 << 24) + 1), dict(c=0), dict(c=48), dict(c=(1 << 17) + 32), dict(t=3), dict(t=-1))
    for f, ok in ((lib.gs_quantise_fp4, quant), (lib.gs_dequantise_fp4, back), (lib.gs_linear_fp4, linear)):
        for bad in sizes:
            assert call(f, ok, **bad) == INV, bad
        assert call(f, ok, rows=0) == OK
    odd = ctypes.c_void_p(4104)
    for bad in (dict(x=None), dict(x=mat(0)), dict(codes=None), dict(scales=None)):
        assert call(lib.gs_quantise_fp4, quant, **bad) == INV, bad
    for bad in (dict(x=mat(4104)), dict(x=mat(stride=1028)), dict(x=mat(stride=-8)), dict(x=mat(stride=1 << 21)), dict(codes=odd),
                dict(scales=ctypes.c_void_p(4098))):
        assert call(lib.gs_quantise_fp4, quant, **bad) == UNS, bad
    for bad in (dict(codes=None), dict(scales=None), dict(codes=mat(0)), dict(scales=mat(0)), dict(out=None)):
        assert call(lib.gs_dequantise_fp4, back, **bad) == INV, bad
    for bad in (dict(codes=mat(4104)), dict(codes=mat(stride=1032)), dict(scales=mat(4098)), dict(scales=mat(stride=1026)),
                dict(out=odd)):
        assert call(lib.gs_dequantise_fp4, back, **bad) == UNS, bad
    for bad in (dict(x=None), dict(codes=None), dict(scales=None), dict(x=mat(0)), dict(codes=mat(0)), dict(scales=mat(0)),
                dict(n=0), dict(n=(1 << 17) + 1), dict(y=None), dict(ws=None), dict(ws=ctypes.c_void_p(4100)),
                dict(wsb=need - 1)):
        assert call(lib.gs_linear_fp4, linear, **bad) == INV, bad
    for bad in (dict(x=mat(4104)), dict(x=mat(stride=1028)), dict(codes=mat(4104)), dict(codes=mat(stride=1032)),
                dict(scales=mat(4098)), dict(scales=mat(stride=1026)), dict(scales=mat(stride=1 << 21)), dict(codes=mat(stride=16)),
                dict(y=ctypes.c_void_p(4097)), dict(rows=1 << 24, n=1 << 17)):
        assert call(lib.gs_linear_fp4, linear, **bad, **({"wsb": 1 << 60} if "rows" in bad else {})) == UNS, bad


def test_tensor_functions_refuse(lib):
    """Shapes, types and devices, before the library is called."""
    cpu = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        T.layer_norm(cpu)
    with pytest.raises(ValueError):
        T.layer_norm(torch.zeros(64))
    with pytest.raises(ValueError):
        T.layer_norm_backward(cpu, cpu, None, torch.zeros(2, 4))
    w = torch.zeros(8, 64)
    for act in ("silu", "relu"):
        with pytest.raises(ValueError):
            T.gated_ff(cpu, w, w, torch.zeros(64, 8), act)
    with pytest.raises(ValueError):
        T.gated_ff_backward(cpu, cpu, w, w, torch.zeros(64, 8), torch.zeros(4, 8), torch.zeros(4, 16))
    for bad in (lambda: T.quantise4(cpu), lambda: T.linear4(cpu, (cpu, cpu)), lambda: T.dequantise4((cpu, cpu))):
        with pytest.raises(ValueError):
            bad()


def test_gated_ff_bwd_refuses_one_row_for_all(lib):
    """Sums run over the rows of every operand."""
    need = L.gated_ff_bwd_workspace_bytes(10, 64, 128, 64)
    bwd = dict(gy=mat(), x=mat(), wg=mat(), wu=mat(), wd=mat(), h=FAKE, kept=FAKE, rows=10, c=64, hid=128, co=64, act=L.GS_SILU,
               t=L.GS_BF16, gx=FAKE, gwg=FAKE, gwu=FAKE, gwd=FAKE, ws=FAKE, wsb=need, s=None)
    for name in ("gy", "x", "wg", "wu", "wd"):
        assert call(lib.gs_gated_ff_bwd, bwd, **{name: mat(stride=0)}) == UNS, name
