"""Refusals of the 16-bit and 8-bit expert products, on the host before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from weight_only_bit_route_b200 import moe

P = ctypes.c_void_p
A = P(0x10000)             # aligned, never dereferenced by the host checks
MIS = P(0x10008)           # 8-byte aligned only
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -5


def mm(x=A, off=A, rows=4, w=A, E=2, out=64, inn=64, f16=0, y=A, ws=A, wsb=1024):
    return moe.lib.moe_grouped_mm(x, off, rows, w, E, out, inn, f16, y, ws, wsb, None)


def dgrad(dy=A, off=A, rows=4, w=A, E=2, out=64, inn=64, f16=0, dx=A, ws=A, wsb=1024):
    return moe.lib.moe_grouped_mm_dgrad(dy, off, rows, w, E, out, inn, f16, dx, ws, wsb, None)


def wgrad(dy=A, x=A, off=A, rows=4, E=2, out=64, inn=64, f16=0, dw=A, f32=0, acc=0, ws=A, wsb=1024):
    return moe.lib.moe_grouped_mm_wgrad(dy, x, off, rows, E, out, inn, f16, dw, f32, acc, ws, wsb, None)


@pytest.mark.parametrize("call,row_args,big", [(mm, ("x", "y"), "w"), (dgrad, ("dy", "dx"), "w"),
                                               (wgrad, ("dy", "x"), "dw")])
def test_product_argument_errors(call, row_args, big):
    for bad in (dict(rows=-1), dict(E=0), dict(out=0), dict(inn=-8), dict(off=None), {big: None}, {big: MIS}):
        assert call(**bad) == INVALID, bad
    for name in row_args:
        assert call(**{name: None}) == INVALID
        assert call(**{name: MIS}) == INVALID
    for bad in (dict(E=1025), dict(out=60), dict(inn=12), dict(rows=2 ** 31 - 1)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws=P(0x10080)), dict(wsb=1023)):
        assert call(**bad) == WORKSPACE, bad


def test_product_without_rows_launches_nothing():
    assert mm(rows=0, x=None, y=None) == OK
    assert dgrad(rows=0, dy=None, dx=None) == OK
    assert wgrad(rows=0, dy=None, x=None, f32=1, acc=1) == OK


def test_accumulation_needs_fp32():
    assert wgrad(acc=1, f32=0) == UNSUPPORTED


def bank(E=32, out=256, inn=1024, packed=A, scales=A, fmt=moe.FMT_INT8, inscale=None):
    return moe.QWeight(fmt, E, out, inn, packed, scales, None, inscale)


def swiglu(g, u, T=4, H=1024, k=8, limit=0.0, ws=A, wsb=1 << 30, x=A):
    return moe.lib.moe_grouped_w4a16_swiglu(x, T, H, A, A, k, ctypes.byref(g), ctypes.byref(u), limit, A, ws, wsb, None)


def down(d, rows=32, ws=A, wsb=1 << 30, h=A):
    return moe.lib.moe_grouped_w4a16_down(h, A, A, None, rows, ctypes.byref(d), A, ws, wsb, None)


def test_int8_bank_argument_errors():
    g = bank()
    assert swiglu(g, g, T=0) == OK
    assert swiglu(bank(scales=None), g) == INVALID
    assert swiglu(bank(packed=MIS), g) == INVALID
    assert swiglu(g, bank(E=31)) == INVALID
    assert swiglu(g, bank(fmt=0)) == UNSUPPORTED                 # mixed formats
    assert swiglu(bank(inscale=A), g) == UNSUPPORTED             # W4A4's input scale
    assert swiglu(g, g, limit=1.0) == UNSUPPORTED
    assert swiglu(g, g, x=MIS) == INVALID
    assert swiglu(g, g, ws=None) == WORKSPACE
    assert swiglu(g, g, wsb=1024) == WORKSPACE
    wide = bank(inn=131072)
    assert swiglu(wide, wide, H=131072) == UNSUPPORTED           # 128 * 128 * in reaches 2^31
    assert down(bank(out=1024, inn=256), rows=0) == OK
    assert down(bank(out=1024, inn=131072)) == UNSUPPORTED
    assert down(bank(out=1000, inn=256)) == UNSUPPORTED
    assert down(bank(out=1024, inn=256), wsb=2048) == WORKSPACE


def test_unknown_bank_formats_are_refused():
    for fmt in (3, 4, 6, -1):                                     # 3 and 4 name internal variants, not banks
        assert swiglu(bank(fmt=fmt), bank(fmt=fmt)) == UNSUPPORTED
        assert down(bank(fmt=fmt, out=1024, inn=256)) == UNSUPPORTED


def test_int8_layer_argument_errors():
    E, H, F = 32, 1024, 256
    z = moe.QWeight(0, 0, 0, 0, None, None, None, None)

    def call(gate=bank(), up=bank(), dn=bank(out=H, inn=F), sh=(z, z, z), T=4, wsb=1 << 34):
        L = moe.Layer(gate, up, dn, *sh, A, None, E, H, F, 8, 0.0, 0)
        return moe.lib.moe_layer_forward(A, T, ctypes.byref(L), A, A, wsb, None)

    assert call(T=0) == OK
    assert call(dn=bank(out=H, inn=F, fmt=0)) == UNSUPPORTED     # mixed formats
    assert call(gate=bank(scales=None)) == INVALID
    assert call(sh=(bank(E=1), bank(E=1), bank(E=1, out=H, inn=F))) == UNSUPPORTED                     # the shared expert is bf16
    assert call(wsb=4096) == WORKSPACE


def test_quantize_int8_argument_errors():
    q = lambda x=A, rows=4, cols=64, codes=A, scales=A: moe.lib.moe_quantize_int8(x, rows, cols, 0, codes, scales, None)
    assert q(rows=0) == OK and q(cols=0) == OK
    assert q(rows=-1) == INVALID and q(cols=-16) == INVALID
    assert q(cols=24) == UNSUPPORTED and q(rows=1 << 31) == UNSUPPORTED
    for bad in (dict(x=None), dict(codes=None), dict(scales=None), dict(x=MIS), dict(codes=MIS)):
        assert q(**bad) == INVALID, bad


def test_binding_refuses_before_the_call():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    off, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(1024, dtype=torch.uint8)
    for call in (lambda: moe.grouped_mm(x, w, off, ws),                       # not on a GPU
                 lambda: moe.grouped_mm(x.float(), w, off, ws),
                 lambda: moe.grouped_mm_dgrad(x, w.half(), off, ws),
                 lambda: moe.grouped_mm_wgrad(x, x, off, ws),
                 lambda: moe.quantize_int8(x)):
        with pytest.raises(moe.MoEError) as err:
            call()
        assert err.value.code == INVALID
