"""Host-side tests of the experts' linear layers, the gated activation and the 8-bit rows: refusals (no compute
call is made), and calls with no rows."""
import math

import pytest
import torch

from tp_reduce_residual_gb300 import beamnorm as bn
from tp_reduce_residual_gb300 import build as nbuild
from tp_reduce_residual_gb300 import experts

A = 0x100000       # 16-byte aligned fake device addresses, never dereferenced


@pytest.fixture(scope="module")
def L():
    nbuild.build()
    return bn.load()


def at(i):
    return A * (i + 1) << 8


def refuses(L, fn, status, needle, *args):
    assert getattr(L, fn)(*args) == status
    assert needle in L.bn_last_error().decode(), L.bn_last_error()


LINEAR = dict(x=at(0), dtype=0, ld=64, x_rows=20, rows=at(1), M=40, w=at(2), E=4, N=32, K=64, offsets=at(3), y=at(4), ws=at(5), bytes=5120,
              stream=None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=2), 1, "dtype 2"), (dict(dtype=7), 1, "dtype 7"), (dict(M=-1), 1, "M=-1"), (dict(E=0), 1, "E=0"), (dict(E=1025), 2, "E=1025"),
    (dict(N=12), 1, "N=12"), (dict(N=0), 1, "N=0"), (dict(K=60), 1, "K=60"), (dict(K=1 << 21, ld=1 << 21), 2, "above the served"),
    (dict(N=1 << 21), 2, "above the served"), (dict(N=1 << 20, K=1 << 18, ld=1 << 18), 2, "N * K"), (dict(M=2 ** 31 - 8), 2, "M="), (dict(ld=60), 1, "ld=60"), (dict(ld=68), 1, "ld=68"),
    (dict(ld=1 << 40), 2, "ld="), (dict(rows=None), 1, "no rows are given"), (dict(x_rows=0), 1, "no rows"), (dict(x_rows=-1), 1, "x_rows=-1"),
    (dict(offsets=None), 1, "offsets is NULL"), (dict(offsets=at(3) + 2), 1, "offsets is not"), (dict(x=None), 1, "x is NULL"),
    (dict(x=at(0) + 8), 1, "x is not 16-byte"), (dict(rows=at(1) + 1), 1, "rows"), (dict(w=None), 1, "w is NULL"), (dict(y=None), 1, "y is NULL"),
    (dict(ws=at(5) + 4), 1, "workspace"), (dict(y=at(0)), 1, "y overlaps x"), (dict(y=at(2)), 1, "y overlaps w"), (dict(ws=at(0)), 1, "workspace overlaps x"),
    (dict(ws=at(4)), 1, "overlaps"),
])
def test_linear_refuses(L, kw, status, needle):
    refuses(L, "bn_expert_linear", status, needle, *dict(LINEAR, **kw).values())


DX = dict(dy=at(0), dtype=1, ld=32, M=40, w=at(2), E=4, N=32, K=64, offsets=at(3), dx=at(4), stream=None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=2), 1, "dtype"), (dict(ld=24), 1, "ld=24"), (dict(N=20, ld=24), 1, "N=20"), (dict(K=4), 1, "K=4"), (dict(dy=None), 1, "dy is NULL"),
    (dict(w=at(2) + 2), 1, "w is not"), (dict(dx=None), 1, "dx is NULL"), (dict(dx=at(0)), 1, "dx overlaps dy"), (dict(offsets=None), 1, "offsets"),
])
def test_linear_dx_refuses(L, kw, status, needle):
    refuses(L, "bn_expert_linear_dx", status, needle, *dict(DX, **kw).values())


DW = dict(dy=at(0), dtype=0, ld_dy=32, M=40, x=at(1), ld=64, x_rows=20, rows=at(2), E=4, N=32, K=64, offsets=at(3), dw=at(4), dw_dtype=2,
          accumulate=1, ws=at(5), bytes=5120, stream=None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dw_dtype=1), 1, "dw_dtype"), (dict(dw_dtype=0), 1, "accumulate"), (dict(ld_dy=24), 1, "dy: ld=24"), (dict(ld=72 + 4), 1, "x: ld=76"),
    (dict(rows=None), 1, "no rows are given"), (dict(dw=None), 1, "dw is NULL"), (dict(dw=at(4) + 4), 1, "dw is not"), (dict(dw=at(1)), 1, "dw overlaps x"),
    (dict(dw=at(0)), 1, "dw overlaps dy"), (dict(x_rows=0), 1, "x has no rows"), (dict(M=0, dw=None), 1, "dw is NULL"),
])
def test_linear_dw_refuses(L, kw, status, needle):
    refuses(L, "bn_expert_linear_dw", status, needle, *dict(DW, **kw).values())


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=3), 1, "dtype"), (dict(M=-2), 1, "M=-2"), (dict(F=0), 1, "F=0"), (dict(ld=95), 1, "ld=95"), (dict(F=1 << 29, ld=1 << 31), 2, "F="),
    (dict(x=None), 1, "x is NULL"), (dict(x=at(0) + 1), 1, "x is not 2-byte"), (dict(y=None), 1, "y is NULL"), (dict(y=at(0) + 2), 1, "y overlaps x"),
])
def test_swiglu_refuses(L, kw, status, needle):
    refuses(L, "bn_swiglu", status, needle, *dict(dict(x=at(0), dtype=0, ld=96, M=10, F=48, y=at(1), stream=None), **kw).values())


@pytest.mark.parametrize("kw,status,needle", [
    (dict(ld_dy=47), 1, "ld_dy=47"), (dict(dy=None), 1, "dy is NULL"), (dict(dx=None), 1, "dx is NULL"), (dict(dx=at(2)), 1, "dx overlaps dy"),
    (dict(dx=at(0)), 1, "dx overlaps x"), (dict(dtype=2, dy=at(2) + 2), 1, "dy is not 4-byte"),
])
def test_swiglu_backward_refuses(L, kw, status, needle):
    args = dict(x=at(0), dtype=0, ld=96, M=10, F=48, dy=at(2), ld_dy=48, dx=at(1), stream=None)
    refuses(L, "bn_swiglu_backward", status, needle, *dict(args, **kw).values())


INT8 = dict(x=at(0), dtype=0, ld=64, x_rows=20, rows=at(1), M=40, K=64, data=at(2), scales=at(3), ws=at(4), bytes=1360, stream=None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=4), 1, "dtype"), (dict(K=24, ld=24), 1, "K=24"), (dict(K=0), 1, "K=0"), (dict(K=131072, ld=131072), 2, "K=131072"), (dict(ld=56), 1, "ld=56"),
    (dict(ld=68), 1, "ld=68"), (dict(dtype=2, ld=66), 1, "ld=66"), (dict(M=-1), 1, "M=-1"), (dict(rows=None), 1, "no rows are given"),
    (dict(x_rows=0), 1, "no rows"), (dict(x=at(0) + 4), 1, "x is not"), (dict(data=None), 1, "data is NULL"), (dict(scales=at(3) + 2), 1, "scales"),
    (dict(data=at(0)), 1, "data overlaps x"), (dict(ws=at(4) + 8), 1, "workspace is not"), (dict(ws=at(0)), 1, "workspace overlaps x"), (dict(scales=at(2)), 1, "overlaps"),
])
def test_quantize_int8_refuses(L, kw, status, needle):
    refuses(L, "bn_quantize_int8", status, needle, *dict(INT8, **kw).values())


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=9), 1, "dtype"), (dict(K=8), 1, "K=8"), (dict(out=None), 1, "out is NULL"), (dict(out=at(0)), 1, "out overlaps data"),
])
def test_dequantize_int8_refuses(L, kw, status, needle):
    refuses(L, "bn_dequantize_int8", status, needle, *dict(dict(data=at(0), scales=at(1), M=40, K=64, out=at(2), dtype=0, stream=None), **kw).values())


PRODUCT = dict(a=at(0), a_scales=at(1), M=40, w=at(2), w_scales=at(3), E=4, N=32, K=64, offsets=at(4), alpha=1.0, out=at(5), ws=at(6),
               bytes=40 * 64 * 2, stream=None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(M=-1), 1, "M=-1"), (dict(E=0), 1, "E=0"), (dict(E=2000), 2, "E=2000"), (dict(N=12), 1, "N=12"), (dict(N=1 << 21), 2, "N="), (dict(K=40), 1, "K=40"),
    (dict(K=131072), 2, "K=131072"), (dict(offsets=None), 1, "offsets"), (dict(alpha=math.inf), 1, "alpha"), (dict(a=None), 1, "a is NULL"),
    (dict(a_scales=at(1) + 2), 1, "a_scales"), (dict(w=at(2) + 8), 1, "w is not"), (dict(w_scales=None), 1, "w_scales is NULL"), (dict(out=None), 1, "out is NULL"),
    (dict(ws=at(6) + 8), 1, "workspace is not"), (dict(ws=at(0)), 1, "workspace overlaps a"),
    (dict(out=at(2)), 1, "out overlaps w"),
])
def test_product_int8_refuses(L, kw, status, needle):
    refuses(L, "bn_expert_product_int8", status, needle, *dict(PRODUCT, **kw).values())


def test_no_rows_is_no_work(L):
    assert L.bn_expert_linear(*dict(LINEAR, M=0, x=None, w=None, y=None, ws=None).values()) == bn.OK
    assert L.bn_expert_linear_dx(*dict(DX, M=0, dy=None, w=None, dx=None).values()) == bn.OK
    assert L.bn_expert_linear_dw(*dict(DW, M=0, dy=None, x=None, ws=None).values()) == bn.OK  # accumulates nothing
    assert L.bn_swiglu(None, 0, 96, 0, 48, None, None) == bn.OK
    assert L.bn_swiglu_backward(None, 0, 96, 0, 48, None, 48, None, None) == bn.OK
    assert L.bn_quantize_int8(*dict(INT8, M=0, x=None, data=None, scales=None).values()) == bn.OK
    assert L.bn_dequantize_int8(None, None, 0, 64, None, 0, None) == bn.OK
    assert L.bn_expert_product_int8(*dict(PRODUCT, M=0, a=None, w=None, out=None, ws=None).values()) == bn.OK


def test_workspace_bytes(L):
    assert experts.linear_workspace_bytes(32, 64) == 0 and experts.linear_workspace_bytes(33, 64) == 33 * 128
    assert experts.linear_workspace_bytes(100, 60) == 0
    assert experts.product_int8_workspace_bytes(30, 4, 4096, 8192) == 0 and experts.product_int8_workspace_bytes(0, 1, 64, 64) == 0
    assert experts.product_int8_workspace_bytes(2 ** 20, 8, 4096, 131056) == 2 ** 21 * 131056
    assert experts.product_int8_workspace_bytes(800, 256, 6144, 1024) == 0  # a few rows for every expert


def test_binding_refuses_what_is_not_on_a_gpu():
    x, w = torch.ones(4, 16, dtype=torch.bfloat16), torch.ones(2, 8, 16, dtype=torch.bfloat16)
    for call in (lambda: experts.expert_linear(x, w), lambda: experts.expert_linear_dx(x, w), lambda: experts.expert_linear_dw(x, x),
                 lambda: experts.swiglu(x), lambda: experts.swiglu_backward(x, x), lambda: experts.quantize_int8(x),
                 lambda: experts.expert_product(experts.Int8(x.to(torch.int8), torch.ones(4)), experts.Int8(w.to(torch.int8), torch.ones(2, 8)))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError):
        experts.quantize_int8([1.0])
    with pytest.raises(TypeError):
        experts.dequantize_int8(x)
