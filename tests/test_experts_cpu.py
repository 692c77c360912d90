"""Host-side tests of the operators around the experts: refusals (no compute call is made) and the
64-bit definitions that the GPU tests compare with."""
import math

import pytest
import torch

from tests import experts_reference as ref
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


ROUTE = dict(logits=at(0), dtype=0, ld=64, T=4, E=64, k=8, bias=at(1), score=1, groups=8, top=4, gtop=2,
             renorm=1, scale=1.0, R=2, ids=at(2), w=at(3), stream=None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=3), 1, "dtype"), (dict(T=-1), 1, "T=-1"), (dict(E=0), 1, "E=0"), (dict(k=0), 1, "k=0"),
    (dict(k=17), 1, "k=17"), (dict(E=4, ld=64, groups=1, top=1), 1, "k=8 above E=4"), (dict(R=0), 1, "R=0"),
    (dict(R=17), 1, "R=17"), (dict(ld=63), 1, "ld=63"), (dict(score=2), 1, "score"),
    (dict(groups=7), 1, "equal groups"), (dict(groups=0), 1, "groups=0"), (dict(top=9), 1, "top_groups=9"),
    (dict(top=0), 1, "top_groups=0"), (dict(gtop=3), 1, "group_top=3"), (dict(scale=math.nan), 1, "scale"),
    (dict(groups=64, top=4), 1, "k=8 above the 4 experts"), (dict(groups=64, top=64), 2, "groups=64"),
    (dict(E=2048, ld=2048), 2, "E=2048"), (dict(T=2 ** 28), 2, "T*k"),
    (dict(logits=None), 1, "logits is NULL"), (dict(logits=at(0) + 1), 1, "logits is not 2-byte"),
    (dict(bias=at(1) + 2), 1, "bias"), (dict(ids=None), 1, "ids is NULL"), (dict(w=at(3) + 2), 1, "w is not"),
    (dict(ids=at(0)), 1, "ids overlaps logits"), (dict(w=at(1)), 1, "w overlaps bias"), (dict(w=at(2)), 1, "ids overlaps w"),
])
def test_route_refuses(L, kw, status, needle):
    refuses(L, "bn_route", status, needle, *dict(ROUTE, **kw).values())


def test_no_tokens_is_no_work(L):
    assert L.bn_route(*dict(ROUTE, T=0, logits=None, ids=None, w=None).values()) == bn.OK
    assert L.bn_route_backward(None, 0, 64, 0, 64, 8, None, None, 1, 0, 1, 1.0, None, None) == bn.OK
    assert L.bn_quantize_fp4(None, 0, 64, 0, None, 0, 64, None, 1, 0, 1.0, None, None, None, 0, None) == bn.OK
    assert L.bn_dequantize_fp4(None, None, 0, 64, None, 1, 0, 1.0, None, 0, None) == bn.OK
    assert L.bn_expert_product(None, None, 0, None, None, 4, 64, 64, at(0), 0, 1.0, None, None) == bn.OK


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=5), 1, "dtype"), (dict(k=0), 1, "k=0"), (dict(ids=None), 1, "ids is NULL"),
    (dict(dw=at(3) + 1), 1, "dw is not"), (dict(out=at(4) + 1), 1, "dlogits is not"), (dict(out=at(0)), 1, "dlogits overlaps logits"),
    (dict(out=at(3)), 1, "dlogits overlaps dw"), (dict(scale=math.inf), 1, "scale"), (dict(E=1025, ld=1025), 2, "E=1025"),
])
def test_route_backward_refuses(L, kw, status, needle):
    a = dict(logits=at(0), dtype=0, ld=64, T=4, E=64, k=8, ids=at(2), dw=at(3), R=2, score=0, renorm=1, scale=1.0,
             out=at(4), stream=None)
    refuses(L, "bn_route_backward", status, needle, *dict(a, **kw).values())


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), 1, "T=-1"), (dict(k=17), 1, "k=17"), (dict(E=0), 1, "E=0"), (dict(E=1025), 2, "E=1025"), (dict(R=17), 1, "R=17"),
    (dict(T=2 ** 28), 2, "T*k"), (dict(T=2 ** 31 - 1000, k=1), 2, "T*k"), (dict(ids=None), 1, "ids is NULL"), (dict(offsets=None), 1, "offsets is NULL"),
    (dict(rows=at(0)), 1, "rows overlaps ids"), (dict(perm=at(2)), 1, "perm overlaps offsets"), (dict(perm=at(1) + 2), 1, "perm is not"),
])
def test_plan_refuses(L, kw, status, needle):
    a = dict(ids=at(0), T=4, k=8, E=64, R=2, perm=at(1), offsets=at(2), rows=at(3), stream=None)
    refuses(L, "bn_expert_plan", status, needle, *dict(a, **kw).values())


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=2), 1, "dtype"), (dict(format=2), 1, "format"), (dict(M=-1), 1, "M=-1"), (dict(K=48), 1, "K=48"), (dict(K=0), 1, "K=0"),
    (dict(ld=60), 1, "ld=60"), (dict(ld=68), 1, "ld=68"), (dict(groups=0), 1, "groups=0"), (dict(groups=3, offsets=None), 1, "equal groups"),
    (dict(groups=1025), 2, "groups=1025"), (dict(K=2 ** 21, ld=2 ** 21), 2, "K="),
    (dict(tensor_scale=3.0), 1, "power of two"), (dict(tensor_scale=0.0), 1, "power of two"), (dict(tensor_scale=-1.0), 1, "power of two"),
    (dict(tensor_scale=math.nan), 1, "power of two"), (dict(tensor_scale=2.0 ** 65), 1, "power of two"),
    (dict(rows=None), 1, "no rows are given"), (dict(x_rows=0), 1, "x has no rows"), (dict(x=at(0) + 2), 1, "x is not 16-byte"),
    (dict(data=None), 1, "data is NULL"), (dict(scales=at(2) + 4), 1, "scales is not"), (dict(data=at(0)), 1, "data overlaps x"),
    (dict(scales=at(4)), 1, "scales overlaps offsets"), (dict(work=at(5) + 8), 1, "workspace is not 16-byte"),
    (dict(work=at(0)), 1, "workspace overlaps x"), (dict(work=at(1)), 1, "data overlaps workspace"),
])
def test_quantize_refuses(L, kw, status, needle):
    a = dict(x=at(0), dtype=0, ld=64, x_rows=5, rows=at(3), M=8, K=64, offsets=at(4), groups=4, format=0, tensor_scale=0.5,
             data=at(1), scales=at(2), work=at(5), work_bytes=64, stream=None)
    refuses(L, "bn_quantize_fp4", status, needle, *dict(a, **kw).values())


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=7), 1, "dtype"), (dict(K=40), 1, "K=40"), (dict(out=at(0)), 1, "out overlaps data"), (dict(scales=None), 1, "scales is NULL"),
    (dict(tensor_scale=1.5), 1, "power of two"),
])
def test_dequantize_refuses(L, kw, status, needle):
    a = dict(data=at(0), scales=at(1), M=8, K=64, offsets=at(2), groups=4, format=0, tensor_scale=0.5, out=at(3), dtype=2, stream=None)
    refuses(L, "bn_dequantize_fp4", status, needle, *dict(a, **kw).values())


@pytest.mark.parametrize("kw,status,needle", [
    (dict(N=12), 1, "N=12"), (dict(N=0), 1, "N=0"), (dict(K=63), 1, "K=63"), (dict(E=0), 1, "E=0"), (dict(E=1025), 2, "E=1025"),
    (dict(offsets=None), 1, "offsets is NULL"), (dict(offsets=at(4) + 2), 1, "offsets is not"), (dict(alpha=math.inf), 1, "alpha"),
    (dict(a=at(0) + 8), 1, "a is not 16-byte"), (dict(w=None), 1, "w is NULL"), (dict(out=at(2)), 1, "out overlaps w"),
    (dict(out=at(0)), 1, "out overlaps a"), (dict(E=1024, N=2 ** 21), 2, "E*N"), (dict(format=9), 1, "format"),
    (dict(E=1024, N=2 ** 20, K=2 ** 20), 2, "scale tiles"), (dict(M=2 ** 31 - 1), 2, "M=2147483647"),
])
def test_product_refuses(L, kw, status, needle):
    a = dict(a=at(0), a_scales=at(1), M=8, w=at(2), w_scales=at(3), E=4, N=64, K=64, offsets=at(4), format=0, alpha=1.0, out=at(5),
             stream=None)
    refuses(L, "bn_expert_product", status, needle, *dict(a, **kw).values())


def test_scale_bytes(L):
    f = L.bn_fp4_scale_bytes
    assert f(1, 64, 1, 0, 0) == 512 and f(129, 64, 1, 0, 0) == 2 * 512 and f(1, 96, 1, 0, 0) == 2 * 512
    assert f(1, 128, 1, 0, 1) == 512 and f(1, 160, 1, 0, 1) == 2 * 512
    assert f(256, 64, 2, 0, 0) == 2 * 512 and f(260, 64, 2, 0, 0) == 4 * 512
    assert f(300, 64, 7, 1, 0) == (2 + 7 + 1) * 512
    for bad in ((-1, 64, 1, 0, 0), (4, 48, 1, 0, 0), (4, 64, 0, 0, 0), (5, 64, 2, 0, 0), (4, 64, 1, 0, 2)):
        assert f(*bad) == 0, bad
    for fmt in experts.FORMATS:
        for M, K, g, ragged in ((1, 64, 1, False), (300, 160, 7, True), (260, 2048, 2, False)):
            n = experts.fp4_scales_shape(M, K, fmt, g, ragged)
            assert n[0] * n[1] * n[2] == f(M, K, g, int(ragged), experts.FORMATS[fmt])


def test_quantize_workspace_bytes(L):
    f = L.bn_quantize_fp4_workspace_bytes
    assert f(4096, 32768, 5120, 1) == 4096 * (2560 + 40 * 4) and f(4096, 32768, 5120, 0) == 4096 * (2560 + 80 * 4)
    assert f(5, 50, 8192, 0) == 0 and f(16384, 32768, 5120, 0) == 0      # little work; rows taken twice
    assert f(0, 32768, 5120, 0) == 0 and f(64, 32768, 5100, 0) == 0 and f(64, 32768, 5120, 3) == 0
    assert experts.quantize_workspace_bytes(4096, 32768, 5120, "mxfp4") == f(4096, 32768, 5120, 1)


def test_ragged_tiles_never_meet():
    """Group g's row tiles start at (offsets[g] >> 7) + g: no two groups share one, and all lie inside
    M // 128 + groups + 1 tiles."""
    g = torch.Generator().manual_seed(0)
    for _ in range(200):
        n = int(torch.randint(1, 12, (1,), generator=g))
        counts = torch.randint(0, 400, (n,), generator=g) * torch.randint(0, 2, (n,), generator=g)
        offsets = torch.cat((torch.zeros(1, dtype=torch.long), counts.cumsum(0)))
        M = int(offsets[-1]) + int(torch.randint(0, 200, (1,), generator=g))  # rows past the last group
        owner = {}
        for m, (tile, r) in enumerate(ref.row_tiles(M, offsets)):
            group = sum(1 for v in offsets[1:].tolist() if v <= m)
            assert owner.setdefault(tile, group) == group and 0 <= r < 128
            assert tile < M // 128 + n + 1


@pytest.mark.parametrize("call", [
    lambda c: experts.route(c["x"], 2), lambda c: experts.route_backward(c["x"], c["ids"], c["dw"]),
    lambda c: experts.plan(c["ids"], 8), lambda c: experts.quantize_fp4(c["x"], "nvfp4"),
    lambda c: experts.dequantize_fp4(experts.FP4(c["q"], c["s"], "nvfp4")),
    lambda c: experts.expert_product(experts.FP4(c["q"], c["s"], "nvfp4"), experts.FP4(c["q"], c["s"], "nvfp4")),
])
def test_binding_refuses_cpu_tensors(L, call):
    c = dict(x=torch.zeros(4, 64, dtype=torch.bfloat16), ids=torch.zeros(4, 2, dtype=torch.int32), dw=torch.zeros(1, 4, 2),
             q=torch.zeros(4, 32, dtype=torch.uint8), s=torch.zeros(1, 1, 512, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        call(c)


def test_binding_refuses_unknown_names():
    with pytest.raises(ValueError, match="format"):
        experts.quantize_fp4(torch.zeros(4, 64), "fp8")
    with pytest.raises(TypeError, match="FP4"):
        experts.dequantize_fp4(torch.zeros(4, 64))
    with pytest.raises(ValueError, match="ids"):
        experts.plan(torch.zeros(4, dtype=torch.int32), 8)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_formula_against_differences(score, renormalize):
    """The derivative that the GPU tests use (autograd of the 64-bit weights) against central differences:
    their error is h^2 / 6 of a third derivative below 10, plus 2^-52 / h."""
    g = torch.Generator().manual_seed(1)
    T, E, k, h = 3, 9, 4, 1e-4
    x = torch.randn(T, E, generator=g, dtype=torch.float64, requires_grad=True)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    ids[1, 2] = -1
    dw = torch.randn(T, k, generator=g, dtype=torch.float64)
    f = lambda v: (ref.route_weights(v, ids, score, renormalize, 2.5) * dw).sum()
    f(x).backward()
    for t in range(T):
        for e in range(E):
            d = torch.zeros_like(x)
            d[t, e] = h
            diff = float(f(x.detach() + d) - f(x.detach() - d)) / (2 * h)
            assert abs(diff - float(x.grad[t, e])) < 10 * h * h + 1e-10
