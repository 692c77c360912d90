"""The gated activation with its gradient, and rows in 8-bit integers, against their definitions in 64 bits.

Tolerances.  z = exp(-|gate|) is within 2^-22 of itself (and 2^-149, its smallest step), 1 + z and the fast
division add 2^-24 and 2^-22, so s, 1 - s and gate * s are within 2^-20; y within 2^-19, as one more
product rounds.  dgate sums two such terms that may cancel: 2^-19 of |dy up| (s + |gate s (1 - s)|).
The rounding to the output's type is eps / 2 of the value, or half its smallest step.  Codes and scales are exact."""

import pytest
import torch

from tp_reduce_residual_gb300 import beamnorm as bn
from tp_reduce_residual_gb300 import build as nbuild
from tp_reduce_residual_gb300 import experts

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
STEP = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the smallest step


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    nbuild.build()
    bn.load()
    bn.check_device_error(raise_on_error=False)
    yield
    assert bn.check_device_error() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def within(got, want, tol, what):
    t = got.dtype
    off = (got.double() - want).abs()
    tol = tol + torch.finfo(t).eps / 2 * want.abs() + STEP[t]
    assert not torch.isnan(got).any() and (off <= tol).all(), (what, (off - tol).max().item())


def check_swiglu(x, dy):
    F = dy.shape[1]
    g, u, d = x[:, :F].double(), x[:, F:].double(), dy.double()
    s, t = torch.sigmoid(g), torch.sigmoid(-g)
    y = experts.swiglu(x)
    assert y.shape == dy.shape and y.dtype is x.dtype and y.is_contiguous()
    tiny = 2.0 ** -147 * (g * u).abs()
    within(y, g * s * u, 2.0 ** -19 * (g * s * u).abs() + tiny, "y")
    dx = experts.swiglu_backward(x, dy)
    assert dx.shape == x.shape and dx.is_contiguous()
    within(dx[:, :F], d * u * s * (1 + g * t), 2.0 ** -19 * (d * u).abs() * s * (1 + (g * t).abs()) + 2.0 ** -147 * (d * u).abs() * (1 + g.abs()), "dgate")
    within(dx[:, F:], d * g * s, 2.0 ** -19 * (d * g * s).abs() + 2.0 ** -147 * (d * g).abs(), "dup")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,F", [(1, 1), (1, 8), (3, 7), (2, 1001), (5, 256), (33, 520), (700, 48), (1, 100000), (129, 2048)])
def test_swiglu(dtype, M, F):
    x = (3 * torch.randn(M, 2 * F, generator=gen(M + F), device="cuda")).to(DTYPES[dtype])
    check_swiglu(x, torch.randn(M, F, generator=gen(F), device="cuda").to(DTYPES[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_swiglu_extremes(dtype):
    g = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20, -20, 60, -60, 87, -87, 88.5, -88.5, 95, -95, 104, -104, 500, -500, 1e4, -1e4, -1.2785])
    u = torch.tensor([1.0, -3.0, 1e20, -1e-20, 1e30, 0.0])
    x = torch.cat((g.repeat_interleave(len(u))[None], u.repeat(len(g))[None]), 1).cuda().to(DTYPES[dtype])
    check_swiglu(x, torch.full((1, x.shape[1] // 2), 0.5, device="cuda").to(x.dtype))


def test_swiglu_strides_and_bad_values():
    wide = torch.full((9, 160), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = torch.randn(9, 96, generator=gen(0), device="cuda").bfloat16()
    dy = torch.randn(9, 48, generator=gen(1), device="cuda").bfloat16()
    want, back = experts.swiglu(x), experts.swiglu_backward(x, dy)
    for at in (8, 3):  # aligned rows, and rows that no vector fits
        wide[:, at:at + 96] = x
        strided = torch.full((9, 99), float("inf"), dtype=torch.bfloat16, device="cuda")
        strided[:, at:at + 48] = dy
        assert torch.equal(experts.swiglu(wide[:, at:at + 96]), want)
        assert torch.equal(experts.swiglu_backward(wide[:, at:at + 96], strided[:, at:at + 48]), back)
    x[4, 10] = float("nan")
    y = experts.swiglu(x)
    assert torch.isnan(y[4, 10]) and torch.isnan(y).sum() == 1
    assert experts.swiglu(x[:0]).shape == (0, 48) and experts.swiglu_backward(x[:0], dy[:0]).shape == (0, 96)


def test_swiglu_gradient_against_differences():
    x = torch.randn(4, 64, generator=gen(5), device="cuda")
    dy = torch.randn(4, 32, generator=gen(6), device="cuda")
    dx = experts.swiglu_backward(x, dy).double()
    h = 2.0 ** -7
    v = torch.randn(4, 64, generator=gen(7), device="cuda")
    f = [(experts.swiglu(x + s * h * v).double() * dy.double()).sum() for s in (1, -1)]
    slope = (f[0] - f[1]) / (2 * h)
    # third derivatives of silu(g) u are below 1 |u| + 0.8: h^2 / 6 * |v|^3 of each; the values' roundings over 2 h
    bound = (h * h / 6 * (v[:, :32].abs() + v[:, 32:].abs()) ** 3 * (x[:, 32:].abs() + 2) * dy.abs()).sum() \
        + (2.0 ** -18 * (x[:, :32] * x[:, 32:] * dy).abs()).sum() / h
    assert (slope - (dx * v.double()).sum()).abs() <= bound


# ---- rows in 8-bit integers ------------------------------------------------------------------------

def reference(x):
    """Codes and scales of rows, decided in 64 bits."""
    top = x.float().abs().amax(-1).cpu()
    scale = top / 127  # one IEEE division
    bad = ~torch.isfinite(top)
    y = x.cpu().double() / torch.where((scale > 0) & ~bad, scale, 1).double()[:, None]
    codes = torch.where(((scale > 0) & ~bad)[:, None], torch.round(y), 0).nan_to_num(0).clamp(-127, 127).to(torch.int8)
    return codes.cuda(), torch.where(bad, float("nan"), scale).cuda()


def check_int8(x, rows=None, **kw):
    q = experts.quantize_int8(x, rows=rows, **kw)
    codes, scales = reference(x if rows is None else x[rows.long()])
    assert torch.equal(q.data, codes), (q.data != codes).nonzero()[:5]
    assert torch.equal(q.scales.nan_to_num(-1), scales.nan_to_num(-1))
    for t in DTYPES.values():
        v = experts.dequantize_int8(q, t)
        assert torch.equal(v.nan_to_num(7), (codes.float() * scales[:, None]).to(t).nan_to_num(7))
    return q


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (7, 512), (9, 1040), (50, 2064), (300, 256), (5, 8208), (2, 20000), (1, 131056)])
def test_int8_rows(dtype, M, K):
    x = (torch.randn(M, K, generator=gen(M * K), device="cuda") * torch.exp(torch.randn(K, generator=gen(K), device="cuda"))).to(DTYPES[dtype])
    check_int8(x)


def test_int8_ties_and_near_ties():
    """Halves of a scale that is a power of two go to the even code; FP32 values next to a half do not."""
    n = torch.arange(-127, 127, device="cuda").float() + 0.5
    for s in (1.0, 2.0 ** -20, 2.0 ** 100, 2.0 ** -90, 2.0 ** -126):
        row = torch.cat((torch.tensor([127.0, 0.0], device="cuda"), n)) * s
        q = check_int8(row[None].bfloat16())
        assert (q.data[0, 2:] % 2 == 0).all()
    up, down = (torch.nextafter(n, torch.full_like(n, v)) for v in (1e9, -1e9))
    x = torch.zeros(3, 272, device="cuda")
    for r, v in enumerate((n, up, down)):
        x[r, 0], x[r, 1:255] = 127, v
    check_int8(x)
    x[:, 0] = 126.7  # a scale that is not exact
    check_int8(x * torch.tensor([[1.0], [0.37], [1e-20]], device="cuda"))


def test_int8_small_and_bad_rows():
    x = torch.randn(8, 64, generator=gen(3), device="cuda")
    x[0] = 0
    x[1] *= 2.0 ** -130
    x[2] *= 2.0 ** -145
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    x[5, 7] = -3.3e38
    x[6, 8] = -float("inf")
    q = check_int8(x)
    assert (q.scales[0] == 0) and torch.isnan(q.scales[[3, 4, 6]]).all() and (q.data[[0, 3, 4, 6]] == 0).all()
    check_int8((x * 1e-3).bfloat16())


def test_int8_rows_by_index_and_strides():
    wide = torch.randn(20, 200, generator=gen(4), device="cuda").half()
    x = wide[:, 8:8 + 144]
    rows = torch.randint(0, 20, (75,), generator=gen(5), device="cuda").to(torch.int32)
    offsets = torch.tensor([0, 40, 75], dtype=torch.int32, device="cuda")
    q = check_int8(x, rows=rows, offsets=offsets)
    assert q.offsets is offsets and q.shape == (75, 144)
    rows[3], rows[9] = -1, 20
    again = experts.quantize_int8(x, rows=rows)
    assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_PERM_RANGE
    fixed = rows.clone()
    fixed[3] = fixed[9] = 0
    assert torch.equal(again.data, experts.quantize_int8(x, rows=fixed).data)


def test_int8_weights():
    w = torch.randn(3, 40, 80, generator=gen(6), device="cuda").bfloat16()
    q = experts.quantize_int8(w)
    assert q.data.shape == (3, 40, 80) and q.scales.shape == (3, 40)
    codes, scales = reference(w.view(120, 80))
    assert torch.equal(q.data.view(120, 80), codes) and torch.equal(q.scales.view(-1), scales)
    assert experts.dequantize_int8(q).shape == (3, 40, 80)
    assert experts.quantize_int8(w[0, :0]).data.shape == (0, 80)


@pytest.mark.parametrize("n,M,K", [(500, 5000, 4096), (3000, 9000, 3008), (1, 20000, 1040)])
def test_int8_repeated_rows_through_a_workspace(n, M, K):
    """Rows quantised once and copied: the codes and scales of place by place."""
    x = torch.randn(n, K, generator=gen(n), device="cuda").bfloat16()
    x[0, 3] = float("nan")
    rows = torch.randint(0, n, (M,), generator=gen(M), device="cuda").to(torch.int32)
    rows[7], rows[M - 1] = n, -5
    size = experts.quantize_int8_workspace_bytes(n, M, K)
    assert size == n * (K + 4)
    ws = torch.full((size + 32,), 255, dtype=torch.uint8, device="cuda")
    once = experts.quantize_int8(x, rows=rows, workspace=ws[:size])
    assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_PERM_RANGE and (ws[size:] == 255).all()
    ws.fill_(255)
    each = experts.quantize_int8(x, rows=rows, workspace=ws[:16])
    assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_PERM_RANGE and (ws == 255).all()
    assert torch.equal(once.data, each.data) and torch.equal(once.scales.nan_to_num(-1), each.scales.nan_to_num(-1))
    assert experts.quantize_int8_workspace_bytes(100, 199, 65536) == 0 and experts.quantize_int8_workspace_bytes(100, 800, 1024) == 0


def test_callers_streams():
    """Outputs and workspaces come from the caller's stream's pool; two streams at once."""
    x = torch.randn(600, 1024, generator=gen(1), device="cuda").bfloat16()
    dy = torch.randn(600, 512, generator=gen(2), device="cuda").bfloat16()
    rows = torch.arange(600, device="cuda").repeat(40).to(torch.int32)
    assert experts.quantize_int8_workspace_bytes(600, 24000, 1024) > 0
    want = experts.swiglu(x), experts.swiglu_backward(x, dy), experts.quantize_int8(x, rows=rows)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        for s in streams:
            q = experts.quantize_int8(x, rows=rows, stream=s)
            got.append((experts.swiglu(x, stream=s), experts.swiglu_backward(x, dy, stream=s.cuda_stream), q, experts.dequantize_int8(q, stream=s)))
    for s in streams:
        s.synchronize()
    for y, dx, q, v in got:
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1]) and torch.equal(q.data, want[2].data) and torch.equal(q.scales, want[2].scales)
        assert torch.equal(v, experts.dequantize_int8(want[2]))
