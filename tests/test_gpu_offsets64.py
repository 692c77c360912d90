"""Operands and results past 2^31 elements: the linear layers' gradients and placed rows, the gated activation,
rows in 8-bit integers.

Row addresses that wrapped to 32 bits would read or write other rows, which hold other values here.  Whole numbers
are exact; the activation's rows are compared with the same rows alone, bit for bit (an element's result depends on
no other)."""
import pytest
import torch

from tp_reduce_residual_gb300 import beamnorm as bn
from tp_reduce_residual_gb300 import build as nbuild
from tp_reduce_residual_gb300 import experts

pytestmark = pytest.mark.gpu

PAST = 2 ** 31


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    nbuild.build()
    bn.load()
    bn.check_device_error(raise_on_error=False)
    yield
    assert bn.check_device_error() == 0
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(shape, seed, dtype=torch.bfloat16, top=3):
    return torch.randint(-top, top + 1, shape, generator=gen(seed), device="cuda").to(dtype)


def some(M, width):
    """Rows at both ends, and around every multiple of 2^30 elements."""
    at = {0, 1, M - 2, M - 1}
    for i in range(1, M * width // 2 ** 30 + 1):
        at |= {m for m in range(i * 2 ** 30 // width - 1, i * 2 ** 30 // width + 2) if m < M}
    return torch.tensor(sorted(at), device="cuda")


@pytest.mark.parametrize("ld,ld_dy", [(8200, 16), (16, 8200), (8200, 8200)])
def test_weight_gradient_of_rows_far_apart(ld, ld_dy):
    """Rows of x, of dy, or of both, whose addresses pass 2^31 elements; all but a few hundred are zeros, so that the
    sum is exact: 300 products of at most 9."""
    M, N, K = PAST // 8200 + 1000, 16, 16
    x, dy = (torch.zeros(M, n, dtype=torch.bfloat16, device="cuda")[:, :16] for n in (ld, ld_dy))
    rows = torch.cat((torch.randint(0, M, (270,), generator=gen(1), device="cuda"), some(M, 8200), torch.arange(M - 16, M, device="cuda"))).unique()
    x[rows] = whole((len(rows), K), 2)
    dy[rows] = whole((len(rows), N), 3)
    want = dy[rows].double().T @ x[rows].double()
    assert torch.equal(experts.expert_linear_dw(dy, x, dtype=torch.float32).double(), want)
    assert torch.equal(experts.expert_linear_dw(dy, x), want.bfloat16())
    o = torch.tensor([0, M - 7, M], dtype=torch.int32, device="cuda")
    last = experts.expert_linear_dw(dy, x, o, dtype=torch.float32)[1]
    assert torch.equal(last.double(), dy[-7:].double().T @ x[-7:].double())


@pytest.mark.parametrize("K,M,n", [(8192, 270000, 5000), (16, 300, PAST // 16 + 64)])
def test_rows_by_index(K, M, n):
    """Places past 2^31 elements in the workspace, and rows of x past them."""
    x = torch.zeros(n, K, dtype=torch.bfloat16, device="cuda")
    w = whole((24, K), 5)
    rows = torch.randint(0, n, (M,), generator=gen(6), device="cuda").to(torch.int32)
    rows[-1], rows[0] = n - 1, n // 2
    live = rows.unique().long()
    x[live] = whole((len(live), K), 7)
    at = some(M, K) if M > 1000 else torch.arange(M, device="cuda")
    y = experts.expert_linear(x, w, rows=rows)
    assert torch.equal(y[at], (x[rows[at].long()].double() @ w.double().T).bfloat16())
    dy = torch.zeros(M, 24, dtype=torch.bfloat16, device="cuda")
    dy[at] = whole((len(at), 24), 8)
    want = dy[at].double().T @ x[rows[at].long()].double()
    assert torch.equal(experts.expert_linear_dw(dy, x, rows=rows, dtype=torch.float32).double(), want)


@pytest.mark.parametrize("M,F", [(PAST // 2000 + 500, 2000), (PAST // 2001 + 500, 2001), (3, 2 ** 28)])
def test_activation_and_gradient(M, F):
    """In 16-byte pieces, element by element, and of few very long rows."""
    x = torch.empty(M, 2 * F, dtype=torch.bfloat16, device="cuda")
    dy = torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
    for t in (x, dy):
        for i, part in enumerate(t.view(-1).split(2 ** 28)):
            part.copy_(2 * torch.randn(part.numel(), generator=gen(i), device="cuda"))
    at = some(M, F) if M > 3 else torch.arange(3, device="cuda")
    y = experts.swiglu(x)
    assert torch.equal(y[at], experts.swiglu(x[at]))
    del y
    dx = experts.swiglu_backward(x, dy)
    assert torch.equal(dx[at], experts.swiglu_backward(x[at], dy[at]))
    gate, up = x[at[-1], :F].double(), x[at[-1], F:].double()
    want = gate * torch.sigmoid(gate) * up  # and by the formula: FP32's digits, BF16's rounding
    assert ((experts.swiglu(x[at[-1:]])[0].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -18) * want.abs()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_8_bit_rows_and_back(dtype):
    M, K = PAST // 8192 + 300, 8192
    x = torch.empty(M, K, dtype=dtype, device="cuda")
    for i, part in enumerate(x.split(2 ** 15)):
        part.copy_(torch.randn(part.shape, generator=gen(i), device="cuda"))
    at = some(M, K)
    q = experts.quantize_int8(x)
    few = experts.quantize_int8(x[at])
    scale = x[at].float().abs().amax(-1) / torch.tensor(127.0, device="cuda")  # a division of tensors: rounded once
    assert torch.equal(q.scales[at], scale) and torch.equal(q.data[at], torch.round(x[at].double() / scale[:, None].double()).to(torch.int8))
    assert torch.equal(q.data[at], few.data) and torch.equal(q.scales[at], few.scales)
    del x
    back = experts.dequantize_int8(q, dtype)
    assert torch.equal(back[at], (q.data[at].float() * q.scales[at, None]).to(dtype))


def test_repeated_8_bit_rows():
    """Rows quantised once and copied to places past 2^31 bytes."""
    n, M, K = 1000, PAST // 8192 + 300, 8192
    x = torch.randn(n, K, generator=gen(9), device="cuda").bfloat16()
    rows = torch.randint(0, n, (M,), generator=gen(10), device="cuda").to(torch.int32)
    assert experts.quantize_int8_workspace_bytes(n, M, K) > 0
    q, once = experts.quantize_int8(x, rows=rows), experts.quantize_int8(x)
    at = some(M, K)
    assert torch.equal(q.data[at], once.data[rows[at].long()]) and torch.equal(q.scales, once.scales[rows.long()])
