"""The experts' linear layers over long sums: y over K values, dx over N.

Tolerances.  Small whole numbers: every partial sum is below 2^24 and exact in FP32 in any order, so results are
the exact sum rounded once.  Values of one sign: the tensor core's sums lose at most 2^-23 of themselves for 16
values, over at most 16384 values: 2^-13; R such sums (and up to 8 CTAs' parts) are added with rounding,
(R + 8) * 2^-24; the rounding to FP16 or BF16 is eps / 2.  The mean over n outputs sees a loss below the rounding:
products of two uniform values have the relative spread sqrt(7 / 9), sums of D of them s = sqrt(7 / (9 D)), at least
8.6e-4 here.  Rounded to a step h they are off by h / pi * exp(-2 pi^2 (s / h)^2) in the mean: FP16's h is at most 2^-10,
which gives 1e-10, and of n such roundings of at most eps / 2 the mean is below 6 / sqrt(n) of that.  BF16's h is up
to 2^-7, its sums round alike (1e-3 in the mean), and only single outputs are held."""
import math

import pytest
import torch

from tp_reduce_residual_gb300 import beamnorm as bn
from tp_reduce_residual_gb300 import build as nbuild
from tp_reduce_residual_gb300 import experts

pytestmark = pytest.mark.gpu

RUN = 16384


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    nbuild.build()
    bn.load()
    bn.check_device_error(raise_on_error=False)
    yield
    assert bn.check_device_error() == 0


def outputs(x, w, offsets, rows):
    """The forward (rows fetched by the product and through a workspace, if by index), and the input gradient,
    which is the same sum over transposed weights."""
    grouped = x if rows is None else x[rows.long()]
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    yield "y", experts.expert_linear(x, w, offsets, rows=rows)
    if rows is not None:
        yield "y, rows fetched", experts.expert_linear(x, w, offsets, rows=rows, workspace=small)
    yield "dx", experts.expert_linear_dx(grouped, w.transpose(1, 2).contiguous(), offsets)


def groups(sizes):
    return torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], dtype=torch.int32, device="cuda")


# features F and values D: a cluster's parts, single CTAs, pairs, and what would be tall pairs
WHOLE = [([5], 64, 140000), ([64], 4096, 70000), ([70, 0, 3], 256, 70008), ([300], 6400, 33000), ([100, 0, 150], 2056, 33000),
         ([129, 128, 127, 1, 0, 65] * 4, 520, 16392), ([1200], 2048, 32768), ([4001], 4104, 17000), ([2300, 2600, 90], 264, 49160)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sizes,F,D", WHOLE)
def test_whole_numbers(sizes, F, D, gather, dtype):
    g = torch.Generator(device="cuda").manual_seed(F + D)
    M, o = sum(sizes), groups(sizes)
    n = max(1, M // 3) if gather else M
    rows = torch.randint(0, n, (M,), generator=g, device="cuda").to(torch.int32) if gather else None
    x = torch.randint(-3, 4, (n, D), generator=g, device="cuda").to(dtype)
    w = torch.randint(-3, 4, (len(sizes), F, D), generator=g, device="cuda").to(dtype)
    want = torch.empty(M, F, dtype=dtype, device="cuda")
    at = o.tolist()
    for e in range(len(sizes)):
        s = slice(at[e], at[e + 1])
        want[s] = ((x[s] if rows is None else x[rows[s].long()]).double() @ w[e].double().T).to(dtype)
    for what, got in outputs(x, w, o, rows):
        assert torch.equal(got, want), (what, (got.double() - want.double()).abs().max().item())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,F,D", [(40, 72, 2 ** 20), (40, 4096, 2 ** 18), (1200, 2048, 2 ** 18), (300, 6400, 2 ** 18), (1200, 2048, RUN), (600, 2048, 5 * RUN + 8)])
def test_sums_of_one_sign_keep_their_digits(M, F, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + D)
    x = torch.rand(M, D, generator=g, device="cuda").to(dtype)
    w = torch.empty(1, F, D, dtype=dtype, device="cuda")
    for part in w[0].split(256):
        part.copy_(torch.rand(part.shape, generator=g, device="cuda") * 2.0 ** -10)
    some = torch.arange(0, M, max(1, M // 32), device="cuda")
    want = torch.cat([x[some].double() @ part.double().T for part in w[0].split(512)], dim=1)
    runs, eps = -(-D // RUN), torch.finfo(dtype).eps / 2
    lost = 2.0 ** -13 + (runs + 8) * 2.0 ** -24
    for what, got in outputs(x, w, groups([M]), None):
        off = (got[some].double() - want) / want
        assert off.abs().max() <= eps * (1 + lost) + lost, (what, off.abs().max().item())
        assert dtype is torch.bfloat16 or off.mean().abs() <= lost + 6 * eps / math.sqrt(off.numel()), (what, off.mean().item())
