"""Edges of the experts' linear layers: places of no group, long sums, operands past 2^31 elements.

Whole numbers of small size: every product and partial sum is exact in FP32, so results are the exact sums
rounded once to the output's type."""
import pytest
import torch

from tests.test_gpu_linear import exact, make
from tp_reduce_residual_gb300 import beamnorm as bn
from tp_reduce_residual_gb300 import build as nbuild
from tp_reduce_residual_gb300 import experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    nbuild.build()
    bn.load()
    bn.check_device_error(raise_on_error=False)
    yield
    assert bn.check_device_error() == 0


def workspaces(M, K):
    """The call's own, one that is too small (rows fetched by the product), and one full of NaN."""
    return [None] + [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for size in (16, max(16, M * K * 2))]


@pytest.mark.parametrize("sizes,before,after", [([10, 0, 9], 5, 6), ([20, 0, 70], 9, 30), ([5, 300], 1, 400), ([64] * 40, 128, 0), ([3], 0, 2000)])
@pytest.mark.parametrize("unused", [-1, 2 ** 31 - 1])
def test_places_of_no_group_need_no_row(sizes, before, after, unused):
    """An index at such a place is not looked at, whichever way rows come."""
    d = make(sizes, 136, 264, "bf16", gather=True, before=before, after=after, seed=before)
    y, _, dw = (v.bfloat16() for v in exact(d))
    M = d["rows"].numel()
    d["rows"][:before] = unused
    d["rows"][M - after:] = unused
    for ws in workspaces(M, 264):
        assert torch.equal(experts.expert_linear(d["x"], d["w"], d["offsets"], rows=d["rows"], workspace=ws), y)
        assert torch.equal(experts.expert_linear_dw(d["dy"], d["x"], d["offsets"], rows=d["rows"], workspace=ws), dw)
        assert bn.check_device_error(raise_on_error=False) == 0
    d["rows"][before] = unused
    for ws in workspaces(M, 264):
        experts.expert_linear(d["x"], d["w"], d["offsets"], rows=d["rows"], workspace=ws)
        assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_PERM_RANGE


@pytest.mark.parametrize("offsets", [[10, 30, 5, 9], [0, 40, 20, 20], [-4, 12, 50, 999], [60, 60, 2, 40]])
def test_offsets_that_fall_reach_the_same_rows_by_any_way(offsets):
    """Groups that do not overlap, in any order: reported, and each has its rows."""
    d = make([20, 20, 20], 72, 136, "bf16", gather=True)
    d["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    o = [min(max(v, 0), 60) for v in offsets]
    for ws in workspaces(60, 136):
        y = experts.expert_linear(d["x"], d["w"], d["offsets"], rows=d["rows"], workspace=ws)
        dw = experts.expert_linear_dw(d["dy"], d["x"], d["offsets"], rows=d["rows"], workspace=ws)
        assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_OFFSETS
        for e in range(3):
            s = slice(o[e], max(o[e], o[e + 1]))
            x = d["x"][d["rows"][s].long()].double()
            assert torch.equal(dw[e], (d["dy"][s].double().T @ x).bfloat16())
            if o[e] >= o[0] and o[e + 1] <= o[3]:  # not among the rows that are cleared before and after
                assert torch.equal(y[s], (x @ d["w"][e].double().T).bfloat16())


def test_gradient_of_rows_taken_several_times():
    """Small whole numbers: dx is exact, and so is a sum over three places (below 256, BF16's whole numbers)."""
    g = torch.Generator(device="cuda").manual_seed(4)
    T, E, k, N, K = 50, 8, 3, 24, 264
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k).indices.int()
    plan = experts.plan(ids, E)
    w = torch.randint(-1, 2, (E, N, K), generator=g, device="cuda").bfloat16()
    dy = torch.randint(-1, 2, (T * k, N), generator=g, device="cuda").bfloat16()
    dx = experts.expert_linear_dx(dy, w, plan.offsets)
    got = bn.finalize_reduce_only(dx[None], plan.perm, torch.ones(1, T, k, device="cuda"), None)
    expert = torch.arange(E, device="cuda").repeat_interleave(plan.offsets.diff().long())
    rows = torch.einsum("mn,mnk->mk", dy.double(), w[expert].double())
    want = torch.zeros(T, K, dtype=torch.float64, device="cuda").index_add_(0, plan.rows.long(), rows)
    assert got.dtype is torch.float32 and torch.equal(got.double(), want)
    for fn in (bn.finalize_reduce_only, bn.finalize_only):  # rows in FP16 are refused
        with pytest.raises(TypeError, match="bfloat16"):
            fn(dx[None].half(), plan.perm, torch.ones(1, T, k, device="cuda"), None)
