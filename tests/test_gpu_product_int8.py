"""The experts' product of 8-bit integers: sums are exact, so results are those of the same three FP32
operations on the exact sum: float(sum) * a_scale * (alpha * w_scale), rounded to BF16."""
import pytest
import torch

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


def make(sizes, N, K, seed=0, before=0, after=0, lo=-128):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M = before + sum(sizes) + after
    E = len(sizes)
    o = torch.tensor([before] + [before + sum(sizes[:i + 1]) for i in range(E)], dtype=torch.int32, device="cuda")
    a = torch.randint(lo, 128, (M, K), generator=g, device="cuda").to(torch.int8)
    w = torch.randint(lo, 128, (E, N, K), generator=g, device="cuda").to(torch.int8)
    sa = torch.rand(M, generator=g, device="cuda") + 0.01
    sw = torch.rand(E, N, generator=g, device="cuda") + 0.01
    return experts.Int8(a, sa, offsets=o), experts.Int8(w, sw)


def expected(a, w, alpha=1.0):
    o = a.offsets.tolist()
    E, N, _ = w.data.shape
    out = torch.zeros(a.data.shape[0], N, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        s = slice(o[e], o[e + 1])
        sums = a.data[s].double() @ w.data[e].double().T  # whole numbers below 2^53
        out[s] = (sums.float() * a.scales[s, None] * (torch.tensor(alpha, device="cuda") * w.scales[e])).bfloat16()
    return out


def check(a, w, alpha=1.0, **kw):
    got = experts.expert_product(a, w, scale=alpha, **kw)
    want = expected(a, w, alpha)
    assert torch.equal(got, want), ((got.float() - want.float()).abs().max().item(), (got != want).nonzero()[:4].tolist())


SHAPES = [([1], 8, 16), ([3], 16, 48), ([0, 5, 0], 72, 64), ([1, 1, 1], 128, 128), ([16, 17, 15], 136, 144), ([33, 0, 64, 65], 256, 272),
          ([127, 128, 129], 264, 528), ([300], 520, 1040), ([7, 250, 1, 0, 96], 640, 1024), ([1000], 128, 2064), ([513, 511], 256, 256)]


@pytest.mark.parametrize("sizes,N,K", SHAPES)
def test_small(sizes, N, K):
    check(*make(sizes, N, K, seed=N + K, before=2, after=5), alpha=0.37)


@pytest.mark.parametrize("sizes,N,K", [([700, 1300, 40, 2000], 1024, 2320), ([900] * 16, 1000, 528), ([256, 512, 257, 4000, 31, 96], 2048, 1040),
                                       ([129, 128, 127, 1, 0, 65] * 4, 4096, 640)])
def test_large_groups(sizes, N, K):
    """Enough tiles for pairs of CTAs, with odd last tiles."""
    check(*make(sizes, N, K, seed=7, before=3, after=200))


@pytest.mark.parametrize("sizes,N,K", [([1], 64, 8192), ([0, 7, 0, 9], 512, 4096), ([16], 2048, 3008), ([40], 128, 2064), ([64], 4096, 2048),
                                       ([1] * 10, 512, 2048), ([70], 128, 4112), ([2], 8, 131056)])
def test_split_sums(sizes, N, K):
    check(*make(sizes, N, K, seed=3, after=1))


@pytest.mark.parametrize("sizes,N", [([20], 40), ([200] * 20, 1024)])
def test_sums_past_24_bits(sizes, N):
    """The largest sums, and large ones that cancel to a few units."""
    K = 4096 if len(sizes) > 1 else 131056
    a, w = make(sizes, N, K)
    a.data.fill_(-128)
    w.data.fill_(-128)
    check(a, w)
    a.data.fill_(127)
    w.data.fill_(127)
    w.data[:, :, K // 2:] = -127
    w.data[:, ::3, K // 3] = 126
    a.data[1::2, 5] = -3
    check(a, w)


def test_one_expert_without_offsets_and_bad_scales():
    a, w = make([75], 200, 96)
    want = expected(a, w)
    one = experts.Int8(a.data, a.scales)
    assert torch.equal(experts.expert_product(one, experts.Int8(w.data[0], w.scales[0])), want)
    a.scales[3] = float("nan")
    a.scales[9] = 0
    w.scales[0, 7] = float("inf")
    got = experts.expert_product(a, w)
    assert torch.isnan(got[3]).all() and (got[9, :7] == 0).all() and torch.isnan(got[9, 7])
    rows = [i for i in range(75) if i not in (3, 9)]
    assert torch.equal(got[rows][:, 8:], want[rows][:, 8:])


def test_quantised_rows_and_weights():
    """The run as it is used: rows by index to 8 bits, the product, against 64-bit values of the codes."""
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(30, 512, generator=g, device="cuda").bfloat16()
    wt = (torch.randn(4, 256, 512, generator=g, device="cuda") / 512 ** 0.5).bfloat16()
    ids = torch.randn(30, 4, generator=g, device="cuda").topk(2).indices.to(torch.int32)
    plan = experts.plan(ids, 4)
    a, w = experts.quantize_int8(h, rows=plan.rows, offsets=plan.offsets), experts.quantize_int8(wt)
    out = experts.expert_product(a, w)
    va, vw = experts.dequantize_int8(a, torch.float32).double(), experts.dequantize_int8(w, torch.float32).double()
    e = torch.arange(4, device="cuda").repeat_interleave(plan.offsets.diff().long())
    want = torch.einsum("mk,mnk->mn", va, vw[e])
    # values are rounded products of code and scale, 2^-24 each; three FP32 roundings; BF16's
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -21 * torch.einsum("mk,mnk->mn", va.abs(), vw[e].abs())
    assert ((out.double() - want).abs() <= tol).all()
    full = torch.einsum("mk,mnk->mn", h[plan.rows.long()].double(), wt[e].double())
    assert float((out.double() - full).norm() / full.norm()) < 0.02


def test_workspace_and_offsets():
    a, w = make([2000, 3000], 1024, 64)
    n = experts.product_int8_workspace_bytes(5000, 2, 1024, 64)
    assert n == 5000 * 64 * 2
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
    check(a, w, workspace=ws[:n])
    assert (ws[n:] == 255).all()
    ws.fill_(255)
    check(a, w, workspace=ws[:n - 16])  # too small: not used
    assert (ws == 255).all()
    a, w = make([20, 30], 64, 64)
    experts.expert_product(experts.Int8(a.data, a.scales, torch.tensor([0, 60, 50], dtype=torch.int32, device="cuda")), w)
    assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_OFFSETS
    empty = experts.Int8(a.data[:0], a.scales[:0], torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert experts.expert_product(empty, w).shape == (0, 64)


def test_offsets_past_32_bits():
    M, N, K = 270000, 8192, 16
    a, w = make([M], N, K)
    out = experts.expert_product(a, w)
    for lo, hi in ((0, 3), (131070, 131080), (262140, 262150), (M - 3, M)):
        part = experts.Int8(a.data[lo:hi], a.scales[lo:hi], torch.tensor([0, hi - lo], dtype=torch.int32))
        assert torch.equal(out[lo:hi], expected(part, w))
    del a, w, out
    E, N, K = 40, 8192, 8192
    w = experts.Int8(torch.zeros(E, N, K, dtype=torch.int8, device="cuda"), torch.ones(E, N, device="cuda"))
    w.data[-1] = torch.randint(-128, 128, (N, K), device="cuda").to(torch.int8)
    o = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    o[E - 1], o[E] = 2, 40
    a = experts.Int8(torch.randint(-128, 128, (40, K), device="cuda").to(torch.int8), torch.rand(40, device="cuda"), o)
    check(a, w)


def test_streams_and_graphs():
    a, w = make([300, 0, 500], 512, 256)
    want = expected(a, w)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [experts.expert_product(a, w, stream=x) for _ in range(4) for x in (s, t)]
    s.synchronize()
    t.synchronize()
    assert all(torch.equal(x, want) for x in got)
    graphs = []
    for _ in range(2):  # two graphs with workspaces of their own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = experts.expert_product(a, w)
        graphs.append((g, out))
    for seed in range(3):
        n, _ = make([300, 0, 500], 512, 256, seed=seed + 9)
        a.data.copy_(n.data)
        for g, _ in graphs:
            g.replay()
        assert all(torch.equal(out, expected(a, w)) for _, out in graphs)


def test_many_experts():
    g = torch.Generator().manual_seed(3)
    sizes = [0] * 1024
    for e in torch.randint(0, 1024, (300,), generator=g).tolist():
        sizes[e] += 1
    sizes[5], sizes[1023] = 300, 40
    check(*make(sizes, 72, 48, before=1, after=2))
    check(*make([0] * 1023 + [3], 128, 2048))


def test_no_row_in_any_group():
    check(*make([0, 0, 0], 64, 512, before=3, after=300))
    check(*make([0, 0, 0], 64, 512, after=9000))
