"""The experts' linear layers in 16 bits and their gradients against sums in 64 bits.

Tolerances.  Small whole numbers: every product and partial sum is a whole number below 2^24, exact in
FP32 in any order, so results equal the exact sum rounded once to the output's type.  Other values: D
additions in 32 bits, 2^-23 each of the sum of |a b|, and the rounding, eps / 2 of the value (FP16's
smallest step is 2^-24)."""
import pytest
import torch

from tp_reduce_residual_gb300 import beamnorm as bn
from tp_reduce_residual_gb300 import build as nbuild
from tp_reduce_residual_gb300 import experts

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    nbuild.build()
    bn.load()
    bn.check_device_error(raise_on_error=False)
    yield
    assert bn.check_device_error() == 0


def values(shape, dtype, g, whole):
    if whole:
        return torch.randint(-3, 4, shape, generator=g, device="cuda").to(dtype)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def make(sizes, N, K, dtype, whole=True, seed=0, before=0, after=0, gather=False, E=None):
    """x [n,K], w [E,N,K], dy [M,N], offsets, rows for groups of these sizes, with rows of no group around them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[dtype]
    M = before + sum(sizes) + after
    o = torch.tensor([before] + [before + sum(sizes[:i + 1]) for i in range(len(sizes))], dtype=torch.int32, device="cuda")
    rows = None
    n = M
    if gather:
        n = max(1, M // 3)
        rows = torch.randint(0, n, (M,), generator=g, device="cuda").to(torch.int32)
    return dict(x=values((n, K), dt, g, whole), w=values((len(sizes), N, K), dt, g, whole), dy=values((M, N), dt, g, whole),
                offsets=o, rows=rows)


def exact(d):
    x = d["x"].double() if d["rows"] is None else d["x"][d["rows"].long()].double()
    w, dy, o = d["w"].double(), d["dy"].double(), d["offsets"].tolist()
    M = dy.shape[0]
    y = torch.zeros(M, w.shape[1], dtype=torch.float64, device="cuda")
    dx = torch.zeros(M, w.shape[2], dtype=torch.float64, device="cuda")
    dw = torch.zeros_like(w)
    for e in range(w.shape[0]):
        s = slice(o[e], o[e + 1])
        y[s], dx[s], dw[e] = x[s] @ w[e].T, dy[s] @ w[e], dy[s].T @ x[s]
    return y, dx, dw


def sizes_abs(d):
    a = {k: d[k].abs() if k in ("x", "w", "dy") else d[k] for k in d}
    return exact(a)


def close(got, want, total, depth, what):
    t = got.dtype
    tol = depth * 2.0 ** -23 * total + torch.finfo(t).eps / 2 * want.abs() + (2.0 ** -24 if t is torch.float16 else 0.0)
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all() and (off <= tol).all(), (what, (off - tol).max().item(), got.shape)


def run(d, dw_dtype=None):
    y = experts.expert_linear(d["x"], d["w"], d["offsets"], rows=d["rows"])
    dx = experts.expert_linear_dx(d["dy"], d["w"], d["offsets"])
    dw = experts.expert_linear_dw(d["dy"], d["x"], d["offsets"], rows=d["rows"], dtype=dw_dtype)
    return y, dx, dw


def check(d, whole, dw_dtype=None):
    got = run(d, dw_dtype)
    want = exact(d)
    total = None if whole else sizes_abs(d)
    for i, what in enumerate(("y", "dx", "dw")):
        if whole:
            assert torch.equal(got[i], want[i].to(got[i].dtype)), (what, (got[i].double() - want[i]).abs().max().item())
        else:
            depth = (d["w"].shape[2], d["w"].shape[1], d["dy"].shape[0])[i]
            close(got[i], want[i], total[i], depth, what)


SHAPES = [
    ([1], 8, 8), ([3], 16, 24), ([0, 5, 0], 72, 64), ([1, 1, 1], 128, 128), ([16, 17, 15], 136, 72), ([33, 0, 64, 65], 256, 200),
    ([127, 128, 129], 264, 136), ([300], 520, 328), ([7, 250, 1, 0, 96], 640, 512), ([1000], 128, 64), ([513, 511], 256, 256),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sizes,N,K", SHAPES)
def test_whole_numbers(sizes, N, K, dtype, gather):
    check(make(sizes, N, K, dtype, gather=gather, seed=N + K, before=2, after=5), whole=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("sizes,N,K", SHAPES[3:8])
def test_real_numbers(sizes, N, K, dtype):
    check(make(sizes, N, K, dtype, whole=False, gather=True, seed=K), whole=False)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sizes,N,K", [([700, 1300, 40, 2000], 1024, 768), ([900] * 16, 1000, 520), ([256, 512, 257, 4000, 31, 96], 2048, 1032)])
def test_large_groups(sizes, N, K, gather):
    """Enough tiles for pairs of CTAs in every product, with odd last tiles."""
    check(make(sizes, N, K, "bf16", gather=gather, seed=7, before=3, after=200), whole=True)


def test_long_sum():
    check(make([20, 40], 64, 8200, "bf16", gather=True), whole=True)
    check(make([20000, 3], 264, 72, "bf16"), whole=True)


@pytest.mark.parametrize("sizes,N,K", [([5, 0, 70], 72, 136), ([400, 0, 900], 512, 520)])
def test_weight_gradient_in_32_bits_accumulates(sizes, N, K):
    d = make(sizes, N, K, "bf16", gather=True)
    want = exact(d)[2]
    dw = experts.expert_linear_dw(d["dy"], d["x"], d["offsets"], rows=d["rows"], dtype=torch.float32)
    assert dw.dtype is torch.float32 and torch.equal(dw.double(), want)
    again = experts.expert_linear_dw(d["dy"], d["x"], d["offsets"], rows=d["rows"], dw=dw, accumulate=True)
    assert again is dw and torch.equal(dw.double(), 2 * want)
    assert (dw[1] == 0).all()


def test_one_expert_without_offsets():
    d = make([150], 200, 96, "fp16")
    y, dx, dw = exact(d)
    assert torch.equal(experts.expert_linear(d["x"], d["w"][0]), y.half())
    assert torch.equal(experts.expert_linear_dx(d["dy"], d["w"][0]), dx.half())
    got = experts.expert_linear_dw(d["dy"], d["x"])
    assert got.shape == (200, 96) and torch.equal(got, dw[0].half())


def test_row_strides():
    d = make([40, 90], 128, 72, "bf16")
    want = run(d)
    wide = torch.full((130, 200), float("nan"), dtype=torch.bfloat16, device="cuda")
    x, dy = wide[:, 8:80], torch.full((130, 160), float("inf"), dtype=torch.bfloat16, device="cuda")[:, 16:144]
    x.copy_(d["x"])
    dy.copy_(d["dy"])
    got = run(dict(d, x=x, dy=dy))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_group(bad):
    """What is not in a group's rows, features or sums adds nothing to it, not even 0 * NaN."""
    d = make([37, 5, 70, 0, 3], 72, 104, "bf16", before=9, after=11)
    want = exact(d)
    o = d["offsets"].tolist()
    d["x"][:9] = bad
    d["dy"][:9] = bad
    d["x"][o[-1]:] = bad
    d["dy"][o[-1]:] = bad
    d["x"][o[1]:o[2]] = bad
    d["dy"][o[1]:o[2]] = bad
    d["w"][1] = bad
    got = run(d)
    for e in (0, 2, 3, 4):
        s = slice(o[e], o[e + 1])
        assert torch.equal(got[0][s], want[0][s].bfloat16()) and torch.equal(got[1][s], want[1][s].bfloat16())
        assert torch.equal(got[2][e], want[2][e].bfloat16())
    s = slice(o[1], o[2])
    assert not torch.isfinite(got[0][s]).any() and not torch.isfinite(got[2][1]).any()
    assert (got[0][:9] == 0).all() and (got[0][o[-1]:] == 0).all() and (got[1][o[-1]:] == 0).all()


def test_bad_rows_and_offsets_are_reported():
    d = make([20, 30], 64, 64, "bf16", gather=True)
    rows = d["rows"].clone()
    rows[3], rows[40] = -1, d["x"].shape[0]
    fixed = rows.clone()
    fixed[3] = fixed[40] = 0
    for fn in (lambda r: experts.expert_linear(d["x"], d["w"], d["offsets"], rows=r),
               lambda r: experts.expert_linear_dw(d["dy"], d["x"], d["offsets"], rows=r)):
        got = fn(rows)
        assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_PERM_RANGE
        assert torch.equal(got, fn(fixed))
    wrong = torch.tensor([0, 60, 50], dtype=torch.int32, device="cuda")
    experts.expert_linear(d["x"], d["w"], wrong, rows=d["rows"])
    assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_OFFSETS


def test_no_rows():
    w = torch.ones(3, 16, 24, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = (torch.empty(0, n, dtype=torch.bfloat16, device="cuda") for n in (24, 16))
    assert experts.expert_linear(x, w, o).shape == (0, 16)
    assert experts.expert_linear_dx(dy, w, o).shape == (0, 24)
    assert (experts.expert_linear_dw(dy, x, o) == 0).all()
    dw = torch.full((3, 16, 24), 2.0, device="cuda")
    experts.expert_linear_dw(dy, x, o, dw=dw, accumulate=True)
    assert (dw == 2).all()


@pytest.mark.parametrize("M", [32, 33, 300])
def test_rows_with_and_without_a_workspace(M):
    """The product fetches rows itself where it gets no workspace, or one that is too small."""
    d = make([M // 3, 0, M - M // 3], 136, 264, "bf16", gather=True, before=2)
    y, _, dw = exact(d)
    n = experts.linear_workspace_bytes(M + 2, 264)
    assert n == (0 if M + 2 <= 32 else (M + 2) * 264 * 2)
    for size in (16, n, n + 160):
        ws = torch.full((max(size, 16),), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(experts.expert_linear(d["x"], d["w"], d["offsets"], rows=d["rows"], workspace=ws), y.bfloat16())
        assert torch.equal(experts.expert_linear_dw(d["dy"], d["x"], d["offsets"], rows=d["rows"], workspace=ws), dw.bfloat16())
        if size == 16:
            assert (ws == 255).all()


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sizes,N,K", [([1], 64, 8192), ([0, 7, 0, 9], 512, 4096), ([16], 2048, 3000), ([40], 128, 2056), ([64], 4096, 2048),
                                       ([1, 1, 1, 1, 1, 1, 1, 1, 1, 1], 512, 2048), ([70], 128, 4104)])
def test_split_sums(sizes, N, K, gather):
    """Few tiles and a long sum: clusters of CTAs that each sum a part, by 2 to 8."""
    d = make(sizes, N, K, "bf16", gather=gather, seed=3, after=1)
    check(d, whole=True)
    t = dict(d, w=d["w"].transpose(1, 2).contiguous(), x=d["dy"], dy=d["x"] if not gather else d["x"][d["rows"].long()], rows=None)
    check(t, whole=True)
    check(make(sizes, N, K, "fp16", whole=False, gather=gather), whole=False)


def test_offsets_past_32_bits():
    """Rows, weights and gradients whose elements lie beyond 2^31."""
    g = torch.Generator(device="cuda").manual_seed(5)
    M, N, K = 270000, 8192, 16
    x, w = values((M, K), torch.bfloat16, g, True), values((N, K), torch.bfloat16, g, True)
    y = experts.expert_linear(x, w)
    for s in (slice(0, 3), slice(131070, 131080), slice(262140, 262150), slice(M - 3, M)):
        assert torch.equal(y[s], (x[s].double() @ w.double().T).bfloat16())
    wide = experts.expert_linear_dw(y[:, :64], y)  # rows of dy and x far apart
    assert wide.shape == (64, N) and torch.isfinite(wide).all()
    dx = experts.expert_linear_dx(y, w)  # sums past 2^24: to FP32 rounding
    want = y[M - 2:].double() @ w.double()
    assert ((dx[M - 2:].double() - want).abs() <= 2.0 ** -8 * want.abs() + N * 2.0 ** -23 * (y[M - 2:].double().abs() @ w.double().abs())).all()
    del x, w, y, wide, dx
    E, N, K = 40, 8192, 8192
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    w[-1] = values((N, K), torch.bfloat16, g, True)
    o = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    o[E - 1], o[E] = 2, 40
    x, dy = values((40, K), torch.bfloat16, g, True), values((40, N), torch.bfloat16, g, True)
    y, dx = experts.expert_linear(x, w, o), experts.expert_linear_dx(dy, w, o)
    dw = experts.expert_linear_dw(dy, x, o)
    assert torch.equal(y[2:], (x[2:].double() @ w[-1].double().T).bfloat16()) and torch.equal(dx[2:], (dy[2:].double() @ w[-1].double()).bfloat16())
    assert (y[:2] == 0).all() and (dx[:2] == 0).all() and (dw[0] == 0).all()
    assert torch.equal(dw[-1], (dy[2:].double().T @ x[2:].double()).bfloat16())


def test_streams():
    """Calls on a stream of the caller's, with outputs and workspace from its pool, and two at once."""
    d = make([300, 0, 500], 512, 256, "bf16", gather=True)
    want = [v.bfloat16() for v in exact(d)]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in (a, b):
            got.append((s, experts.expert_linear(d["x"], d["w"], d["offsets"], rows=d["rows"], stream=s),
                        experts.expert_linear_dx(d["dy"], d["w"], d["offsets"], stream=s.cuda_stream),
                        experts.expert_linear_dw(d["dy"], d["x"], d["offsets"], rows=d["rows"], stream=s)))
    a.synchronize()
    b.synchronize()
    for _, *v in got:
        assert all(torch.equal(x, y) for x, y in zip(v, want))


def test_equal_calls_give_equal_bits():
    for sizes, N, K in (([200, 31, 900], 264, 1032), ([5], 72, 4096)):
        d = make(sizes, N, K, "bf16", whole=False)
        first = run(d, torch.float32)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(run(d, torch.float32), first))


def test_gradients_against_differences():
    """The forward's own change along the gradients, in FP32 sums of BF16 values."""
    d = make([30, 0, 50], 64, 96, "bf16", whole=False, seed=11)
    y, dx, dw = run(d, torch.float32)
    x, w, dy = d["x"].double(), d["w"].double(), d["dy"].double()
    o = d["offsets"].tolist()

    def value(x, w):
        return sum((x[o[e]:o[e + 1]] @ w[e].T * dy[o[e]:o[e + 1]]).sum() for e in range(3))

    for which, v in (("x", dx.double()), ("w", dw.double())):
        v = v / v.norm()
        ends = [value(x + s * v, w) if which == "x" else value(x, w + s * v) for s in (0.5, -0.5)]  # linear: any step
        want = ((dx if which == "x" else dw).double() * v).sum()
        assert abs(ends[0] - ends[1] - want) <= 2.0 ** -8 * abs(want)


def test_captured_and_replayed():
    d = make([90, 0, 40], 136, 264, "bf16", gather=True)
    run(d)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs with workspaces of their own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(d)
        graphs.append((g, out))
    for seed in range(3):
        n = make([90, 0, 40], 136, 264, "bf16", gather=True, seed=seed + 20)
        for k in ("x", "w", "dy", "rows"):
            d[k].copy_(n[k])
        for g, _ in graphs:
            g.replay()
        want = exact(d)
        for _, out in graphs:
            assert all(torch.equal(a, b.bfloat16()) for a, b in zip(out, want))


@pytest.mark.parametrize("sizes,N,K", [([4001], 4104, 520), ([4001], 520, 4104), ([3000, 0, 5000], 2056, 264), ([2300, 2600, 90], 264, 4096)])
def test_tall_tiles(sizes, N, K):
    """A few large groups: pairs whose tiles have 512 rows, with odd last tiles of one block and of two."""
    check(make(sizes, N, K, "bf16", seed=13, before=1, after=40), whole=True)


@pytest.mark.parametrize("N,K", [(72, 200), (2048, 1536)])
def test_long_gradients_keep_32_bits(N, K):
    """Sums of one sign over 8192 rows.  The tensor core's sums lose at most 2^-23 a step of 16 rows, in runs of
    256 rows: 16 * 2^-23 of a run; 32 runs are added, 2^-24 of the sum each: 32 * 2^-24."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.rand(8200, n, generator=g, device="cuda").bfloat16() for n in (K, N))
    o = torch.tensor([0, 8192, 8200], dtype=torch.int32, device="cuda")
    dw = experts.expert_linear_dw(dy, x, o, dtype=torch.float32)
    for e, s in ((0, slice(0, 8192)), (1, slice(8192, 8200))):
        want = dy[s].double().T @ x[s].double()
        assert ((dw[e].double() - want).abs() <= (16 * 2.0 ** -23 + 32 * 2.0 ** -24) * want).all()
    want = dy[:8192].double().T @ x[:8192].double()
    half = experts.expert_linear_dw(dy, x, o)[0].double()  # runs of 4096 rows: 256 steps
    assert ((half - want).abs() <= (2.0 ** -8 + 256 * 2.0 ** -23 + 2.0 ** -23) * want).all()


def test_many_experts():
    """1024 experts, most of them empty, a few large."""
    g = torch.Generator().manual_seed(3)
    sizes = [0] * 1024
    for e in torch.randint(0, 1024, (300,), generator=g).tolist():
        sizes[e] += 1
    sizes[5], sizes[1023] = 300, 40
    for gather in (False, True):
        check(make(sizes, 72, 40, "bf16", gather=gather, before=1, after=2), whole=True)
    check(make([0] * 1023 + [3], 128, 1024, "fp16", gather=True), whole=True)


def test_no_row_in_any_group():
    for gather in (False, True):
        check(make([0, 0, 0], 64, 512, "bf16", before=3, after=300, gather=gather), whole=True)
    d = make([0, 0], 64, 512, "bf16", after=7)
    dw = torch.full((2, 64, 512), 3.0, device="cuda")
    experts.expert_linear_dw(d["dy"], d["x"], d["offsets"], dw=dw, accumulate=True)
    assert (dw == 3).all()
