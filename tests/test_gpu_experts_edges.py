"""The operators around the experts at the edges of their ranges, against the 64-bit definitions.

Tolerances are those of ``test_gpu_experts`` except where a test states its own."""
import math

import pytest
import torch

from tests import experts_reference as ref
from tests.test_gpu_experts import DTYPES, _gpu, check_route, gen  # noqa: F401
from tp_reduce_residual_gb300 import beamnorm as bn
from tp_reduce_residual_gb300 import experts

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min


# ---- routing: masks of the type's lowest value in small groups ---------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,gtop", [(64, 32, 8, 1), (64, 32, 8, 2), (96, 32, 5, 1), (96, 32, 5, 2), (60, 20, 4, 2), (6, 3, 2, 1),
                                               (24, 8, 3, 2), (40, 8, 2, 1), (256, 8, 4, 1), (256, 8, 4, 2)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_route_groups_masked_by_the_lowest_value(score, E, groups, top, gtop, dtype):
    """Experts masked by the type's lowest value, whole groups among them, with -inf beside them: a group may
    have four keys or fewer left, and the sum of its two is past 32 bits."""
    g = gen(E + groups)
    x = torch.randn(24, E, generator=g).to(DTYPES[dtype])
    low = torch.finfo(DTYPES[dtype]).min
    x[torch.rand(24, E, generator=g) < 0.6] = low
    x[torch.rand(24, E, generator=g) < 0.3] = -math.inf
    x[0] = low
    x[1, :E // groups] = low
    x[2] = low
    x[2, ::2] = -math.inf
    x[3, E // groups:] = -math.inf
    x[4] = -math.inf
    check_route(x, min(3, top * (E // groups)), score=score, groups=groups, top_groups=top, group_top=gtop, renormalize=False)
    check_route(x[:1], 2, score=score, groups=groups, top_groups=top, group_top=gtop, renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,gtop", [(64, 32, 8, 2), (96, 32, 5, 2), (60, 20, 4, 2), (6, 3, 2, 1), (256, 8, 4, 2)])
@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_route_groups_masked_by_the_bias(score, E, groups, top, gtop, dtype):
    """The same masks held by the bias, and biases so high that sums of two pass 32 bits upwards."""
    g = gen(E + top)
    x = torch.randn(8, E, generator=g).to(DTYPES[dtype])
    x[torch.rand(8, E, generator=g) < 0.3] = -math.inf
    for value in (LOWEST, -LOWEST):
        bias = 0.1 * torch.randn(E, generator=g)
        bias[torch.rand(E, generator=g) < 0.5] = value
        bias[:E // groups] = value
        bias[E - 1] = -math.inf
        check_route(x, min(3, top * (E // groups)), bias=bias, score=score, groups=groups, top_groups=top, group_top=gtop,
                    renormalize=False)


# ---- the product: what is in flight when a pair of CTAs leaves -----------------------------------------

def test_products_back_to_back():
    """Short products on pairs of CTAs, each followed at once by kernels that take over its shared memory (a
    product on single CTAs and one on pairs): an arrival that came after its CTA had left would land on one
    of their barriers.  Every output has the bits of the first, and no wait gave up."""
    g = gen(40)

    def operands(rows, N, K):
        a = experts.quantize_fp4(torch.randn(rows, K, generator=g).bfloat16().cuda(), "nvfp4")
        b = experts.quantize_fp4(torch.randn(N, K, generator=g).bfloat16().cuda(), "nvfp4")
        return a, b

    calls = [operands(2100, 2056, 32), operands(130, 264, 64), operands(900, 4360, 96)]
    want = [experts.expert_product(a, b) for a, b in calls]
    outs = [[torch.empty_like(w) for w in want] for _ in range(2)]
    torch.cuda.synchronize()
    off = torch.zeros((), dtype=torch.long, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(100):
            for set_ in outs:  # six products without another kernel between them
                for (a, b), o in zip(calls, set_):
                    experts.expert_product(a, b, out=o)
            for set_ in outs:
                for o, w in zip(set_, want):
                    off += (o != w).sum()
                    o.zero_()
    side.synchronize()
    assert off.item() == 0


# ---- routing: 16-bit floats with sums ------------------------------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top,gtop", [
    (40, 256, 8, 8, 4, 2), (17, 256, 8, 8, 3, 1), (9, 160, 6, 8, 3, 2), (11, 56, 5, 8, 5, 2), (5, 24, 4, 24, 7, 2),
    (3, 1024, 16, 32, 4, 2), (8, 512, 10, 2, 1, 1), (4, 40, 2, 1, 1, 1), (6, 513, 16, 1, 1, 1)])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("strided", [False, True])
def test_route_fp16_sums(score, T, E, k, groups, top, gtop, biased, strided):
    """FP16 logits with a bias, with sums of group scores, and rows with masks, subnormals and the type's
    extremes among them."""
    g = gen(E + k + 1)
    x = torch.randn(T, E, generator=g)
    x[1] *= 2.0 ** -20
    x[2, torch.rand(E, generator=g) < 0.5] = -math.inf
    x = x.half()
    x[0, 3], x[0, E - 1] = torch.finfo(torch.float16).min, -0.0
    bias = 0.1 * torch.randn(E, generator=g) if biased else None
    check_route(x, k, bias=bias, score=score, groups=groups, top_groups=top, group_top=gtop, shards=2, strided=strided)


# ---- routing: infinite logits --------------------------------------------------------------------------

@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [False, True])
def test_route_infinite_logit(renormalize, biased):
    """exp(inf - inf): a softmax with an infinite logit has no weights, as with a NaN; a sigmoid of it is 1."""
    x = torch.randn(5, 64, generator=gen(60))
    x[1, 7] = math.inf
    x[3, 9] = x[3, 40] = math.inf
    x[4, 8:] = -math.inf
    x[4, 3] = math.inf
    bias = torch.zeros(64, device="cuda") if biased else None
    ids, w = experts.route(x.cuda(), 10, bias=bias, renormalize=renormalize)
    clean = experts.route(x[[0, 2]].cuda(), 10, bias=bias, renormalize=renormalize)
    assert torch.isnan(w[0, [1, 3, 4]]).all() and torch.equal(w[0, [0, 2]], clean[1][0])
    assert torch.equal(ids[[0, 2]], clean[0])
    ids, w = experts.route(x.cuda(), 10, bias=bias, score="sigmoid", renormalize=False)
    assert ids[1, 0].item() == 7 and ids[3, :2].tolist() == [9, 40] and ids[4, 0].item() == 3
    assert w[0, 1, 0].item() == 1.0 and torch.isfinite(w).all()


# ---- normalised sigmoids of small scores ---------------------------------------------------------------

def small_scores(dtype, seed):
    """Rows whose largest chosen logit is far below 0, to where the scores leave 32 bits, and mixed ones."""
    g = gen(seed)
    x = torch.randn(12, 40, generator=g)
    for t, shift in enumerate((-20, -60, -69, -75, -87, -90, -104, -200, -650)):
        x[t] += shift
    x[9] -= 75
    x[9, ::3] -= 300
    x[10] -= 90
    x[10, 7] = 3.0
    x[11] = -90.0
    return x.to(DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_normalised_sigmoids_of_small_scores(dtype, groups):
    """The weights are s over their sum however small the scores are."""
    x = small_scores(dtype, 50)
    _, w = check_route(x, 8, score="sigmoid", scale=2.5, groups=groups, top_groups=min(groups, 2))
    assert ((w.sum(-1) - 2.5).abs() < 2.5 * 2.0 ** -18).all()


def test_route_normalised_sigmoids_past_64_bits_are_zero():
    """Rows whose chosen logits are all below -709.78, where exp(-x) passes 64 bits, count as masked; beside a
    larger one such a logit has weight 0."""
    x = torch.full((4, 32), -709.0)
    x[1] = -710.0
    x[2] = -65504.0
    x[3] = LOWEST
    x[3, 4] = -709.5
    _, w = experts.route(x.cuda(), 8, score="sigmoid")
    w = w[0].cpu()
    assert ((w[0] - 0.125).abs() <= 2.0 ** -18).all()
    assert (w[1] == 0).all() and (w[2] == 0).all()
    assert w[3].tolist() == [1.0] + [0.0] * 7
    dw = torch.randn(1, 4, 8, generator=gen(51)).cuda()
    ids = torch.arange(8, dtype=torch.int32).repeat(4, 1).cuda()
    d = experts.route_backward(x.cuda(), ids, dw, score="sigmoid").cpu()
    assert torch.isfinite(d).all() and (d[1] == 0).all() and (d[2] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_route_backward_normalised_sigmoids_of_small_scores(dtype):
    """dx_j = w_j (c_j - sum_i w_i c_i) (1 - s_j): each w within 2^-18 (32-bit exponentials of differences of at
    most 8, or weights that are nothing beside the others), so 2^-16 of w_j (|c_j| + sum_i w_i |c_i|)."""
    x = small_scores(dtype, 52)
    ids, _ = ref.route(x, 8, score="sigmoid")
    c = torch.randn(12, 8, generator=gen(53))
    x64 = x.double().requires_grad_()
    (ref.route_weights(x64, ids, "sigmoid", True, 1.0) * c.double()).sum().backward()
    got = experts.route_backward(x.cuda(), ids.cuda(), c[None].cuda(), score="sigmoid").cpu().double()
    w = ref.route_weights(x.double(), ids, "sigmoid", True, 1.0)
    size = w * (c.double().abs() + (w * c.double().abs()).sum(-1, keepdim=True))
    tol = torch.zeros_like(got).scatter_(1, ids.long(), 2.0 ** -16 * size)
    tol += torch.finfo(DTYPES[dtype]).eps / 2 * x64.grad.abs() + (2.0 ** -25 if dtype == "fp16" else 1e-37)
    assert ((got - x64.grad).abs() <= tol).all()


# ---- gradients of saturated rows -----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True)])
@pytest.mark.parametrize("gap", [4, 8, 12, 20, 40, 80])
def test_route_backward_of_a_dominant_expert(dtype, score, renormalize, gap):
    """One expert (or two) far ahead: its gradient w_j sum_i w_i (c_j - c_i) is as exact as the others'.  Logits
    are whole numbers, so exponentials are the only errors of w: 2^-18 with their sum.  With D the largest,
    2^-16 of w_j (|c_j - c_D| + sum_i w_i |c_i - c_D|) and the rounding to the logits' type."""
    g = gen(gap)
    T, E, k = 10, 48, 6
    x = torch.randint(-3, 1, (T, E), generator=g).float() - (gap if score == "sigmoid" else 0)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    for t in range(T):
        x[t, ids[t, t % k]] += gap
    x[8, ids[8, 0]] = x[8, ids[8, 2]]  # two of them
    x[9, (set(range(E)) - set(ids[9].tolist())).pop()] = gap + 5.0  # one that was not chosen
    c = torch.randint(-8, 9, (T, k), generator=g).float()
    c[0] = torch.tensor([1.0, 0, 0, 0, 0, 0])
    ids[1, 3] = -1
    ids[1, 2], ids[1, 4] = ids[1, 1], ids[1, 1]  # an expert chosen again
    x, up = x.to(DTYPES[dtype]), torch.zeros(T, E, dtype=torch.float64)
    got = experts.route_backward(x.cuda(), ids.cuda(), c[None].cuda(), score=score, renormalize=renormalize).cpu().double()
    want, size = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        on = [j for j in range(k) if ids[t, j] >= 0]
        e = [int(ids[t, j]) for j in on]
        cc = [float(c[t, j]) for j in on]
        if not renormalize:  # every expert of the row, with the sum of its slots' c
            cc = [sum(v for i, v in zip(e, cc) if i == n) for n in range(E)]
            e = list(range(E))
        z = x[t, e].double()
        w = torch.softmax(z, 0) if score == "softmax" else torch.softmax(torch.nn.functional.logsigmoid(z), 0)
        cc = torch.tensor(cc, dtype=torch.float64)
        d = w * (w * (cc[:, None] - cc)).sum(1)
        far = cc - cc[w.argmax()]
        s = w * (far.abs() + (w * far.abs()).sum())
        if score == "sigmoid":
            d, s = d * torch.sigmoid(-z), s * torch.sigmoid(-z)
        for i, n in enumerate(e):
            want[t, n] += d[i]
            size[t, n] += s[i]
    tol = 2.0 ** -16 * size + torch.finfo(DTYPES[dtype]).eps / 2 * want.abs() + 1e-37
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E", [8, 100, 1024])
@pytest.mark.parametrize("spread", [0, 1, 3])
def test_route_backward_of_light_experts(dtype, E, spread):
    """No expert has much of the weight, the largest is chosen and its c is far above the others': the others'
    gradients p_e (c_e - sum_i p_i c_i) are as exact as without it.  Whole logits, so 2^-16 of
    p_e (|c_e| + sum_i p_i |c_i|), and with an expert D of more than a quarter of p (at 8 experts) of
    4 p_e (|c_e - c_D| + sum_i p_i |c_i - c_D|)."""
    g = gen(E + spread)
    T, k = 12, 4
    x = torch.randint(-spread, 1, (T, E), generator=g).float()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    x[torch.arange(T), ids[:, 0].long()] = 0.0
    c = torch.randint(-4, 5, (T, k), generator=g).float()
    c[:, 0] = 4096.0
    c[::2, 0] = 1.0
    c[1::4, 1:] = 0.0
    x = x.to(DTYPES[dtype])
    got = experts.route_backward(x.cuda(), ids.cuda(), c[None].cuda(), renormalize=False).cpu().double()
    p = torch.softmax(x.double(), 1)
    u = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ids.long(), c.double())
    want = p * (p[:, None, :] * (u[:, :, None] - u[:, None, :])).sum(-1)
    heavy, at = p.max(1)
    off = torch.where(heavy > 0.25 - 2.0 ** -20, u.gather(1, at[:, None])[:, 0], 0.0)[:, None]
    plain = p * (u.abs() + (p * u.abs()).sum(1, keepdim=True))
    less = 4 * p * ((u - off).abs() + (p * (u - off).abs()).sum(1, keepdim=True))
    size = torch.where(heavy[:, None] > 0.25 - 2.0 ** -20, torch.maximum(plain, less), plain)
    tol = 2.0 ** -16 * size + torch.finfo(DTYPES[dtype]).eps / 2 * want.abs() + 1e-37
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()


# ---- outputs on a caller's stream ----------------------------------------------------------------------

def pool_of(t):
    """The stream whose allocator pool a tensor's memory comes from."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


def calls():
    """Every binding that allocates an output, by name."""
    g = gen(70)
    R, T, k, H, E, K = 2, 6, 2, 256, 4, 64
    part = torch.randn(R, T, H, generator=g).bfloat16().cuda()
    eo = torch.randn(R, T * k, H, generator=g).bfloat16().cuda()
    perm = torch.arange(T * k, dtype=torch.int32).view(1, T, k).repeat(R, 1, 1).cuda()
    w = torch.rand(R, T, k, generator=g).cuda()
    sum_ = torch.randn(T, H, generator=g).cuda()
    gamma = torch.ones(H, device="cuda")
    logits = torch.randn(T, E, generator=g).cuda()
    ids = torch.randint(0, E, (T, k), generator=g).to(torch.int32).cuda()
    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    a = experts.quantize_fp4(x, "nvfp4")
    b = experts.quantize_fp4(torch.randn(16, K, generator=g).bfloat16().cuda(), "nvfp4")
    res = lambda: torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    r = [res() for _ in range(8)]
    return dict(
        reduce_norm=lambda s: [bn.reduce_norm(part, r[0], gamma, gamma, 1e-6, stream=s)],
        finalize_reduce_norm=lambda s: [bn.finalize_reduce_norm(eo, perm, w, None, r[1], gamma, gamma, 1e-6, stream=s)],
        finalize_reduce_norm_noalloc=lambda s: [bn.finalize_reduce_norm_noalloc(eo, perm, w, None, r[2], gamma, gamma, 1e-6, stream=s)],
        reduce_residual_norm=lambda s: [bn.reduce_residual_norm(part, r[3], gamma, 1e-6, stream=s)],
        finalize_reduce_residual_norm=lambda s: [bn.finalize_reduce_residual_norm(eo, perm, w, None, r[4], gamma, 1e-6, stream=s)],
        reduce_only=lambda s: [bn.reduce_only(part, stream=s)],
        finalize_reduce_only=lambda s: [bn.finalize_reduce_only(eo, perm, w, None, stream=s)],
        norm_only=lambda s: [bn.norm_only(sum_, r[5], gamma, gamma, 1e-6, stream=s)],
        residual_norm_only=lambda s: [bn.residual_norm_only(sum_, r[6], gamma, 1e-6, stream=s)],
        finalize_only=lambda s: [bn.finalize_only(eo, perm, w, None, stream=s)],
        route=lambda s: list(experts.route(logits, 2, stream=s)),
        route_backward=lambda s: [experts.route_backward(logits, ids, w[:1], stream=s)],
        plan=lambda s: list(experts.plan(ids, E, stream=s)),
        quantize_fp4=lambda s: (lambda q: [q.data, q.scales])(experts.quantize_fp4(x, "nvfp4", stream=s)),
        dequantize_fp4=lambda s: [experts.dequantize_fp4(a, stream=s)],
        expert_product=lambda s: [experts.expert_product(a, b, stream=s)])


@pytest.mark.parametrize("form", ["stream", "address"])
@pytest.mark.parametrize("name", ["reduce_norm", "finalize_reduce_norm", "finalize_reduce_norm_noalloc", "reduce_residual_norm",
                                  "finalize_reduce_residual_norm", "reduce_only", "finalize_reduce_only", "norm_only",
                                  "residual_norm_only", "finalize_only", "route", "route_backward", "plan", "quantize_fp4",
                                  "dequantize_fp4", "expert_product"])
def test_new_outputs_come_from_the_calls_stream(name, form):
    """A block of the current stream's pool may still be in use there when another stream writes it."""
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side if form == "stream" else side.cuda_stream)
    side.synchronize()
    for t in got:
        assert pool_of(t) == side.cuda_stream
    for t in call(torch.cuda.current_stream().cuda_stream) + call(0):
        assert pool_of(t) == torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    if not name.endswith("norm") and "norm_" not in name:  # the others change their residual
        for a, b in zip(got, want[:1] if name == "quantize_fp4" else want):  # scale places of no row are not written
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["reduce_only", "route"])
def test_new_outputs_are_not_the_current_streams_blocks(name):
    """The current stream is busy and has freed blocks that it will still write: outputs of a call on another
    stream keep their values."""
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.empty(1 << 28, dtype=torch.float32, device="cuda")
    for _ in range(20):  # some milliseconds
        busy.fill_(1.0)
    for t in want:  # freed at once, filled after that
        for _ in range(4):
            torch.empty_like(t).fill_(7)
    got = call(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_fallback_runs_on_an_address():
    """The unfused pieces of a declined shape run on the stream whose address is given, copies included."""
    R, T, H = 2, 2, 40960
    g = gen(71)
    part = torch.randn(R, T, H, generator=g).bfloat16().cuda()
    gamma = torch.ones(H, device="cuda")
    side = torch.cuda.Stream()
    outs = []
    for stream in (None, side.cuda_stream):
        res = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
        debug = bn.Debug(sum=torch.zeros(T, H, device="cuda"))
        torch.cuda.synchronize()
        if stream is not None:  # the current stream is busy: what went there would come late
            busy = torch.empty(1 << 28, dtype=torch.float32, device="cuda")
            for _ in range(20):
                busy.fill_(1.0)
        out = bn.reduce_norm(part, res, gamma, gamma, 1e-6, debug=debug, stream=stream, on_decline="fallback")
        (side if stream is not None else torch.cuda.current_stream()).synchronize()
        with torch.cuda.stream(side):
            outs.append((out.clone(), debug.sum.clone()))
        torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# ---- groups that are a part of a longer list ------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("first", [1, 50, 128, 300])
@pytest.mark.parametrize("counts,tail", [([3, 0, 130, 1], 5), ([0, 257], 0), ([0, 0], 40)])
@pytest.mark.parametrize("repeated", [False, True])
def test_rows_before_the_first_group(fmt, first, counts, tail, repeated):
    """Offsets that do not begin at 0, as one of several holders of the experts has them: its groups' rows are
    what they are without the rows before them, and those are zeros."""
    g = gen(first + tail)
    K, n = (608, 20) if repeated else (96, 40)
    scale = 40 if repeated else 1  # enough work that rows are quantised once into the workspace
    counts, tail = [c * scale for c in counts], tail * scale
    first += max(0, 29000 - sum(counts) - tail) if repeated else 0
    M, E, N = first + sum(counts) + tail, len(counts), 40
    offsets = (first + torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist())).to(torch.int32)
    x = torch.randn(n, K, generator=g).bfloat16().cuda()
    rows = torch.randint(0, n, (M,), generator=g).to(torch.int32).cuda()
    assert (experts.quantize_workspace_bytes(n, M, K, fmt) > 0) == repeated
    part = experts.quantize_fp4(x, fmt, rows=rows[first:], offsets=(offsets - first).cuda())
    shape = experts.fp4_scales_shape(M, K, fmt, E, True)
    got = []
    for work in (None, torch.empty(16, dtype=torch.uint8, device="cuda")):
        scales = torch.full(shape, 85, dtype=torch.uint8, device="cuda")
        q = experts.quantize_fp4(x, fmt, rows=rows, offsets=offsets.cuda(), scales=scales, workspace=work)
        assert torch.equal(q.data[first:], part.data)
        assert (scales[:first // 128] == 85).all()  # no row's places
        got.append(scales)
        v = experts.dequantize_fp4(q, dtype=torch.float32)
        assert (v[:first] == 0).all() and torch.equal(v[first:], experts.dequantize_fp4(part, dtype=torch.float32))
    assert torch.equal(got[0], got[1])
    w = experts.quantize_fp4((torch.randn(E, N, K, generator=g) / 8).bfloat16().cuda(), fmt)
    out = torch.full((M, N), math.nan, dtype=torch.bfloat16, device="cuda")
    experts.expert_product(q, w, out=out)
    assert bn.check_device_error() == 0
    assert (out[:first] == 0).all() and torch.equal(out[first:], experts.expert_product(part, w))
    assert (out[M - tail:] == 0).all()


def test_rows_before_the_first_group_on_pairs_of_ctas():
    """The same where the product runs on pairs of CTAs."""
    g = gen(81)
    first, counts, tail, N, K = 300, [900, 1300], 70, 2312, 96
    M = first + sum(counts) + tail
    offsets = torch.tensor([300, 1200, 2500], dtype=torch.int32, device="cuda")
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    w = experts.quantize_fp4((torch.randn(2, N, K, generator=g) / 8).bfloat16().cuda(), "nvfp4")
    out = torch.full((M, N), math.nan, dtype=torch.bfloat16, device="cuda")
    experts.expert_product(experts.quantize_fp4(x, "nvfp4", offsets=offsets), w, out=out)
    part = experts.expert_product(experts.quantize_fp4(x[first:], "nvfp4", offsets=offsets - first), w)
    assert bn.check_device_error() == 0
    assert (out[:first] == 0).all() and torch.equal(out[first:], part) and (out[2500:] == 0).all()
    experts.expert_product(experts.quantize_fp4(x, "nvfp4", offsets=offsets[:2]),
                           experts.FP4(w.data[:1], w.scales[:19], "nvfp4"), out=out.fill_(math.nan))
    assert bn.check_device_error() == 0
    assert (out[:first] == 0).all() and torch.equal(out[first:1200], part[:900]) and (out[1200:] == 0).all()
