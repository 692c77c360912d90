"""The operators around the experts on the GPU against their 64-bit definitions.

Tolerances.  Routing weights: a score is within 1.5 * 2^-22 (sigmoid: expf 2^-22, an addition, a
division) or 2^-18 + |x - max| 2^-24 (softmax: the sum of up to 1024 terms) of itself, and a
normalisation adds a sum of at most 16 terms and a division, 2^-21: under 2^-17 relative for the logits
here (|x - max| < 30).  Gradients: a sum of terms that may cancel, each as exact as that, so 2^-16 of the
row's largest |c s|, plus the rounding to the logits' type, eps / 2 of the value.  Quantised values are
exact.  Products: K additions in 32 bits, 2^-23 each of the sum of |a w|, and the rounding to BF16, 2^-8."""
import math

import pytest
import torch

from tests import experts_reference as ref
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


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---- routing ---------------------------------------------------------------------------------------

def check_route(logits, k, bias=None, shards=1, strided=False, **kw):
    T, E = logits.shape
    x = logits.cuda()
    if strided:  # rows of a wider, misaligned buffer
        wide = torch.full((T, E + 7), 1e4, dtype=logits.dtype, device="cuda")
        wide[:, 3:3 + E] = x
        x = wide[:, 3:3 + E]
    ids, w = experts.route(x, k, bias=None if bias is None else bias.cuda(), shards=shards, **kw)
    assert ids.shape == (T, k) and w.shape == (shards, T, k)
    rids, rw = ref.route(logits, k, bias=bias, **kw)
    assert torch.equal(ids.cpu(), rids), (ids.cpu()[(ids.cpu() != rids).any(1)], rids[(ids.cpu() != rids).any(1)])
    for r in range(shards):
        got = w[r].cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(rw))
        ok = ~torch.isnan(rw)
        assert ((got - rw).abs()[ok] <= 2.0 ** -17 * rw.abs()[ok] + 1e-37).all()
    return ids, w


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (5, 7, 7), (3, 33, 16), (67, 64, 2), (9, 100, 10), (6, 200, 8),
                                   (4, 513, 16), (3, 1024, 5), (130, 128, 6)])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route(dtype, T, E, k, score, renormalize):
    logits = (2 * torch.randn(T, E, generator=gen(T * E + k))).to(DTYPES[dtype])
    check_route(logits, k, score=score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,E,k,groups,top,gtop", [
    (40, 256, 8, 8, 4, 2), (17, 256, 8, 8, 3, 1), (9, 160, 6, 8, 3, 2), (11, 56, 5, 8, 5, 2), (5, 24, 4, 24, 7, 2),
    (6, 96, 8, 3, 2, 2), (3, 1024, 16, 32, 4, 2), (7, 60, 3, 4, 4, 2), (8, 512, 10, 2, 1, 1), (4, 40, 2, 1, 1, 1)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_groups(score, dtype, T, E, k, groups, top, gtop, biased):
    g = gen(E + k)
    logits = torch.randn(T, E, generator=g).to(DTYPES[dtype])
    bias = 0.1 * torch.randn(E, generator=g) if biased else None
    check_route(logits, k, bias=bias, score=score, groups=groups, top_groups=top, group_top=gtop, shards=3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route_strides(dtype):
    logits = torch.randn(21, 88, generator=gen(5)).to(DTYPES[dtype])
    check_route(logits, 6, score="sigmoid", bias=0.1 * torch.randn(88, generator=gen(6)), strided=True)
    check_route(logits, 6, strided=True)


@pytest.mark.parametrize("bias", [None, 0.0, 0.25])
@pytest.mark.parametrize("groups,top,gtop", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lowest_index(bias, groups, top, gtop, score):
    """Logits from four values only, all equal in one row, +0 beside -0 in another."""
    g = gen(3)
    logits = torch.randint(0, 4, (24, 64), generator=g).float()
    logits[3] = 1.0
    logits[4] = torch.where(torch.rand(64, generator=g) < 0.5, 0.0, -0.0)
    b = None if bias is None else torch.full((64,), bias)
    check_route(logits.bfloat16(), 8, bias=b, score=score, groups=groups, top_groups=top, group_top=gtop)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scores_closer_than_32_bits(score):
    """Biases that lift unequal scores to within a few 2^-30 of one another: the order is that of 64 bits."""
    g = gen(11)
    E, k = 96, 8
    x = torch.randn(64, E, generator=g)
    x[:] = x[0]
    s = ref.scores(x[0].double(), score)
    bias = (1.0 - s).float()  # s + bias = 1 up to the rounding of the bias, 2^-25
    check_route(x, k, bias=bias, score=score)
    check_route(x, k, bias=bias, score=score, groups=8, top_groups=3, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("levels", [1, 2, 3])
@pytest.mark.parametrize("E,groups,top,gtop", [(256, 8, 4, 2), (256, 8, 3, 1), (96, 3, 2, 2), (60, 4, 2, 2)])
def test_route_many_ties_in_groups(score, levels, E, groups, top, gtop):
    """Logits and biases of one to three values: groups whose best are many equal experts."""
    g = gen(E + levels)
    x = torch.randint(0, levels, (24, E), generator=g).float() / 2
    x[5, ::3] = -math.inf
    bias = torch.randint(0, levels, (E,), generator=g).float() / 8
    for b in (None, torch.zeros(E), bias):
        check_route(x, 8, bias=b, score=score, groups=groups, top_groups=top, group_top=gtop)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 2, 3])
def test_route_a_third_key_crosses_two_equal_ones(score, k):
    """Two experts of one logit and bias, and a third whose logit passes by them in steps of one unit in the
    last place: 2^-26 of its score at a step."""
    T = 1024
    x = torch.full((T, 40), -3.0)
    x[:, 17] = x[:, 30] = 0.25
    x[:, 35] = 0.7 + torch.arange(-T // 2, T // 2) * 2.0 ** -24
    s = ref.scores(x[T // 2].double(), score)
    bias = torch.zeros(40)
    bias[17] = bias[30] = float(s[35] - s[17])
    check_route(x, k, bias=bias, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("copies,masked", [(2, 0.0), (3, 0.0), (1, 0.8), (2, 0.6)])
@pytest.mark.parametrize("k,groups,top,gtop", [(1, 1, 1, 1), (5, 1, 1, 1), (8, 8, 3, 2), (6, 8, 2, 1), (3, 4, 1, 2), (8, 24, 8, 2)])
def test_route_equal_and_close_scores_at_the_border(score, copies, masked, k, groups, top, gtop):
    """Scores within 2^-25 of one another, each held by several experts: the k-th and the next may be equal and
    a third between them and the bound on 32-bit errors; groups of nearly equal rank with few experts left."""
    g = gen(100 * copies + k + groups)
    E = 96
    x = torch.randn(80, E // copies, generator=g).repeat_interleave(copies, 1)
    x[:] = x[0, :, ].clone()
    s = ref.scores(x[0].double(), score)
    bias = (1.0 - s).float()
    order = torch.stack([torch.randperm(E, generator=g) for _ in range(80)])
    for t in range(80):
        b, row = bias[order[t]], x[t][order[t]].clone()
        if masked:
            row[torch.rand(E, generator=g) < masked] = -math.inf
        if t % 4 == 0:  # one token a call, each with a bias of its own
            check_route(row[None], k, bias=b, score=score, groups=groups, top_groups=top, group_top=gtop)


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masked_rows(score, renormalize, biased, groups):
    """-inf takes experts out; fewer than k, one or none may be left; the type's lowest value is no mask."""
    g = gen(7)
    x = torch.randn(40, 64, generator=g)
    x[torch.rand(40, 64, generator=g) < 0.7] = -math.inf
    x[4] = -math.inf
    x[5] = -math.inf
    x[5, 13] = -3.0
    x[6, :60] = -math.inf
    x[7] = torch.finfo(torch.float32).min
    x[8] = torch.finfo(torch.float32).min
    x[8, 9] = 1.0
    bias = 0.1 * torch.randn(64, generator=g) if biased else None
    if biased:
        bias[11] = -math.inf
    check_route(x, 8, bias=bias, score=score, renormalize=renormalize, groups=groups, top_groups=min(groups, 2), group_top=2)


@pytest.mark.parametrize("biased", [False, True])
def test_route_nan_shows_in_the_weights(biased):
    x = torch.randn(6, 64, generator=gen(8))
    x[2, 5] = math.nan
    x[3] = math.nan
    x[4, ::2] = math.nan
    check_route(x, 40 % 16, bias=torch.zeros(64) if biased else None, score="sigmoid")


def test_route_large_logits():
    x = torch.tensor([[80.0, -80.0, 79.5, 0.0, 30.0, -200.0, 200.0, 100.0]])
    check_route(x, 4, score="sigmoid")
    check_route(x, 8, score="sigmoid", renormalize=False)
    ids, w = experts.route(x.cuda(), 3)
    assert ids.tolist() == [[6, 7, 0]]
    assert w[0, 0, 0].item() == 1.0


def test_route_no_tokens_and_streams():
    ids, w = experts.route(torch.empty(0, 64, device="cuda"), 4, shards=2)
    assert ids.shape == (0, 4) and w.shape == (2, 0, 4)
    x = torch.randn(50, 64, generator=gen(9))
    side = torch.cuda.Stream()
    xc = x.cuda()
    torch.cuda.synchronize()
    ids, w = experts.route(xc, 4, stream=side)
    dw = torch.ones(1, 50, 4, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(ids.cpu(), ref.route(x, 4)[0])
    with torch.cuda.stream(side):
        d = experts.route_backward(xc, ids, dw)
    side.synchronize()
    assert d.abs().max().item() < 2.0 ** -16  # a constant gradient of normalised weights is none


# ---- its gradient ------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,k,shards", [(1, 256, 8, 1), (5, 7, 7, 2), (3, 33, 16, 1), (70, 64, 2, 8), (4, 1000, 10, 3), (9, 100, 1, 1),
                                          (2, 1, 1, 1), (6, 512, 4, 16)])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_backward(dtype, T, E, k, shards, score, renormalize):
    g = gen(T + E)
    x = (2 * torch.randn(T, E, generator=g)).to(DTYPES[dtype])
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    if k > 2:
        ids[0, 1] = -1
    if T > 2:
        ids[2] = -1  # a token without experts
    dw = torch.randn(shards, T, k, generator=g)
    x64 = x.double().requires_grad_()
    on = (ids >= 0).any(1)
    (ref.route_weights(x64, ids, score, renormalize, 2.5)[on] * dw.double().sum(0)[on]).sum().backward()
    want = torch.nan_to_num(x64.grad) * on[:, None]
    got = experts.route_backward(x.cuda(), ids.cuda(), dw.cuda(), score=score, renormalize=renormalize, scale=2.5).cpu().double()
    assert got.shape == (T, E)
    s = ref.scores(x.double(), score)
    largest = 2.5 * dw.double().abs().sum(0).amax(-1, keepdim=True) * (1.0 if renormalize else s.amax(-1, keepdim=True))
    tol = 2.0 ** -16 * largest + torch.finfo(DTYPES[dtype]).eps / 2 * want.abs() + (2.0 ** -25 if dtype == "fp16" else 0)
    assert ((got - want).abs() <= tol).all()
    dead = torch.ones(T, E, dtype=torch.bool)
    if renormalize or score == "sigmoid":  # no gradient but at the chosen experts
        for t in range(T):
            dead[t, ids[t][ids[t] >= 0].long()] = False
        assert (got[dead] == 0).all()


def test_route_backward_strides_and_bad_ids():
    g = gen(2)
    x = torch.randn(10, 40, generator=g)
    wide = torch.zeros(10, 50, device="cuda")
    wide[:, 5:45] = x.cuda()
    ids, _ = experts.route(x.cuda(), 4)
    dw = torch.randn(1, 10, 4, generator=g).cuda()
    a = experts.route_backward(x.cuda(), ids, dw)
    b = experts.route_backward(wide[:, 5:45], ids, dw)
    assert torch.equal(a, b)
    ids2 = ids.clone()
    ids2[3, 1] = 40
    ids2[4, 0] = -7
    c = experts.route_backward(x.cuda(), ids2, dw)
    assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_EXPERT_RANGE
    ids2[3, 1] = -1
    ids2[4, 0] = -1
    assert torch.equal(c, experts.route_backward(x.cuda(), ids2, dw))


def test_route_backward_saturated_and_masked():
    """Sigmoids near 1 keep their slope; a softmax row with masked logits has no gradient there."""
    x = torch.tensor([[20.0, 15.0, -30.0, 0.0]])
    ids = torch.tensor([[0, 1]], dtype=torch.int32)
    dw = torch.ones(1, 1, 2)
    got = experts.route_backward(x.cuda(), ids.cuda(), dw.cuda(), score="sigmoid", renormalize=False).cpu().double()
    s = torch.sigmoid(x.double()) * torch.sigmoid(-x.double())
    assert (got[0, :2] - s[0, :2]).abs().max() <= 2.0 ** -20 * s[0, 1] and (got[0, 2:] == 0).all()
    x = torch.tensor([[1.0, -math.inf, 0.5, -math.inf], [-math.inf] * 4])
    ids = torch.tensor([[0, 2], [-1, -1]], dtype=torch.int32)
    dw = torch.tensor([[[1.0, -1.0], [1.0, 1.0]]])
    for renorm in (True, False):
        got = experts.route_backward(x.cuda(), ids.cuda(), dw.cuda(), renormalize=renorm).cpu()
        assert torch.isfinite(got).all() and (got[1] == 0).all() and got[0, 1] == 0 and got[0, 3] == 0 and got[0, 0] > 0


# ---- the plan ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,E,shards", [(0, 8, 16, 2), (1, 1, 1, 1), (1, 10, 256, 8), (33, 16, 40, 1), (61, 10, 256, 4), (200, 3, 1024, 2),
                                          (700, 8, 7, 1), (1500, 8, 256, 1), (5000, 6, 512, 1), (9000, 4, 3, 1)])
@pytest.mark.parametrize("dropped", [0.0, 0.2])
def test_plan(T, k, E, shards, dropped):
    g = gen(T + E)
    ids = torch.randint(0, E, (T, k), generator=g).to(torch.int32)
    ids[torch.rand(T, k, generator=g) < dropped] = -1
    p = experts.plan(ids.cuda(), E, shards=shards)
    flat = torch.where(ids.reshape(-1) < 0, E, ids.reshape(-1).long())
    order = torch.sort(flat, stable=True).indices
    perm = torch.empty(T * k, dtype=torch.long)
    perm[order] = torch.arange(T * k)
    counts = torch.bincount(flat, minlength=E + 1)
    offsets = torch.cat((torch.zeros(1, dtype=torch.long), counts[:E].cumsum(0)))
    assert torch.equal(p.offsets.cpu().long(), offsets)
    assert torch.equal(p.rows.cpu().long(), order // k)
    assert p.perm.shape == (shards, T, k)
    for r in range(shards):
        assert torch.equal(p.perm[r].cpu().long().reshape(-1), perm)
    if T * k <= 700:
        want = ref.plan(ids, E)
        assert torch.equal(p.perm[0].cpu(), want[0]) and torch.equal(p.offsets.cpu(), want[1]) and torch.equal(p.rows.cpu(), want[2])


def test_plan_many_slots_one_expert():
    ids = torch.full((40000, 8), 5, dtype=torch.int32)
    ids[::3, 0] = 2
    p = experts.plan(ids.cuda(), 9)
    n = int((ids == 2).sum())
    assert p.offsets.tolist() == [0, 0, 0, n, n, n, 320000, 320000, 320000, 320000]
    assert torch.equal(torch.sort(p.perm.reshape(-1)).values.cpu(), torch.arange(320000, dtype=torch.int32))


def test_plan_takes_bad_ids_as_none():
    ids = torch.tensor([[0, 9], [-5, 1]], dtype=torch.int32)
    p = experts.plan(ids.cuda(), 4)
    assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_EXPERT_RANGE
    assert p.offsets.tolist() == [0, 1, 2, 2, 2] and p.perm.tolist() == [[[0, 2], [3, 1]]]


# What 1 becomes in a block of ones: 6 times the e4m3 value next to 1/6 (11/64), or 4 times a quarter.
ONE = {"nvfp4": 6 * 11 / 64, "mxfp4": 1.0}


# ---- 4-bit quantisation --------------------------------------------------------------------------------

def values(M, K, dtype, seed):
    """Rows over many scales, with zero blocks, ties and the type's extremes."""
    g = gen(seed)
    x = torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-6, 7, (M, 1), generator=g).float())
    x[0, :32] = 0.0
    x[0, 32:64] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0] * 2)[:K - 32][:32] \
        if K >= 64 else 1.0
    if M > 1:
        x[1] = torch.randint(-12, 13, (K,), generator=g).float() / 4
    if M > 2:
        x[2] = torch.finfo(dtype).tiny * torch.randint(-9, 10, (K,), generator=g).float() / 8
    if M > 3:
        x[3] = torch.finfo(dtype).max * torch.rand(K, generator=g)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,K", [(1, 32), (4, 64), (5, 96), (130, 160), (3, 1024), (33, 544), (7, 8192)])
@pytest.mark.parametrize("tensor_scale", [1.0, 0.0078125])
def test_quantize(dtype, fmt, M, K, tensor_scale):
    x = values(M, K, DTYPES[dtype], M + K)
    if dtype == "bf16" and tensor_scale < 1 and M > 3:
        x[3] /= 256  # dividing by the tensor scale stays within 32 bits
    q = experts.quantize_fp4(x.cuda(), fmt, tensor_scale=tensor_scale)
    codes, scale = ref.encode(x, fmt, tensor_scale)
    got = q.data.cpu()
    got = torch.stack((got & 15, got >> 4), -1).view(M, K).long()
    dead = torch.isnan(scale).repeat_interleave(ref.BLOCK[fmt], 1) | (scale == 0).repeat_interleave(ref.BLOCK[fmt], 1)
    assert torch.equal(got[~dead] & 7, codes[~dead] & 7)
    live = ~dead & (codes & 7 != 0)
    assert torch.equal(got[live], codes[live])
    want = (ref.LEVELS[codes & 7] * torch.where(codes >= 8, -1.0, 1.0)).view(M, -1, ref.BLOCK[fmt]) * (scale * tensor_scale)[..., None]
    assert torch.equal(ref.decode(q.data, q.scales, fmt, tensor_scale), want.view(M, K))
    back = experts.dequantize_fp4(q, dtype=torch.float32)
    assert torch.equal(back.cpu().double(), want.view(M, K).float().double())
    b16 = experts.dequantize_fp4(q)
    assert torch.equal(b16.cpu(), want.view(M, K).float().bfloat16())
    h16 = experts.dequantize_fp4(q, dtype=torch.float16)
    assert torch.equal(h16.cpu(), want.view(M, K).float().half())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantize_scales_past_a_row_are_zero(fmt):
    scales = torch.full(experts.fp4_scales_shape(5, 32, fmt), 255, dtype=torch.uint8, device="cuda")
    experts.quantize_fp4(torch.ones(5, 32, dtype=torch.bfloat16, device="cuda"), fmt, scales=scales)
    t = scales.cpu().view(32, 4, 4)
    used = 32 // ref.BLOCK[fmt]
    assert (t[:5, 0, used:] == 0).all() and (t[:5, 0, :used] != 255).all()
    assert (t[5:] == 255).all() and (t[:, 1:] == 255).all()  # places of no row are not written


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantize_infinity_and_nan_spoil_their_block_only(fmt):
    x = torch.ones(3, 128, dtype=torch.bfloat16)
    x[0, 5] = math.inf
    x[1, 100] = math.nan
    x[2, 70] = -math.inf
    q = experts.quantize_fp4(x.cuda(), fmt)
    v = experts.dequantize_fp4(q).cpu()
    B = ref.BLOCK[fmt]
    for r, c in ((0, 5), (1, 100), (2, 70)):
        bad = torch.zeros(128, dtype=torch.bool)
        bad[c // B * B:c // B * B + B] = True
        assert torch.isnan(v[r][bad]).all() and (v[r][~bad] == ONE[fmt]).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("counts,tail", [([3, 0, 130, 1, 0, 257], 5), ([0, 0, 1], 0), ([128, 128], 0), ([0, 0], 3), ([127, 129, 0], 200)])
def test_quantize_grouped_rows(fmt, counts, tail):
    g = gen(sum(counts))
    M, K = sum(counts) + tail, 96
    offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32)
    x = torch.randn(11, K, generator=g).bfloat16()
    wide = torch.zeros(11, K + 24, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + K] = x.cuda()
    rows = torch.randint(0, 11, (M,), generator=g).to(torch.int32)
    q = experts.quantize_fp4(wide[:, 8:8 + K], fmt, rows=rows.cuda(), offsets=offsets.cuda())
    plain = experts.quantize_fp4(x.cuda(), fmt)
    want = ref.decode(plain.data, plain.scales, fmt)[rows.long()]
    assert torch.equal(ref.decode(q.data, q.scales, fmt, offsets=offsets), want)
    assert torch.equal(experts.dequantize_fp4(q).cpu().double(), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("K", [544, 2048])
def test_quantize_repeated_rows_through_the_workspace(fmt, dtype, K):
    """Places that take a row many times: the same bytes with the workspace and without."""
    g = gen(K)
    n, M = 300, 31000
    x = torch.randn(n, K, generator=g).to(DTYPES[dtype]).cuda()
    rows = torch.randint(0, n, (M,), generator=g).to(torch.int32)
    rows[17] = -3
    rows[M - 1] = n
    counts = torch.randint(0, 2 * M // 50, (50,), generator=g)
    offsets = torch.cat((torch.zeros(1, dtype=torch.long), counts.cumsum(0))).clamp_max(M - 5).to(torch.int32)
    need = experts.quantize_workspace_bytes(n, M, K, fmt)
    assert (need > 0) == (M * K >= 1 << 24)
    shape = experts.fp4_scales_shape(M, K, fmt, 50, True)
    got = []
    for work in (None, torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"), torch.empty(16, dtype=torch.uint8, device="cuda")):
        scales = torch.full(shape, 85, dtype=torch.uint8, device="cuda")
        q = experts.quantize_fp4(x, fmt, rows=rows.cuda(), offsets=offsets.cuda(), scales=scales, workspace=work)
        assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_PERM_RANGE
        got.append((q.data.clone(), scales))
    for data, scales in got[1:]:
        assert torch.equal(data, got[0][0]) and torch.equal(scales, got[0][1])
    plain = experts.quantize_fp4(x, fmt)
    want = experts.dequantize_fp4(plain)[rows.long().where((rows >= 0) & (rows < n), torch.zeros(1, dtype=torch.long)).cuda()]
    assert torch.equal(experts.dequantize_fp4(experts.FP4(got[0][0], got[0][1], fmt, offsets.cuda())), want)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantize_weights_and_bad_rows(fmt):
    w = torch.randn(3, 136, 64, generator=gen(1)).bfloat16().cuda()
    q = experts.quantize_fp4(w, fmt)
    assert q.shape == (3, 136, 64)
    flat = experts.quantize_fp4(w.view(-1, 64), fmt)
    want = ref.decode(flat.data, flat.scales, fmt)
    assert torch.equal(ref.decode(q.data, q.scales, fmt, groups=3), want)
    assert torch.equal(experts.dequantize_fp4(q).cpu().double().view(-1, 64), want)
    rows = torch.tensor([1, 408, -1], dtype=torch.int32, device="cuda")
    b = experts.quantize_fp4(w.view(-1, 64), fmt, rows=rows)
    assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_PERM_RANGE
    assert torch.equal(ref.decode(b.data, b.scales, fmt), want[[1, 0, 0]])
    assert experts.dequantize_fp4(experts.quantize_fp4(w.view(-1, 64)[:0], fmt)).shape == (0, 64)


# ---- the experts' product --------------------------------------------------------------------------------

def check_product(counts, tail, N, K, fmt, seed=0, tensor_scale=1.0, offsets=None):
    g = gen(seed + N + K)
    E, M = len(counts), sum(counts) + tail
    if offsets is None:
        offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32)
    x = torch.randn(M, K, generator=g).bfloat16()
    w = (torch.randn(E, N, K, generator=g) / 8).bfloat16()
    a = experts.quantize_fp4(x.cuda(), fmt, offsets=offsets.cuda())
    b = experts.quantize_fp4(w.cuda(), fmt, tensor_scale=tensor_scale)
    out = torch.full((M, N), math.nan, dtype=torch.bfloat16, device="cuda")
    assert experts.expert_product(a, b, scale=0.5, out=out) is out
    assert bn.check_device_error() == 0
    av = experts.dequantize_fp4(a, dtype=torch.float32).cpu().double()
    wv = experts.dequantize_fp4(b, dtype=torch.float32).cpu().double()
    want, size = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    o = offsets.tolist()
    for e in range(E):
        want[o[e]:o[e + 1]] = 0.5 * av[o[e]:o[e + 1]] @ wv[e].T
        size[o[e]:o[e + 1]] = 0.5 * av[o[e]:o[e + 1]].abs() @ wv[e].abs().T
    got = out.cpu().double()
    err = (got - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + K * 2.0 ** -23 * size).all(), float((err / size.clamp_min(1e-30)).max())
    assert (got[o[E]:] == 0).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("counts,tail,N,K", [
    ([1], 0, 128, 256), ([128], 0, 128, 64), ([16], 0, 128, 32), ([128], 0, 128, 256), ([128], 0, 128, 512),
    ([5, 0, 17], 0, 256, 96), ([1, 1, 1, 1], 2, 8, 160), ([33, 64, 0, 129], 0, 136, 288), ([200, 300], 100, 264, 1056),
    ([0, 0], 3, 64, 64), ([2, 0, 1, 0, 0, 7, 0, 1], 0, 512, 2048), ([700], 0, 384, 2304)])
def test_product(fmt, counts, tail, N, K):
    check_product(counts, tail, N, K, fmt, tensor_scale=0.015625)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("counts,tail,N,K", [
    # where tiles of one CTA take more than one round over the device, pairs of CTAs run: 256 features by
    # 256 rows, in halves
    ([129], 0, 136, 64), ([256, 257, 255], 0, 256, 288), ([1, 600, 0, 31, 513], 0, 392, 1312), ([0, 1000], 40, 904, 160),
    ([383, 385, 128], 0, 2056, 96), ([2500, 3], 0, 264, 512), ([700], 0, 4360, 160), ([0, 1300, 31, 257], 50, 2312, 96),
    ([33] * 40 + [900, 0, 513], 0, 1544, 288), ([2100, 1], 7, 1288, 1312),
    ([300, 0, 511, 257, 1, 256, 129, 385], 30, 2056, 352)])
def test_product_of_large_groups(fmt, counts, tail, N, K):
    check_product(counts, tail, N, K, fmt, seed=3)


@pytest.mark.parametrize("rows", [4, 300])
def test_product_on_another_stream(rows):
    """Operands made on the current stream, the product on a side stream that waits for it."""
    a = experts.quantize_fp4(torch.ones(rows, 256, dtype=torch.bfloat16, device="cuda"), "mxfp4")
    b = experts.quantize_fp4(torch.ones(264, 256, dtype=torch.bfloat16, device="cuda"), "mxfp4")
    out = torch.zeros(rows, 264, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    experts.expert_product(a, b, out=out, stream=side)
    side.synchronize()
    assert (out == 256).all()


def test_product_no_rows_and_binding_refusals():
    b = experts.quantize_fp4(torch.ones(2, 16, 64, dtype=torch.bfloat16, device="cuda"), "nvfp4")
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    none = experts.quantize_fp4(torch.ones(0, 64, dtype=torch.bfloat16, device="cuda"), "nvfp4", offsets=offsets)
    assert experts.expert_product(none, b).shape == (0, 16)
    a = experts.quantize_fp4(torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), "nvfp4", offsets=offsets)
    assert (experts.expert_product(a, b) == 0).all()  # rows of no group
    one = experts.quantize_fp4(torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), "nvfp4")
    with pytest.raises(ValueError, match="1 groups, w has 2 experts"):
        experts.expert_product(one, b)
    with pytest.raises(ValueError, match="no offsets"):
        experts.expert_product(a, a)
    mx = experts.quantize_fp4(torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), "mxfp4", offsets=offsets)
    with pytest.raises(ValueError, match="mxfp4 values"):
        experts.expert_product(mx, b)
    with pytest.raises(ValueError, match="shape"):
        experts.expert_product(a, b, out=torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda"))
    x = torch.randn(4, 64, device="cuda")
    with pytest.raises(TypeError, match="bfloat16"):
        experts.quantize_fp4(x, "nvfp4")
    with pytest.raises(ValueError, match="contiguous rows"):
        experts.route(x.T, 2)
    with pytest.raises(ValueError, match="do not overlap"):
        experts.route(x.as_strided((4, 64), (32, 1)), 2)
    with pytest.raises(TypeError, match="bias must be"):
        experts.route(x, 2, bias=torch.zeros(64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(bn.BeamNormError, match="k=17"):
        experts.route(x, 17)
    with pytest.raises(ValueError, match="multiple of 32"):
        experts.quantize_fp4(torch.ones(4, 40, dtype=torch.bfloat16, device="cuda"), "nvfp4")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_product_many_experts_and_tiles(fmt):
    g = gen(4)
    counts = torch.randint(0, 40, (150,), generator=g).tolist()
    check_product(counts, 0, 520, 320, fmt)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_product_of_one_matrix_needs_no_offsets(fmt):
    g = gen(12)
    x, w = torch.randn(45, 192, generator=g).bfloat16().cuda(), torch.randn(72, 192, generator=g).bfloat16().cuda()
    a, b = experts.quantize_fp4(x, fmt), experts.quantize_fp4(w, fmt)
    out = experts.expert_product(a, b).cpu().double()
    av, wv = (experts.dequantize_fp4(q, dtype=torch.float32).cpu().double() for q in (a, b))
    assert ((out - av @ wv.T).abs() <= 2.0 ** -8 * (av @ wv.T).abs() + 192 * 2.0 ** -23 * (av.abs() @ wv.abs().T)).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_product_nan_stays_in_its_row(fmt):
    x = torch.ones(20, 128, dtype=torch.bfloat16)
    x[7, 3] = math.nan
    a = experts.quantize_fp4(x.cuda(), fmt)
    b = experts.quantize_fp4(torch.ones(128, 128, dtype=torch.bfloat16, device="cuda"), fmt)
    out = experts.expert_product(a, b).cpu()
    assert torch.isnan(out[7]).all()
    out[7] = 128 * ONE[fmt] ** 2
    assert (out == torch.tensor(128 * ONE[fmt] ** 2).bfloat16()).all()


def test_product_bad_offsets_are_reported():
    a = experts.quantize_fp4(torch.ones(10, 64, dtype=torch.bfloat16, device="cuda"), "nvfp4",
                             offsets=torch.tensor([0, 4, 10], dtype=torch.int32, device="cuda"))
    b = experts.quantize_fp4(torch.ones(2, 16, 64, dtype=torch.bfloat16, device="cuda"), "nvfp4")
    a.offsets = torch.tensor([0, 12, 10], dtype=torch.int32, device="cuda")
    experts.expert_product(a, b)
    assert bn.check_device_error(raise_on_error=False) == bn.DEVERR_OFFSETS


def test_offsets_past_32_bits():
    """Logits, codes, values and products whose last elements lie past 2^31 elements or bytes."""
    g = gen(30)
    T, ld, E = 520, 1 << 22, 64
    x = torch.randn(T, E, generator=g)
    far = torch.empty((T - 1) * ld + E, dtype=torch.bfloat16, device="cuda").as_strided((T, E), (ld, 1))
    far.copy_(x)
    ids, w = experts.route(far, 4)
    near = experts.route(x.bfloat16().cuda(), 4)
    assert torch.equal(ids, near[0]) and torch.equal(w, near[1])
    dw = torch.randn(1, T, 4, generator=g).cuda()
    assert torch.equal(experts.route_backward(far, ids, dw), experts.route_backward(x.bfloat16().cuda(), ids, dw))
    del far
    n, M, K = 9, 140000, 32768  # 2.3 GB of codes, 9.2 GB of values
    x = torch.randn(n, K, generator=g).bfloat16().cuda()
    rows = torch.randint(0, n, (M,), generator=g).to(torch.int32).cuda()
    offsets = torch.tensor([0, 70001, M], dtype=torch.int32, device="cuda")
    small = experts.dequantize_fp4(experts.quantize_fp4(x, "mxfp4"))
    for work in (None, torch.empty(16, dtype=torch.uint8, device="cuda")):
        q = experts.quantize_fp4(x, "mxfp4", rows=rows, offsets=offsets, workspace=work)
        v = experts.dequantize_fp4(q)
        for lo in (0, 65536, 70000, 131072, M - 100):
            assert torch.equal(v[lo:lo + 100], small[rows[lo:lo + 100].long()])
        del q, v
    M, N, K = 300000, 8192, 64  # 2.5 G products
    x = torch.randn(n, K, generator=g).bfloat16().cuda()
    rows = torch.randint(0, n, (M,), generator=g).to(torch.int32).cuda()
    b = experts.quantize_fp4(torch.randn(N, K, generator=g).bfloat16().cuda(), "nvfp4")
    want = experts.expert_product(experts.quantize_fp4(x, "nvfp4"), b)
    got = experts.expert_product(experts.quantize_fp4(x, "nvfp4", rows=rows), b)
    for lo in (0, 131072, 262100, M - 100):
        assert torch.equal(got[lo:lo + 100], want[rows[lo:lo + 100].long()])


def test_layer_in_a_graph_matches_eager():
    """Route, plan, quantise, product and finalize, captured once and replayed on new inputs."""
    g = gen(20)
    T, E, k, H, K = 24, 16, 4, 256, 128
    w = (torch.randn(E, H, K, generator=g) / 8).bfloat16().cuda()
    wq = experts.quantize_fp4(w, "mxfp4")
    logits, x = torch.randn(T, E, generator=g).cuda(), torch.randn(T, K, generator=g).bfloat16().cuda()
    gamma = torch.ones(H, device="cuda")
    res0 = torch.randn(T, H, generator=g).bfloat16().cuda()

    def layer(res):
        ids, wt = experts.route(logits, k, score="sigmoid")
        p = experts.plan(ids, E)
        q = experts.quantize_fp4(x, "mxfp4", rows=p.rows, offsets=p.offsets)
        y = experts.expert_product(q, wq)
        return bn.finalize_reduce_norm(y[None], p.perm, wt, None, res, gamma, gamma, 1e-6)

    res = res0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(res)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(res)
    for seed in (1, 2):
        logits.copy_(torch.randn(T, E, generator=gen(seed)))
        x.copy_(torch.randn(T, K, generator=gen(seed + 50)).bfloat16())
        res.copy_(res0)
        graph.replay()
        torch.cuda.synchronize()
        got, got_res = out.clone(), res.clone()
        eager_res = res0.clone()
        eager = layer(eager_res)
        assert torch.equal(got, eager) and torch.equal(got_res, eager_res)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_example_layer(fmt):
    """The example's layer against 32-bit activations: rounding a value to 4 bits moves it by at most a
    quarter (half the step from 1 to 1.5), about a tenth in the mean square; two roundings in a row and
    the residual, which is as large as the normed sum and exact, leave under a quarter."""
    from examples import moe_layer
    assert moe_layer.main(["--format", fmt, "--tokens", "37", "--hidden", "512", "--width", "256"]) < 0.25
    assert moe_layer.main(["--format", fmt, "--tokens", "3", "--hidden", "256", "--width", "128", "--shards", "1", "--experts", "6",
                           "--topk", "2"]) < 0.25
