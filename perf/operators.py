"""The operators around the experts of a mixture-of-experts layer, as measured: routing and its
gradient, the plan that groups token slots by expert, 4-bit microscaled quantisation, and the experts'
product of 4-bit operands.

``listed()`` are the cases, ``prepare`` makes one case's tensors from a seed, ``run`` is one pass: with
``own`` the framework's kernels, else elementary torch operations in 32 bits (64 bits where a choice
between nearly equal scores is made).  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    """H and k are those of the finalize workloads (H = 5120, 6144, 8192; k = 8, 10; 256 experts); 2048 is
    the width of one expert's hidden layer."""
    return [
        # one decoded token: 256 experts in 8 groups, sigmoid scores with a balance bias, weights for 8 shards
        dict(name="route one token", op="route", T=1, E=256, k=8, dtype="bf16", score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5, shards=8, masked=0.0),
        # a decode batch whose requests may only use some experts: softmax over an odd expert count, some rows empty
        dict(name="route masked batch", op="route", T=333, E=200, k=10, dtype="fp32", score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0, shards=1, masked=0.5),
        # a long prompt through the first case's router
        dict(name="route prompt", op="route", T=16384, E=256, k=8, dtype="bf16", score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5, shards=1, masked=0.0),
        # training, one sequence: normalised sigmoid weights that 8 shards used
        dict(name="route grad sigmoid", op="route_grad", T=4096, E=256, k=8, dtype="bf16", score="sigmoid",
             renorm=True, scale=2.5, shards=8, masked=0.0),
        # training, a larger batch: plain softmax weights, a dense gradient
        dict(name="route grad softmax", op="route_grad", T=16384, E=128, k=10, dtype="fp32", score="softmax",
             renorm=False, scale=1.0, shards=1, masked=0.0),
        # a decode batch's slots grouped by expert, for 8 shards
        dict(name="plan decode", op="plan", T=61, E=256, k=10, shards=8, masked=0.05),
        # a long prompt's slots
        dict(name="plan prompt", op="plan", T=16384, E=256, k=8, shards=1, masked=0.0),
        # a few tokens' rows repeated for their experts, scales of 16 values
        dict(name="quantize decode", op="quantize", T=5, E=256, k=10, H=8192, dtype="bf16", format="nvfp4", tensor_scale=0.0078125),
        # a prompt's rows, scales of 32 values
        dict(name="quantize prompt", op="quantize", T=4096, E=256, k=8, H=5120, dtype="bf16", format="mxfp4", tensor_scale=1.0),
        # one decoded token through 10 experts: a stream of weights
        dict(name="product one token", op="product", T=1, E=256, k=10, N=8192, K=2048, format="nvfp4"),
        # a decode batch that reaches nearly every expert with a few rows each
        dict(name="product decode batch", op="product", T=100, E=256, k=8, N=6144, K=2048, format="mxfp4"),
        # a prompt: large ragged groups
        dict(name="product prompt", op="product", T=4096, E=64, k=8, N=4096, K=5120, format="nvfp4"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("route", "route", "route_grad", "plan", "quantize", "product", "product"))
    k = rng.choice((1, 2, 4, 6, 8, 10, 16))
    T = _log_int(rng, 1, 16384)
    if op in ("route", "route_grad"):
        score = rng.choice(("softmax", "sigmoid"))
        c = dict(op=op, T=T, k=k, dtype=rng.choice(("bf16", "fp16", "fp32")), score=score, renorm=rng.random() < 0.6,
                 scale=rng.choice((1.0, 2.5)), shards=rng.choice((1, 1, 4, 8)), masked=rng.choice((0.0, 0.0, 0.4)))
        if op == "route_grad":
            c["E"] = _log_int(rng, k, 512 if T <= 4096 else 256)
            return c
        groups = rng.choice((1, 1, 4, 8))
        if groups == 1:
            c |= dict(E=_log_int(rng, k, 512 if T <= 4096 else 256), groups=1, top_groups=1, group_top=1)
        else:
            top = rng.randint(1, groups)
            c |= dict(E=groups * rng.randint(max(2, -(-k // top)), 32), groups=groups, top_groups=top, group_top=rng.choice((1, 2)))
        c["bias"] = rng.random() < 0.5
        return c
    if op == "plan":
        return dict(op=op, T=T, E=_log_int(rng, k, 512), k=k, shards=rng.choice((1, 4, 8)), masked=rng.choice((0.0, 0.1)))
    if op == "quantize":
        T = _log_int(rng, 1, 4096)
        k = min(k, 8) if T > 2048 else k
        H = 32 * _log_int(rng, 1, 256 if T * k <= 16384 else 128)
        return dict(op=op, T=T, E=_log_int(rng, k, 256), k=k, H=H, dtype=rng.choice(("bf16", "fp16")),
                    format=rng.choice(("nvfp4", "mxfp4")), tensor_scale=rng.choice((1.0, 0.0078125)))
    T = _log_int(rng, 1, 2048)
    k = min(k, 8)
    while True:
        N, K = 8 * _log_int(rng, 16, 512), 32 * _log_int(rng, 4, 256)
        if 3072 not in (N, K, K // 2):
            return dict(op=op, T=T, E=rng.choice((8, 16, 32, 64)), k=k, N=N, K=K, format=rng.choice(("nvfp4", "mxfp4")))


def work(case):
    c = case
    T, E, k = c["T"], c["E"], c["k"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}.get(c.get("dtype"), 2)
    if c["op"] == "route":     # the logits and the bias in, the ids and every shard's weights out; a score is about 8 operations
        return {"bytes": T * E * size + 4 * E * c["bias"] + 4 * T * k * (1 + c["shards"]), "flops": 8 * T * E}
    if c["op"] == "route_grad":  # sigmoid and renormalised softmax need the chosen logits alone; the gradient is written whole
        need = T * E if c["score"] == "softmax" and not c["renorm"] else T * k
        return {"bytes": need * size + 4 * T * k * (1 + c["shards"]) + T * E * size, "flops": 8 * need + 2 * c["shards"] * T * k}
    if c["op"] == "plan":
        return {"bytes": 4 * T * k * (2 + c["shards"]) + 4 * (E + 1), "flops": T * k}
    if c["op"] == "quantize":  # tokens in, codes and scales out and in again, the values that they stand for out
        M, H = T * k, c["H"]
        q = M * H // 2 + M * H // BLOCK[c["format"]]
        return {"bytes": T * H * size + 4 * M + 4 * (E + 1) + 2 * q + M * H * 2, "flops": 6 * M * H}
    M, N, K = T * k, c["N"], c["K"]
    active = E * (1 - (1 - k / E) ** T)  # experts that T tokens reach when each takes k of E
    byte = 0.5 + 1 / BLOCK[c["format"]]
    return {"bytes": int(active * N * K * byte + M * K * byte + 2 * M * N + 4 * (E + 1)), "flops": 2 * M * N * K}


# ---- inputs --------------------------------------------------------------------------------------

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = {"nvfp4": 16, "mxfp4": 32}   # values that share a scale
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _ids(g, T, E, k):
    """Each token's k experts: some experts are more popular than others."""
    u = torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
    return u.topk(k, dim=1).indices.to(torch.int32)


def _grouped(ids, E):
    """offsets [E+1] and the token of every slot, slots in the order of their experts."""
    order = torch.sort(ids.reshape(-1), stable=True).indices
    counts = torch.bincount(ids.reshape(-1), minlength=E)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return offsets, (order // ids.shape[1]).to(torch.int32), int(counts.max())


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    T, E, k = c["T"], c["E"], c["k"]
    state = {"case": c}
    if c["op"] in ("route", "route_grad"):
        logits = torch.randn(T, E, generator=g, device=DEV)
        if c["masked"]:  # a token may use some experts only; every 16th none at all
            off = torch.rand(T, E, generator=g, device=DEV) < c["masked"]
            off[5::16] = True
            logits = logits.masked_fill(off, -math.inf)
        state["logits"] = logits.to(DTYPES[c["dtype"]])
        if c["op"] == "route":
            state["bias"] = 0.05 * torch.randn(E, generator=g, device=DEV) if c["bias"] else None
        else:
            ids = state["logits"].float().topk(k, dim=1)
            state["ids"] = torch.where(ids.values > -math.inf, ids.indices, -1).to(torch.int32)
            state["dw"] = torch.randn(c["shards"], T, k, generator=g, device=DEV)
        return state
    ids = _ids(g, T, E, k)
    if c["op"] == "plan":
        if c["masked"]:  # padding tokens have no experts
            ids[torch.rand(T, generator=g, device=DEV) < c["masked"]] = -1
        return state | {"ids": ids}
    offsets, rows, most = _grouped(ids, E)
    state["offsets"], state["most"] = offsets, most
    if c["op"] == "quantize":  # normed activations: some channels are far larger than the rest
        channel = torch.exp(torch.randn(c["H"], generator=g, device=DEV))
        x = (torch.randn(T, c["H"], generator=g, device=DEV) * channel).to(DTYPES[c["dtype"]])
        return state | {"x": x, "rows": rows}
    M, N, K, fmt = T * k, c["N"], c["K"], c["format"]
    codes, scales = _encode(torch.randn(M, K, generator=g, device=DEV), fmt, 1.0)
    state["a"], state["a_scales"] = _pack(codes), _tiled(scales, fmt, offsets)
    state["w"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    each = torch.arange(0, 2 * N, N, dtype=torch.int32, device=DEV)  # one expert's rows are one group
    parts = []
    for e in range(E):
        codes, scales = _encode(torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K), fmt, WEIGHT_SCALE)
        state["w"][e] = _pack(codes)
        parts.append(_tiled(scales, fmt, each)[:-(-N // 128)])
    state["w_scales"] = torch.cat(parts)
    return state


WEIGHT_SCALE = 2.0 ** -6  # the weights' tensor scale


# ---- the plain form ------------------------------------------------------------------------------

def _order(v):
    """Indexes by falling value, equal ones by rising index."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices


def _scores(x, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.amax(-1, keepdim=True).clamp_min(torch.finfo(x.dtype).min)
    e = torch.exp(x - top)
    return e / e.sum(-1, keepdim=True).clamp_min(torch.finfo(x.dtype).tiny)


def _route(s):
    c, x, bias = s["case"], s["logits"].float(), s["bias"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    choice = x
    if bias is not None or c["group_top"] > 1:  # scores that differ past 32 bits still have an order
        choice = torch.where(x > -math.inf, _scores(x.double(), c["score"]), -math.inf)
        choice = choice if bias is None else choice + bias.double()
    if G > 1:
        by = choice.view(T, G, E // G)
        best = by.topk(min(c["group_top"], E // G), dim=-1).values
        rank = torch.where(best[..., 0] > -math.inf, torch.where(best > -math.inf, best, 0).sum(-1), -math.inf)
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, _order(rank)[:, :c["top_groups"]], True)
        choice = by.masked_fill(~keep[..., None], -math.inf).view(T, E)
    ids = _order(choice)[:, :k]
    chosen = choice.gather(1, ids) > -math.inf
    w = _scores(x, c["score"]).gather(1, ids)
    if c["renorm"] and c["score"] == "softmax":
        w = _scores(x.gather(1, ids).masked_fill(~chosen, -math.inf), "softmax")
    w = w * chosen
    if c["renorm"] and c["score"] == "sigmoid":
        w = w / w.sum(-1, keepdim=True).clamp_min(1e-30)
    w = w * c["scale"]
    return {"ids": torch.where(chosen, ids, -1).to(torch.int32), "w": w.expand(c["shards"], T, k).contiguous()}


def _route_grad(s):
    c, x = s["case"], s["logits"].float()
    chosen = s["ids"] >= 0
    ids = s["ids"].clamp_min(0).long()
    dw = s["dw"].sum(0) * chosen * c["scale"]
    out = torch.zeros_like(x)
    if c["score"] == "softmax" and not c["renorm"]:
        p = _scores(x, "softmax")
        dp = out.scatter_add(1, ids, dw)
        d = p * (dp - (p * dp).sum(-1, keepdim=True))
    else:
        z = x.gather(1, ids).masked_fill(~chosen, -math.inf)
        if c["score"] == "softmax":
            w = _scores(z, "softmax")
            dz = w * (dw - (w * dw).sum(-1, keepdim=True))
        else:
            v = _scores(z, "sigmoid")
            if c["renorm"]:
                total = v.sum(-1, keepdim=True).clamp_min(1e-30)
                dw = (dw - (v / total * dw).sum(-1, keepdim=True)) / total
            dz = dw * v * _scores(-z, "sigmoid")
        d = out.scatter_add(1, ids, torch.where(chosen, dz, 0))
    return d.to(s["logits"].dtype)


def _plan(s):
    c = s["case"]
    E, k = c["E"], c["k"]
    flat = s["ids"].reshape(-1).long()
    flat = torch.where(flat < 0, E, flat)  # slots without an expert come last
    order = torch.sort(flat, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.long, device=flat.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat((counts.new_zeros(1), counts[:E].cumsum(0)))
    perm = torch.empty_like(flat).scatter_(0, order, torch.arange(flat.numel(), device=flat.device))
    perm = perm.to(torch.int32).view(c["T"], k).expand(c["shards"], c["T"], k).contiguous()
    return {"perm": perm, "offsets": offsets.to(torch.int32), "rows": (order // k).to(torch.int32)}


def _power(code):
    """2 to the (code - 127), from its bits: exp2 is not exact on every device."""
    return torch.where(code > 0, code << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _encode(x, fmt, tensor_scale):
    """Codes (sign and 3 bits, a byte each) and scale bytes of rows of values."""
    v = x.float() / tensor_scale
    v = v.view(x.shape[0], -1, BLOCK[fmt])
    most = v.abs().amax(-1)
    if fmt == "nvfp4":  # the scale is the 8-bit float (4 exponent bits) next to the largest value's sixth
        s8 = (most / 6).clamp_max(448.0).to(torch.float8_e4m3fn)
        scale, code = s8.float(), s8.view(torch.uint8)
    else:               # the scale is a power of two: the largest value's exponent less 2
        e = torch.frexp(most).exponent.to(torch.int32) - 3
        e = torch.where(most > 0, e, -127).clamp(-127, 127)
        scale, code = _power(e + 127), (e + 127).to(torch.uint8)
    y = torch.where(scale[..., None] > 0, v.abs() / scale[..., None], 0)
    # half-way values go to the code whose last bit is 0
    m = (y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)
    return (m + 8 * torch.signbit(v)).to(torch.uint8).view(x.shape), code


def _decode(codes, scales, fmt, tensor_scale):
    """The values of codes [.., K] and their scale bytes [.., K / block], in 32 bits."""
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    v = level[codes.int()].view(*scales.shape, BLOCK[fmt])
    s = scales.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else _power(scales.int())
    return (v * (s * tensor_scale)[..., None]).view(codes.shape)


def _pack(codes):
    """Two codes a byte, the even one in the low half."""
    return codes[..., ::2] | (codes[..., 1::2] << 4)


def _unpack(data):
    return torch.stack((data & 15, data >> 4), -1).view(*data.shape[:-1], -1)


def _row_tiles(M, offsets):
    """Each row's scale tile and its place there: a group starts at tile (offset // 128) + group."""
    m = torch.arange(M, device=offsets.device)
    group = torch.searchsorted(offsets[1:].contiguous(), m.to(offsets.dtype), right=True)
    start = offsets.long()[group]
    r = m - start
    return start // 128 + group + r // 128, r % 128


def _tiled(scales, fmt, offsets):
    """Row-major scale bytes laid out in tiles of 128 rows by 4 scales: [tiles, chunks, 32, 4, 4], row r at
    [.., r % 32, r // 32, ..], unused places 0."""
    M, J = scales.shape
    chunks = -(-J // 4)
    tile, r = _row_tiles(M, offsets)
    out = torch.zeros(M // 128 + offsets.numel(), chunks, 32, 4, 4, dtype=torch.uint8, device=scales.device)
    padded = torch.nn.functional.pad(scales, (0, 4 * chunks - J)).view(M, chunks, 4)
    out[tile, :, r % 32, r // 32] = padded
    return out.view(-1, chunks, 512)


def _untiled(tiles, J, tile, r):
    t = tiles.view(tiles.shape[0], tiles.shape[1], 32, 4, 4)
    return t[tile, :, r % 32, r // 32].reshape(tile.numel(), -1)[:, :J]


def _quantize(s):
    c = s["case"]
    x = s["x"][s["rows"].long()]
    codes, scales = _encode(x, c["format"], c["tensor_scale"])
    return _decode(codes, scales, c["format"], c["tensor_scale"]).to(torch.bfloat16)


def _product(s):
    c = s["case"]
    M, N, K, E, fmt = c["T"] * c["k"], c["N"], c["K"], c["E"], c["format"]
    J = K // BLOCK[fmt]
    tile, r = _row_tiles(M, s["offsets"])
    a = _decode(_unpack(s["a"]), _untiled(s["a_scales"], J, tile, r), fmt, 1.0)
    m = torch.arange(M, device=a.device)
    group = torch.searchsorted(s["offsets"][1:].contiguous(), m.to(torch.int32), right=True)
    n = torch.arange(N, device=a.device)
    per = -(-N // 128)
    few = M <= 32
    pick = group if few else torch.arange(E, device=a.device)  # few rows: their own experts' weights alone
    wt = (pick[:, None] * per + n // 128).reshape(-1)
    ws = _untiled(s["w_scales"], J, wt, (n % 128).repeat(pick.numel()))
    w = _decode(_unpack(s["w"][pick] if few else s["w"]).view(-1, K), ws, fmt, WEIGHT_SCALE).view(-1, N, K)
    if few:
        return (w @ a[:, :, None])[:, :, 0].to(torch.bfloat16)
    at = m - s["offsets"].long()[group]  # every group's rows in a block of its own
    blocks = torch.zeros(E, s["most"], K, device=a.device)
    blocks[group, at] = a
    return torch.bmm(blocks, w.transpose(1, 2))[group, at].to(torch.bfloat16)


# ---- one pass ------------------------------------------------------------------------------------

def run(state):
    c, s = state["case"], state
    if not own:
        return {"route": _route, "route_grad": _route_grad, "plan": _plan, "quantize": _quantize, "product": _product}[c["op"]](s)
    from tp_reduce_residual_gb300 import experts
    if c["op"] == "route":
        ids, w = experts.route(s["logits"], c["k"], bias=s["bias"], score=c["score"], groups=c["groups"], top_groups=c["top_groups"],
                               group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"], shards=c["shards"])
        return {"ids": ids, "w": w}
    if c["op"] == "route_grad":
        return experts.route_backward(s["logits"], s["ids"], s["dw"], score=c["score"], renormalize=c["renorm"], scale=c["scale"])
    if c["op"] == "plan":
        p = experts.plan(s["ids"], c["E"], shards=c["shards"])
        return {"perm": p.perm, "offsets": p.offsets, "rows": p.rows}
    if c["op"] == "quantize":
        q = experts.quantize_fp4(s["x"], c["format"], rows=s["rows"], offsets=s["offsets"], tensor_scale=c["tensor_scale"])
        return experts.dequantize_fp4(q)
    a = experts.FP4(s["a"], s["a_scales"], c["format"], offsets=s["offsets"])
    w = experts.FP4(s["w"], s["w_scales"], c["format"], tensor_scale=WEIGHT_SCALE)
    return experts.expert_product(a, w)


# ---- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    c, s = case, prepare(case, seed)
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "route":
        x = s["logits"].double()
        if c["score"] == "sigmoid":
            p = torch.sigmoid(x)
        else:
            p = torch.nan_to_num(torch.softmax(x, -1))
        key = x if s["bias"] is None and c["group_top"] == 1 else p if s["bias"] is None else p + s["bias"].double()
        left = torch.isfinite(x)
        if c["groups"] > 1:
            G = c["groups"]
            by = torch.where(left, key, -math.inf).view(T, G, -1)
            a = by.amax(-1)
            if c["group_top"] == 2:
                b = by.scatter(-1, by.argmax(-1, keepdim=True), -math.inf).amax(-1)
                a = a + torch.where(torch.isfinite(b), b, 0)
            beat = (a[:, None, :] > a[:, :, None]) | ((a[:, None, :] == a[:, :, None]) & torch.ones(G, G, device=DEV).tril(-1).bool())
            left = (left.view(T, G, -1) & (beat.sum(-1) < c["top_groups"])[..., None]).view(T, E)
        ids, w = torch.full((T, k), -1, dtype=torch.int32, device=DEV), torch.zeros(T, k, dtype=torch.float64, device=DEV)
        at = torch.arange(E, device=DEV)
        for j in range(k):  # the largest that is left, the first of equal ones
            rest = torch.where(left, key, -math.inf)
            best = torch.where(left & (rest == rest.amax(-1, keepdim=True)), at, E).amin(-1)
            some = best < E
            i = best.clamp_max(E - 1)[:, None]
            ids[:, j] = torch.where(some, best, -1)
            w[:, j] = torch.where(some, p.gather(1, i)[:, 0], 0)
            left = left & (at != best[:, None])
        if c["renorm"]:
            w = torch.nan_to_num(w / w.sum(-1, keepdim=True))
        return {"ids": ids, "w": (c["scale"] * w)[None].repeat(c["shards"], 1, 1)}
    if c["op"] == "route_grad":
        x = s["logits"].double()
        on = s["ids"] >= 0
        pick = torch.zeros(T, k, E, dtype=torch.float64, device=DEV)
        pick.scatter_(2, s["ids"].clamp_min(0).long()[..., None], on.double()[..., None])
        d = s["dw"].double().sum(0)
        if c["score"] == "sigmoid":
            p = torch.sigmoid(x)
            slope = torch.sigmoid(x) * torch.sigmoid(-x)
            v = torch.einsum("tke,te->tk", pick, p)
            if c["renorm"]:
                total = v.sum(-1, keepdim=True)
                d = torch.nan_to_num((d * total - (d * v).sum(-1, keepdim=True)) / total ** 2)
            return c["scale"] * torch.einsum("tke,tk->te", pick, d) * slope
        if c["renorm"]:
            x = x.masked_fill(pick.sum(1) == 0, -math.inf)
        p = torch.nan_to_num(torch.softmax(x, -1))
        up = torch.einsum("tke,tk->te", pick, d)
        return c["scale"] * (p * up - p * (p * up).sum(-1, keepdim=True))
    if c["op"] == "plan":
        flat = [E if i < 0 else i for i in s["ids"].reshape(-1).tolist()]
        order = sorted(range(T * k), key=lambda i: (flat[i], i))
        perm, starts = [0] * (T * k), [0] * (E + 1)
        for at, i in enumerate(order):
            perm[i] = at
        for i in flat:
            if i < E:
                starts[i + 1] += 1
        for e in range(E):
            starts[e + 1] += starts[e]
        whole = dict(dtype=torch.int32, device=DEV)
        return {"perm": torch.tensor(perm, **whole).view(1, T, k).repeat(c["shards"], 1, 1), "offsets": torch.tensor(starts, **whole),
                "rows": torch.tensor([i // k for i in order], **whole)}
    level = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)

    def exponent(v):
        return (v.contiguous().view(torch.int64) >> 52) - 1023

    def two_to(e):
        return (e + 1023 << 52).view(torch.float64)

    if c["op"] == "quantize":
        n, size = c["H"] // BLOCK[c["format"]], BLOCK[c["format"]]
        token = torch.empty(T, c["H"], dtype=torch.float64, device=DEV)
        for t in range(0, T, 64):
            v = s["x"][t:t + 64].double().view(-1, n, size) / c["tensor_scale"]
            top = v.abs().amax(-1, keepdim=True)
            if c["format"] == "nvfp4":  # 3 bits after the leading one, steps of 2^-9 at the least
                want = (top / 6).clamp_max(448)
                step = two_to(exponent(want.clamp_min(2.0 ** -6)) - 3)
                scale = torch.round(want / step) * step
            else:
                scale = two_to(exponent(top.clamp_min(2.0 ** -125)) - 2) * (top > 0)
            y = torch.where(scale > 0, v.abs() / scale, 0)
            gap = (y[..., None] - level).abs()
            near = gap == gap.amin(-1, keepdim=True)
            # of two levels equally near, the one with an even number
            code = torch.where(near, torch.arange(8, device=DEV) + 100 * (torch.arange(8, device=DEV) % 2), 1000).amin(-1) % 100
            token[t:t + 64] = (level[code] * torch.sign(v) * scale * c["tensor_scale"]).view(-1, c["H"])
        return token[s["rows"].long()]
    M, N, K, fmt = T * k, c["N"], c["K"], c["format"]
    both = torch.cat((level, -level))

    def values(data, tiles, first, rows):
        """Rows of packed codes whose scale tiles start at tile `first`, in 64 bits."""
        byte = tiles[first:first + -(-rows // 128)]
        q = torch.arange(rows, device=DEV)
        j = torch.arange(K // BLOCK[fmt], device=DEV)
        b = byte.view(-1)[((q // 128)[:, None] * byte.shape[1] + j // 4) * 512 + (q % 32)[:, None] * 16 + (q % 128 // 32)[:, None] * 4 + j % 4].int()
        if fmt == "nvfp4":
            e, f = b >> 3, (b & 7).double()
            scale = torch.where(e > 0, two_to(e.long() - 7) * (1 + f / 8), f * 2.0 ** -9)
        else:
            scale = two_to(b.long() - 127)
        v = torch.empty(rows, K, dtype=torch.float64, device=DEV)
        v[:, 0::2], v[:, 1::2] = both[(data % 16).int()], both[(data // 16).int()]
        return (v.view(rows, -1, BLOCK[fmt]) * scale[..., None]).view(rows, K)

    at = s["offsets"].tolist()
    out = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    for e in range(E):
        lo, hi = at[e], at[e + 1]
        if hi > lo:
            a = values(s["a"][lo:hi], s["a_scales"], lo // 128 + e, hi - lo)
            w = values(s["w"][e], s["w_scales"], e * -(-N // 128), N)
            out[lo:hi] = a @ w.T * WEIGHT_SCALE
    return out
