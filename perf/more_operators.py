"""Further operators around the experts, as measured: the experts' linear layers in 16 bits over ragged
groups of rows, with their gradients; the gated activation between the two layers of an expert, with its
gradient; rows in 8-bit integers with a scale a row; and the experts' product of such rows and weights.

``listed()`` are the cases, ``prepare`` makes one case's tensors from a seed, ``run`` is one pass: with
``own`` the framework's kernels, else elementary torch operations in 32 bits (64 where a rounding to a
whole number is decided).  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    """H and k are those of the finalize workloads (H = 5120, 6144, 8192; k = 8, 10; 256 experts); an expert's
    hidden layer is 2048 wide, or an eighth of it on one of 8 shards; its first layer is gate and up side by side."""
    return [
        # one decoded token: the first layer of its experts on one of 8 shards, a stream of weights
        dict(name="linear one token", op="linear", T=1, E=256, k=10, N=512, K=8192, dtype="bf16", gather=True, masked=0.0),
        # a decode batch with a few padding tokens: the second layer of nearly every expert on one of 4 shards
        dict(name="linear decode batch", op="linear", T=100, E=256, k=8, N=6144, K=512, dtype="bf16", gather=False, masked=0.05),
        # a prompt: large ragged groups through the first layer, rows taken from their tokens
        dict(name="linear prompt", op="linear", T=4096, E=64, k=8, N=4096, K=5120, dtype="bf16", gather=True, masked=0.0),
        # training, a short odd sequence on a small layer
        dict(name="linear grad short", op="linear_grad", T=333, E=16, k=4, N=1024, K=2048, dtype="fp16", out="fp32", gather=True,
             masked=0.05),
        # training, one sequence through the second layer of all experts
        dict(name="linear grad sequence", op="linear_grad", T=4096, E=64, k=8, N=5120, K=2048, dtype="bf16", out="bf16", gather=False,
             masked=0.0),
        # the activation of a decode batch on one of 8 shards
        dict(name="swiglu decode", op="swiglu", M=100, F=256, dtype="bf16"),
        # its gradient for a training sequence's slots
        dict(name="swiglu grad sequence", op="swiglu_grad", M=32768, F=2048, dtype="bf16"),
        # a few tokens' rows repeated for their experts
        dict(name="int8 rows decode", op="quantize", T=5, E=256, k=10, H=8192, dtype="bf16"),
        # a prompt's rows repeated for their experts
        dict(name="int8 rows prompt", op="quantize", T=4096, E=256, k=8, H=5120, dtype="bf16"),
        # one decoded token through 10 experts: a stream of weights
        dict(name="int8 product one token", op="product", T=1, E=256, k=10, N=1024, K=8192, masked=0.0),
        # a decode batch that reaches nearly every expert with a few rows each
        dict(name="int8 product decode batch", op="product", T=100, E=256, k=8, N=6144, K=1024, masked=0.05),
        # a prompt: large ragged groups
        dict(name="int8 product prompt", op="product", T=4096, E=64, k=8, N=4096, K=5120, masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_grad", "linear_grad", "swiglu", "swiglu_grad", "quantize", "product", "product"))
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    if op in ("swiglu", "swiglu_grad"):
        return dict(op=op, M=_log_int(rng, 1, 16384), F=_log_int(rng, 8, 4096), dtype=rng.choice((dtype, "fp32")))
    k = rng.choice((1, 2, 4, 6, 8, 10))
    T = _log_int(rng, 1, 4096)
    if op == "quantize":
        return dict(op=op, T=T, E=_log_int(rng, k, 256), k=min(k, 8), H=16 * _log_int(rng, 4, 320), dtype=rng.choice((dtype, "fp32")))
    while True:  # no more weights, nor more products, than the largest listed case of the kind
        E = rng.choice((8, 16, 32, 64, 128, 256))
        if E < k:
            continue
        N = 8 * _log_int(rng, 8, 1024)
        K = 16 * _log_int(rng, 4, 512) if op == "product" else 8 * _log_int(rng, 8, 1024)
        if E * N * K <= 64 * 4096 * 5120 // (2 if op == "linear_grad" else 1) \
                and T * k * N * K <= 32768 * 4096 * 5120 // (2 if op == "linear_grad" else 1):
            break
    c = dict(op=op, T=T, E=E, k=k, N=N, K=K, masked=rng.choice((0.0, 0.0, 0.1)))
    if op != "product":
        c |= dict(dtype=dtype, gather=rng.random() < 0.5)
    if op == "linear_grad":
        c["out"] = rng.choice((dtype, "fp32"))
    return c


SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def work(case):
    c = case
    if c["op"] in ("swiglu", "swiglu_grad"):  # gate, up (and the output's gradient) in, the output (or both gradients) out
        n = c["M"] * c["F"] * SIZE[c["dtype"]]
        return {"bytes": (3 if c["op"] == "swiglu" else 5) * n, "flops": (8 if c["op"] == "swiglu" else 16) * c["M"] * c["F"]}
    T, E, k = c["T"], c["E"], c["k"]
    M = T * k
    if c["op"] == "quantize":  # tokens in, codes and scales out and in again, the values that they stand for out
        return {"bytes": T * c["H"] * SIZE[c["dtype"]] + 4 * M + 2 * M * (c["H"] + 4) + 2 * M * c["H"], "flops": 5 * M * c["H"]}
    N, K = c["N"], c["K"]
    live = M * (1 - c["masked"])
    active = E * (1 - (1 - k / E) ** (T * (1 - c["masked"])))  # experts that T tokens reach when each takes k of E
    if c["op"] == "product":
        return {"bytes": int(active * N * (K + 4) + live * (K + 4) + 2 * M * N + 4 * (E + 1)), "flops": int(2 * live * N * K)}
    x = (T * K * 2 + 4 * M) if c["gather"] else live * K * 2
    if c["op"] == "linear":
        return {"bytes": int(active * N * K * 2 + x + 2 * M * N + 4 * (E + 1)), "flops": int(2 * live * N * K)}
    return {"bytes": int(active * N * K * 2 + x + live * N * 2 + 2 * M * K + E * N * K * SIZE[c["out"]] + 4 * (E + 1)),
            "flops": int(4 * live * N * K)}


# ---- inputs --------------------------------------------------------------------------------------

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _groups(g, c):
    """The slots' order when they are grouped by expert: offsets [E+1], the token at every place, the largest
    group.  Some experts are more popular than others; padding tokens' slots come after the last group."""
    T, E, k = c["T"], c["E"], c["k"]
    u = torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
    ids = u.topk(k, dim=1).indices
    if c.get("masked"):
        ids[torch.rand(T, generator=g, device=DEV) < c["masked"]] = E
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return offsets, (order // k).to(torch.int32), int(counts.max())


def _activations(g, n, width):
    """Normed activations: some channels are far larger than the rest."""
    return torch.randn(n, width, generator=g, device=DEV) * torch.exp(0.5 * torch.randn(width, generator=g, device=DEV))


def _codes(x):
    """8-bit codes of rows and their scales."""
    scale = x.abs().amax(-1) / 127
    q = torch.round(x.double() / scale.double().clamp_min(1e-300)[..., None]).clamp(-127, 127)
    return q.to(torch.int8), scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    state = {"case": c}
    if c["op"] in ("swiglu", "swiglu_grad"):
        state["x"] = (2 * torch.randn(c["M"], 2 * c["F"], generator=g, device=DEV)).to(DTYPES[c["dtype"]])
        if c["op"] == "swiglu_grad":
            state["dy"] = torch.randn(c["M"], c["F"], generator=g, device=DEV).to(DTYPES[c["dtype"]])
        return state
    T, E, k = c["T"], c["E"], c["k"]
    M = T * k
    state["offsets"], rows, state["most"] = _groups(g, c)
    if c["op"] == "quantize":
        return state | {"x": _activations(g, T, c["H"]).to(DTYPES[c["dtype"]]), "rows": rows}
    N, K = c["N"], c["K"]
    if c["op"] == "product":
        state["a"], state["a_scales"] = _codes(_activations(g, M, K))
        state["w"] = torch.empty(E, N, K, dtype=torch.int8, device=DEV)
        state["w_scales"] = torch.empty(E, N, device=DEV)
        for e in range(E):
            state["w"][e], state["w_scales"][e] = _codes(torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K))
        return state
    dtype = DTYPES[c["dtype"]]
    state["rows"] = rows if c["gather"] else None
    state["x"] = _activations(g, T if c["gather"] else M, K).to(dtype)
    state["w"] = torch.empty(E, N, K, dtype=dtype, device=DEV)
    for e in range(E):
        state["w"][e] = torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K)
    if c["op"] == "linear_grad":
        state["dy"] = torch.randn(M, N, generator=g, device=DEV).to(dtype)
    return state


# ---- the plain form ------------------------------------------------------------------------------

def _places(s, M):
    """Each place's group and its position there, for the places that are in a group."""
    o = s["offsets"].long()
    m = torch.arange(M, device=o.device)
    m = m[m < o[-1]]
    group = torch.searchsorted(o[1:].contiguous(), m, right=True)
    return m, group, m - o[group]


def _blocks(v, s, m, group, at):
    """Every group's rows in a block of its own, in 32 bits: [E, the largest group, width]."""
    out = torch.zeros(s["case"]["E"], s["most"], v.shape[1], device=v.device)
    out[group, at] = v[m].float()
    return out


def _taken(s):
    return s["x"] if s["rows"] is None else s["x"][s["rows"].long()]


def _grouped(a, w, s, M, width):
    """Rows [M, ..] times their group's [.., width], in 32 bits; rows of no group are zeros."""
    m, group, at = _places(s, M)
    out = torch.zeros(M, width, device=a.device)
    if M <= 32:  # few rows: their own experts' weights alone
        out[m] = torch.bmm(a[m].float()[:, None], w(group))[:, 0]
    else:
        out[m] = torch.bmm(_blocks(a, s, m, group, at), w(slice(None)))[group, at]
    return out


def _linear(s):
    c = s["case"]
    return _grouped(_taken(s), lambda e: s["w"][e].float().transpose(1, 2), s, c["T"] * c["k"], c["N"]).to(s["x"].dtype)


def _linear_grad(s):
    c = s["case"]
    M = c["T"] * c["k"]
    dx = _grouped(s["dy"], lambda e: s["w"][e].float(), s, M, c["K"]).to(s["x"].dtype)
    m, group, at = _places(s, M)
    dw = torch.bmm(_blocks(s["dy"], s, m, group, at).transpose(1, 2), _blocks(_taken(s), s, m, group, at))
    return {"dx": dx, "dw": dw.to(DTYPES[c["out"]])}


def _sigmoid(x):
    z = torch.exp(-x.abs())
    return torch.where(x >= 0, 1 / (1 + z), z / (1 + z))


def _swiglu(s):
    gate, up = s["x"].float().chunk(2, dim=-1)
    return (gate * _sigmoid(gate) * up).to(s["x"].dtype)


def _swiglu_grad(s):
    gate, up = s["x"].float().chunk(2, dim=-1)
    dy, p = s["dy"].float(), _sigmoid(gate)
    dgate = dy * up * (p + gate * p * _sigmoid(-gate))
    return torch.cat((dgate, dy * (gate * p)), dim=-1).to(s["x"].dtype)


def _quantize(s):
    codes, scales = _codes(s["x"].float())
    rows = s["rows"].long()
    return {"values": (codes[rows].float() * scales[rows, None]).to(torch.bfloat16), "scales": scales[rows]}


def _product(s):
    c = s["case"]
    M = c["T"] * c["k"]
    out = _grouped(s["a"], lambda e: s["w"][e].float().transpose(1, 2), s, M, c["N"])
    m, group, _ = _places(s, M)
    out[m] *= s["a_scales"][m, None] * s["w_scales"][group]
    return out.to(torch.bfloat16)


# ---- one pass ------------------------------------------------------------------------------------

def run(state):
    c, s = state["case"], state
    if not own:
        return {"linear": _linear, "linear_grad": _linear_grad, "swiglu": _swiglu, "swiglu_grad": _swiglu_grad,
                "quantize": _quantize, "product": _product}[c["op"]](s)
    from tp_reduce_residual_gb300 import experts
    if c["op"] == "linear":
        return experts.expert_linear(s["x"], s["w"], s["offsets"], rows=s["rows"])
    if c["op"] == "linear_grad":
        dx = experts.expert_linear_dx(s["dy"], s["w"], s["offsets"])
        return {"dx": dx, "dw": experts.expert_linear_dw(s["dy"], s["x"], s["offsets"], rows=s["rows"], dtype=DTYPES[c["out"]])}
    if c["op"] == "swiglu":
        return experts.swiglu(s["x"])
    if c["op"] == "swiglu_grad":
        return experts.swiglu_backward(s["x"], s["dy"])
    if c["op"] == "quantize":
        q = experts.quantize_int8(s["x"], rows=s["rows"], offsets=s["offsets"])
        return {"values": experts.dequantize_int8(q), "scales": q.scales}
    a = experts.Int8(s["a"], s["a_scales"], offsets=s["offsets"])
    return experts.expert_product(a, experts.Int8(s["w"], s["w_scales"]))


# ---- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    c, s = case, prepare(case, seed)
    real = dict(dtype=torch.float64, device=DEV)
    if c["op"] in ("swiglu", "swiglu_grad"):
        F = c["F"]
        gate, up = s["x"][:, :F].double(), s["x"][:, F:].double()
        if c["op"] == "swiglu":
            return gate / (1 + torch.exp(-gate)) * up
        dy = s["dy"].double()
        out = torch.empty(c["M"], 2 * F, **real)
        z = torch.exp(-gate)
        out[:, :F] = dy * up * (1 + z + gate * z) / (1 + z) ** 2
        out[:, F:] = dy * gate / (1 + z)
        return out
    if c["op"] == "quantize":
        values, scales = [], []
        for x in s["x"].split(256):
            x = x.double()
            scale = (torch.linalg.vector_norm(x, ord=math.inf, dim=1) / 127).to(torch.float32).double()
            y = (x / scale[:, None]).clamp(-127, 127)
            low = torch.floor(y)
            part = y - low  # the nearer whole number, the even one of two
            up = (part > 0.5) | ((part == 0.5) & (low % 2 != 0))
            values.append((low + up) * scale[:, None])
            scales.append(scale)
        rows = s["rows"].long()
        return {"values": torch.cat(values)[rows], "scales": torch.cat(scales)[rows]}
    M, N, K = c["T"] * c["k"], c["N"], c["K"]
    bounds = s["offsets"].tolist()
    if c["op"] == "linear_grad":
        out = {"dx": torch.zeros(M, K, **real), "dw": torch.zeros(c["E"], N, K, dtype=torch.float64, device=DEV)}
    else:
        out = torch.zeros(M, N, **real)
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if lo == hi:
            continue
        w = s["w"][e].double()
        if c["op"] == "product":
            a = s["a"][lo:hi].double() * s["a_scales"][lo:hi, None].double()
            out[lo:hi] = a @ (w * s["w_scales"][e][:, None].double()).T
            continue
        x = s["x"][lo:hi] if s["rows"] is None else s["x"].index_select(0, s["rows"][lo:hi])
        if c["op"] == "linear":
            out[lo:hi] = x.double() @ w.T
        else:
            dy = s["dy"][lo:hi].double()
            out["dx"][lo:hi] = dy @ w
            out["dw"][e] = dy.T @ x.double()
    return out
