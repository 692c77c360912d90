"""Plain 64-bit definitions of the operators around the experts, for the tests (CPU torch)."""
from __future__ import annotations

import math

import torch

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
BLOCK = {"nvfp4": 16, "mxfp4": 32}
CHUNK = {"nvfp4": 64, "mxfp4": 128}


def scores(x, score):
    """64-bit scores of logits; a row without a finite logit has softmax scores 0."""
    if score == "sigmoid":
        return torch.sigmoid(x)
    return torch.nan_to_num(torch.softmax(x, -1), nan=0.0)


def route(logits, k, bias=None, score="softmax", groups=1, top_groups=1, group_top=1,
          renormalize=True, scale=1.0):
    """ids [T,k] int32 and w [T,k] float64, one token and one choice at a time."""
    x = logits.double()
    T, E = x.shape
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        row = x[t]
        s = scores(torch.where(torch.isnan(row), -math.inf, row), score)
        if bias is None and not (groups > 1 and group_top > 1):
            key = row.tolist()
        else:
            key = (s + (0.0 if bias is None else bias.double())).tolist()
        nan = bool(torch.isnan(row).any()) or any(math.isnan(v) for v in key)
        left = [not math.isnan(float(row[e])) and float(row[e]) > -math.inf and not math.isnan(key[e])
                and key[e] > -math.inf for e in range(E)]
        if groups > 1 and top_groups < groups:
            size = E // groups
            rank = []
            for g in range(groups):
                have = sorted((key[e] for e in range(g * size, (g + 1) * size) if left[e]), reverse=True)
                rank.append(sum(have[:group_top]) if have else -math.inf)
            keep = sorted(range(groups), key=lambda g: (-rank[g], g))[:top_groups]
            left = [ok and e // size in keep for e, ok in enumerate(left)]
        order = sorted((e for e in range(E) if left[e]), key=lambda e: (-key[e], e))[:k]
        for j, e in enumerate(order):
            ids[t, j] = e
            w[t, j] = s[e]
        if renormalize and order:
            if score == "softmax":
                w[t, :len(order)] = torch.softmax(row[order], -1)
            else:
                total = float(w[t].sum())
                w[t] = w[t] / total if total > 0 else 0.0
        w[t] *= scale
        if nan:
            w[t] = math.nan
    return ids, w


def route_weights(x, ids, score, renormalize, scale):
    """w [T,k] of chosen ids, differentiable in x (64 bits); ids of -1 give 0."""
    on = ids >= 0
    i = ids.clamp_min(0).long()
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, -1)
    v = torch.where(on, s.gather(1, i), 0.0)
    if renormalize:
        v = v / v.sum(-1, keepdim=True)
    return scale * v


def plan(ids, E):
    """perm [T,k], offsets [E+1], rows [T*k] as int32."""
    T, k = ids.shape
    flat = [e if 0 <= e < E else E for e in ids.reshape(-1).tolist()]
    order = sorted(range(T * k), key=lambda i: (flat[i], i))
    perm = torch.empty(T * k, dtype=torch.int32)
    for at, i in enumerate(order):
        perm[i] = at
    offsets = torch.tensor([sum(1 for b in flat if b < e) for e in range(E + 1)], dtype=torch.int32)
    return perm.view(T, k), offsets, torch.tensor([i // k for i in order], dtype=torch.int32)


def encode(x, fmt, tensor_scale=1.0):
    """(codes [M,K] int, scales [M,K/block] float64) of BF16 or FP16 rows by search over the levels."""
    B = BLOCK[fmt]
    v = x.double() / tensor_scale
    M, K = v.shape
    v = v.view(M, K // B, B)
    top = v.abs().amax(-1)
    bad = ~torch.isfinite(v).all(-1)
    if fmt == "nvfp4":
        grid = torch.tensor([m * 2.0 ** -9 for m in range(8)]
                            + [(8 + m) / 8 * 2.0 ** e for e in range(-6, 9) for m in range(8) if not (e == 8 and m == 7)],
                            dtype=torch.float64)
        want = torch.where(bad, 1.0, top / 6).clamp_max(448.0)
        # the nearest, of two the one with an even index (the index is the byte)
        hi = torch.searchsorted(grid, want).clamp_max(len(grid) - 1)
        lo = (hi - 1).clamp_min(0)
        a, b = want - grid[lo], grid[hi] - want
        scale = torch.where((a < b) | ((a == b) & (lo % 2 == 0)), grid[lo], grid[hi])
    else:
        e = torch.frexp(torch.where(bad | (top == 0), 1.0, top)).exponent - 3  # floor(log2) - 2
        scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), e.clamp(-127, 127)), 2.0 ** -127)
    safe = torch.where(scale > 0, scale, 1.0)[..., None]
    y = torch.where((scale > 0)[..., None] & ~bad[..., None], v.abs() / safe, 0.0).clamp_max(8.0)  # past 6 is 6
    gap = (y[..., None] - LEVELS).abs()
    near = gap == gap.amin(-1, keepdim=True)
    odd = torch.arange(8) % 2
    code = torch.where(near, torch.arange(8) + 100 * odd, 1000).amin(-1) % 100
    code = code + 8 * (torch.signbit(v) & ~bad[..., None])
    return code.view(M, K), torch.where(bad, math.nan, scale)


def row_tiles(M, offsets=None, groups=1):
    """(tile, row in the tile) of each row."""
    if offsets is None:
        per = M // groups
        return [((m // per) * (-(-per // 128)) + m % per // 128, m % per % 128) for m in range(M)]
    o = offsets.tolist()
    out = []
    for m in range(M):
        g = sum(1 for v in o[1:] if v <= m)
        r = m - o[g]
        out.append((o[g] // 128 + g + r // 128, r % 128))
    return out


def decode(data, scales, fmt, tensor_scale=1.0, offsets=None, groups=1):
    """Values (float64 [M,K]) of packed codes and tiled scale bytes."""
    data, scales = data.cpu().reshape(-1, data.shape[-1]), scales.cpu()
    M, K = data.shape[0], 2 * data.shape[1]
    codes = torch.stack((data & 15, data >> 4), -1).view(M, K).long()
    value = torch.cat((LEVELS, -LEVELS))[codes]
    where = row_tiles(M, None if offsets is None else offsets.cpu(), groups)
    J = K // BLOCK[fmt]
    b = torch.empty(M, J, dtype=torch.long)
    j = torch.arange(J)
    for m, (tile, r) in enumerate(where):
        b[m] = scales[tile].view(-1)[j // 4 * 512 + r % 32 * 16 + r // 32 * 4 + j % 4].long()
    if fmt == "nvfp4":
        e, f = b >> 3, (b & 7).double()
        s = torch.where(e > 0, torch.ldexp(1 + f / 8, e - 7), f * 2.0 ** -9)
        s = torch.where(b == 127, math.nan, s)
    else:
        s = torch.where(b == 255, math.nan, torch.ldexp(torch.ones(1, dtype=torch.float64), b - 127))
    return (value.view(M, J, -1) * (s * tensor_scale)[..., None]).view(M, K)
