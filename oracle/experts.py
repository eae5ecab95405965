"""The expert layer in 64 bits, written from the definitions in include/reshard_ops.h: what the kernels are compared with.

Plain torch on whatever device the inputs are on; loops where they are the shortest form. Independent of the library.
"""
from __future__ import annotations

import torch

F64 = torch.float64
NONE = float("-inf")


# ----------------------------------------------------------------------------------------------------------- routing

def scores(logits: torch.Tensor, score: str) -> torch.Tensor:
    z = logits.to(F64)
    z = torch.where(torch.isnan(z), NONE, z)
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - torch.where(top == NONE, 0.0, top))
    return e / e.sum(1, keepdim=True)


def route_keys(logits, score, bias):
    """What orders the experts; -inf for what cannot be chosen."""
    z = logits.to(F64)
    z = torch.where(torch.isnan(z), NONE, z)
    if bias is None:
        return z
    key = scores(logits, score) + bias.to(F64)
    return torch.where((z == NONE) | torch.isnan(key), NONE, key)


def route(logits, k, score="softmax", bias=None, groups=1, groups_kept=1, group_top=1, renormalize=True, scale=1.0):
    """(weights [T, k] 64 bits, ids [T, k]) one row at a time."""
    s, key = scores(logits, score), route_keys(logits, score, bias)
    T, E = key.shape
    weights, ids = torch.zeros(T, k, dtype=F64), torch.full((T, k), -1, dtype=torch.int64)
    for t in range(T):
        row = key[t].tolist()
        rank = row if bias is not None else [v if r > NONE else NONE for v, r in zip(s[t].tolist(), row)]
        if groups > 1:
            size = E // groups
            total = []
            for g in range(groups):
                best = sorted((v for v in rank[g * size:(g + 1) * size] if v > NONE), reverse=True)[:group_top]
                total.append(sum(best) if best else NONE)
            kept = sorted(range(groups), key=lambda g: (-total[g], g))[:groups_kept]
            row = [v if e // size in kept else NONE for e, v in enumerate(row)]
        order = [e for e in sorted(range(E), key=lambda e: (-row[e], e)) if row[e] > NONE][:k]
        w = s[t, order] if order else s[t, :0]
        if renormalize and len(order):
            if score == "softmax":        # the row's divisor cancels, also where it underflows
                z = logits[t].to(F64)[order]
                w = torch.softmax(z, 0)
            else:
                total = w.sum()
                w = w / total if total > 0 else w * 0
        weights[t, :len(order)] = w.cpu() * scale
        ids[t, :len(order)] = torch.tensor(order, dtype=torch.int64)
    return weights, ids


def route_weights(logits, ids, score, renormalize, scale):
    """The weights of a fixed choice, differentiable in the logits."""
    z = logits
    valid = (ids >= 0) & (ids < z.shape[1])
    chosen = torch.gather(z, 1, torch.where(valid, ids, 0))
    if score == "softmax" and renormalize:
        e = torch.exp(chosen - chosen.detach().masked_fill(~valid, NONE).max(1, keepdim=True).values.nan_to_num(0, 0, 0)) * valid
    elif score == "softmax":
        e = torch.gather(torch.softmax(z, 1), 1, torch.where(valid, ids, 0)) * valid
    else:
        e = torch.sigmoid(chosen) * valid
    if renormalize:
        total = e.sum(1, keepdim=True)
        e = e / torch.where(total == 0, 1.0, total)
    return e * scale


def route_backward(grad, logits, ids, score, renormalize, scale):
    """The gradient by the formulas (rows without masked logits), summed slot by slot."""
    z, g = logits.to(F64), grad.to(F64) * scale
    T, E = z.shape
    out = torch.zeros(T, E, dtype=F64, device=z.device)
    s = scores(logits, score)
    for t in range(T):
        slots = [(j, int(e)) for j, e in enumerate(ids[t].tolist()) if 0 <= e < E]
        if not slots:
            continue
        e = torch.tensor([x for _, x in slots])
        gj = g[t, [j for j, _ in slots]]
        sj = s[t, e]
        if score == "softmax" and not renormalize:
            dot = (gj * sj).sum()
            row = -s[t] * dot
            row.index_add_(0, e.to(row.device), gj * sj)
            out[t] = row
            continue
        if renormalize:
            r = torch.softmax(z[t, e], 0) if score == "softmax" else sj / sj.sum()
            d = r * (gj - (gj * r).sum())
        else:
            d = gj * sj
        if score == "sigmoid":
            d = d * (1.0 / (1.0 + torch.exp(z[t, e])))
        out[t].index_add_(0, e.to(out.device), d)
    return out


def dispatch(ids, experts, first=0):
    """(offsets, order, position): slots by expert, ascending."""
    flat = ids.reshape(-1).tolist()
    per = [[i for i, x in enumerate(flat) if x == first + e] for e in range(experts)]
    offsets, order, position = [0], [], [-1] * len(flat)
    for p in per:
        for i in p:
            position[i] = len(order)
            order.append(i)
        offsets.append(len(order))
    return offsets, order, position


# ------------------------------------------------------------------------------------------------------ quantization

def e4m3(v: torch.Tensor) -> torch.Tensor:
    """v rounded to the nearest e4m3 value, ties to even, +-448 at most; NaN stays. Values, in v's type."""
    _, e = torch.frexp(v.abs().to(F64))
    # 2^n from its bits: a device's power function may be off in the last place
    step = (((e.long() - 1).clamp(-6, 100) - 3 + 1023) << 52).view(F64)
    return (torch.round(v.to(F64) / step) * step).clamp(-448, 448).to(v.dtype)


def _blocks(x, rows):
    *lead, M, K = x.shape
    m, k = -(-M // rows), -(-K // 128)
    pad = torch.zeros(*lead, m * rows, k * 128, dtype=torch.float32, device=x.device)
    pad[..., :M, :K] = x.float()
    return pad.reshape(*lead, m, rows, k, 128).transpose(-3, -2)


def quantize(x: torch.Tensor, rows: int):
    """(values, scale) in blocks of rows x 128, by the definition's fp32 steps: exact, so that codes can be compared."""
    b = _blocks(x, rows)
    a = b.abs().amax((-2, -1))
    a = torch.where(torch.isfinite(a), a.clamp(min=2.0 ** -100), float("nan"))
    one = torch.ones((), dtype=torch.float32, device=x.device)
    inv = torch.div(one, a) * (one * 448)
    scale = a * torch.div(one, one * 448)
    q = e4m3(b * inv[..., None, None])
    *lead, M, K = x.shape
    q = q.transpose(-3, -2).reshape(*lead, b.shape[-4] * rows, b.shape[-3] * 128)[..., :M, :K]
    return q, scale


def dequantize(q: torch.Tensor, scale: torch.Tensor, rows: int) -> torch.Tensor:
    M, K = q.shape[-2:]
    s = scale.to(F64).repeat_interleave(rows, -2)[..., :M, :].repeat_interleave(128, -1)[..., :K]
    return q.to(F64) * s


def values(q: torch.Tensor) -> torch.Tensor:
    """float8 codes (or their bytes) as 64-bit values."""
    return (q.view(torch.float8_e4m3fn) if q.dtype == torch.uint8 else q).float().to(F64)


# ------------------------------------------------------------------------------------------------------- expert layer

def experts(x, ids, weights, w13, w13_scale, w2, w2_scale, first=0):
    """The routed feed-forward in 64 bits; only the two quantizations round."""
    xq, xs = quantize(x, 1)
    xv = dequantize(xq, xs, 1)
    E, H, I = w2.shape
    out = torch.zeros(x.shape[0], H, dtype=F64, device=x.device)
    for e in range(E):
        t, j = torch.nonzero(ids == first + e, as_tuple=True)
        if len(t) == 0:
            continue
        gu = xv[t] @ dequantize(values(w13[e]), w13_scale[e], 128).t()
        g, u = gu[:, :I], gu[:, I:]
        hq, hs = quantize(g / (1 + torch.exp(-g)) * u, 1)
        y = dequantize(hq, hs, 1) @ dequantize(values(w2[e]), w2_scale[e], 128).t()
        out.index_add_(0, t, y * weights[t, j].to(F64)[:, None])
    return out
