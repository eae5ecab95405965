"""Rows moved by an index, their gradients, and the norm and clipping of many tensors in 64 bits, written from the
definitions in include/reshard_ops.h: what the kernels are compared with.

Plain torch on whatever device the inputs are on. Independent of the library.
"""
from __future__ import annotations

import torch

F64 = torch.float64


def sort(ids: torch.Tensor, experts: int, first: int = 0):
    """(offsets, order, position) of the slots by expert, as reshard_dispatch defines them; order ends with the last place."""
    flat = ids.reshape(-1).tolist()
    order = [s for e in range(experts) for s, i in enumerate(flat) if i == first + e]
    position = [-1] * len(flat)
    for p, s in enumerate(order):
        position[s] = p
    counts = [sum(1 for i in flat if i == first + e) for e in range(experts)]
    offsets = [sum(counts[:e]) for e in range(experts + 1)]
    return tuple(torch.tensor(v, dtype=torch.int32, device=ids.device) for v in (offsets, order, position))


def _slots(position: torch.Tensor, rows: int):
    """(slots that have a place among the rows, their places)"""
    s = torch.nonzero((position >= 0) & (position < rows)).view(-1)
    return s, position[s].long()


def permute(x: torch.Tensor, position: torch.Tensor, into: torch.Tensor) -> torch.Tensor:
    """`into` with every placed slot's row replaced (places are distinct)."""
    out = into.clone()
    s, p = _slots(position, into.shape[0])
    out[p] = x[s // (position.numel() // x.shape[0])]
    return out


def combine(y: torch.Tensor, position: torch.Tensor, weights, k: int, magnitudes: bool = False) -> torch.Tensor:
    """sum_j w y; with `magnitudes` the sum of the terms' magnitudes instead."""
    s, p = _slots(position, y.shape[0])
    terms = y.to(F64)[p]
    if weights is not None:
        terms = terms * weights.to(F64).view(-1)[s].unsqueeze(1)
    out = torch.zeros(position.numel() // k, y.shape[1], dtype=F64, device=y.device)
    return out.index_add_(0, s // k, terms.abs() if magnitudes else terms)


def combine_backward(grad: torch.Tensor, y: torch.Tensor, position: torch.Tensor, weights, k: int, magnitudes: bool = False):
    """(gradient to y, gradient to the weights); with `magnitudes` the sums of the products' magnitudes as the latter."""
    s, p = _slots(position, y.shape[0])
    g = grad.to(F64)[s // k]
    w = torch.ones(position.numel(), dtype=F64, device=y.device) if weights is None else weights.to(F64).view(-1)
    dy = torch.zeros(y.shape, dtype=F64, device=y.device)
    dy[p] = g * w[s].unsqueeze(1)
    dw = torch.zeros(position.numel(), dtype=F64, device=y.device)
    products = g * y.to(F64)[p]
    dw[s] = (products.abs() if magnitudes else products).sum(1)
    return dy, dw.view(-1, k)


def embedding(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0, first: int = 0) -> torch.Tensor:
    r = ids.long() - first
    here = (r >= 0) & (r < table.shape[0])
    out = torch.zeros(*ids.shape, table.shape[1], dtype=F64, device=table.device)
    out[here] = table.to(F64)[r[here]] * scale
    return out


def embedding_backward(grad: torch.Tensor, ids: torch.Tensor, rows: int, scale: float = 1.0, first: int = 0, magnitudes: bool = False) -> torch.Tensor:
    r = ids.long().reshape(-1) - first
    t = torch.nonzero((r >= 0) & (r < rows)).view(-1)
    g = grad.reshape(-1, grad.shape[-1]).to(F64)[t]
    out = torch.zeros(rows, grad.shape[-1], dtype=F64, device=grad.device)
    return out.index_add_(0, r[t], g.abs() if magnitudes else g) * scale


def norm(tensors) -> torch.Tensor:
    """The root of the sum of squares; squares of fp32 values fit 64 bits."""
    return sum((t.to(F64).square().sum() for t in tensors), torch.zeros((), dtype=F64)).sqrt()


def clip(tensors, limit: float, whole=None):
    n = norm(tensors) if whole is None else torch.as_tensor(whole, dtype=F64)
    f = limit / (n + 1e-6)
    f = torch.ones_like(f) if limit == float("inf") else torch.where(f >= 1, torch.ones_like(f), f)
    return [t.to(F64) * f.to(t.device) for t in tensors]
