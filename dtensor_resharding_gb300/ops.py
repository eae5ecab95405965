"""The expert layer over resharded weights: the calls of include/reshard_ops.h on torch tensors.

Routing to experts and its gradient, quantization to 8-bit floating point in blocks of 128, the matrix product over
such blocks, and the routed expert feed-forward; tokens to their experts and back and the rows of a vocabulary's shard, with
their gradients, and the norm and clipping of many gradients. A refit leaves a generation rank with FP8 weights and their fp32 block
scales (``reshard_plan_blockwise_fp8``), or with BF16 weights that ``reshard_quantize_blocks`` brings to that form;
these calls compute with them.

Argument marshalling only, as in ``binding``: the checks on values are the library's, which lists every violation.
Outputs are allocated unless given (``out``, written in place as far as autograd knows). Work is enqueued on ``stream`` (a cudaStream_t as int, or a
``torch.cuda.Stream``; the current stream if None) and is asynchronous. What a call allocates belongs to that stream; an
input made on another stream must be ready there (an event), as for any torch operation.

A wait inside a product kernel that gives up (it does not on a working GPU) leaves an incomplete output and a status that no call
looks at: ``reshard_ops_status`` reads it.

Gradients: ``reshard_route``'s weights carry the gradient to its logits (``reshard_route_backward``); ``reshard_permute``,
``reshard_combine`` and ``reshard_embedding`` carry theirs, which are also calls of their own. ``reshard_linear_fp8``,
``reshard_experts_fp8``, ``reshard_grad_norm`` and the gradients' own calls have none (that of ``reshard_permute`` is a
``reshard_combine``): of an input that requires one, their result raises when a gradient is asked of it. Codes and
scales (the quantizations, ``reshard_matmul_fp8`` over them) carry none. In forward mode (``torch.autograd.forward_ad``) there
are no derivatives: an input with a tangent is refused.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache
from struct import Struct
from typing import Iterable, Optional, Tuple, Union

import torch
from torch.autograd import forward_ad as _forward
from torch.autograd.graph import increment_version as _written

from .binding import LIB, ReshardError, RESHARD_ERR_INVALID_ARG, RESHARD_ERR_UNSUPPORTED, _check, reshard_last_error

RESHARD_SCORE_SOFTMAX = 0
RESHARD_SCORE_SIGMOID = 1
SCORES = {"softmax": RESHARD_SCORE_SOFTMAX, "sigmoid": RESHARD_SCORE_SIGMOID}
OPS_EXPORTED = ("reshard_route", "reshard_route_backward", "reshard_dispatch", "reshard_quantize_rows", "reshard_quantize_blocks",
                "reshard_matmul_fp8", "reshard_linear_fp8_workspace", "reshard_linear_fp8", "reshard_experts_fp8_workspace",
                "reshard_experts_fp8", "reshard_permute", "reshard_combine", "reshard_combine_backward", "reshard_embedding",
                "reshard_embedding_backward_workspace", "reshard_embedding_backward", "reshard_tensors_create", "reshard_tensors_destroy",
                "reshard_grad_norm_workspace", "reshard_grad_norm", "reshard_clip_grads", "reshard_ops_call", "reshard_ops_status")
_CODES = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}   # RESHARD_BF16, RESHARD_F16, RESHARD_F32
_FP8 = torch.float8_e4m3fn

_i, _l, _p, _f, _d = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_double
_SIGNATURES = {
    "reshard_route": [_p, _i, _l, _i, _l, _p, _i, _i, _i, _i, _i, _i, _f, _p, _p, _p],
    "reshard_route_backward": [_p, _p, _i, _l, _i, _l, _p, _i, _i, _i, _f, _p, _l, _p],
    "reshard_dispatch": [_p, _l, _i, _i, _p, _p, _p, _p],
    "reshard_quantize_rows": [_p, _i, _l, _l, _l, _p, _l, _p, _l, _l, _p],
    "reshard_quantize_blocks": [_p, _i, _l, _l, _l, _l, _l, _p, _l, _l, _p, _p],
    "reshard_matmul_fp8": [_p, _l, _p, _l, _l, _p, _l, _l, _p, _p, _i, _l, _l, _l, _p, _i, _l, _p],
    "reshard_linear_fp8_workspace": [_l, _l],
    "reshard_linear_fp8": [_p, _i, _l, _l, _l, _p, _l, _p, _l, _p, _l, _p, _l, _p],
    "reshard_experts_fp8_workspace": [_l, _i, _i, _l, _l, _i],
    "reshard_experts_fp8": [_p, _i, _l, _l, _l, _p, _p, _i, _i, _i, _l, _p, _l, _l, _p, _p, _l, _l, _p, _p, _l, _p, _l, _p],
    "reshard_permute": [_p, _i, _l, _l, _l, _p, _p, _i, _p, _l, _l, _i, _p],
    "reshard_combine": [_p, _i, _l, _l, _l, _p, _p, _l, _i, _p, _i, _l, _p],
    "reshard_combine_backward": [_p, _i, _l, _p, _i, _l, _l, _l, _p, _p, _p, _l, _i, _p, _l, _p, _p],
    "reshard_embedding": [_p, _i, _l, _p, _i, _l, _l, _l, _l, _f, _p, _l, _p],
    "reshard_embedding_backward_workspace": [_l, _l],
    "reshard_embedding_backward": [_p, _i, _l, _l, _l, _p, _i, _l, _l, _f, _p, _i, _l, _i, _p, _l, _p],
    "reshard_tensors_create": [_p, _p, _p, _l, _p],
    "reshard_tensors_destroy": [_p],
    "reshard_grad_norm_workspace": [],
    "reshard_grad_norm": [_p, _p, _p, _l, _p],
    "reshard_clip_grads": [_p, _p, _d, _p, _p, _p, _l, _p],
    "reshard_ops_call": [_i, ctypes.c_char_p],
    "reshard_ops_status": [_p, _i],
}
for _name, _args in _SIGNATURES.items():
    getattr(LIB, _name).argtypes = _args
    getattr(LIB, _name).restype = _l if _name.endswith("_workspace") else _i


# The calls' arguments as 64-bit words (reshard_ops_call): packing them takes a third of what ctypes takes for each.
_ROUTE = Struct("=12qd3q").pack
_ROUTE_BACKWARD = Struct("=10qd3q").pack
_DISPATCH = Struct("=8q").pack
_QUANTIZE_ROWS = Struct("=11q").pack
_QUANTIZE_BLOCKS = Struct("=12q").pack
_MATMUL_FP8 = Struct("=18q").pack
_LINEAR_FP8 = Struct("=14q").pack
_EXPERTS_FP8 = Struct("=24q").pack
_PERMUTE = Struct("=13q").pack
_COMBINE = Struct("=13q").pack
_COMBINE_BACKWARD = Struct("=17q").pack
_EMBEDDING = Struct("=9qd3q").pack
_EMBEDDING_BACKWARD = Struct("=9qd7q").pack
_GRAD_NORM = Struct("=5q").pack
_CLIP_GRADS = Struct("=2qd5q").pack


def _call(op: int, words: bytes) -> None:
    rc = LIB.reshard_ops_call(op, words)
    if rc:
        raise ReshardError(rc, reshard_last_error())


def _bad(what: str) -> None:
    raise ReshardError(RESHARD_ERR_INVALID_ARG, what)


# The checks below cover what the C call cannot see (types, shapes, layout and device of a tensor). They are on the path
# of calls that take a few microseconds on the GPU, so each looks at a tensor once.

def _code(t: torch.Tensor, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        _bad(f"{name} must be bfloat16, float16 or float32, not {t.dtype}")
    return code


def _matrix(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """(rows, columns, row stride); a single row's stride may be anything."""
    shape = t.shape
    if len(shape) != 2:
        _bad(f"{name} must have 2 dimensions, not {len(shape)}")
    rows, cols = shape
    step, inner = t.stride()
    if inner != 1 and cols > 1:
        _bad(f"{name} must have contiguous rows")
    return rows, cols, step if rows > 1 or step > cols else cols


def _dense(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, like: torch.Tensor) -> int:
    """The address of a contiguous tensor of that type and shape on `like`'s device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != like.get_device():
        _bad(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {like.device}, not {t.dtype} of shape "
             f"{tuple(t.shape)}, strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _output(out: Optional[torch.Tensor], rows: int, cols: int, dtype: torch.dtype, like: torch.Tensor) -> Tuple[torch.Tensor, int]:
    """(the output, its row stride)"""
    if out is None:
        return torch.empty((rows, cols), dtype=dtype, device=like.device), cols
    if out.dtype is not dtype or out.shape != (rows, cols) or out.get_device() != like.get_device():
        _bad(f"out must be {dtype} of shape {(rows, cols)} on {like.device}, not {out.dtype} of shape {tuple(out.shape)} on {out.device}")
    step = _matrix(out, "out")[2]
    if _forward._current_level >= 0:
        _no_tangent("what is written to out", out)
    _written(out)      # a backward pass that kept what was there is told, as by torch's own operations
    return out, step


# Workspace sizes by sizes: asking the library each time costs a call.
_linear_space = lru_cache(maxsize=4096)(LIB.reshard_linear_fp8_workspace)
_experts_space = lru_cache(maxsize=4096)(LIB.reshard_experts_fp8_workspace)
_embedding_space = lru_cache(maxsize=4096)(LIB.reshard_embedding_backward_workspace)
_norm_space = LIB.reshard_grad_norm_workspace()


def _here(t: torch.Tensor, stream) -> Optional[int]:
    """The raw stream of a call if `t`'s device and that stream are the current ones; None otherwise."""
    if not t.is_cuda:
        _bad(f"tensors must be on a CUDA device, not on {t.device}")
    index = t.get_device()
    if index != torch._C._cuda_getDevice():
        return None
    raw = torch._C._cuda_getCurrentRawStream(index)
    if stream is None or raw == (stream if isinstance(stream, int) else stream.cuda_stream):
        return raw
    return None


class _on:
    """Makes a tensor's device, and a stream, the current ones."""

    def __init__(self, t: torch.Tensor, stream):
        self.enter = [torch.cuda.device(t.device)]
        if stream is not None:
            raw = stream if isinstance(stream, int) else stream.cuda_stream
            self.enter.append(torch.cuda.stream(torch.cuda.ExternalStream(raw, device=t.device)))

    def __enter__(self):
        for e in self.enter:
            e.__enter__()

    def __exit__(self, *exc):
        for e in reversed(self.enter):
            e.__exit__(*exc)


# Forward mode reads a result without a tangent as one that does not depend on its inputs. The calls ask for tangents only
# inside a level of forward mode (the number of the innermost, -1 outside).

def _no_tangent(name: str, *inputs: Optional[torch.Tensor]) -> None:
    if any(t is not None and _forward.unpack_dual(t).tangent is not None for t in inputs):
        raise ReshardError(RESHARD_ERR_UNSUPPORTED, f"{name} has no derivative in forward mode: call it on the primal, or use reverse mode")


def _score(score) -> int:
    if isinstance(score, str):
        if score not in SCORES:
            _bad(f"unknown score function {score!r}")
        return SCORES[score]
    return int(score)


def reshard_route(logits: torch.Tensor, k: int, *, score="softmax", bias: Optional[torch.Tensor] = None, groups: int = 1,
                  groups_kept: int = 1, group_top: int = 1, renormalize: bool = True, scale: float = 1.0,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(weights [tokens, k] float32, ids [tokens, k] int32) of logits [tokens, experts].

    Experts are ordered by score (softmax or sigmoid of the logits) + ``bias``, the lowest index first among equals; with
    ``groups`` only the ``groups_kept`` groups whose ``group_top`` best experts have the largest sum take part. The weights are
    the chosen scores without the bias, divided by their sum if ``renormalize``, times ``scale``. A logit of -inf or NaN
    is never chosen: missing choices have id -1 and weight 0. The weights are differentiable in the logits, the choice and
    the bias that makes it are not."""
    if _forward._current_level >= 0:
        _no_tangent("reshard_route", logits, bias)
    here = _here(logits, stream)
    if here is None:
        with _on(logits, stream):
            return reshard_route(logits, k, score=score, bias=bias, groups=groups, groups_kept=groups_kept, group_top=group_top,
                                 renormalize=renormalize, scale=scale)
    if logits.requires_grad and torch.is_grad_enabled():
        return _Route.apply(logits, k, score, bias, groups, groups_kept, group_top, renormalize, scale)
    T, E, step = _matrix(logits, "logits")
    code = _code(logits, "logits")
    at_bias = 0 if bias is None else _dense(bias, "bias", torch.float32, (E,), logits)
    device = logits.device
    weights = torch.empty((T, max(0, k)), dtype=torch.float32, device=device)
    ids = torch.empty((T, max(0, k)), dtype=torch.int32, device=device)
    _call(0, _ROUTE(logits.data_ptr(), code, T, E, step, at_bias, _score(score), groups, groups_kept, group_top, k,
                    renormalize, scale, weights.data_ptr(), ids.data_ptr(), here))
    return weights, ids


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, score, bias, groups, groups_kept, group_top, renormalize, scale):
        weights, ids = reshard_route(logits.detach(), k, score=score, bias=bias, groups=groups, groups_kept=groups_kept,
                                     group_top=group_top, renormalize=renormalize, scale=scale)
        ctx.save_for_backward(logits, ids)
        ctx.how = dict(score=score, renormalize=renormalize, scale=scale)
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_weights, _):
        logits, ids = ctx.saved_tensors
        return (reshard_route_backward(grad_weights, logits, ids, **ctx.how), *[None] * 8)


class _Undifferentiable(torch.autograd.Function):
    """A call's result that depends on inputs that require a gradient, where the call has none."""

    @staticmethod
    def forward(ctx, name, out, *inputs):
        ctx.name = name
        return out.view_as(out)

    @staticmethod
    def backward(ctx, *grads):
        raise ReshardError(RESHARD_ERR_UNSUPPORTED, f"{ctx.name} has no gradient: call it under torch.no_grad(), or detach its inputs")



def reshard_route_backward(grad_weights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, *, score="softmax",
                           renormalize: bool = True, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """The gradient to ``logits`` of ``reshard_route``'s weights, the choice ``ids`` held fixed, in the logits' type.

    ``grad_weights`` is copied where it is not contiguous (a broadcast gradient)."""
    if _forward._current_level >= 0:
        _no_tangent("reshard_route_backward", grad_weights, logits)
    here = _here(logits, stream)
    if here is None:
        with _on(logits, stream):
            return reshard_route_backward(grad_weights, logits, ids, score=score, renormalize=renormalize, scale=scale, out=out)
    T, E, step = _matrix(logits, "logits")
    code = _code(logits, "logits")
    k = _matrix(ids, "ids")[1]
    at_ids = _dense(ids, "ids", torch.int32, (T, k), logits)
    grad_weights = grad_weights.contiguous()
    at_grad = _dense(grad_weights, "grad_weights", torch.float32, (T, k), logits)
    out, to_step = _output(out, T, E, logits.dtype, logits)
    _call(1, _ROUTE_BACKWARD(at_grad, logits.data_ptr(), code, T, E, step, at_ids, k, _score(score), renormalize, scale,
                             out.data_ptr(), to_step, here))
    if (grad_weights.requires_grad or logits.requires_grad) and torch.is_grad_enabled():
        return _Undifferentiable.apply("reshard_route_backward", out, grad_weights, logits)
    return out


def reshard_dispatch(ids: torch.Tensor, experts: int, first_expert: int = 0, stream=None) -> Tuple[torch.Tensor, ...]:
    """(offsets [experts + 1], order [slots], position [slots]) int32: the slots (flat indices of ``ids``) sorted by expert, for
    experts first_expert .. first_expert + experts - 1. Expert e's slots are order[offsets[e]:offsets[e + 1]], ascending;
    position is a slot's place in order, -1 for an id outside the range. Places from offsets[experts] on are not written."""
    here = _here(ids, stream)
    if here is None:
        with _on(ids, stream):
            return reshard_dispatch(ids, experts, first_expert)
    at_ids = _dense(ids, "ids", torch.int32, ids.shape, ids)
    n, device = ids.numel(), ids.device
    offsets = torch.empty(max(0, experts) + 1, dtype=torch.int32, device=device)
    order = torch.empty(n, dtype=torch.int32, device=device)
    position = torch.empty(n, dtype=torch.int32, device=device)
    _call(2, _DISPATCH(at_ids, n, first_expert, experts, offsets.data_ptr(), order.data_ptr(), position.data_ptr(), here))
    return offsets, order, position


def reshard_quantize_rows(x: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(values [rows, cols] float8_e4m3fn, scale [rows, ceil(cols / 128)] float32) of x [rows, cols] in blocks of 1 x 128.

    The values' rows start every multiple of 16 bytes; the scales are stored block by block (a transposed view)."""
    here = _here(x, stream)
    if here is None:
        with _on(x, stream):
            return reshard_quantize_rows(x)
    M, K, step = _matrix(x, "x")
    code = _code(x, "x")
    device, pitch, rows = x.device, -(-K // 16) * 16, M or 1
    q = torch.empty_strided((M, K), (pitch, 1), dtype=_FP8, device=device)
    scale = torch.empty_strided((M, -(-K // 128)), (1, rows), dtype=torch.float32, device=device)
    _call(3, _QUANTIZE_ROWS(x.data_ptr(), code, M, K, step, q.data_ptr(), pitch, scale.data_ptr(), 1, rows, here))
    return q, scale


def reshard_quantize_blocks(w: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(values float8_e4m3fn, scale float32) of w [rows, cols] or [batch, rows, cols] in blocks of 128 x 128: the scale has the
    last two extents divided by 128, rounded up, the layout that ``reshard_plan_blockwise_fp8`` moves."""
    here = _here(w, stream)
    if here is None:
        with _on(w, stream):
            return reshard_quantize_blocks(w)
    shape, stride = w.shape, w.stride()
    if len(shape) not in (2, 3):
        _bad(f"w must have 2 or 3 dimensions, not {len(shape)}")
    N, K = shape[-2:]
    if K > 1 and stride[-1] != 1:
        _bad("w must have contiguous rows")
    code = _code(w, "w")
    pitch, blocks, device = -(-K // 16) * 16, (-(-N // 128), -(-K // 128)), w.device
    step = stride[-2] if N > 1 or stride[-2] > K else K
    if len(shape) == 3:
        E, batch = shape[0], stride[0]
        q = torch.empty_strided(shape, (N * pitch, pitch, 1), dtype=_FP8, device=device)
        scale = torch.empty((E, *blocks), dtype=torch.float32, device=device)
    else:
        E, batch = 1, 0
        q = torch.empty_strided(shape, (pitch, 1), dtype=_FP8, device=device)
        scale = torch.empty(blocks, dtype=torch.float32, device=device)
    _call(4, _QUANTIZE_BLOCKS(w.data_ptr(), code, E, N, K, batch, step, q.data_ptr(), N * pitch, pitch, scale.data_ptr(), here))
    return q, scale


def _weights(w: torch.Tensor, scale: torch.Tensor, name: str, dim: int, like: torch.Tensor) -> Tuple[int, ...]:
    """(address, batch stride, row stride, scale's address) of 8-bit weights."""
    shape, stride = w.shape, w.stride()
    if len(shape) != dim:
        _bad(f"{name} must have {dim} dimensions, not {len(shape)}")
    if w.dtype is not _FP8 and w.dtype is not torch.uint8:
        _bad(f"{name} must be float8_e4m3fn (or its bytes as uint8), not {w.dtype}")
    N, K = shape[-2:]
    if stride[-1] != 1 and K > 1:
        _bad(f"{name} must have contiguous rows")
    if w.get_device() != like.get_device():
        _bad(f"{name} is on {w.device}, not on {like.device}")
    at_scale = _dense(scale, f"{name}'s scale", torch.float32, (*shape[:-2], -(-N // 128), -(-K // 128)), like)
    # one row has no pitch of its own: the next multiple of 16
    return w.data_ptr(), stride[0] if dim == 3 else 0, stride[-2] if N > 1 else -(-K // 16) * 16, at_scale


def reshard_matmul_fp8(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, *,
                       offsets: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                       out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out [m, n] = a [m, k] w^T over values quantized by rows (``a``) and by blocks (``w``).

    ``w`` is [n, k], or [groups, n, k] with ``offsets`` [groups + 1] int32 (on the device): rows offsets[g]:offsets[g + 1] of
    ``a`` meet w[g], rows beyond the last offset are left as they are in ``out``. float8 values may also come as the
    uint8 bytes that a reshard moved. ``a_scale`` may have any strides: one scale a row or one in all may come expanded."""
    here = _here(a, stream)
    if here is None:
        with _on(a, stream):
            return reshard_matmul_fp8(a, a_scale, w, w_scale, offsets=offsets, out_dtype=out_dtype, out=out)
    M, K, step = _matrix(a, "a")
    if a.dtype is not _FP8 and a.dtype is not torch.uint8:
        _bad(f"a must be float8_e4m3fn (or its bytes as uint8), not {a.dtype}")
    at_w, batch, pitch, at_ws = _weights(w, w_scale, "w", 2 if offsets is None else 3, a)
    N = w.shape[-2]
    if w.shape[-1] != K:
        _bad(f"a has {K} columns, w {w.shape[-1]}")
    groups = 1 if offsets is None else w.shape[0]
    at_offsets = 0 if offsets is None else _dense(offsets, "offsets", torch.int32, (groups + 1,), a)
    if a_scale.dtype is not torch.float32 or a_scale.shape != (M, -(-K // 128)) or a_scale.device != a.device:
        _bad(f"a_scale must be float32 of shape {(M, -(-K // 128))} on {a.device}, not {a_scale.dtype} of shape {tuple(a_scale.shape)}")
    out, to_step = _output(out, M, N, out_dtype if out is None else out.dtype, a)
    _call(5, _MATMUL_FP8(a.data_ptr(), step if M > 1 else -(-step // 16) * 16, a_scale.data_ptr(), *a_scale.stride(), at_w, batch, pitch, at_ws,
                         at_offsets, groups, M, N, K, out.data_ptr(), _code(out, "out"), to_step, here))
    return out


def reshard_linear_fp8(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """out [m, n] = Q(x) w^T in x's type: x [m, k] is quantized by rows, ``w`` [n, k] holds 8-bit values and block scales."""
    if _forward._current_level >= 0:
        _no_tangent("reshard_linear_fp8", x, w_scale)
    here = _here(x, stream)
    if here is None:
        with _on(x, stream):
            return reshard_linear_fp8(x, w, w_scale, out=out)
    M, K, step = _matrix(x, "x")
    code = _code(x, "x")
    at_w, _, pitch, at_ws = _weights(w, w_scale, "w", 2, x)
    N = w.shape[0]
    if w.shape[1] != K:
        _bad(f"x has {K} columns, w {w.shape[1]}")
    out, to_step = _output(out, M, N, x.dtype, x)
    need = _linear_space(M, K)
    space = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    _call(6, _LINEAR_FP8(x.data_ptr(), code, M, K, step, at_w, pitch, at_ws, N, out.data_ptr(), to_step,
                         space.data_ptr() if need else 0, need, here))
    if x.requires_grad and torch.is_grad_enabled():
        return _Undifferentiable.apply("reshard_linear_fp8", out, x)
    return out


def reshard_experts_fp8(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w13: torch.Tensor, w13_scale: torch.Tensor,
                        w2: torch.Tensor, w2_scale: torch.Tensor, *, first_expert: int = 0, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] W2[e] Q(silu(g) * u), [g; u] = W13[e] Q(x[t]), e = ids[t, j] - first_expert.

    x [tokens, hidden]; ids int32 and weights float32 [tokens, k] (``reshard_route``); w13 [experts, 2 ffn, hidden] (gate rows,
    then up rows) and w2 [experts, hidden, ffn] with their block scales; ffn a multiple of 128. Ids outside this
    rank's experts first_expert .. first_expert + experts - 1 add nothing."""
    if _forward._current_level >= 0:
        _no_tangent("reshard_experts_fp8", x, weights, w13_scale, w2_scale)
    here = _here(x, stream)
    if here is None:
        with _on(x, stream):
            return reshard_experts_fp8(x, ids, weights, w13, w13_scale, w2, w2_scale, first_expert=first_expert, out=out)
    T, H, step = _matrix(x, "x")
    code = _code(x, "x")
    k = _matrix(ids, "ids")[1]
    at_ids = _dense(ids, "ids", torch.int32, (T, k), x)
    at_weights = _dense(weights, "weights", torch.float32, (T, k), x)
    at_w13, batch13, pitch13, at_s13 = _weights(w13, w13_scale, "w13", 3, x)
    at_w2, batch2, pitch2, at_s2 = _weights(w2, w2_scale, "w2", 3, x)
    E, _, I = w2.shape
    if w13.shape != (E, 2 * I, H) or w2.shape[1] != H:
        _bad(f"w13 {tuple(w13.shape)} and w2 {tuple(w2.shape)} do not fit x with {H} columns: [experts, 2 ffn, hidden] and "
             "[experts, hidden, ffn]")
    out, to_step = _output(out, T, H, x.dtype, x)
    need = _experts_space(T, k, E, H, I, code)
    space = torch.empty(need, dtype=torch.uint8, device=x.device)
    _call(7, _EXPERTS_FP8(x.data_ptr(), code, T, H, step, at_ids, at_weights, k, first_expert, E, I, at_w13, batch13, pitch13,
                          at_s13, at_w2, batch2, pitch2, at_s2, out.data_ptr(), to_step, space.data_ptr(), need, here))
    if (x.requires_grad or weights.requires_grad) and torch.is_grad_enabled():
        return _Undifferentiable.apply("reshard_experts_fp8", out, x, weights)
    return out


# ------------------------------------------------------------------------------- tokens to their experts and back

Sort = Tuple[torch.Tensor, torch.Tensor, torch.Tensor]


def _sorted(sort: Sort, like: torch.Tensor) -> Tuple[int, int, int, int]:
    """(address of order, its length, address of position, its length) of what reshard_dispatch gave."""
    _, order, position = sort
    device = like.get_device()
    for t, name in ((order, "the sort's order"), (position, "the sort's position")):
        if t.dtype is not torch.int32 or not t.is_contiguous() or t.get_device() != device:
            _dense(t, name, torch.int32, t.shape, like)      # which says what is wrong
    return order.data_ptr(), order.numel(), position.data_ptr(), position.numel()


def _choices(slots: int, tokens: int) -> int:
    """k of a sort of so many slots, of so many tokens."""
    if tokens == 0 and slots == 0:
        return 1
    if tokens == 0 or slots == 0 or slots % tokens:
        _bad(f"a sort of {slots} slots does not fit {tokens} tokens")
    return slots // tokens


def _tokens(sort: Sort, weights: Optional[torch.Tensor], k: Optional[int]) -> Tuple[int, int]:
    """(tokens, k) of a sort, from its weights [tokens, k] or a k given."""
    slots = sort[2].numel()
    if weights is not None:
        tokens, choices, _ = _matrix(weights, "weights")
        if k is not None and k != choices:
            _bad(f"k is {k}, the weights have {choices} columns")
        if tokens * choices != slots:
            _bad(f"weights {tuple(weights.shape)} do not fit a sort of {slots} slots")
        return tokens, max(choices, 1)
    if k is None or k < 1 or slots % k:
        _bad(f"without weights k must be given and divide the sort's {slots} slots")
    return slots // k, k


def _rows(t: torch.Tensor) -> torch.Tensor:
    """A gradient as autograd brings it (expanded, transposed): copied if its rows are not rows of a matrix."""
    return t if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1] else t.contiguous()


def _no_out(out, *inputs) -> None:
    if out is not None and torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs):
        raise ReshardError(RESHARD_ERR_UNSUPPORTED, "a result that carries a gradient cannot be written to out: call under torch.no_grad(), or without out")


def reshard_permute(x: torch.Tensor, sort: Sort, *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y [slots, cols] with y[position[t * k + j]] = x[t]: each token's row at the places of its experts.

    ``sort`` is what ``reshard_dispatch`` gave for these tokens' ids. Rows of no slot (from offsets[-1] on: other ranks' experts') are
    left as they are in ``out``, which may have more or fewer rows than slots, and 0 in a new tensor (all tokens * k rows are
    written then: for a small share of the experts an ``out`` saves most of that). Values are copied bit for bit;
    differentiable in ``x``."""
    if _forward._current_level >= 0:
        _no_tangent("reshard_permute", x)
    here = _here(x, stream)
    if here is None:
        with _on(x, stream):
            return reshard_permute(x, sort, out=out)
    if x.requires_grad and torch.is_grad_enabled():
        _no_out(out, x)
        return _Permute.apply(x, *sort)
    T, H, step = _matrix(x, "x")
    code = _code(x, "x")
    at_order, places, at_position, slots = _sorted(sort, x)
    k = _choices(slots, T)
    rows, zero_rest = (places, 1) if out is None else (out.shape[0], 0)
    out, to_step = _output(out, rows, H, x.dtype, x)
    if rows > places:      # places that the sort does not have are nobody's
        rows = places
    _call(8, _PERMUTE(x.data_ptr(), code, T, H, step, at_order, at_position, k, out.data_ptr(), rows, to_step, zero_rest, here))
    return out


def reshard_permute_backward(grad: torch.Tensor, sort: Sort, k: int, *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient to ``x`` of ``reshard_permute``: each token's sum over its k places, in ``grad``'s type; differentiable in
    ``grad``, as ``reshard_combine`` is."""
    return reshard_combine(grad, sort, k=k, out=out, stream=stream)


class _Permute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, *sort):
        ctx.save_for_backward(*sort)
        ctx.k = _choices(sort[2].numel(), x.shape[0])
        return reshard_permute(x.detach(), sort)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        return (reshard_permute_backward(_rows(grad), ctx.saved_tensors, ctx.k), None, None, None)


def reshard_combine(y: torch.Tensor, sort: Sort, weights: Optional[torch.Tensor] = None, *, k: Optional[int] = None,
                    out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * y[position[t * k + j]]: experts' rows back to their tokens.

    ``weights`` [tokens, k] float32 (``reshard_route``), or None with ``k`` given: plain sums. Slots without a place add nothing.
    ``y`` may have more rows than the sort has places (a padded buffer): those belong to no slot and their gradient is 0. The sum
    is fp32 and rounded once, to ``out_dtype`` (y's type if None). Differentiable in ``y`` and ``weights``."""
    if _forward._current_level >= 0:
        _no_tangent("reshard_combine", y, weights)
    here = _here(y, stream)
    if here is None:
        with _on(y, stream):
            return reshard_combine(y, sort, weights, k=k, out_dtype=out_dtype, out=out)
    if torch.is_grad_enabled() and (y.requires_grad or (weights is not None and weights.requires_grad)):
        _no_out(out, y, weights)
        return _Combine.apply(y, weights, k, out_dtype, *sort)
    rows, H, step = _matrix(y, "y")
    code = _code(y, "y")
    T, k = _tokens(sort, weights, k)
    _, _, at_position, _ = _sorted(sort, y)
    at_weights = 0 if weights is None else _dense(weights, "weights", torch.float32, (T, k), y)
    out, to_step = _output(out, T, H, (out_dtype or y.dtype) if out is None else out.dtype, y)
    _call(9, _COMBINE(y.data_ptr(), code, rows, H, step, at_position, at_weights, T, k, out.data_ptr(), _code(out, "out"), to_step, here))
    return out


def reshard_combine_backward(grad: torch.Tensor, y: torch.Tensor, sort: Sort, weights: Optional[torch.Tensor] = None, *,
                             k: Optional[int] = None, needs: Tuple[bool, bool] = (True, True),
                             stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(grad_y in y's type, grad_weights float32) of ``reshard_combine`` for ``grad`` [tokens, cols].

    Rows of ``y`` that belong to no slot have gradient 0, and so have weights of slots without a place. ``needs``: which of the two
    are wanted (the other is None). Without ``weights`` there is no gradient to them."""
    if _forward._current_level >= 0:
        _no_tangent("reshard_combine_backward", grad, y, weights)
    rows, places = _matrix(y, "y")[0], sort[1].numel()
    if places < rows:
        _bad(f"y has {rows} rows, the sort {places} places")
    grad_y, grad_weights = _combine_gradients(grad, y, (y.shape, y.dtype), sort, weights, k, needs, stream)
    if (grad.requires_grad or y.requires_grad or (weights is not None and weights.requires_grad)) and torch.is_grad_enabled():
        grad_y, grad_weights = (t if t is None else _Undifferentiable.apply("reshard_combine_backward", t, grad, y, weights) for t in (grad_y, grad_weights))
    return grad_y, grad_weights


def _combine_gradients(grad: torch.Tensor, y: Optional[torch.Tensor], like: Tuple[torch.Size, torch.dtype], sort: Sort, weights: Optional[torch.Tensor],
                       k: Optional[int], needs: Tuple[bool, bool], stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(grad_y, grad_weights), the one that is not needed None. Rows of y behind the sort's places are no slot's. `like`: y's shape
    and type; y itself is read for grad_weights only."""
    here = _here(grad, stream)
    if here is None:
        with _on(grad, stream):
            return _combine_gradients(grad, y, like, sort, weights, k, needs)
    grad = _rows(grad)
    T, k = _tokens(sort, weights, k)
    G, H, grad_step = _matrix(grad, "grad")
    (rows, cols), dtype = like
    if (G, H) != (T, cols):
        _bad(f"grad {tuple(grad.shape)} does not fit {T} tokens and y {(rows, cols)}")
    at_y, step = 0, cols
    if y is not None:
        at_y, step = y.data_ptr(), _matrix(y, "y")[2]
        if y.get_device() != grad.get_device():
            _bad(f"y is on {y.device}, not on {grad.device}")
    code = _CODES.get(dtype)
    if code is None:
        _bad(f"y must be bfloat16, float16 or float32, not {dtype}")
    at_order, places, at_position, _ = _sorted(sort, grad)
    at_weights = 0 if weights is None else _dense(weights, "weights", torch.float32, (T, k), grad)
    grad_y = torch.empty((rows, H), dtype=dtype, device=grad.device) if needs[0] else None
    if rows > places:
        if needs[0]:
            grad_y[places:].zero_()
        rows = places
    grad_weights = torch.empty((T, k), dtype=torch.float32, device=grad.device) if needs[1] and weights is not None else None
    _call(10, _COMBINE_BACKWARD(grad.data_ptr(), _code(grad, "grad"), grad_step, at_y, code, rows, H, step, at_order, at_position,
                                at_weights, T, k, 0 if grad_y is None else grad_y.data_ptr(), H,
                                0 if grad_weights is None else grad_weights.data_ptr(), here))
    return grad_y, grad_weights


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, k, out_dtype, *sort):
        # y is kept only for a gradient that reads it: tokens * k rows
        keep = y if weights is not None and ctx.needs_input_grad[1] else None
        ctx.save_for_backward(keep, weights, *sort)
        ctx.k, ctx.like = k, (y.shape, y.dtype)
        return reshard_combine(y.detach(), sort, None if weights is None else weights.detach(), k=k, out_dtype=out_dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        y, weights, *sort = ctx.saved_tensors
        grad_y, grad_weights = _combine_gradients(grad, y, ctx.like, tuple(sort), weights, ctx.k, ctx.needs_input_grad[:2])
        return (grad_y, grad_weights, *[None] * 5)


# ----------------------------------------------------------------------------------------- a shard of a vocabulary

def _id_bits(ids: torch.Tensor, like: torch.Tensor) -> int:
    if ids.dtype is not torch.int64 and ids.dtype is not torch.int32:
        _bad(f"ids must be int64 or int32, not {ids.dtype}")
    if ids.get_device() != like.get_device():
        _bad(f"ids are on {ids.device}, not on {like.device}")
    return 64 if ids.dtype is torch.int64 else 32


def reshard_embedding(ids: torch.Tensor, table: torch.Tensor, *, scale: float = 1.0, first_row: int = 0,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out [*ids.shape, cols] = scale * table[ids - first_row], 0 where the id's row is not in ``table`` (another rank's shard).

    ``ids`` int64 or int32 of any shape (copied where not contiguous), ``table`` [rows, cols] the rows first_row .. first_row +
    rows - 1 of the vocabulary: the shards' results sum to the whole lookup. Differentiable in ``table``."""
    if _forward._current_level >= 0:
        _no_tangent("reshard_embedding", table)
    here = _here(table, stream)
    if here is None:
        with _on(table, stream):
            return reshard_embedding(ids, table, scale=scale, first_row=first_row, out=out)
    if table.requires_grad and torch.is_grad_enabled():
        _no_out(out, table)
        return _Embedding.apply(ids, table, scale, first_row)
    rows, H, step = _matrix(table, "table")
    code, bits = _code(table, "table"), _id_bits(ids, table)
    ids = ids.contiguous()
    T, shape = ids.numel(), ids.shape
    if out is None:
        out = to = torch.empty((*shape, H), dtype=table.dtype, device=table.device)
        to_step = H
    else:
        if out.shape != (*shape, H):
            _bad(f"out must be of shape {(*shape, H)}, not {tuple(out.shape)}")
        if len(shape) != 1 and not out.is_contiguous():
            _bad("out must be contiguous for ids of more than one dimension")
        to, to_step = _output(out if len(shape) == 1 else out.view(T, H), T, H, table.dtype, table)
    _call(11, _EMBEDDING(ids.data_ptr(), bits, T, table.data_ptr(), code, first_row, rows, H, step, scale, to.data_ptr(), to_step, here))
    return out


def reshard_embedding_backward(grad: torch.Tensor, ids: torch.Tensor, rows: int, *, scale: float = 1.0, first_row: int = 0,
                               dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None, accumulate: bool = False,
                               stream=None) -> torch.Tensor:
    """The gradient [rows, cols] to ``reshard_embedding``'s table: scale * the sum of ``grad`` over each row's tokens.

    Sums are fp32, rounded once to ``dtype`` (``grad``'s if None): runs of a row's tokens in their order, then the runs; the same
    ids, columns and types give the same bits (tokens of other rows can regroup a row's). Rows without a token get 0; with
    ``accumulate`` the sums are added to ``out`` instead (a main gradient of a training step), and other rows not touched."""
    if _forward._current_level >= 0:
        _no_tangent("reshard_embedding_backward", grad, out if accumulate else None)
    here = _here(grad, stream)
    if here is None:
        with _on(grad, stream):
            return reshard_embedding_backward(grad, ids, rows, scale=scale, first_row=first_row, dtype=dtype, out=out, accumulate=accumulate)
    if grad.shape[:-1] != ids.shape:
        _bad(f"grad {tuple(grad.shape)} does not fit ids {tuple(ids.shape)}")
    bits, ids = _id_bits(ids, grad), ids.contiguous()
    grad = _rows(grad if grad.dim() == 2 else grad.reshape(ids.numel(), grad.shape[-1]))
    T, H, step = _matrix(grad, "grad")
    if accumulate and out is None:
        _bad("accumulate needs out")
    out, to_step = _output(out, max(0, rows), H, (dtype or grad.dtype) if out is None else out.dtype, grad)
    need = _embedding_space(T, H)
    space = torch.empty(need, dtype=torch.uint8, device=grad.device) if need else None
    _call(12, _EMBEDDING_BACKWARD(grad.data_ptr(), _code(grad, "grad"), T, H, step, ids.data_ptr(), bits, first_row, rows, scale, out.data_ptr(),
                                  _code(out, "out"), to_step, accumulate, space.data_ptr() if need else 0, need, here))
    if grad.requires_grad and torch.is_grad_enabled():
        return _Undifferentiable.apply("reshard_embedding_backward", out, grad)
    return out


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale, first_row):
        ctx.save_for_backward(ids)
        ctx.how = dict(rows=table.shape[0], scale=scale, first_row=first_row, dtype=table.dtype)
        return reshard_embedding(ids, table.detach(), scale=scale, first_row=first_row)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        return (None, reshard_embedding_backward(grad, ctx.saved_tensors[0], **ctx.how), None, None)


# ------------------------------------------------------------------------------------------ many tensors' norm and clipping

def _packed(t: torch.Tensor) -> bool:
    """Whether the tensor's elements fill its storage from the first to the last, in some order of its dimensions."""
    expect = 1
    for step, size in sorted(zip(t.stride(), t.shape)):
        if size > 1:
            if step != expect:
                return False
            expect *= size
    return True


class TensorList:
    """Dense tensors of one device for ``reshard_grad_norm`` and ``reshard_clip_grads``, looked over once: for tensors that
    stay where they are from step to step (``zero_grad(set_to_none=False)``). The list keeps them and their memory alive, and
    goes on with that memory where a tensor is given other (``t.data = ...``) or a parameter another gradient: then make a new
    list. Storages that are resized in place must not be in one."""

    is_cuda = True

    def __init__(self, tensors: Iterable[torch.Tensor]):
        self._handle = None
        self.tensors = tensors = list(tensors)
        at, sizes, types, self._order, self._memory, self._wanting = [], [], [], {}, [], []
        self.device = device = tensors[0].device if tensors else torch.device("cuda", torch.cuda.current_device())
        if device.type != "cuda":
            _bad(f"tensors must be on a CUDA device, not on {device}")
        for i, t in enumerate(tensors):
            if t.layout is not torch.strided:
                _bad(f"tensor {i} is not strided but {t.layout}")
            if t.device != device:
                _bad(f"tensor {i} is on {t.device}, the first on {device}")
            if not t.is_contiguous():
                if not _packed(t):
                    _bad(f"tensor {i} of shape {tuple(t.shape)}, strides {t.stride()} is not dense")
                self._order[i] = (t.shape, t.stride())
            at.append(t.data_ptr())
            self._memory.append(t.untyped_storage())      # what the addresses are of, whatever the tensor is given later
            if t.requires_grad:
                self._wanting.append(t)
            sizes.append(t.numel())
            types.append(_code(t, "a tensor"))
        n, handle = len(tensors), ctypes.c_void_p()
        with torch.cuda.device(device):
            _check(LIB.reshard_tensors_create((ctypes.c_void_p * n)(*at), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*types), n, ctypes.byref(handle)))
        self._handle = handle.value

    def __reduce__(self):
        """A copy, deep copy or pickle is a list of its own: the library's list is freed with the object that made it."""
        return type(self), (self.tensors,)

    def get_device(self) -> int:
        return self.device.index

    def __len__(self) -> int:
        return len(self.tensors)

    def __del__(self):
        if getattr(self, "_handle", None) is not None and LIB is not None:      # (None while the interpreter ends)
            LIB.reshard_tensors_destroy(self._handle)


def reshard_tensor_list(tensors: Iterable[torch.Tensor]) -> TensorList:
    """A list of tensors for the calls below (bfloat16, float16 and float32, mixed as they come; dense in any order of dimensions).
    Making one looks at each tensor (10,000: some 9 ms), so lists that are used again are worth keeping."""
    return TensorList(tensors)


Tensors = Union[TensorList, Iterable[torch.Tensor]]


def reshard_grad_norm(tensors: Tensors, *, stream=None) -> torch.Tensor:
    """The norm sqrt(sum x^2) over all elements of ``tensors`` (a ``TensorList`` or tensors), a float32 scalar on their device.

    Other ranks' shards: the root of the sum of their norms' squares is the whole norm. It has no gradient: of tensors that
    require one (when their list is made) the result raises when it is asked for, outside ``torch.no_grad()``."""
    if not isinstance(tensors, TensorList):
        tensors = TensorList(tensors)
    if _forward._current_level >= 0:
        _no_tangent("reshard_grad_norm", *tensors.tensors)
    here = _here(tensors, stream)
    if here is None:
        with _on(tensors, stream):
            return reshard_grad_norm(tensors)
    norm = torch.empty((), dtype=torch.float32, device=tensors.device)
    space = torch.empty(_norm_space, dtype=torch.uint8, device=tensors.device)
    _call(13, _GRAD_NORM(tensors._handle, norm.data_ptr(), space.data_ptr(), _norm_space, here))
    if tensors._wanting and torch.is_grad_enabled():
        return _Undifferentiable.apply("reshard_grad_norm", norm, *tensors._wanting)
    return norm


def reshard_clip_grads(tensors: Tensors, limit: float, *, norm: Optional[torch.Tensor] = None, out: Optional[Tensors] = None,
                       stream=None) -> torch.Tensor:
    """Scales ``tensors`` by min(1, limit / (norm + 1e-6)), in place or into ``out`` (other types are fine); returns the norm.

    ``norm``: a float32 scalar on the device (the norm over all ranks), or None: ``reshard_grad_norm`` of the tensors. Nothing is
    read back: a step with a NaN norm makes every value NaN, one with an infinite norm 0 (see include/reshard_ops.h). As with
    any write through a pointer, autograd is not told: neither what is written nor the norm carries a gradient."""
    if not isinstance(tensors, TensorList):
        tensors = TensorList(tensors)
    if out is not None and not isinstance(out, TensorList):
        out = TensorList(out)
    if _forward._current_level >= 0:
        _no_tangent("reshard_clip_grads", *tensors.tensors, norm, *(() if out is None else out.tensors))
    here = _here(tensors, stream)
    if here is None:
        with _on(tensors, stream):
            return reshard_clip_grads(tensors, limit, norm=norm, out=out)
    into = 0
    if out is not None:
        if len(out) != len(tensors) or out.device != tensors.device:
            _bad(f"out has {len(out)} tensors on {out.device}, not {len(tensors)} on {tensors.device}")
        if out._order != tensors._order:
            _bad("a tensor of out has another order of dimensions than its source")
        into = out._handle
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=tensors.device)
        space = torch.empty(_norm_space, dtype=torch.uint8, device=tensors.device)
        _call(14, _CLIP_GRADS(tensors._handle, into, limit, 0, norm.data_ptr(), space.data_ptr(), _norm_space, here))
    else:
        if norm.dtype is not torch.float32 or norm.numel() != 1 or norm.device != tensors.device:
            _bad(f"norm must be one float32 on {tensors.device}, not {norm.dtype} of shape {tuple(norm.shape)} on {norm.device}")
        _call(14, _CLIP_GRADS(tensors._handle, into, limit, norm.data_ptr(), 0, 0, 0, here))
    return norm


def reshard_ops_status(reset: bool = False) -> int:
    """The product kernels' status word on the current device (0 = fine); synchronizes the device."""
    st = ctypes.c_int32()
    _check(LIB.reshard_ops_status(ctypes.byref(st), 1 if reset else 0))
    return int(st.value)
