"""The expert layer over resharded weights: the calls of include/reshard_ops.h on torch tensors.

Routing to experts and its gradient, quantization to 8-bit floating point in blocks of 128, the matrix product over
such blocks, and the routed expert feed-forward. A refit leaves a generation rank with FP8 weights and their fp32 block
scales (``reshard_plan_blockwise_fp8``), or with BF16 weights that ``reshard_quantize_blocks`` brings to that form;
these calls compute with them.

Argument marshalling only, as in ``binding``: the checks on values are the library's, which lists every violation.
Outputs are allocated unless given (``out``). Work is enqueued on ``stream`` (a cudaStream_t as int, or a
``torch.cuda.Stream``; the current stream if None) and is asynchronous. What a call allocates belongs to that stream; an
input made on another stream must be ready there (an event), as for any torch operation.

A wait inside a product kernel that gives up (it does not on a working GPU) leaves an incomplete output and a status that no call
looks at: ``reshard_ops_status`` reads it.

Gradients: ``reshard_route``'s weights carry the gradient to its logits (``reshard_route_backward``). ``reshard_linear_fp8`` and
``reshard_experts_fp8`` have none: of an input that requires one, their result raises when a gradient is asked of it. Codes and
scales (the quantizations, ``reshard_matmul_fp8`` over them) carry none.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache
from struct import Struct
from typing import Optional, Tuple

import torch

from .binding import LIB, ReshardError, RESHARD_ERR_INVALID_ARG, RESHARD_ERR_UNSUPPORTED, _check, reshard_last_error

RESHARD_SCORE_SOFTMAX = 0
RESHARD_SCORE_SIGMOID = 1
SCORES = {"softmax": RESHARD_SCORE_SOFTMAX, "sigmoid": RESHARD_SCORE_SIGMOID}
OPS_EXPORTED = ("reshard_route", "reshard_route_backward", "reshard_dispatch", "reshard_quantize_rows", "reshard_quantize_blocks",
                "reshard_matmul_fp8", "reshard_linear_fp8_workspace", "reshard_linear_fp8", "reshard_experts_fp8_workspace",
                "reshard_experts_fp8", "reshard_ops_call", "reshard_ops_status")
_CODES = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}   # RESHARD_BF16, RESHARD_F16, RESHARD_F32
_FP8 = torch.float8_e4m3fn

_i, _l, _p, _f = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
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
    return out, _matrix(out, "out")[2]


# Workspace sizes by sizes: asking the library each time costs a call.
_linear_space = lru_cache(maxsize=4096)(LIB.reshard_linear_fp8_workspace)
_experts_space = lru_cache(maxsize=4096)(LIB.reshard_experts_fp8_workspace)


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


def reshard_ops_status(reset: bool = False) -> int:
    """The product kernels' status word on the current device (0 = fine); synchronizes the device."""
    st = ctypes.c_int32()
    _check(LIB.reshard_ops_status(ctypes.byref(st), 1 if reset else 0))
    return int(st.value)
