"""The expert layer over resharded weights: the calls of include/reshard_ops.h on torch tensors.

Routing to experts and its gradient, quantization to 8-bit floating point in blocks of 128, the matrix product over
such blocks, and the routed expert feed-forward. A refit leaves a generation rank with FP8 weights and their fp32 block
scales (``reshard_plan_blockwise_fp8``), or with BF16 weights that ``reshard_quantize_blocks`` brings to that form;
these calls compute with them.

Argument marshalling only, as in ``binding``: the checks on values are the library's, which lists every violation.
Outputs are allocated unless given (``out``). Work is enqueued on ``stream`` (a cudaStream_t as int, or a
``torch.cuda.Stream``; the current stream if None) and is asynchronous. What a call allocates belongs to that stream; an
input made on another stream must be ready there (an event), as for any torch operation.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .binding import LIB, ReshardError, RESHARD_ERR_INVALID_ARG, _check

RESHARD_SCORE_SOFTMAX = 0
RESHARD_SCORE_SIGMOID = 1
SCORES = {"softmax": RESHARD_SCORE_SOFTMAX, "sigmoid": RESHARD_SCORE_SIGMOID}
OPS_EXPORTED = ("reshard_route", "reshard_route_backward", "reshard_dispatch", "reshard_quantize_rows", "reshard_quantize_blocks",
                "reshard_matmul_fp8", "reshard_linear_fp8_workspace", "reshard_linear_fp8", "reshard_experts_fp8_workspace",
                "reshard_experts_fp8", "reshard_ops_status")
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
    "reshard_ops_status": [_p, _i],
}
for _name, _args in _SIGNATURES.items():
    getattr(LIB, _name).argtypes = _args
    getattr(LIB, _name).restype = _l if _name.endswith("_workspace") else _i


def _bad(what: str) -> None:
    raise ReshardError(RESHARD_ERR_INVALID_ARG, what)


def _code(t: torch.Tensor, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        _bad(f"{name} must be bfloat16, float16 or float32, not {t.dtype}")
    return code


def _want(t: torch.Tensor, name: str, dim: int, dtype: Optional[torch.dtype] = None, dense: bool = False,
          shape: Optional[tuple] = None, device: Optional[torch.device] = None) -> None:
    """What ctypes cannot see: dimensions, type, layout and device of a tensor."""
    if t.dim() != dim:
        _bad(f"{name} must have {dim} dimensions, not {t.dim()}")
    if dtype is not None and t.dtype != dtype:
        _bad(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and tuple(t.shape) != shape:
        _bad(f"{name} must have shape {shape}, not {tuple(t.shape)}")
    if device is not None and t.device != device:
        _bad(f"{name} is on {t.device}, not on {device}")
    if dense:
        if not t.is_contiguous():
            _bad(f"{name} must be contiguous")
    elif t.shape[-1] > 1 and t.stride(-1) != 1:
        _bad(f"{name} must have contiguous rows")


def _row_stride(t: torch.Tensor) -> int:
    """The distance of t's rows; that of a single row (or column) may be anything."""
    return t.stride(-2) if t.shape[-2] > 1 else max(t.stride(-2), t.shape[-1])


class _On:
    """The device and stream of a call: enters them only where they are not the current ones."""

    def __init__(self, t: torch.Tensor, stream):
        if not t.is_cuda:
            _bad(f"tensors must be on a CUDA device, not on {t.device}")
        self.device = t.device
        self.enter = []
        if t.device.index != torch.cuda.current_device():
            self.enter.append(torch.cuda.device(t.device))
        if stream is None:
            self.stream = torch._C._cuda_getCurrentRawStream(t.device.index)
        else:
            self.stream = stream if isinstance(stream, int) else stream.cuda_stream
            if self.stream != torch._C._cuda_getCurrentRawStream(t.device.index):
                self.enter.append(torch.cuda.stream(torch.cuda.ExternalStream(self.stream, device=t.device)))

    def __enter__(self):
        for e in self.enter:
            e.__enter__()
        return self

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
    is never chosen: missing choices have id -1 and weight 0."""
    _want(logits, "logits", 2)
    T, E = logits.shape
    with _On(logits, stream) as on:
        if bias is not None:
            _want(bias, "bias", 1, torch.float32, True, (E,), on.device)
        weights = torch.empty((T, max(0, k)), dtype=torch.float32, device=on.device)
        ids = torch.empty((T, max(0, k)), dtype=torch.int32, device=on.device)
        _check(LIB.reshard_route(logits.data_ptr(), _code(logits, "logits"), T, E, _row_stride(logits),
                                 None if bias is None else bias.data_ptr(), _score(score), groups, groups_kept, group_top, k,
                                 renormalize, scale, weights.data_ptr(), ids.data_ptr(), on.stream))
    return weights, ids


def reshard_route_backward(grad_weights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, *, score="softmax",
                           renormalize: bool = True, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """The gradient to ``logits`` of ``reshard_route``'s weights, the choice ``ids`` held fixed, in the logits' type."""
    _want(logits, "logits", 2)
    _want(ids, "ids", 2, torch.int32, True)
    T, E = logits.shape
    k = ids.shape[1]
    with _On(logits, stream) as on:
        _want(ids, "ids", 2, shape=(T, k), device=on.device, dense=True)
        _want(grad_weights, "grad_weights", 2, torch.float32, True, (T, k), on.device)
        if out is None:
            out = torch.empty((T, E), dtype=logits.dtype, device=on.device)
        else:
            _want(out, "out", 2, logits.dtype, False, (T, E), on.device)
        _check(LIB.reshard_route_backward(grad_weights.data_ptr(), logits.data_ptr(), _code(logits, "logits"), T, E,
                                          _row_stride(logits), ids.data_ptr(), k, _score(score), renormalize, scale,
                                          out.data_ptr(), _row_stride(out), on.stream))
    return out


def reshard_dispatch(ids: torch.Tensor, experts: int, first_expert: int = 0, stream=None) -> Tuple[torch.Tensor, ...]:
    """(offsets [experts + 1], order [slots], position [slots]) int32: the slots (flat indices of ``ids``) sorted by expert, for
    experts first_expert .. first_expert + experts - 1. Expert e's slots are order[offsets[e]:offsets[e + 1]], ascending;
    position is a slot's place in order, -1 for an id outside the range."""
    _want(ids, "ids", ids.dim(), torch.int32, True)
    n = ids.numel()
    with _On(ids, stream) as on:
        offsets = torch.empty(max(0, experts) + 1, dtype=torch.int32, device=on.device)
        order = torch.empty(n, dtype=torch.int32, device=on.device)
        position = torch.empty(n, dtype=torch.int32, device=on.device)
        _check(LIB.reshard_dispatch(ids.data_ptr(), n, first_expert, experts, offsets.data_ptr(), order.data_ptr(),
                                    position.data_ptr(), on.stream))
    return offsets, order, position


def _pitched(shape, device) -> torch.Tensor:
    """Bytes whose rows start every multiple of 16, as the products read them."""
    cols = shape[-1]
    pitch = -(-cols // 16) * 16
    t = torch.empty((*shape[:-1], pitch), dtype=_FP8, device=device)
    return t if pitch == cols else t[..., :cols]


def reshard_quantize_rows(x: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(values [rows, cols] float8_e4m3fn, scale [rows, ceil(cols / 128)] float32) of x [rows, cols] in blocks of 1 x 128.

    The values' rows start every multiple of 16 bytes; the scales are stored block by block (a transposed view)."""
    _want(x, "x", 2)
    M, K = x.shape
    with _On(x, stream) as on:
        q = _pitched((M, K), on.device)
        scale = torch.empty((-(-K // 128), M), dtype=torch.float32, device=on.device)
        _check(LIB.reshard_quantize_rows(x.data_ptr(), _code(x, "x"), M, K, _row_stride(x), q.data_ptr(), q.stride(0),
                                         scale.data_ptr(), 1, max(1, M), on.stream))
    return q, scale.t()


def reshard_quantize_blocks(w: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(values float8_e4m3fn, scale float32) of w [rows, cols] or [batch, rows, cols] in blocks of 128 x 128: the scale has the
    last two extents divided by 128, rounded up, the layout that ``reshard_plan_blockwise_fp8`` moves."""
    if w.dim() not in (2, 3):
        _bad(f"w must have 2 or 3 dimensions, not {w.dim()}")
    _want(w, "w", w.dim())
    N, K = w.shape[-2:]
    E = w.shape[0] if w.dim() == 3 else 1
    with _On(w, stream) as on:
        q = _pitched(tuple(w.shape), on.device)
        scale = torch.empty((*w.shape[:-2], -(-N // 128), -(-K // 128)), dtype=torch.float32, device=on.device)
        _check(LIB.reshard_quantize_blocks(w.data_ptr(), _code(w, "w"), E, N, K, w.stride(0) if w.dim() == 3 else 0,
                                           _row_stride(w), q.data_ptr(), q.stride(0) if w.dim() == 3 else 0, q.stride(-2),
                                           scale.data_ptr(), on.stream))
    return q, scale


def _weights(w: torch.Tensor, scale: torch.Tensor, name: str, dim: int, device) -> None:
    _want(w, name, dim, None, False, None, device)
    if w.dtype not in (_FP8, torch.uint8):
        _bad(f"{name} must be float8_e4m3fn (or its bytes as uint8), not {w.dtype}")
    N, K = w.shape[-2:]
    _want(scale, f"{name}'s scale", dim, torch.float32, True, (*w.shape[:-2], -(-N // 128), -(-K // 128)), device)


def reshard_matmul_fp8(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, *,
                       offsets: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                       out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out [m, n] = a [m, k] w^T over values quantized by rows (``a``) and by blocks (``w``).

    ``w`` is [n, k], or [groups, n, k] with ``offsets`` [groups + 1] int32 (on the device): rows offsets[g]:offsets[g + 1] of
    ``a`` meet w[g], rows beyond the last offset are left as they are in ``out``. float8 values may also come as the
    uint8 bytes that a reshard moved."""
    _want(a, "a", 2)
    if a.dtype not in (_FP8, torch.uint8):
        _bad(f"a must be float8_e4m3fn (or its bytes as uint8), not {a.dtype}")
    M, K = a.shape
    with _On(a, stream) as on:
        _weights(w, w_scale, "w", 2 if offsets is None else 3, on.device)
        N = w.shape[-2]
        if w.shape[-1] != K:
            _bad(f"a has {K} columns, w {w.shape[-1]}")
        groups = w.shape[0] if offsets is not None else 1
        if offsets is not None:
            _want(offsets, "offsets", 1, torch.int32, True, (groups + 1,), on.device)
        if a_scale.dtype != torch.float32 or tuple(a_scale.shape) != (M, -(-K // 128)) or a_scale.device != on.device:
            _bad(f"a_scale must be float32 [{M}, {-(-K // 128)}] on {on.device}")
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype, device=on.device)
        else:
            _want(out, "out", 2, None, False, (M, N), on.device)
        _check(LIB.reshard_matmul_fp8(a.data_ptr(), _row_stride(a) if M > 1 else -(-max(K, a.stride(0)) // 16) * 16,
                                      a_scale.data_ptr(), max(1, a_scale.stride(0)), max(1, a_scale.stride(1)), w.data_ptr(),
                                      w.stride(0) if offsets is not None else 0, _pitch_of(w), w_scale.data_ptr(),
                                      None if offsets is None else offsets.data_ptr(), groups, M, N, K, out.data_ptr(),
                                      _code(out, "out"), _row_stride(out), on.stream))
    return out


def _pitch_of(w: torch.Tensor) -> int:
    """The row pitch of weights; one row has none of its own, and takes the next multiple of 16."""
    return w.stride(-2) if w.shape[-2] > 1 else -(-w.shape[-1] // 16) * 16


def reshard_linear_fp8(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """out [m, n] = Q(x) w^T in x's type: x [m, k] is quantized by rows, ``w`` [n, k] holds 8-bit values and block scales."""
    _want(x, "x", 2)
    M, K = x.shape
    with _On(x, stream) as on:
        _weights(w, w_scale, "w", 2, on.device)
        N = w.shape[0]
        if w.shape[1] != K:
            _bad(f"x has {K} columns, w {w.shape[1]}")
        if out is None:
            out = torch.empty((M, N), dtype=x.dtype, device=on.device)
        else:
            _want(out, "out", 2, x.dtype, False, (M, N), on.device)
        need = LIB.reshard_linear_fp8_workspace(M, K)
        space = torch.empty(need, dtype=torch.uint8, device=on.device)
        _check(LIB.reshard_linear_fp8(x.data_ptr(), _code(x, "x"), M, K, _row_stride(x), w.data_ptr(), _pitch_of(w), w_scale.data_ptr(),
                                      N, out.data_ptr(), _row_stride(out), space.data_ptr(), need, on.stream))
    return out


def reshard_experts_fp8(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w13: torch.Tensor, w13_scale: torch.Tensor,
                        w2: torch.Tensor, w2_scale: torch.Tensor, *, first_expert: int = 0, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] W2[e] Q(silu(g) * u), [g; u] = W13[e] Q(x[t]), e = ids[t, j] - first_expert.

    x [tokens, hidden]; ids int32 and weights float32 [tokens, k] (``reshard_route``); w13 [experts, 2 ffn, hidden] (gate rows,
    then up rows) and w2 [experts, hidden, ffn] with their block scales; ffn a multiple of 128. Ids outside this
    rank's experts first_expert .. first_expert + experts - 1 add nothing."""
    _want(x, "x", 2)
    T, H = x.shape
    with _On(x, stream) as on:
        _want(ids, "ids", 2, torch.int32, True, None, on.device)
        k = ids.shape[1]
        if ids.shape[0] != T:
            _bad(f"ids must have {T} rows, not {ids.shape[0]}")
        _want(weights, "weights", 2, torch.float32, True, (T, k), on.device)
        _weights(w13, w13_scale, "w13", 3, on.device)
        _weights(w2, w2_scale, "w2", 3, on.device)
        E, I = w2.shape[0], w2.shape[2]
        if tuple(w13.shape) != (E, 2 * I, H) or w2.shape[1] != H:
            _bad(f"w13 {tuple(w13.shape)} and w2 {tuple(w2.shape)} do not fit x with {H} columns: [experts, 2 ffn, hidden] and "
                 "[experts, hidden, ffn]")
        if out is None:
            out = torch.empty((T, H), dtype=x.dtype, device=on.device)
        else:
            _want(out, "out", 2, x.dtype, False, (T, H), on.device)
        code = _code(x, "x")
        need = LIB.reshard_experts_fp8_workspace(T, k, E, H, I, code)
        space = torch.empty(need, dtype=torch.uint8, device=on.device)
        _check(LIB.reshard_experts_fp8(x.data_ptr(), code, T, H, _row_stride(x), ids.data_ptr(), weights.data_ptr(), k, first_expert, E, I,
                                       w13.data_ptr(), w13.stride(0), _pitch_of(w13), w13_scale.data_ptr(), w2.data_ptr(),
                                       w2.stride(0), _pitch_of(w2), w2_scale.data_ptr(), out.data_ptr(), _row_stride(out),
                                       space.data_ptr(), need, on.stream))
    return out


def reshard_ops_status(reset: bool = False) -> int:
    """The product kernels' status word on the current device (0 = fine); synchronizes the device."""
    st = ctypes.c_int32()
    _check(LIB.reshard_ops_status(ctypes.byref(st), 1 if reset else 0))
    return int(st.value)
