"""GB300-native DTensor -> DTensor reshard executor (single GPU, sm_103a).

The public calls mirror the C ABI in include/reshard.h:
``reshard_plan_create``, ``reshard_plan_batch``, ``reshard_execute``, ``reshard_execute_pack`` /
``reshard_execute_unpack``, ``reshard_plan_partition`` / ``reshard_plan_transfers`` (the multi-process
exchange, driven by ``exchange``), ``reshard_plan_stats``, ``reshard_plan_regions``,
``reshard_plan_group_members``, ``reshard_plan_destroy``, ``reshard_last_error``. Importing the
package loads libreshard.so and raises if it is not built.

The expert layer over resharded weights (``ops``, include/reshard_ops.h) takes torch tensors: ``reshard_route`` /
``reshard_route_backward``, ``reshard_dispatch``, ``reshard_quantize_rows`` / ``reshard_quantize_blocks``,
``reshard_matmul_fp8``, ``reshard_linear_fp8``, ``reshard_experts_fp8``, ``reshard_ops_status``; around it, for training,
``reshard_permute`` / ``reshard_combine`` (tokens to their experts and back), ``reshard_embedding`` (a vocabulary's shard), their
``_backward`` calls, and ``reshard_grad_norm`` / ``reshard_clip_grads`` over a ``reshard_tensor_list``. It is imported (and torch
with it) at the first use of one of its names.
"""
from .binding import (  # noqa: F401
    Plan, ReshardError, Spec, View, LIB_PATH, EXPORTED, STATS_FIELDS, pointer_array,
    reshard_plan_create, reshard_plan_batch, reshard_plan_blockwise_fp8, reshard_execute, reshard_execute_pack, reshard_execute_unpack,
    reshard_plan_partition, reshard_plan_transfers, reshard_execute_static, reshard_plan_stats, reshard_plan_regions,
    reshard_plan_group_members, reshard_plan_items, reshard_plan_slabs, reshard_plan_status,
    reshard_plan_destroy, reshard_last_error, make_spec,
    RESHARD_OK, RESHARD_ERR_INVALID_ARG, RESHARD_ERR_UNSUPPORTED, RESHARD_ERR_CUDA, RESHARD_ERR_OOM,
    RESHARD_ERR_COVERAGE, RESHARD_DIRECT, RESHARD_PACKED, RESHARD_QUANT_NONE, RESHARD_QUANT_MXFP8,
    RESHARD_STRIPED, RESHARD_SEND, RESHARD_RECV, RESHARD_SEND_BUF, RESHARD_RECV_BUF,
)
from .workload import plan_workload, workload_pointers  # noqa: F401

_OPS = ("reshard_route", "reshard_route_backward", "reshard_dispatch", "reshard_quantize_rows", "reshard_quantize_blocks",
        "reshard_matmul_fp8", "reshard_linear_fp8", "reshard_experts_fp8", "reshard_permute", "reshard_permute_backward", "reshard_combine",
        "reshard_combine_backward", "reshard_embedding", "reshard_embedding_backward", "reshard_tensor_list", "TensorList",
        "reshard_grad_norm", "reshard_clip_grads", "reshard_ops_status",
        "RESHARD_SCORE_SOFTMAX", "RESHARD_SCORE_SIGMOID")


def __getattr__(name):
    if name in _OPS:
        from . import ops
        globals().update({n: getattr(ops, n) for n in _OPS})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted([*globals(), *_OPS])
