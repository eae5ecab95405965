"""The expert layer without a GPU: the calls' refusals, and the 64-bit oracle against other definitions of the same things."""
import ctypes
import os
import re

import pytest
import torch

import dtensor_resharding_gb300 as R
from dtensor_resharding_gb300 import binding as B, ops
from oracle import experts as X

from conftest import ROOT

F64 = torch.float64
NULL = None


def test_library_exports_every_declared_operator():
    hdr = open(os.path.join(ROOT, "include", "reshard_ops.h")).read()
    declared = set(re.findall(r"^(?:int|int64_t)\s+(reshard_\w+)\(", hdr, flags=re.M))
    assert declared == set(ops.OPS_EXPORTED)
    for name in declared:
        assert hasattr(B.LIB, name)
    for name in R._OPS:
        assert getattr(R, name) is getattr(ops, name)


def refused(rc, code, *words):
    assert rc == code
    text = R.reshard_last_error()
    for w in words:
        assert w in text, text


def test_empty_calls_need_no_device():
    L = B.LIB
    assert L.reshard_route(NULL, 1, 0, 8, 8, NULL, 0, 1, 1, 1, 2, 1, 1.0, NULL, NULL, NULL) == 0
    assert L.reshard_route_backward(NULL, NULL, 1, 0, 8, 8, NULL, 2, 0, 1, 1.0, NULL, 8, NULL) == 0
    assert L.reshard_quantize_rows(NULL, 1, 0, 256, 256, NULL, 256, NULL, 1, 1, NULL) == 0
    assert L.reshard_quantize_blocks(NULL, 1, 0, 128, 128, 0, 128, NULL, 0, 128, NULL, NULL) == 0
    assert L.reshard_matmul_fp8(NULL, 256, NULL, 1, 1, NULL, 0, 256, NULL, NULL, 1, 0, 128, 256, NULL, 1, 128, NULL) == 0
    assert L.reshard_linear_fp8(NULL, 1, 0, 256, 256, NULL, 256, NULL, 128, NULL, 128, NULL, 0, NULL) == 0
    assert L.reshard_experts_fp8(NULL, 1, 0, 256, 256, NULL, NULL, 2, 0, 4, 128, NULL, 0, 256, NULL, NULL, 0, 128, NULL, NULL, 256, NULL, 0, NULL) == 0


def test_every_violation_is_listed():
    L, bad, unsup = B.LIB, B.RESHARD_ERR_INVALID_ARG, B.RESHARD_ERR_UNSUPPORTED
    refused(L.reshard_route(NULL, 4, 3, 8, 4, NULL, 7, 3, 4, 5, 9, 1, 1.0, NULL, NULL, NULL), bad, "k at most experts", "row stride", "dtype",
            "score", "divide", "groups_kept", "group_top")
    refused(L.reshard_route(NULL, 1, 3, 8, 8, NULL, 0, 4, 1, 1, 4, 1, 1.0, NULL, NULL, NULL), bad, "fewer than k")
    refused(L.reshard_route(NULL, 1, 3, 8, 8, NULL, 0, 8, 8, 2, 4, 1, 1.0, NULL, NULL, NULL), bad, "group_top exceeds")
    refused(L.reshard_route(NULL, 1, 3, 2048, 2048, NULL, 0, 1, 1, 1, 2, 1, 1.0, NULL, NULL, NULL), unsup, "1024")
    refused(L.reshard_route(NULL, 1, 3, 8, 8, NULL, 0, 1, 1, 1, 2, 1, 1.0, NULL, NULL, NULL), bad, "logits is NULL", "weights is NULL", "ids is NULL")
    refused(L.reshard_route_backward(NULL, NULL, 1, 1, 8, 8, NULL, 2, 0, 1, 1.0, NULL, 4, NULL), bad, "row stride")
    refused(L.reshard_dispatch(NULL, 4, -1, 0, NULL, NULL, NULL, NULL), bad, "first_expert")
    refused(L.reshard_dispatch(NULL, 4, 0, 513, NULL, NULL, NULL, NULL), unsup, "512")
    refused(L.reshard_quantize_rows(NULL, 0, 2, 256, 128, NULL, 128, NULL, 0, 1, NULL), bad, "dtype", "row stride", "scale strides")
    refused(L.reshard_quantize_blocks(NULL, 1, 2, 128, 128, -1, 64, NULL, 0, 128, NULL, NULL), bad, "row stride", "batch strides")
    refused(L.reshard_matmul_fp8(NULL, 250, NULL, 1, 1, NULL, 0, 256, NULL, NULL, 2, 4, 128, 256, NULL, 1, 64, NULL), bad, "groups", "row stride", "multiple of 16")
    refused(L.reshard_matmul_fp8(NULL, 256, NULL, 1, 1, NULL, 0, 256, NULL, NULL, 1, 4, 128, 256, NULL, 1, 128, NULL), bad, "a is NULL", "w is NULL")
    refused(L.reshard_linear_fp8(NULL, 1, 4, 0, 0, NULL, 0, NULL, 4, NULL, 4, NULL, 0, NULL), bad, "k >= 1")
    refused(L.reshard_experts_fp8(NULL, 1, 4, 256, 256, NULL, NULL, 2, 0, 4, 100, NULL, 0, 256, NULL, NULL, 0, 100, NULL, NULL, 256, NULL, 0, NULL),
            unsup, "multiple of 128")
    refused(L.reshard_ops_status(None, 0), bad, "status is NULL")


def test_workspace_sizes():
    L = B.LIB
    assert L.reshard_linear_fp8_workspace(1 << 62, 1 << 62) == 0 and L.reshard_experts_fp8_workspace(1 << 62, 8, 4, 256, 128, 1) == 0
    assert L.reshard_linear_fp8_workspace(-1, 4) == 0 and L.reshard_experts_fp8_workspace(4, 0, 4, 256, 128, 1) == 0
    # values at a 16-byte pitch and one fp32 scale for each 128, each part rounded up to 256 bytes
    assert L.reshard_linear_fp8_workspace(30, 300) == 30 * 304 // 256 * 256 + 256 + 512 and L.reshard_linear_fp8_workspace(3, 300) == 0
    assert L.reshard_experts_fp8_workspace(0, 2, 4, 256, 128, 1) >= 0


@pytest.mark.parametrize("call", [
    lambda: R.reshard_route(torch.zeros(2, 8), 2),
    lambda: R.reshard_route_backward(torch.zeros(2, 2), torch.zeros(2, 8), torch.zeros(2, 2, dtype=torch.int32)),
    lambda: R.reshard_dispatch(torch.zeros(2, 2, dtype=torch.int32), 4),
    lambda: R.reshard_quantize_rows(torch.zeros(2, 8)),
    lambda: R.reshard_quantize_blocks(torch.zeros(2, 8)),
    lambda: R.reshard_linear_fp8(torch.zeros(2, 8), torch.zeros(4, 8), torch.zeros(1, 1)),
])
def test_host_tensors_are_refused(call):
    with pytest.raises(R.ReshardError) as e:
        call()
    assert e.value.code == R.RESHARD_ERR_INVALID_ARG and "CUDA device" in str(e.value)


# ------------------------------------------------------------------------------------------------ the oracle itself

def test_e4m3_against_every_code():
    codes = torch.arange(256, dtype=torch.uint8)
    v = codes.view(torch.float8_e4m3fn).float()
    v = torch.unique(v[~torch.isnan(v)]).to(F64)
    assert torch.equal(X.e4m3(v), v)
    mid = (v[1:] + v[:-1]) / 2
    even = torch.where(((v[1:].float().to(torch.float8_e4m3fn).view(torch.uint8)) & 1) == 0, v[1:], v[:-1])
    assert torch.equal(X.e4m3(mid), even)
    eps = (v[1:] - v[:-1]) * 1e-9
    assert torch.equal(X.e4m3(mid + eps), v[1:]) and torch.equal(X.e4m3(mid - eps), v[:-1])
    assert torch.equal(X.e4m3(torch.tensor([1e9, -1e9], dtype=F64)), torch.tensor([448.0, -448.0], dtype=F64))


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_recovers_its_input(rows):
    """|x - q scale| is at most half an e4m3 step of the block's largest (relative 2^-4 or the subnormal step 2^-10), with
    the few fp32 roundings of scale and factor."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(130, 300, generator=g) * torch.logspace(-6, 3, 300)
    q, s = X.quantize(x, rows)
    back = X.dequantize(q.to(F64), s, rows)
    step = X.dequantize(torch.ones_like(q, dtype=F64), s, rows)
    assert bool(((back - x.to(F64)).abs() <= (x.abs().to(F64) * 2 ** -4 + step * 2 ** -10) * (1 + 1e-5)).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_backward_against_differences(score, renormalize):
    """The formulas against central differences of the weights of a fixed choice in 64 bits: error O(h^2) + eps / h."""
    g = torch.Generator().manual_seed(5)
    z = torch.randn(6, 9, generator=g, dtype=F64) * 1.5
    ids = torch.stack([torch.randperm(9, generator=g)[:4] for _ in range(6)])
    ids[2, 3] = -1
    ids[4, :] = torch.tensor([1, 5, 5, 2])           # a repeated expert: both slots' gradients
    grad = torch.randn(6, 4, generator=g, dtype=F64)
    got = X.route_backward(grad, z, ids, score, renormalize, 2.5)
    h = 1e-6
    for e in range(9):
        d = torch.zeros_like(z)
        d[:, e] = h
        diff = (X.route_weights(z + d, ids, score, renormalize, 2.5) - X.route_weights(z - d, ids, score, renormalize, 2.5)) / (2 * h)
        want = (diff * grad).sum(1)
        assert torch.allclose(got[:, e], want, rtol=1e-7, atol=1e-7), e


def test_route_groups_by_hand():
    z = torch.tensor([[3.0, 0.0, 2.0, 2.0, 1.9, 1.8, -9.0, -9.0]])
    # sums of the two best scores of each pair: softmax keeps the order of the sums of exponentials
    assert X.route(z, 2, groups=4, groups_kept=1, group_top=1)[1].tolist() == [[0, 1]]
    assert X.route(z, 3, groups=4, groups_kept=2, group_top=2)[1].tolist() == [[0, 2, 3]]
    masked = z.clone()
    masked[0, :6] = float("-inf")
    masked[0, 7] = float("nan")
    w, ids = X.route(masked, 2)
    assert ids.tolist() == [[6, -1]] and w.tolist() == [[1.0, 0.0]]


def test_packed_arguments_reach_the_same_calls():
    """The word form refuses what the plain form refuses, and takes no number or value that it cannot hold."""
    words = (ctypes.c_int64 * 24)()
    refused(B.LIB.reshard_ops_call(99, bytes(words)), B.RESHARD_ERR_INVALID_ARG, "unknown operator")
    refused(B.LIB.reshard_ops_call(0, None), B.RESHARD_ERR_INVALID_ARG, "NULL")
    for op in range(8):
        rc = B.LIB.reshard_ops_call(op, bytes(words))
        assert rc == B.RESHARD_ERR_INVALID_ARG, (op, rc)
    words[:5] = [0, 1, 1, 1 << 40, 1 << 40]         # experts beyond 32 bits
    words[11] = 2
    assert B.LIB.reshard_ops_call(0, bytes(words)) != 0
    with pytest.raises(R.ReshardError):
        ops._call(2, ops._DISPATCH(0, 4, -1, 0, 0, 0, 0, 0))
