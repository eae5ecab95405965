"""Rows by index, embedding, norm and clipping without a GPU: the calls' refusals, the words that the binding hands over, and
the 64-bit oracle against other definitions of the same things."""
import contextlib
import copy
import ctypes
import pickle
import struct

import pytest
import torch
from torch.autograd import forward_ad

import dtensor_resharding_gb300 as R
from dtensor_resharding_gb300 import binding as B, ops
from oracle import rows as X

F64 = torch.float64
L = B.LIB
BAD, UNSUP = B.RESHARD_ERR_INVALID_ARG, B.RESHARD_ERR_UNSUPPORTED


def refused(rc, code, *words):
    assert rc == code, (rc, R.reshard_last_error())
    text = R.reshard_last_error()
    for w in words:
        assert w in text, text


def test_empty_calls_need_no_device():
    assert L.reshard_permute(None, 1, 0, 8, 8, None, None, 2, None, 4, 8, 0, None) == 0
    assert L.reshard_permute(None, 1, 4, 8, 8, None, None, 2, None, 0, 8, 0, None) == 0
    assert L.reshard_combine(None, 1, 4, 8, 8, None, None, 0, 2, None, 1, 8, None) == 0
    assert L.reshard_combine_backward(None, 1, 8, None, 1, 0, 8, 8, None, None, None, 0, 2, None, 8, None, None) == 0
    assert L.reshard_combine_backward(None, 1, 8, None, 1, 4, 8, 8, None, None, None, 2, 2, None, 8, None, None) == 0      # neither is wanted
    assert L.reshard_embedding(None, 64, 0, None, 1, 0, 9, 8, 8, 1.0, None, 8, None) == 0
    assert L.reshard_embedding(None, 64, 5, None, 1, 0, 9, 0, 0, 1.0, None, 0, None) == 0
    assert L.reshard_embedding_backward(None, 1, 0, 8, 8, None, 64, 0, 9, 1.0, None, 1, 8, 1, None, 0, None) == 0
    assert L.reshard_embedding_backward(None, 1, 5, 8, 8, None, 64, 0, 0, 1.0, None, 1, 8, 0, None, 0, None) == 0
    assert L.reshard_tensors_destroy(None) == 0


def test_gradients_of_no_columns_are_nothing():
    """Rows of no columns have no slices: their gradients are calls without work, of few tokens and of many, whole or accumulated."""
    for tokens in (1, 5, 256, 257, 300, 1 << 30):
        for rows in (0, 9):
            for accumulate in (0, 1):
                assert L.reshard_embedding_backward(None, 1, tokens, 0, 0, None, 64, 0, rows, 1.0, None, 1, 0, accumulate, None, 0, None) == 0
    assert L.reshard_embedding_backward_workspace(300, 0) == 0
    assert L.reshard_combine_backward(None, 1, 0, None, 1, 4, 0, 0, None, None, None, 0, 2, None, 0, None, None) == 0


def test_every_violation_is_listed():
    refused(L.reshard_permute(None, 4, 2, 8, 4, None, None, 0, None, 4, 7, 0, None), BAD, "k >= 1", "dtype", "row stride")
    refused(L.reshard_permute(None, 1, 2, 8, 8, None, None, 2, None, 4, 8, 0, None), BAD, "x is NULL", "order is NULL", "position is NULL", "out is NULL")
    refused(L.reshard_permute(None, 1, 1 << 31, 8, 8, None, None, 2, None, 4, 8, 0, None), UNSUP, "2^30")
    refused(L.reshard_permute(None, 1, 1 << 30, 8, 8, None, None, 2, None, 4, 8, 0, None), UNSUP, "2^30 slots")
    refused(L.reshard_permute(None, 1, 1 << 62, 1 << 62, 1 << 62, None, None, 1 << 30, None, 4, 1 << 62, 0, None), UNSUP, "2^30")
    refused(L.reshard_permute(None, 1, 1 << 28, 1 << 30, 1 << 30, None, None, 2, None, 4, 1 << 30, 0, None), UNSUP, "one launch")
    refused(L.reshard_combine(None, 0, -1, 8, 4, None, None, 3, 2, None, 9, 4, None), BAD, ">= 0", "dtype", "row stride")
    refused(L.reshard_combine(None, 1, 4, 8, 8, None, None, 3, 2, None, 1, 8, None), BAD, "y is NULL", "position is NULL", "out is NULL")
    refused(L.reshard_combine_backward(None, 7, 4, None, 1, 4, 8, 4, None, None, None, 3, 2, 16, 4, 16, None), BAD, "grad_dtype", "row stride")
    refused(L.reshard_combine_backward(None, 1, 8, None, 1, 4, 8, 8, None, None, None, 3, 2, 1, 8, 2, None), BAD, "grad is NULL", "y is NULL",
            "position is NULL", "order is NULL", "grad_y is not aligned", "grad_weights is not aligned")
    refused(L.reshard_embedding(None, 16, -2, None, 5, -1, 9, 8, 4, 1.0, None, 4, None), BAD, "first_row", "id_bits", "dtype", "row stride")
    refused(L.reshard_embedding(None, 64, 2, None, 1, 0, 9, 8, 8, 1.0, None, 8, None), BAD, "ids is NULL", "table is NULL", "out is NULL")
    refused(L.reshard_embedding(4, 64, 2, 1, 1, 0, 9, 8, 8, 1.0, 1, 8, None), BAD, "ids is not aligned to 8", "table is not aligned", "out is not aligned")
    refused(L.reshard_embedding(None, 64, 1 << 31, None, 1, 0, 9, 8, 8, 1.0, None, 8, None), UNSUP, "2^30")
    refused(L.reshard_embedding_backward(None, 0, 2, 8, 4, None, 8, -1, 9, 1.0, None, 0, 4, 0, None, 0, None), BAD, "first_row", "id_bits", "grad_dtype", "row stride")
    refused(L.reshard_embedding_backward(None, 1, 300, 8, 8, None, 64, 0, 9, 1.0, None, 1, 8, 0, None, 0, None), BAD, "grad_table is NULL", "grad is NULL",
            "ids is NULL", "workspace is NULL", "workspace is smaller")
    refused(L.reshard_embedding_backward(None, 1, 2, 8, 8, None, 64, 0, 9, 1.0, None, 1, 8, 0, None, 0, None), BAD, "grad is NULL", "ids is NULL")
    assert "workspace" not in R.reshard_last_error()
    refused(L.reshard_grad_norm(None, None, None, 0, None), BAD, "list is NULL")
    refused(L.reshard_clip_grads(None, None, -1.0, 4, 4, None, 0, None), BAD, "list is NULL", "limit", "give one")
    refused(L.reshard_clip_grads(None, None, float("nan"), None, None, None, 0, None), BAD, "limit")
    handle = ctypes.c_void_p()
    one, size, kind = (ctypes.c_void_p * 1)(None), (ctypes.c_int64 * 1)(4), (ctypes.c_int32 * 1)(3)
    refused(L.reshard_tensors_create(one, size, kind, 1, None), BAD, "list is NULL")
    refused(L.reshard_tensors_create(None, None, None, 1, ctypes.byref(handle)), BAD, "not NULL")
    refused(L.reshard_tensors_create(one, size, kind, -1, ctypes.byref(handle)), BAD, "count")
    refused(L.reshard_tensors_create(one, size, kind, 1, ctypes.byref(handle)), BAD, "a tensor is NULL")
    refused(L.reshard_tensors_create(one, size, (ctypes.c_int32 * 1)(0), 1, ctypes.byref(handle)), BAD, "type")
    refused(L.reshard_tensors_create(one, (ctypes.c_int64 * 1)(-1), kind, 1, ctypes.byref(handle)), BAD, "elements")
    refused(L.reshard_tensors_create(one, (ctypes.c_int64 * 1)(1 << 50), kind, 1, ctypes.byref(handle)), UNSUP, "2^40")
    assert not handle.value


def test_a_list_of_nothing():
    """Lists of no tensors and of empty ones need no device; calls on them still want where to put the norm."""
    for n in (0, 3):
        handle = ctypes.c_void_p()
        assert L.reshard_tensors_create((ctypes.c_void_p * n)(), (ctypes.c_int64 * n)(), (ctypes.c_int32 * n)(*[1] * n), n, ctypes.byref(handle)) == 0
        refused(L.reshard_grad_norm(handle, None, None, 0, None), BAD, "norm is NULL", "workspace is NULL", "workspace is smaller")
        refused(L.reshard_clip_grads(handle, None, 1.0, None, None, None, 0, None), BAD, "norm_out is NULL")
        assert L.reshard_tensors_destroy(handle) == 0


def test_copies_of_a_list_are_lists_of_their_own(monkeypatch):
    """A list that is copied, deeply copied or pickled (with the optimizer that holds it) makes another in the library, and each is
    freed once."""
    freed = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(ops, "LIB", type("Lib", (), {"reshard_tensors_create": staticmethod(L.reshard_tensors_create),
                                                     "reshard_tensors_destroy": staticmethod(lambda h: freed.append(h) or L.reshard_tensors_destroy(h))}))
    first = R.reshard_tensor_list([])
    lists = [first, copy.copy(first), copy.deepcopy({"of": [first]})["of"][0], pickle.loads(pickle.dumps(first))]
    handles = {t._handle for t in lists}
    assert len(handles) == 4 and all(type(t) is R.TensorList and t.tensors == [] for t in lists)
    del first
    while lists:
        lists.pop()
    assert sorted(freed) == sorted(handles)


def test_workspace_sizes():
    assert L.reshard_embedding_backward_workspace(0, 8) == 0 and L.reshard_embedding_backward_workspace(-1, 8) == 0
    assert L.reshard_embedding_backward_workspace(1 << 31, 8) == 0 and L.reshard_embedding_backward_workspace(8, 1 << 31) == 0
    # pairs twice, their number, and two fp32 rows a run: everything that the tokens alone decide
    assert L.reshard_embedding_backward_workspace(256, 64) == 0                # a few tokens need none
    small = L.reshard_embedding_backward_workspace(257, 1)
    assert 2 * 8 * 257 < small <= 16384
    assert L.reshard_embedding_backward_workspace(1 << 30, 1 << 30) > 1 << 34 and L.reshard_grad_norm_workspace() > 0


@pytest.mark.parametrize("call", [
    lambda: R.reshard_permute(torch.zeros(2, 8), tuple(torch.zeros(4, dtype=torch.int32) for _ in range(3))),
    lambda: R.reshard_combine(torch.zeros(4, 8), tuple(torch.zeros(4, dtype=torch.int32) for _ in range(3)), torch.zeros(2, 2)),
    lambda: R.reshard_combine_backward(torch.zeros(2, 8), torch.zeros(4, 8), tuple(torch.zeros(4, dtype=torch.int32) for _ in range(3)), torch.zeros(2, 2)),
    lambda: R.reshard_permute_backward(torch.zeros(4, 8), tuple(torch.zeros(4, dtype=torch.int32) for _ in range(3)), 2),
    lambda: R.reshard_embedding(torch.zeros(3, dtype=torch.int64), torch.zeros(2, 8)),
    lambda: R.reshard_embedding_backward(torch.zeros(3, 8), torch.zeros(3, dtype=torch.int64), 4),
    lambda: R.reshard_tensor_list([torch.zeros(3)]),
    lambda: R.reshard_grad_norm([torch.zeros(3)]),
    lambda: R.reshard_clip_grads([torch.zeros(3)], 1.0),
])
def test_host_tensors_are_refused(call):
    with pytest.raises(R.ReshardError) as e:
        call()
    assert e.value.code == BAD and "CUDA device" in str(e.value)


def test_packed_arguments_reach_the_same_calls():
    """Each number calls its operator: the refusal of arguments that are all 0 names it."""
    words = bytes(8 * 24)
    for op, name in ((8, "reshard_permute"), (9, "reshard_combine"), (10, "reshard_combine_backward"), (11, "reshard_embedding"),
                     (12, "reshard_embedding_backward"), (13, "reshard_grad_norm"), (14, "reshard_clip_grads")):
        refused(L.reshard_ops_call(op, words), BAD, name + ":")


@pytest.fixture
def words(monkeypatch):
    """A list that receives (operator number, words) of each call in place of the library; host tensors pass for the device's."""
    seen = []
    monkeypatch.setattr(ops, "_here", lambda t, stream: 0)
    monkeypatch.setattr(ops, "_call", lambda op, w: seen.append((op, struct.unpack(f"={len(w) // 8}q", w))))
    return seen


def test_words_of_the_row_calls(words):
    x = torch.zeros(3, 24, dtype=torch.bfloat16)[:, :16]
    sort = (torch.zeros(3, dtype=torch.int32), torch.zeros(6, dtype=torch.int32), torch.zeros(6, dtype=torch.int32))
    out = torch.zeros(9, 40, dtype=torch.bfloat16)[:, :16]
    R.reshard_permute(x, sort, out=out)
    y, w = torch.zeros(6, 16), torch.zeros(3, 2)
    back = R.reshard_combine(y, sort, w, out_dtype=torch.float16)
    dy, dw = R.reshard_combine_backward(x, y, sort, w)
    assert [op for op, _ in words] == [8, 9, 10]
    at_order, at_position = sort[1].data_ptr(), sort[2].data_ptr()
    # places that the sort does not have are left out
    assert words[0][1] == (x.data_ptr(), 1, 3, 16, 24, at_order, at_position, 2, out.data_ptr(), 6, 40, 0, 0)
    assert words[1][1] == (y.data_ptr(), 3, 6, 16, 16, at_position, w.data_ptr(), 3, 2, back.data_ptr(), 2, 16, 0)
    assert words[2][1] == (x.data_ptr(), 1, 24, y.data_ptr(), 3, 6, 16, 16, at_order, at_position, w.data_ptr(), 3, 2, dy.data_ptr(), 16, dw.data_ptr(), 0)


def test_words_of_the_embedding_calls(words):
    ids, table = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(9, 20)[:, :16]
    out = R.reshard_embedding(ids, table, scale=2.0, first_row=5)
    grad = R.reshard_embedding_backward(out, ids, 9, first_row=5, dtype=torch.bfloat16)
    two = struct.unpack("=q", struct.pack("=d", 2.0))[0]
    one = struct.unpack("=q", struct.pack("=d", 1.0))[0]
    assert out.shape == (2, 3, 16) and grad.shape == (9, 16) and grad.dtype is torch.bfloat16
    assert words[0] == (11, (ids.data_ptr(), 32, 6, table.data_ptr(), 3, 5, 9, 16, 20, two, out.data_ptr(), 16, 0))
    op, w = words[1]
    assert op == 12 and w[:14] == (out.data_ptr(), 3, 6, 16, 16, ids.data_ptr(), 32, 5, 9, one, grad.data_ptr(), 1, 16, 0)
    assert w[15] == L.reshard_embedding_backward_workspace(6, 16) and w[16] == 0


def test_a_given_output_counts_as_written(words):
    """Autograd keeps tensors by their version: a buffer that a call writes has another one afterwards, through any of its views."""
    x, sort = torch.zeros(2, 8), _sort()
    logits, ids2, tokens = torch.zeros(2, 4), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    w8, s8 = torch.zeros(8, 128, dtype=torch.uint8), torch.zeros(1, 1)
    calls = [(torch.zeros(4, 8), lambda o: R.reshard_permute(x, sort, out=o)), (torch.zeros(2, 8), lambda o: R.reshard_combine(torch.zeros(4, 8), sort, k=2, out=o)),
             (torch.zeros(2, 8), lambda o: R.reshard_permute_backward(torch.zeros(4, 8), sort, 2, out=o)), (torch.zeros(3, 8), lambda o: R.reshard_embedding(tokens, x, out=o)),
             (torch.zeros(1, 3, 8), lambda o: R.reshard_embedding(tokens.view(1, 3), x, out=o)), (torch.zeros(2, 8), lambda o: R.reshard_embedding_backward(torch.zeros(3, 8), tokens, 2, out=o)),
             (torch.zeros(2, 8), lambda o: R.reshard_embedding_backward(torch.zeros(3, 8), tokens, 2, out=o, accumulate=True)),
             (torch.zeros(2, 4), lambda o: R.reshard_route_backward(torch.zeros(2, 2), logits, ids2, out=o)), (torch.zeros(2, 8), lambda o: R.reshard_linear_fp8(torch.zeros(2, 128), w8, s8, out=o)),
             (torch.zeros(2, 8), lambda o: R.reshard_matmul_fp8(torch.zeros(2, 128, dtype=torch.uint8), torch.zeros(2, 1), w8, s8, out=o))]
    for i, (out, call) in enumerate(calls):
        base = torch.zeros(4, *out.shape)
        for to in (out, base[2]):
            leaf = torch.ones(out.shape, requires_grad=True)
            product = leaf * to                       # keeps `to`
            version = to._version
            assert call(to) is to and to._version > version and len(words) > 0, i
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                product.sum().backward()
        with torch.inference_mode():
            assert call(torch.zeros(out.shape)).is_inference()


def test_dense_in_any_order():
    x = torch.zeros(4, 6, 5)
    for t in (x, x.permute(2, 0, 1), x.transpose(0, 1), x[:1], x[:, :, :1].contiguous(), torch.zeros(()), torch.zeros(0)):
        assert t.is_contiguous() or ops._packed(t), t.shape
    for t in (x[:, ::2], x[:, :, :3], x[:, :, :1], x.expand(2, 4, 6, 5), torch.zeros(3, 1).expand(3, 4), x.permute(2, 0, 1)[:3]):
        assert not t.is_contiguous() and not ops._packed(t), (t.shape, t.stride())


# ---------------------------------------------------------------------------------------------------------- derivatives

def _sort():
    return tuple(torch.zeros(4, dtype=torch.int32) for _ in range(3))


TANGENTS = {
    "reshard_route": lambda d: R.reshard_route(d(2, 4), 2),
    "reshard_route bias": lambda d: R.reshard_route(torch.zeros(2, 4), 2, bias=d(4)),
    "reshard_route_backward": lambda d: R.reshard_route_backward(d(2, 2), torch.zeros(2, 4), torch.zeros(2, 2, dtype=torch.int32)),
    "reshard_route_backward logits": lambda d: R.reshard_route_backward(torch.zeros(2, 2), d(2, 4), torch.zeros(2, 2, dtype=torch.int32)),
    "reshard_linear_fp8": lambda d: R.reshard_linear_fp8(d(2, 128), torch.zeros(8, 128, dtype=torch.uint8), torch.zeros(1, 1)),
    "reshard_experts_fp8": lambda d: R.reshard_experts_fp8(torch.zeros(2, 128), torch.zeros(2, 1, dtype=torch.int32), d(2, 1), None, None, None, None),
    "reshard_permute": lambda d: R.reshard_permute(d(2, 8), _sort()),
    "reshard_permute_backward": lambda d: R.reshard_permute_backward(d(4, 8), _sort(), 2),
    "reshard_combine": lambda d: R.reshard_combine(d(4, 8), _sort(), torch.zeros(2, 2)),
    "reshard_combine weights": lambda d: R.reshard_combine(torch.zeros(4, 8), _sort(), d(2, 2)),
    "reshard_combine_backward": lambda d: R.reshard_combine_backward(torch.zeros(2, 8), d(4, 8), _sort(), torch.zeros(2, 2)),
    "reshard_embedding": lambda d: R.reshard_embedding(torch.zeros(3, dtype=torch.int64), d(2, 8)),
    "reshard_embedding_backward": lambda d: R.reshard_embedding_backward(d(3, 8), torch.zeros(3, dtype=torch.int64), 4),
    "reshard_embedding_backward out": lambda d: R.reshard_embedding_backward(torch.zeros(3, 8), torch.zeros(3, dtype=torch.int64), 4, out=d(4, 8), accumulate=True),
}


@pytest.mark.parametrize("name", TANGENTS)
@pytest.mark.parametrize("requires_grad", [False, True])
def test_tangents_are_refused(name, requires_grad):
    """Forward mode would read a result without a tangent as a constant; without a tangent, or outside the level, nothing is
    refused for it."""
    call = TANGENTS[name]

    def dual(*shape):
        return forward_ad.make_dual(torch.zeros(*shape, requires_grad=requires_grad), torch.ones(*shape))

    with forward_ad.dual_level():
        for grad in (True, False):
            with torch.set_grad_enabled(grad), pytest.raises(R.ReshardError, match="forward mode") as e:
                call(dual)
            assert e.value.code == UNSUP
        with pytest.raises(R.ReshardError, match="CUDA device"):
            call(torch.zeros)
    with pytest.raises(R.ReshardError, match="CUDA device"):
        call(torch.zeros)


def test_a_given_output_has_no_tangent(words):
    """What is written is not what the tangent was of."""
    with forward_ad.dual_level():
        out = forward_ad.make_dual(torch.zeros(4, 8), torch.ones(4, 8))
        for call in (lambda: R.reshard_permute(torch.zeros(2, 8), _sort(), out=out), lambda: R.reshard_embedding(torch.zeros(4, dtype=torch.int64), torch.zeros(2, 8), out=out),
                     lambda: R.reshard_combine(torch.zeros(4, 8), _sort(), k=1, out=out), lambda: R.reshard_embedding_backward(torch.zeros(3, 8), torch.zeros(3, dtype=torch.int64), 4, out=out)):
            with pytest.raises(R.ReshardError, match="forward mode"):
                call()
        assert words == [] and R.reshard_permute(torch.zeros(2, 8), _sort(), out=torch.zeros(4, 8)).shape == (4, 8)


# ------------------------------------------------------------------------------------------------ the oracle itself

def test_oracle_sort_and_rows_by_hand():
    ids = torch.tensor([[1, 0], [2, 1], [0, -1]], dtype=torch.int32)
    offsets, order, position = X.sort(ids, 2)
    assert offsets.tolist() == [0, 2, 4] and order.tolist() == [1, 4, 0, 3] and position.tolist() == [2, 0, -1, 3, 1, -1]
    x = torch.tensor([[1.0], [2.0], [3.0]])
    assert X.permute(x, position, torch.zeros(5, 1)).view(-1).tolist() == [1, 3, 1, 2, 0]
    y, w = torch.tensor([[10.0], [20.0], [30.0], [40.0], [50.0]]), torch.tensor([[0.5, 2.0], [9.0, 1.0], [3.0, 9.0]])
    assert X.combine(y, position, w, 2).view(-1).tolist() == [0.5 * 30 + 2 * 10, 40, 3 * 20]
    dy, dw = X.combine_backward(x, y, position, w, 2)
    assert dy.view(-1).tolist() == [2, 9, 0.5, 2, 0] and dw.tolist() == [[30, 10], [0, 80], [60, 0]]


def test_oracle_gradients_are_autograds():
    g = torch.Generator().manual_seed(1)
    ids = torch.stack([torch.randperm(5, generator=g)[:3] for _ in range(7)]).int()
    _, _, position = X.sort(ids, 3, 1)
    held = int((position >= 0).sum())
    y = torch.randn(21, 4, generator=g, dtype=F64).requires_grad_()
    w = torch.rand(7, 3, generator=g, dtype=F64).requires_grad_()
    grad = torch.randn(7, 4, generator=g, dtype=F64)
    place = torch.where(position >= 0, position, held).long().view(7, 3)
    masked = torch.where(torch.arange(21)[:, None] < held, y, 0.0)
    out = (masked[place] * (w * (position.view(7, 3) >= 0))[..., None]).sum(1)
    assert torch.allclose(out, X.combine(y, position, w, 3), rtol=1e-14)
    out.backward(grad)
    dy, dw = X.combine_backward(grad, y.detach(), position, w.detach(), 3)
    assert torch.allclose(y.grad, dy, rtol=1e-14) and torch.allclose(w.grad, dw, rtol=1e-13)
    table = torch.randn(6, 4, generator=g, dtype=F64).requires_grad_()
    tokens = torch.randint(0, 6, (3, 5), generator=g)
    pull = torch.randn(3, 5, 4, generator=g, dtype=F64)
    (torch.nn.functional.embedding(tokens, table) * 3.0).backward(pull)
    assert torch.allclose(X.embedding(tokens + 4, table.detach(), 3.0, 4), torch.nn.functional.embedding(tokens, table) * 3.0)
    assert torch.allclose(table.grad, X.embedding_backward(pull, tokens + 4, 6, 3.0, 4), rtol=1e-14)


def test_oracle_clip_is_torchs():
    g = torch.Generator().manual_seed(2)
    for limit in (0.5, 1e3):
        ts = [torch.nn.Parameter(torch.zeros(n, dtype=F64)) for n in (1, 7, 30)]
        for t in ts:
            t.grad = torch.randn(t.shape, generator=g, dtype=F64)
        want = X.clip([t.grad for t in ts], limit)
        norm = X.norm([t.grad for t in ts])
        assert torch.allclose(torch.nn.utils.clip_grad_norm_(ts, limit), norm)
        assert all(torch.allclose(t.grad, v, rtol=1e-12) for t, v in zip(ts, want))
