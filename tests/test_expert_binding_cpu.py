"""What the binding of the expert layer hands to the library, seen without a GPU: the packed words of a call."""
import struct

import pytest
import torch

import dtensor_resharding_gb300 as R
from dtensor_resharding_gb300 import binding as B, ops


@pytest.fixture
def words(monkeypatch):
    """A list that receives (operator number, words) of each call in place of the library; host tensors pass for the device's."""
    seen = []
    monkeypatch.setattr(ops, "_here", lambda t, stream: 0)
    monkeypatch.setattr(ops, "_call", lambda op, w: seen.append((op, struct.unpack(f"={len(w) // 8}q", w))))
    return seen


def matmul(a_scale, M, K):
    a = torch.zeros(M, -(-K // 16) * 16, dtype=torch.uint8)[:, :K]
    w = torch.zeros(128, -(-K // 16) * 16, dtype=torch.uint8)[:, :K]
    return R.reshard_matmul_fp8(a, a_scale, w, torch.zeros(1, -(-K // 128)))


@pytest.mark.parametrize("M,kb", [(8, 4), (8, 1), (1, 4), (1, 1)])
@pytest.mark.parametrize("form", ["rows", "blocks", "by row", "by block", "whole"])
def test_matmul_scale_strides_reach_the_scales(words, M, kb, form):
    """Whatever the strides of a_scale (0 where it is broadcast), element [m, b] is read at m * row + b * block, and the
    last of them lies in the storage."""
    s = {"rows": torch.rand(M, kb), "blocks": torch.rand(kb, M).t(), "by row": torch.rand(M, 1).expand(M, kb),
         "by block": torch.rand(1, kb).expand(M, kb), "whole": torch.rand(()).expand(M, kb)}[form]
    matmul(s, M, kb * 128)
    (op, w), = words
    assert op == 5
    row, block = w[3], w[4]
    flat = s.as_strided((s.untyped_storage().nbytes() // 4,), (1,), 0)
    for m in range(M):
        for b in range(kb):
            at = m * row + b * block
            assert 0 <= at < len(flat) and flat[at] == s[m, b], (m, b, row, block)


def test_matmul_takes_broadcast_scales_and_no_negative_strides():
    call = lambda row, block: B.LIB.reshard_matmul_fp8(None, 256, None, row, block, None, 0, 256, None, None, 1, 4, 128, 256, None, 1, 128, None)  # noqa: E731
    for row, block in ((0, 0), (0, 1), (1, 0)):
        assert call(row, block) == B.RESHARD_ERR_INVALID_ARG and "stride" not in R.reshard_last_error()      # only the missing buffers
    for row, block in ((-1, 1), (1, -1)):
        assert call(row, block) == B.RESHARD_ERR_INVALID_ARG and "scale strides" in R.reshard_last_error()


def test_interleaved_weight_matrices_are_named():
    """[rows, experts, cols] seen as [experts, rows, cols]: such matrices do not overlap, and the refusal does not say so."""
    E, N, K = 4, 128, 256
    rc = B.LIB.reshard_matmul_fp8(None, K, None, 1, 1, None, K, E * K, None, 16, E, 8, N, K, None, 1, N, None)
    text = R.reshard_last_error()
    assert rc != 0 and "interleave" in text and "one after another" in text
    rc = B.LIB.reshard_matmul_fp8(None, K, None, 1, 1, None, N * K, K, None, 16, E, 8, N, K, None, 1, N, None)
    assert rc != 0 and "interleave" not in R.reshard_last_error()
