"""The expert layer's kernels on the paths, values and layouts that the sizes of test_experts_gpu.py do not reach.

Tolerances are those of that file, by the same arithmetic, unless a test derives its own.
"""
import pytest
import torch

from oracle import experts as X

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dtensor_resharding_gb300 as R

F64 = torch.float64
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _status():
    yield
    assert R.reshard_ops_status() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def weights(g, *shape):
    return R.reshard_quantize_blocks(randn(g, *shape) * 0.02)


# --------------------------------------------------------------------------------- experts' outputs before their sum

@pytest.mark.parametrize("T", [3, 400])
def test_experts_outputs_beyond_the_output_type(T):
    """An expert's output of 100,000 is no float16, an eighth of it is: the sum is taken before the rounding."""
    g = gen(T)
    E, k, H, I = 4, 2, 256, 512
    x = randn(g, T, H).half()
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    w13, s13 = weights(g, E, 2 * I, H)
    w2, s2 = weights(g, E, H, I)
    one = torch.ones(T, 1, device="cuda")
    s2 *= 100000.0 / max(float(X.experts(x, ids[:, j:j + 1], one, w13, s13, w2, s2).abs().amax()) for j in range(k))
    share = torch.full((T, k), 0.125, device="cuda")
    want = X.experts(x, ids, share, w13, s13, w2, s2)
    out = R.reshard_experts_fp8(x, ids, share, w13, s13, w2, s2)
    assert bool(torch.isfinite(out).all())
    assert bool(((out.to(F64) - want).norm(dim=1) <= 6 * 2.5e-3 * want.norm(dim=1)).all())


@pytest.mark.parametrize("T", [2, 500])
def test_experts_outputs_that_cancel(T):
    """Two experts whose second matrices are opposite but for 16 of 1,024 columns: the sum is those columns', some eighth of
    either output. Hidden codes are the same for both. Tolerance, of the norm: codes 2e-3, the output's rounding 1.2e-3, the
    fp32 sums (128 + 24) 2^-23 of sums of magnitudes 160 times the result's, 3e-3: 7e-3 in all. Rounding either output to 16
    bits before the sum would leave 1.3e-2."""
    g = gen(T)
    H, I = 512, 1024
    x = randn(g, T, H).bfloat16()
    w13, s13 = weights(g, 1, 2 * I, H)
    w2, s2 = weights(g, 1, H, I)
    other = (-X.values(w2)).float()
    other[:, :, ::64] = 0.0
    w2 = torch.cat([w2, other.to(torch.float8_e4m3fn)])
    w13, s13, s2 = (t.repeat(2, 1, 1) if t.dtype != torch.float8_e4m3fn else t.view(torch.uint8).repeat(2, 1, 1) for t in (w13, s13, s2))
    ids = torch.tensor([0, 1], dtype=torch.int32, device="cuda").repeat(T, 1)
    ones = torch.ones(T, 2, device="cuda")
    want = X.experts(x, ids, ones, w13, s13, w2, s2)
    err = R.reshard_experts_fp8(x, ids, ones, w13, s13, w2, s2).to(F64) - want
    assert float(err.norm()) <= 7e-3 * float(want.norm()), float(err.norm() / want.norm())
