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


# ------------------------------------------------------------------------------------------ strides of the rows' scales

@pytest.mark.parametrize("M,groups", [(1, 0), (3, 0), (40, 0), (300, 0), (2000, 0), (20, 4), (700, 4)])
@pytest.mark.parametrize("K", [128, 1000])
def test_product_scales_of_any_strides(M, groups, K):
    """Scales stored row by row, block by block, one a row, one a block and one in all, through each product kernel: what
    their copies give."""
    g = gen(M + K)
    kb, N = -(-K // 128), 200
    q, s = R.reshard_quantize_rows(randn(g, M, K).bfloat16())
    wq, ws = weights(g, groups, N, K) if groups else weights(g, N, K)
    kw = {"offsets": torch.tensor([M * i // groups for i in range(groups + 1)], dtype=torch.int32, device="cuda")} if groups else {}
    rows = torch.rand(M, 2 * kb + 3, generator=g, device="cuda") + 0.5
    for scale in (rows[:, :kb], rows[:, 1:2 * kb + 1:2], rows[:, :1].expand(M, kb), rows[:1, :kb].expand(M, kb), rows[0, 0].expand(M, kb),
                  rows[:, :kb].t().contiguous().t()):
        got = R.reshard_matmul_fp8(q, scale, wq, ws, out_dtype=torch.float32, **kw)
        copy = torch.empty_strided((M, kb), (1, M), device="cuda").copy_(scale)       # as the quantization stores them
        assert torch.equal(got, R.reshard_matmul_fp8(q, copy, wq, ws, out_dtype=torch.float32, **kw))
        a, w = X.dequantize(X.values(q), scale.contiguous(), 1), X.dequantize(X.values(wq), ws, 128)
        for e in range(groups or 1):
            r = slice(M * e // groups, M * (e + 1) // groups) if groups else slice(None)
            we = w[e] if groups else w
            tol = (min(K, 128) + 3 * kb) * 2.0 ** -23 * (a[r].abs() @ we.abs().t()) + 2.0 ** -24 * (a[r] @ we.t()).abs()
            assert bool(((got[r].to(F64) - a[r] @ we.t()).abs() <= tol).all())


# --------------------------------------------------------------------------------------------------- rows of 2^31 bytes

def test_product_columns_beyond_2_31_bytes():
    """fp32 rows of 2^29 + 300 columns, whole quarters of a tile's rows: the first, the last and those around byte 2^31 are written."""
    N, K, M = 2 ** 29 + 300, 16, 32
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 * 2 ** 30:
        pytest.skip("needs 100 GiB of device memory")
    g = gen(29)
    q, s = R.reshard_quantize_rows(randn(g, M, K).bfloat16())
    w = torch.zeros(1, N, K, dtype=torch.uint8, device="cuda")
    ws = torch.ones(1, -(-N // 128), 1, device="cuda")
    at = [0, 2 ** 28, 2 ** 29 - 256, N - 300]
    for c in at:
        w[0, c:c + 300] = (randn(g, 300, K) * 100).to(torch.float8_e4m3fn).view(torch.uint8)
    out = torch.empty(M, -(-N // 4) * 4, device="cuda")[:, :N]
    for c in at:
        out[:, c:c + 300] = float("nan")
    R.reshard_matmul_fp8(q, s, w, ws, offsets=torch.tensor([0, M], dtype=torch.int32, device="cuda"), out=out)
    a = X.dequantize(X.values(q), s, 1)
    for c in at:
        v = X.values(w[0, c:c + 300])
        tol = (K + 3) * 2.0 ** -23 * (a.abs() @ v.abs().t()) + 2.0 ** -24 * (a @ v.t()).abs()
        assert bool(((out[:, c:c + 300].to(F64) - a @ v.t()).abs() <= tol).all()), c
    del out, w, ws
    torch.cuda.empty_cache()


# ------------------------------------------------------------------------------------------ offsets that are not ascending

@pytest.mark.parametrize("offsets", [[0, 40, 10, 40], [0, 30, 5, 20, 35, 12, 40], [40, 0, 40], [-3, 25, 90, 7, 31], [0] + [33, 1] * 80 + [40]])
@pytest.mark.parametrize("K", [256, 2048])
@pytest.mark.parametrize("times", [1, 20])
def test_grouped_product_of_descending_offsets(offsets, K, times):
    """Offsets below one before them count as that one: no row is of two groups, and a repeated call gives the same."""
    g = gen(len(offsets) + K)
    E, M, N = len(offsets) - 1, 40 * times, 130
    q, s = R.reshard_quantize_rows(randn(g, M, K).bfloat16())
    wq, ws = weights(g, E, N, K)
    given = torch.tensor(offsets, dtype=torch.int32, device="cuda") * times
    raised = given.clamp(0, M).cummax(0).values.int()
    out = torch.full((M, N), 7.0, device="cuda")
    R.reshard_matmul_fp8(q, s, wq, ws, offsets=given, out=out)
    want = torch.full((M, N), 7.0, device="cuda")
    R.reshard_matmul_fp8(q, s, wq, ws, offsets=raised, out=want)
    assert torch.equal(out, want)
    a, w = X.dequantize(X.values(q), s, 1), X.dequantize(X.values(wq), ws, 128)
    for e in range(E):
        r = slice(int(raised[e]), int(raised[e + 1]))
        tol = (128 + 3 * (K // 128)) * 2.0 ** -23 * (a[r].abs() @ w[e].abs().t()) + 2.0 ** -24 * (a[r] @ w[e].t()).abs()
        assert bool(((out[r].to(F64) - a[r] @ w[e].t()).abs() <= tol).all())


# ------------------------------------------------------------------------------------ experts switched off by their bias

@pytest.mark.parametrize("E,groups,kept,k", [(32, 4, 2, 12), (256, 32, 6, 32), (60, 4, 3, 20)])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_bias_of_the_lowest_value(E, groups, kept, k, top, score):
    """Biases of fp32's lowest value put experts behind all others and switch no group off: a sum of two of them is below
    every fp32 number, and its group still comes before none."""
    size = E // groups
    z = torch.arange(E, device="cuda").float()[torch.randperm(E, generator=gen(E), device="cuda")][None].repeat(3, 1) * (4.0 / E)
    bias = torch.full((E,), torch.finfo(torch.float32).min, device="cuda")
    bias[size:2 * size] = 0.0
    for renormalize in (True, False):
        w, ids = R.reshard_route(z, k, score=score, bias=bias, groups=groups, groups_kept=kept, group_top=top, renormalize=renormalize)
        ww, want = X.route(z, k, score=score, bias=bias, groups=groups, groups_kept=kept, group_top=top, renormalize=renormalize)
        assert bool((want >= 0).all()) and torch.equal(ids.cpu().long(), want)
        assert bool(((w.cpu().to(F64) - ww).abs() <= 64 * 2.0 ** -24 * ww.abs() + 1e-38).all())


# --------------------------------------------------------------------------------------------------------- autograd

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_route_weights_carry_their_gradient(score, renormalize, dtype):
    """A loss of the routing weights reaches the logits and what made them, as reshard_route_backward gives it."""
    g = gen(21)
    x, router = randn(g, 37, 64).to(DT[dtype]), randn(g, 64, 24).to(DT[dtype]).requires_grad_()
    logits = x @ router
    logits.retain_grad()
    grad = randn(g, 37, 4)
    w, ids = R.reshard_route(logits, 4, score=score, renormalize=renormalize, scale=2.5)
    plain, plain_ids = R.reshard_route(logits.detach(), 4, score=score, renormalize=renormalize, scale=2.5)
    assert torch.equal(w, plain) and torch.equal(ids, plain_ids) and w.requires_grad and not ids.requires_grad and not plain.requires_grad
    (w * grad).sum().backward()
    want = R.reshard_route_backward(grad, logits.detach(), ids, score=score, renormalize=renormalize, scale=2.5)
    assert torch.equal(logits.grad, want)
    assert torch.equal(router.grad, x.t() @ want)
    with torch.no_grad():
        assert not R.reshard_route(logits, 4)[0].requires_grad


def test_route_gradient_of_groups_bias_streams_and_broadcasts():
    g = gen(22)
    z, bias = randn(g, 9, 32), randn(g, 32) * 0.1
    kw = dict(score="sigmoid", bias=bias, groups=4, groups_kept=2, group_top=2, renormalize=True, scale=1.5)
    a = z.clone().requires_grad_()
    w, ids = R.reshard_route(a, 5, **kw)
    (w[:, :1].expand(9, 5) * 2.0).sum().backward()
    grad = torch.zeros(9, 5, device="cuda")
    grad[:, 0] = 10.0
    assert torch.equal(a.grad, R.reshard_route_backward(grad, z, ids, score="sigmoid", scale=1.5))
    side, b = torch.cuda.Stream(), z.clone().requires_grad_()
    side.wait_stream(torch.cuda.current_stream())
    w2, ids2 = R.reshard_route(b, 5, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    w2[:, 0].sum().backward()
    torch.cuda.synchronize()
    grad[:, 0] = 1.0
    assert torch.equal(ids, ids2) and torch.equal(b.grad, R.reshard_route_backward(grad, z, ids, score="sigmoid", scale=1.5))


def test_gradients_that_do_not_exist_are_refused():
    g = gen(23)
    x = randn(g, 6, 256).bfloat16().requires_grad_()
    w13, s13 = weights(g, 4, 256, 256)
    w2, s2 = weights(g, 4, 256, 128)
    y = R.reshard_linear_fp8(x, w13[0], s13[0])
    assert torch.equal(y.detach(), R.reshard_linear_fp8(x.detach(), w13[0], s13[0]))
    with pytest.raises(R.ReshardError, match="no gradient") as e:
        y.sum().backward()
    assert e.value.code == R.RESHARD_ERR_UNSUPPORTED
    z = randn(g, 6, 4).requires_grad_()
    for xs, zs in ((x.detach(), z), (x, z.detach())):
        shares, ids = R.reshard_route(zs, 2)
        y = R.reshard_experts_fp8(xs, ids, shares, w13, s13, w2, s2)
        assert torch.equal(y.detach(), R.reshard_experts_fp8(x.detach(), ids, shares.detach(), w13, s13, w2, s2))
        with pytest.raises(R.ReshardError, match="no gradient"):
            y.float().sum().backward()
    with torch.no_grad():
        assert not R.reshard_linear_fp8(x, w13[0], s13[0]).requires_grad


# ------------------------------------------------------------------------------- the gated products' splits and many tiles

def layer(g, T, E, k, H, I, local=None, dtype=torch.bfloat16):
    n = E if local is None else local
    x = randn(g, T, H).to(dtype)
    w, ids = R.reshard_route(randn(g, T, E), k)
    return (x, ids, w, *weights(g, n, 2 * I, H), *weights(g, n, H, I))


def check_layer(args, first=0):
    got = R.reshard_experts_fp8(*args, first_expert=first)
    want = X.experts(*args, first=first)
    tol = 5e-3 if got.dtype == torch.bfloat16 else 2.5e-3
    err = got.to(F64) - want
    assert float(err.norm()) <= tol * float(want.norm()) * (6 if len(got) < 7 else 1), float(err.norm() / want.norm())
    assert bool((err.norm(dim=1) <= 6 * tol * want.norm(dim=1) + 1e-30).all())
    for _ in range(3):
        assert torch.equal(got, R.reshard_experts_fp8(*args, first_expert=first))
    return got


@pytest.mark.parametrize("T,E,k,H,I", [(1, 16, 2, 1024, 256), (3, 16, 2, 1024, 256), (1, 16, 2, 2048, 256), (3, 16, 2, 2048, 256),
                                       (3, 4, 4, 4096, 384), (1, 2, 1, 4224, 128), (9, 16, 2, 1920, 128), (30, 4, 1, 2048, 128), (1, 128, 8, 2048, 768)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_experts_gated_product_split_over_a_cluster(T, E, k, H, I, dtype):
    """Few tiles and a long row: the gated product's K is shared by 2 to 8 CTAs (H / 512 at most), which add gate and up
    before silu and meet for the row's amax."""
    check_layer(layer(gen(T + H + I), T, E, k, H, I, dtype=DT[dtype]))


@pytest.mark.parametrize("T", [1, 16, 17, 64])
def test_experts_a_share_of_a_decode_step(T):
    """16 of 128 experts: most choices are another rank's, and some calls have none here."""
    x, ids, w, w13, s13, w2, s2 = layer(gen(T), T, 128, 8, 2048, 256, local=16)
    for first in (0, 48, 112):
        args = (x, ids, w, w13, s13, w2, s2)
        here = bool(((ids >= first) & (ids < first + 16)).any())
        if here:
            check_layer(args, first)
        else:
            assert not R.reshard_experts_fp8(*args, first_expert=first).any()


@pytest.mark.parametrize("T,E,k,H,I", [(100, 128, 8, 256, 1280), (2000, 16, 8, 256, 768)])
def test_experts_many_gated_tiles_a_cta(T, E, k, H, I):
    """Four tiles and more for each CTA of the narrow and of the wide gated product: the amax buffers, their barriers' parity
    and the boxes on their way out are used again."""
    check_layer(layer(gen(T), T, E, k, H, I))


# ------------------------------------------------------------------------------------------------- the linear's types

@pytest.mark.parametrize("M", [1, 3, 4, 5, 130])
@pytest.mark.parametrize("K", [16, 300, 1000, 1024])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_linear_types_and_rows(M, K, dtype):
    """Every type through the few-row kernel and through quantization and product, rows aligned and not."""
    g = gen(M * K)
    big = randn(g, M, K + 24).to(DT[dtype])
    wq, ws = weights(g, 140, K)
    w = X.dequantize(X.values(wq), ws, 128)
    for off in (0, 8, 1, 3):
        x = big[:, off:off + K]
        got = R.reshard_linear_fp8(x, wq, ws)
        q, s = X.quantize(x, 1)
        a = X.dequantize(q, s, 1)
        want = a @ w.t()
        tol = (min(K, 128) + 3 * s.shape[1]) * 2.0 ** -23 * (a.abs() @ w.abs().t()) + torch.finfo(x.dtype).eps / 2 * want.abs() * (1 + 1e-3)
        assert got.dtype == x.dtype and bool(((got.to(F64) - want).abs() <= tol).all())
        assert torch.equal(got, R.reshard_linear_fp8(x.contiguous(), wq, ws))


@pytest.mark.parametrize("M", [2, 48, 300])
def test_linear_replayed_from_a_graph(M):
    """A captured linear computes with what its input holds at each replay."""
    g = gen(M)
    x, (wq, ws) = randn(g, M, 512).bfloat16(), weights(g, 384, 512)
    inp, side = x.clone(), torch.cuda.Stream()
    R.reshard_linear_fp8(inp, wq, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = R.reshard_linear_fp8(inp, wq, ws)
    for scale in (1.0, -0.5, 3.0):
        inp.copy_(x * scale)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, R.reshard_linear_fp8(inp, wq, ws)) and float(out.float().norm()) > 0


@pytest.mark.parametrize("T", [23, 24, 25, 36, 37])
def test_experts_where_the_product_changes(T):
    """8 experts, 2 choices, so 6 to 9 rows each, and with 4 experts 12 and 13: both sides of the choice between kernels that
    gather tokens and kernels that read copies of them, by the same oracle."""
    for E in (4, 8):
        check_layer(layer(gen(T + E), T, E, 2, 1024, 384))


@pytest.mark.parametrize("rows", [12, 13])
def test_grouped_product_where_the_kernel_changes(rows):
    g = gen(rows)
    E, N, K = 16, 300, 1024
    q, s = R.reshard_quantize_rows(randn(g, rows * E, K).bfloat16())
    wq, ws = weights(g, E, N, K)
    offsets = torch.arange(0, rows * E + 1, rows, dtype=torch.int32, device="cuda")
    got = R.reshard_matmul_fp8(q, s, wq, ws, offsets=offsets, out_dtype=torch.float32).to(F64).view(E, rows, N)
    a, w = X.dequantize(X.values(q), s, 1).view(E, rows, K), X.dequantize(X.values(wq), ws, 128)
    want = a @ w.transpose(1, 2)
    tol = (128 + 3 * 8) * 2.0 ** -23 * (a.abs() @ w.abs().transpose(1, 2)) + 2.0 ** -24 * want.abs()
    assert bool(((got - want).abs() <= tol).all())
