"""The expert layer's kernels against the 64-bit oracle, at the sizes and values where they can go wrong.

Tolerances, from the arithmetic:
- fp32 scores and weights: an exponential (2 ulp), a reciprocal, a division and a sum of at most 1,024 terms added as
  32 per lane and then by halves: fewer than 64 roundings of 2^-24.
- the product: each block's 128 products are exact and summed in fp32 (at most 128 roundings or truncations of 2^-23 of the
  sum of magnitudes), then scaled and added block by block (3 more each); then the output's own rounding.
- the expert layer: h's 32-bit error moves a value across an e4m3 boundary for a share of about 3e-4 of them, by 2^-3 at
  most each (2e-3 of the norm); y and the output round to the type (2^-9 / sqrt(3) each for bf16): 5e-3 of the norm for
  bf16, 2.5e-3 for types of more bits, and six times that for a single row.
Codes, scales, ids, offsets and places are compared exactly.
"""
import pytest
import torch

from oracle import experts as X

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dtensor_resharding_gb300 as R

F64 = torch.float64
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_ULP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
F32 = 64 * 2.0 ** -24


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


# ----------------------------------------------------------------------------------------------------------- routing

def check_route(z, k, bias=None, **kw):
    w, ids = R.reshard_route(z, k, bias=bias, **kw)
    ww, want = X.route(z, k, bias=bias, **kw)
    assert torch.equal(ids.cpu().long(), want)
    assert w.dtype == torch.float32 and ids.dtype == torch.int32
    err = (w.cpu().to(F64) - ww).abs()
    assert bool((err <= F32 * ww.abs() + 1e-38).all()), err.max()
    return w, ids


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (7, 3), (33, 8), (60, 4), (64, 6), (128, 8), (130, 12), (256, 8), (300, 32), (512, 10), (1000, 5), (1024, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_orders_and_weighs(E, k, dtype, score):
    """16-bit logits repeat within a row: equal ones go to the lowest index."""
    z = (randn(gen(E + k), 9, E) * 1.5).to(DT[dtype])
    for renormalize in (True, False):
        check_route(z, k, score=score, renormalize=renormalize, scale=2.5 if renormalize else 1.0)


@pytest.mark.parametrize("E,k", [(32, 32), (60, 20), (128, 32), (256, 8), (300, 32), (1024, 32)])
def test_route_ties_and_neighbours(E, k):
    """Rows of few different logits, and rows whose largest are neighbours (held by one lane) or lie far apart."""
    g = gen(E * k)
    z = torch.randint(0, 3, (40, E), generator=g, device="cuda").float()
    z[0] = 1.0
    for i in range(1, 13):
        at = int(torch.randint(0, max(1, E - 16), (1,), generator=g, device="cuda"))
        z[i] = randn(g, E) - 20
        z[i, at:at + 16] += 20
        z[i + 13, ::(i * 11) % 37 + 1] += 3.0
    z[30, : E - k] = float("-inf")
    z[31, k:] = float("-inf")
    z[32, k // 2:] = float("nan")
    for dtype in (torch.float32, torch.bfloat16):
        check_route(z.to(dtype), k)


def separated(g, T, E, score):
    """f32 logits and a bias whose keys (score + bias) lie far apart against fp32 roundings: a permuted grid for each row."""
    bias = (torch.rand(E, generator=g, device="cuda") - 0.5) * 0.2
    grid = (torch.arange(E, device="cuda", dtype=F64) + 0.5) / E * 0.7 + 0.15
    key = torch.stack([grid[torch.randperm(E, generator=g, device="cuda")] for _ in range(T)])
    s = (key - bias.to(F64)).clamp(0.01, 0.99)
    z = torch.log(s / (1 - s)).float()
    keys = X.route_keys(z, score, bias).sort(1).values
    keep = (keys[:, 1:] - keys[:, :-1]).min(1).values > 1e-5
    assert int(keep.sum()) >= T // 2
    return z[keep], bias


@pytest.mark.parametrize("E,k", [(8, 3), (60, 4), (128, 8), (256, 8)])
def test_route_bias_selects_and_does_not_weigh(E, k):
    z, bias = separated(gen(E), 16, E, "sigmoid")
    check_route(z, k, bias=bias, score="sigmoid")
    soft = torch.log_softmax(z.to(F64), 1).float()      # scores of 1 / E: a bias of that size reorders them
    small = bias / E
    keys = X.route_keys(soft, "softmax", small).sort(1).values
    keep = (keys[:, 1:] - keys[:, :-1]).min(1).values > 1e-6 / E * 8
    check_route(soft[keep], k, bias=small, score="softmax", renormalize=False)


@pytest.mark.parametrize("E,groups,kept,k", [(8, 2, 1, 4), (60, 4, 2, 4), (64, 8, 4, 6), (96, 3, 2, 8), (128, 32, 5, 8), (256, 8, 4, 8), (256, 2, 1, 8), (264, 8, 3, 7),
                                             (1024, 8, 2, 8), (1024, 32, 7, 8)])
@pytest.mark.parametrize("top", [1, 2])
def test_route_groups(E, groups, kept, k, top):
    z = randn(gen(E * groups + top), 12, E) * 1.5
    for score in ("softmax", "sigmoid"):
        check_route(z, k, score=score, groups=groups, groups_kept=kept, group_top=top)
    check_route(z[:, :].bfloat16(), k, groups=groups, groups_kept=kept, group_top=1)      # equal logits, equal groups
    zb, bias = separated(gen(E + top), 12, E, "sigmoid")
    # a group's sum of two keys can come within a rounding of another's: rows where it does are left out
    part = X.route_keys(zb, "sigmoid", bias).view(zb.shape[0], groups, -1).topk(top, 2).values.sum(2).sort(1).values
    keep = (part[:, 1:] - part[:, :-1]).min(1).values > 1e-5
    if bool(keep.any()):
        check_route(zb[keep], k, bias=bias, score="sigmoid", groups=groups, groups_kept=kept, group_top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masked_rows(score, groups):
    """-inf and NaN are never chosen; rows with fewer than k left, and with none; a mask of the type's lowest value is a logit."""
    z = randn(gen(4), 8, 64)
    z[0, :] = float("-inf")
    z[1, 5:] = float("-inf")
    z[2, :] = float("nan")
    z[3, ::2] = float("nan")
    z[4, 3:] = torch.finfo(torch.float32).min
    z[5, :] = torch.finfo(torch.float32).min
    for renormalize in (True, False):
        w, ids = check_route(z, 8, score=score, renormalize=renormalize, groups=groups, groups_kept=groups, group_top=1)
        assert ids[0].tolist() == [-1] * 8 and ids[2].tolist() == [-1] * 8 and not w[0].any() and not w[2].any()
        assert bool(torch.isfinite(w).all())
        assert (ids[1] == -1).sum() == 3 and int(ids[4, 3]) == 3


def test_route_infinite_logits():
    z = torch.zeros(2, 40, device="cuda")
    z[0, 7] = float("inf")
    z[1, :] = -200.0          # sigmoid underflows to 0 with every weight: no division by 0
    w, ids = R.reshard_route(z, 2, score="sigmoid")
    assert ids.tolist() == [[7, 0], [0, 1]] and w[0, 0] > w[0, 1] and w[1].tolist() == [0.0, 0.0]
    w, ids = R.reshard_route(z, 2)
    assert ids.tolist() == [[7, 0], [0, 1]] and bool(torch.isnan(w[0]).any()) and w[1].tolist() == [0.5, 0.5]


@pytest.mark.parametrize("T", [0, 1, 5, 1025])
def test_route_rows_strides_and_alignment(T):
    big = randn(gen(9), T + 2, 201).bfloat16()
    for view in (big[1:T + 1, 3:63], big[1:T + 1, 4:132], big[:T, 1:129]):
        w, ids = R.reshard_route(view, 4)
        w2, ids2 = R.reshard_route(view.contiguous(), 4)
        assert torch.equal(w, w2) and torch.equal(ids, ids2)


@pytest.mark.parametrize("E,k", [(2, 2), (7, 3), (60, 4), (128, 8), (256, 8), (300, 32), (1000, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_route_backward(E, k, score, renormalize, dtype):
    """Against the formulas in 64 bits. An element is a difference of terms of at most scale * max|g|: 64 roundings of that."""
    g = gen(E + k)
    z = (randn(g, 13, E) * 1.5).to(DT[dtype])
    _, ids = R.reshard_route(z, k, score=score)
    ids[3, k - 1] = -1
    ids[4, :] = -1
    ids[5, 0] = E                # no expert: no gradient
    if k > 1:
        ids[6, 1] = ids[6, 0]    # a repeated expert: the sum of both
    grad = randn(g, 13, k)
    got = R.reshard_route_backward(grad, z, ids, score=score, renormalize=renormalize, scale=2.5)
    want = X.route_backward(grad, z, ids, score, renormalize, 2.5)
    assert got.dtype == z.dtype and got.shape == z.shape
    tol = F32 * 2.5 * float(grad.abs().max()) * k + HALF_ULP[z.dtype] * want.abs()
    assert bool(((got.to(F64) - want).abs() <= tol).all())
    assert not got[4].any()


def test_route_backward_against_differences():
    """The kernel's weights, differenced: h = 2^-7 leaves O(h^2) = 1e-4 of third derivatives below 1 and 2^-22 / h = 3e-5 of rounding."""
    g = gen(8)
    z = randn(g, 4, 16)
    grad = randn(g, 4, 3)
    h = 2.0 ** -7
    for score in ("softmax", "sigmoid"):
        _, ids = R.reshard_route(z, 3, score=score)
        got = R.reshard_route_backward(grad, z, ids, score=score)

        def loss(d):
            w = X.route_weights((z + d).to(F64), ids.long(), score, True, 1.0)
            return (w * grad).sum(1)
        for e in range(16):
            d = torch.zeros_like(z)
            d[:, e] = h
            assert torch.allclose(got[:, e].to(F64), (loss(d) - loss(-d)) / (2 * h), rtol=0, atol=2e-4 * float(grad.abs().max()))


def test_route_backward_masked_and_broadcast():
    z = randn(gen(2), 5, 32)
    z[0, :] = float("-inf")
    z[1, 4:] = float("-inf")
    z[2, 9] = float("nan")
    w, ids = R.reshard_route(z, 6, renormalize=False)
    grad = torch.ones(1, 1, device="cuda").expand(5, 6)         # as the gradient of a sum comes
    got = R.reshard_route_backward(grad, z, ids, renormalize=False)
    assert bool(torch.isfinite(got).all()) and not got[0].any() and not got[1, 4:].any() and got[2, 9] == 0
    clean = z[3:]
    want = X.route_backward(torch.ones(2, 6, device="cuda"), clean, ids[3:], "softmax", False, 1.0)
    assert bool(((got[3:].to(F64) - want).abs() <= 6 * F32).all())


# ---------------------------------------------------------------------------------------------------------- dispatch

@pytest.mark.parametrize("slots,E,first,local", [(0, 4, 0, 4), (1, 4, 0, 4), (31, 4, 0, 4), (500, 8, 2, 3), (4096, 128, 0, 128), (4097, 128, 96, 32),
                                                 (30011, 512, 0, 512), (70000, 3, 0, 3)])
def test_dispatch(slots, E, first, local):
    ids = torch.randint(-1, E, (slots,), generator=gen(slots), device="cuda", dtype=torch.int32)
    offsets, order, position = R.reshard_dispatch(ids, local, first)
    wo, wr, wp = X.dispatch(ids, local, first)
    assert offsets.tolist() == wo and order[:len(wr)].tolist() == wr and position.tolist() == wp


def test_dispatch_skewed_and_repeatable():
    ids = torch.full((20000,), 5, dtype=torch.int32, device="cuda")
    ids[7::1000] = 0
    first = [t.clone() for t in R.reshard_dispatch(ids, 8)]
    assert first[0].tolist() == X.dispatch(ids, 8)[0]
    for _ in range(3):
        again = R.reshard_dispatch(ids, 8)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ------------------------------------------------------------------------------------------------------ quantization

def same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 127), (5, 129), (33, 1000), (130, 2048), (2, 5001)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_rows(M, K, dtype):
    x = (randn(gen(M * K), M, K) * torch.logspace(-3, 2, K, device="cuda")).to(DT[dtype])
    q, scale = R.reshard_quantize_rows(x)
    wq, ws = X.quantize(x, 1)
    assert q.dtype == torch.float8_e4m3fn and q.shape == (M, K) and q.stride(0) % 16 == 0
    assert torch.equal(scale, ws) and torch.equal(X.values(q), wq.to(F64))


@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (130, 300), (2, 127, 129), (3, 256, 640), (4, 1, 4096)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_blocks(shape, dtype):
    w = (randn(gen(sum(shape)), *shape) * 0.02).to(DT[dtype])
    q, scale = R.reshard_quantize_blocks(w)
    wq, ws = X.quantize(w, 128)
    assert q.shape == w.shape and torch.equal(scale, ws) and torch.equal(X.values(q), wq.to(F64))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_special_values(dtype):
    """Zero blocks, the smallest and largest numbers of the type, and blocks that hold an infinity or NaN."""
    info = torch.finfo(DT[dtype])
    x = randn(gen(1), 6, 384).to(DT[dtype])
    x[0, :] = 0
    x[0, 130] = -0.0
    x[1, 5] = float("inf")
    x[2, 200] = float("nan")
    x[3, :128] = info.smallest_normal * 2 ** -3
    x[4, 1] = info.max
    x[5, 300:] = -info.max
    q, scale = R.reshard_quantize_rows(x)
    wq, ws = X.quantize(x, 1)
    assert same(scale, ws) and same(X.values(q), wq.to(F64))
    assert bool(scale[1, 0].isnan()) and not scale[1, 1:].isnan().any() and bool(scale[2, 1].isnan())
    assert torch.isfinite(scale[[0, 3, 4, 5]]).all() and X.values(q[4, 1:2]) == 448
    qb, sb = R.reshard_quantize_blocks(x)
    wb, wsb = X.quantize(x, 128)
    assert same(sb, wsb) and same(X.values(qb), wb.to(F64))


def test_quantize_strides_and_alignment():
    big = randn(gen(3), 40, 700).bfloat16()
    for view in (big[1:, 3:259], big[:, 8:264], big[::2, :256], big[:, 1:130]):
        for f in (R.reshard_quantize_rows, R.reshard_quantize_blocks):
            a, b = f(view), f(view.contiguous())
            assert torch.equal(X.values(a[0]), X.values(b[0])) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------------------------------------------- the product

def weights(g, *shape):
    return R.reshard_quantize_blocks(randn(g, *shape) * 0.02)


def check_product(got, q, s, wq, ws, dtype):
    a, w = X.dequantize(X.values(q), s, 1), X.dequantize(X.values(wq), ws, 128)
    want, size = a @ w.t(), a.abs() @ w.abs().t()
    kb = -(-q.shape[1] // 128)
    tol = (min(q.shape[1], 128) + 3 * kb) * 2.0 ** -23 * size + HALF_ULP[dtype] * want.abs() * (1 + 1e-3)
    assert got.dtype == dtype
    err = (got.to(F64) - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 64, 65, 100, 128, 129, 257, 700])
@pytest.mark.parametrize("N,K", [(1, 16), (64, 128), (127, 129), (130, 2048), (300, 1000), (515, 4111)])
def test_product(M, N, K):
    g = gen(M + N + K)
    x = randn(g, M, K).bfloat16()
    q, s = R.reshard_quantize_rows(x)
    wq, ws = weights(g, N, K)
    for dtype in (torch.bfloat16, torch.float32, torch.float16):
        check_product(R.reshard_matmul_fp8(q, s, wq, ws, out_dtype=dtype), q, s, wq, ws, dtype)
    y = R.reshard_linear_fp8(x, wq, ws)
    assert torch.equal(y, R.reshard_matmul_fp8(q, s, wq, ws))
    if K % 16 == 0:     # the bytes a reshard moves
        assert torch.equal(y, R.reshard_linear_fp8(x, wq.contiguous().view(torch.uint8), ws))


@pytest.mark.parametrize("N,K", [(4096, 1024), (2867, 4096), (14336, 512)])
@pytest.mark.parametrize("M", [1, 24, 77, 2000])
def test_product_whole_grid(M, N, K):
    """Sizes that fill the GPU several times over or split K over a cluster."""
    g = gen(N + M)
    x = randn(g, M, K).bfloat16()
    q, s = R.reshard_quantize_rows(x)
    wq, ws = weights(g, N, K)
    first = R.reshard_linear_fp8(x, wq, ws)
    check_product(first, q, s, wq, ws, torch.bfloat16)
    for _ in range(3):
        assert torch.equal(first, R.reshard_linear_fp8(x, wq, ws))


@pytest.mark.parametrize("counts", [[0, 0, 0], [1, 0, 2], [5, 17, 0, 1], [130, 0, 1, 255, 64], [300, 129], [1] * 40, [0, 700, 3],
                                    [0] * 60 + [400, 3], [17] * 40 + [0], [i % 3 for i in range(512)]])
@pytest.mark.parametrize("N,K", [(130, 300), (256, 1024)])
def test_grouped_product(counts, N, K):
    """Empty groups, groups of one row, groups that end inside a tile, rows beyond the last group untouched."""
    g = gen(len(counts) + N)
    E, M = len(counts), sum(counts) + 5
    q, s = R.reshard_quantize_rows(randn(g, M, K).bfloat16())
    wq, ws = weights(g, E, N, K)
    offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    out = torch.full((M, N + 14), 7.0, dtype=torch.bfloat16, device="cuda")[:, 3:N + 3]      # rows at odd places
    R.reshard_matmul_fp8(q, s, wq, ws, offsets=offsets, out=out)
    boxed = R.reshard_matmul_fp8(q, s, wq, ws, offsets=offsets)
    for e, n in enumerate(counts):
        r = slice(int(offsets[e]), int(offsets[e]) + n)
        check_product(out[r], q[r], s[r], wq[e], ws[e], torch.bfloat16)
        assert torch.equal(out[r], boxed[r])
    assert bool((out[sum(counts):] == 7).all())


def test_grouped_product_keeps_offsets_in_bounds():
    """Offsets come from the device: what lies outside the rows is cut off."""
    g = gen(6)
    q, s = R.reshard_quantize_rows(randn(g, 40, 256).bfloat16())
    wq, ws = weights(g, 3, 128, 256)
    out = R.reshard_matmul_fp8(q, s, wq, ws, offsets=torch.tensor([-5, 10, 1000, 2000], dtype=torch.int32, device="cuda"))
    check_product(out[:10], q[:10], s[:10], wq[0], ws[0], torch.bfloat16)
    check_product(out[10:], q[10:], s[10:], wq[1], ws[1], torch.bfloat16)


def test_product_rows_do_not_reach_one_another():
    """A row of NaN (or of infinities, which quantize to it) leaves the others' results as they are."""
    g = gen(7)
    for M in (3, 40, 200):
        x = randn(g, M, 512).bfloat16()
        wq, ws = weights(g, 200, 512)
        clean = R.reshard_linear_fp8(x, wq, ws)
        x[1, 100] = float("inf")
        got = R.reshard_linear_fp8(x, wq, ws)
        assert bool(got[1].isnan().all())
        keep = [i for i in range(M) if i != 1]
        assert torch.equal(got[keep], clean[keep])


def test_product_strides():
    g = gen(11)
    big = randn(g, 70, 1200).bfloat16()
    wq, ws = weights(g, 3, 144, 512)
    x = big[:, 5:517]
    want = R.reshard_linear_fp8(x.contiguous(), wq[1], ws[1])
    assert torch.equal(want, R.reshard_linear_fp8(x, wq[1], ws[1]))
    for off in (1, 8):
        out = torch.zeros(70, 300, dtype=torch.bfloat16, device="cuda")[:, off:off + 144]
        R.reshard_linear_fp8(x, wq[1], ws[1], out=out)
        assert torch.equal(want, out)
    pitched = torch.zeros(144, 1024, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, 16:528]
    pitched.view(torch.uint8).copy_(wq[1].view(torch.uint8))
    assert torch.equal(want, R.reshard_linear_fp8(x, pitched, ws[1]))


def test_input_gradient_is_the_product_with_transposed_blocks():
    """d x = Q(d y) W through the transposed bytes and block scales, against the 64-bit product, and with it differences
    of the loss (linear in x but for its quantization, which is left out: x enters as values)."""
    g = gen(12)
    dy = randn(g, 50, 384).bfloat16()
    wq, ws = weights(g, 384, 256)
    wt = wq.view(torch.uint8).t().contiguous()
    dx = R.reshard_linear_fp8(dy, wt, ws.t().contiguous())
    q, s = R.reshard_quantize_rows(dy)
    check_product(dx, q, s, wt.view(torch.float8_e4m3fn), ws.t(), torch.bfloat16)
    w = X.dequantize(X.values(wq), ws, 128)
    x = randn(g, 50, 256).to(F64)
    d, h = randn(g, 50, 256).to(F64), 2.0 ** -10
    up = X.dequantize(X.values(q), s, 1)
    diff = ((((x + h * d) @ w.t()) * up).sum() - (((x - h * d) @ w.t()) * up).sum()) / (2 * h)
    assert abs(float((dx.to(F64) * d).sum() - diff)) <= 2.0 ** -9 * float((dx.to(F64) * d).abs().sum())


def test_offsets_beyond_32_bits():
    """Weights of more than 2^32 bytes, and an output whose elements lie beyond 2^31."""
    g = gen(13)
    E, N, K = 129, 8192, 4096
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    ws = torch.ones(E, N // 128, K // 128, device="cuda")
    wq, s1 = weights(g, N, K)
    w[E - 1].copy_(wq.view(torch.uint8))
    ws[E - 1].copy_(s1)
    for M in (4, 200):
        q, s = R.reshard_quantize_rows(randn(g, M, K).bfloat16())
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[E] = M
        check_product(R.reshard_matmul_fp8(q, s, w, ws, offsets=offsets), q, s, wq, s1, torch.bfloat16)
    del w
    M, step = 70000, 40000
    x = randn(g, M, 128).bfloat16()
    out = torch.empty(M, step, dtype=torch.bfloat16, device="cuda")[:, :128]
    wq, ws = weights(g, 128, 128)
    R.reshard_linear_fp8(x, wq, ws, out=out)
    assert torch.equal(out[-3000:], R.reshard_linear_fp8(x[-3000:], wq, ws))


# ---------------------------------------------------------------------------------------------------- the expert layer

def layer(g, T, E, k, H, I, local=None, dtype=torch.bfloat16):
    n = E if local is None else local
    x = randn(g, T, H).to(dtype)
    w, ids = R.reshard_route(randn(g, T, E), k)
    return (x, ids, w, *weights(g, n, 2 * I, H), *weights(g, n, H, I))


def check_layer(got, args, first=0):
    want = X.experts(*args, first=first)
    tol = 5e-3 if got.dtype == torch.bfloat16 else 2.5e-3
    err = got.to(F64) - want
    assert float(err.norm()) <= tol * float(want.norm()), float(err.norm() / want.norm())
    assert bool((err.norm(dim=1) <= 6 * tol * want.norm(dim=1) + 1e-30).all())


@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 128, 128), (1, 128, 8, 512, 256), (7, 8, 3, 272, 384), (24, 16, 4, 512, 128), (40, 4, 2, 640, 256),
                                       (100, 4, 4, 384, 256), (300, 4, 2, 512, 384), (513, 16, 1, 1008, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_experts(T, E, k, H, I, dtype):
    args = layer(gen(T + H), T, E, k, H, I, dtype=DT[dtype])
    out = R.reshard_experts_fp8(*args)
    check_layer(out, args)
    assert torch.equal(out, R.reshard_experts_fp8(*args))


@pytest.mark.parametrize("T", [5, 700])
def test_experts_shares_add_up(T):
    """Every rank's share: ids of other ranks and -1 add nothing, a rank without tokens gives zeros."""
    x, ids, w, w13, s13, w2, s2 = layer(gen(T), T, 16, 3, 256, 128)
    ids[::3, 2] = -1
    check_layer(R.reshard_experts_fp8(x, ids, w, w13, s13, w2, s2), (x, ids, w, w13, s13, w2, s2))
    for first, n in ((0, 5), (5, 11), (15, 1)):
        part = slice(first, first + n)
        args = (x, ids, w, w13[part], s13[part], w2[part], s2[part])
        check_layer(R.reshard_experts_fp8(*args, first_expert=first), args, first)
    none = R.reshard_experts_fp8(x, torch.full_like(ids, -1), w, w13, s13, w2, s2)
    assert none.shape == x.shape and not none.any()
    away = R.reshard_experts_fp8(x, ids, w, w13, s13, w2, s2, first_expert=16)
    assert not away.any()


def test_experts_nothing_to_do_and_skew():
    x, ids, w, w13, s13, w2, s2 = layer(gen(1), 600, 8, 2, 256, 128)
    assert R.reshard_experts_fp8(x[:0], ids[:0], w[:0], w13, s13, w2, s2).shape == (0, 256)
    ids[:, 0], ids[:, 1] = 7, 2           # all tokens to two experts
    check_layer(R.reshard_experts_fp8(x, ids, w, w13, s13, w2, s2), (x, ids, w, w13, s13, w2, s2))


def test_stages_equal_the_whole():
    """dispatch, quantization and grouped products by hand give what the layer's own enqueue of them gives."""
    T, k, E, H, I = 200, 2, 4, 384, 256
    x, ids, w, w13, s13, w2, s2 = layer(gen(5), T, E, k, H, I)
    out = R.reshard_experts_fp8(x, ids, w, w13, s13, w2, s2)
    offsets, order, position = R.reshard_dispatch(ids, E)
    q, s = R.reshard_quantize_rows(x[order.long() // k])
    gu = R.reshard_matmul_fp8(q, s, w13, s13, offsets=offsets, out_dtype=torch.float32)
    h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    hq, hs = R.reshard_quantize_rows(h)
    y = R.reshard_matmul_fp8(hq, hs, w2, s2, offsets=offsets)
    want = (y[position.long()].view(T, k, H).float() * w[..., None]).sum(1)
    # the fused silu differs by some 2^-21: a share of about 1e-4 of h moves by an e4m3 step
    assert float((out.float() - want).norm()) <= 4e-3 * float(want.norm())


# ----------------------------------------------------------------------------------------------- streams, graphs, refusals

def test_other_stream_and_graph():
    x, ids, w, w13, s13, w2, s2 = layer(gen(3), 48, 8, 2, 256, 128)
    z = randn(gen(4), 48, 8)
    want = R.reshard_experts_fp8(x, ids, w, w13, s13, w2, s2)
    want_w, want_ids = R.reshard_route(z, 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = R.reshard_experts_fp8(x, ids, w, w13, s13, w2, s2, stream=side.cuda_stream)
    rw, rids = R.reshard_route(z, 2, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(rw, want_w) and torch.equal(rids, want_ids)
    xs = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gw, gids = R.reshard_route(z, 2)
        out = R.reshard_experts_fp8(xs, ids, w, w13, s13, w2, s2)
        lin = R.reshard_linear_fp8(xs, w2[0, :, :].view(torch.uint8).t().contiguous(), s2[0].t().contiguous())
    for scale in (1.0, 0.5):
        xs.copy_(x * scale)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, R.reshard_experts_fp8(xs, ids, w, w13, s13, w2, s2)) and torch.equal(gids, want_ids)
    assert torch.equal(out, out) and lin.shape == (48, 128)


def test_refusals_name_what_is_wrong():
    g = gen(1)
    x = randn(g, 4, 256).bfloat16()
    wq, ws = weights(g, 128, 256)
    z = randn(g, 4, 8)
    _, ids = R.reshard_route(z, 2)
    cases = [
        (lambda: R.reshard_route(z.t(), 2), "contiguous rows"),
        (lambda: R.reshard_route(z.to(F64), 2), "float32"),
        (lambda: R.reshard_route(z, 9), "k at most experts"),
        (lambda: R.reshard_route(z, 2, score="tanh"), "score"),
        (lambda: R.reshard_route(z, 2, bias=torch.zeros(7, device="cuda")), "bias"),
        (lambda: R.reshard_route(z, 2, groups=3, groups_kept=3), "divide"),
        (lambda: R.reshard_route_backward(torch.zeros(4, 3, device="cuda"), z, ids), "grad_weights"),
        (lambda: R.reshard_route_backward(torch.zeros(4, 2, device="cuda"), z, ids.long()), "ids"),
        (lambda: R.reshard_linear_fp8(x, wq, ws.double()), "scale"),
        (lambda: R.reshard_linear_fp8(x, wq, ws[:, :1]), "scale"),
        (lambda: R.reshard_linear_fp8(x[:, :128], wq, ws), "columns"),
        (lambda: R.reshard_linear_fp8(x, wq.float(), ws), "float8"),
        (lambda: R.reshard_linear_fp8(x, wq.view(torch.uint8)[:, :250].contiguous(), ws), "columns"),
        (lambda: R.reshard_linear_fp8(x[:, :250].contiguous(), wq.view(torch.uint8)[:, :250].contiguous(), ws), "multiple of 16"),
        (lambda: R.reshard_linear_fp8(x, wq.view(torch.uint8).flatten()[8:].resize_(1), ws), "dimensions"),
        (lambda: R.reshard_linear_fp8(x, wq, ws, out=torch.zeros(4, 128, device="cuda")), "out"),
        (lambda: R.reshard_matmul_fp8(x, ws, wq, ws), "float8"),
        (lambda: R.reshard_experts_fp8(x, ids, torch.zeros(4, 2, device="cuda"), wq[None], ws[None], wq[None], ws[None]), "fit"),
        (lambda: R.reshard_experts_fp8(x, ids.cpu(), torch.zeros(4, 2, device="cuda"), wq[None], ws[None], wq[None], ws[None]), "ids"),
    ]
    for call, word in cases:
        with pytest.raises(R.ReshardError) as e:
            call()
        assert word in str(e.value), (word, str(e.value))
    # pageable host memory at the C entry: refused, not dereferenced
    host = torch.zeros(4, 8)
    w, i = torch.zeros(4, 2, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    rc = R.binding.LIB.reshard_route(host.data_ptr(), 3, 4, 8, 8, None, 0, 1, 1, 1, 2, 1, 1.0, w.data_ptr(), i.data_ptr(), None)
    assert rc == R.RESHARD_ERR_INVALID_ARG and "pageable" in R.reshard_last_error()


def test_example_refits_and_computes():
    """The example's generation ranks against the layer in one piece: a rank's share rounds to bf16 (2^-8 at most) once more."""
    import importlib.util
    import os

    from conftest import ROOT
    spec = importlib.util.spec_from_file_location("refit_experts", os.path.join(ROOT, "examples", "refit_experts.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main([]) < 2 ** -7
    assert example.main(["--tokens", "3", "--experts", "8", "--hidden", "384", "--ffn", "256", "--train", "4", "--gen", "4", "--k", "2"]) < 2 ** -7
