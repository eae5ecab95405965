"""Rows moved by an index and their gradients against the 64-bit oracle, at the sizes and values where they can go wrong.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32 relative to the value):
- a sum of n terms in fp32, each added by one fused operation: n u of the sum of the terms' magnitudes.
- a dot product over H columns: a lane adds its share of the products, then five additions by shuffles: (H / 32 + 32) u of
  the sum of the products' magnitudes (a lane has up to 8 columns more than H / 32, and 16 where rows start anywhere).
- a product in fp32 is off by u; what is rounded to a type by half a step of it, at least half its smallest number.
What is copied is compared bit for bit.
"""
import pytest
import torch
from torch.autograd import forward_ad

from oracle import rows as X

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dtensor_resharding_gb300 as R

F64 = torch.float64
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def close(got, want, loose):
    """|got - want| <= loose (what the fp32 arithmetic may be off by) + half a step of got's type."""
    info = torch.finfo(got.dtype)
    step = (want.abs() + loose) * (info.eps / 2) + info.smallest_normal * info.eps / 2
    bad = (got.to(F64) - want).abs() - loose - step
    assert bool((bad <= 0).all()), (float(bad.max()), torch.nonzero(bad > 0)[:4].tolist())


def laid(x, how):
    """The same values dense, with a pitch, from an element that is no 16-byte boundary, or with columns between them."""
    rows, cols = x.shape
    if how == "dense":
        return x.contiguous().clone()
    pitch, skip = {"pitch": (-(-cols // 16) * 16 + 16, 0), "odd": (cols + 3, 1)}[how]
    buf = torch.full((rows * pitch + skip + 8,), float("nan"), dtype=x.dtype, device=x.device)
    v = buf[skip:skip + rows * pitch].view(rows, pitch)[:, :cols]
    v.copy_(x)
    return v


def case(seed, T, k, E, H, dtype, first=0, local=None):
    """(x, ids, sort of this rank's experts)"""
    g = gen(seed)
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int() if T else torch.empty(0, k, dtype=torch.int32, device="cuda")
    return randn(g, T, H).to(DT[dtype]), ids, R.reshard_dispatch(ids, local or E, first)


SHAPES = [(1, 1, 1, 1), (1, 8, 16, 2048), (5, 2, 4, 7), (17, 3, 8, 130), (64, 4, 8, 1000), (33, 8, 8, 2867), (300, 2, 16, 64), (9, 12, 40, 8200), (2, 40, 64, 256)]


@pytest.mark.parametrize("T,k,E,H", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("how", ["dense", "pitch", "odd"])
@pytest.mark.parametrize("share", [False, True])
def test_permute(T, k, E, H, dtype, how, share):
    first, local = (E // 4, max(1, E // 2)) if share else (0, E)
    x, ids, sort = case(T + H, T, k, E, H, dtype, first, local)
    x = laid(x, how)
    offsets, order, position = sort
    held = int(offsets[-1])
    got = R.reshard_permute(x, sort)
    assert got.shape == (T * k, H) and torch.equal(got[:held], x[order[:held].long() // k]) and not bool(got[held:].any())
    # rows behind the last expert, of a longer and of a shorter buffer, stay as they were
    for rows in (T * k + 3, max(1, held - 1)):
        to = laid(torch.full((rows, H), 7.0, dtype=x.dtype, device="cuda"), how)
        want = X.permute(x, position, to)
        assert R.reshard_permute(x, sort, out=to) is to and torch.equal(to, want)
        assert bool((to[held:] == 7.0).all())


@pytest.mark.parametrize("H", [64, 67])
def test_permute_copies_bits(H):
    """Every 16-bit pattern, NaN payloads among them."""
    x = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16)
    for dtype in (torch.bfloat16, torch.float16):
        v = x[:65536 // H * H].view(-1, H).view(dtype)
        ids = torch.zeros(v.shape[0], 1, dtype=torch.int32, device="cuda")
        y = R.reshard_permute(v, R.reshard_dispatch(ids, 1))
        assert torch.equal(y.view(torch.int16), v.view(torch.int16))
        table = R.reshard_embedding(torch.arange(v.shape[0], device="cuda"), v)
        assert torch.equal(table.view(torch.int16), v.view(torch.int16))


@pytest.mark.parametrize("H", [64, 67])
def test_sorts_that_are_none(H):
    """Positions beyond the rows, negative ones, several slots at one place, an order that names other slots: nothing outside
    the rows is touched, and only a slot that order names writes its place."""
    T, k = 6, 2
    x = randn(gen(1), T, H)
    position = torch.tensor([0, 0, 5, -1, -7, 12, 2 ** 31 - 1, 3, 3, 1, -2 ** 31, 4], dtype=torch.int32, device="cuda")
    order = torch.tensor([1, 9, -1, 8, 3, 2, 2 ** 31 - 1, 0, 0, 0, 0, 0], dtype=torch.int32, device="cuda")
    sort = (torch.zeros(1, dtype=torch.int32, device="cuda"), order, position)
    owners = {0: 1, 1: 9, 3: 8, 5: 2}                # place: slot; place 4's slot 11 is not the one order names
    to = torch.full((12, H), 7.0, device="cuda")
    R.reshard_permute(x, sort, out=to)
    for p in range(12):
        assert torch.equal(to[p], x[owners[p] // k] if p in owners else torch.full((H,), 7.0, device="cuda")), p
    fresh = R.reshard_permute(x, sort)
    for p in range(12):
        assert torch.equal(fresh[p], x[owners[p] // k] if p in owners else torch.zeros(H, device="cuda")), p
    y, w, g = randn(gen(2), 12, H), randn(gen(3), T, k), randn(gen(4), T, H)
    close(R.reshard_combine(y, sort, w), X.combine(y, position, w, k), k * U * X.combine(y, position, w, k, True))
    dy, dw = R.reshard_combine_backward(g, y, sort, w)
    want = torch.zeros_like(y)
    for p, s in owners.items():
        want[p] = g[s // k] * w.view(-1)[s]
    assert torch.equal(dy, want)
    close(dw, X.combine_backward(g, y, position, w, k)[1], (H / 32 + 32) * U * X.combine_backward(g, y, position, w, k, True)[1])


@pytest.mark.parametrize("T,k,E,H", SHAPES)
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("how", ["dense", "pitch", "odd"])
@pytest.mark.parametrize("share", [False, True])
def test_combine_and_its_gradients(T, k, E, H, types, how, share):
    first, local = (E // 4, max(1, E // 2)) if share else (0, E)
    dtype, out_dtype = types
    g = gen(T * H + k)
    _, ids, sort = case(T + k, T, k, E, 1, "f32", first, local)
    offsets, order, position = sort
    held = int(offsets[-1])
    y = randn(g, T * k, H).to(DT[dtype])
    y[held:] = float("nan")                          # rows of no slot are not read
    y, w, grad = laid(y, how), torch.softmax(randn(g, T, k), 1), laid(randn(g, T, H).to(DT[out_dtype]), how)
    w.view(-1)[position < 0] = float("nan")          # nor are weights of slots without a place
    out = R.reshard_combine(y, sort, w, out_dtype=DT[out_dtype])
    assert out.dtype is DT[out_dtype]
    close(out, X.combine(y, position, w, k), k * U * X.combine(y, position, w, k, True))
    to = laid(torch.zeros(T, H, dtype=DT[out_dtype], device="cuda"), how)
    assert torch.equal(R.reshard_combine(y, sort, w, out=to), out) and torch.equal(to, out)
    dy, dw = R.reshard_combine_backward(grad, y, sort, w)
    wy, ww = X.combine_backward(grad, y, position, w, k)
    assert dy.dtype is y.dtype and dy.shape == y.shape and not bool(dy[held:].any())
    close(dy, wy, U * wy.abs())
    close(dw, ww, (H / 32 + 32) * U * X.combine_backward(grad, y, position, w, k, True)[1])
    assert bool((dw.view(-1)[position < 0] == 0).all())
    only_y, none = R.reshard_combine_backward(grad, y, sort, w, needs=(True, False))
    assert none is None and torch.equal(only_y, dy)
    none, only_w = R.reshard_combine_backward(grad, y, sort, w, needs=(False, True))
    assert none is None and torch.equal(only_w, dw)
    # without weights: the gradient of the permutation
    sums = R.reshard_permute_backward(y, sort, k)
    close(sums, X.combine(y, position, None, k), k * U * X.combine(y, position, None, k, True))


@pytest.mark.parametrize("T", [0, 1, 40])
def test_nothing_is_here(T):
    """No token, or none of a token's experts on this rank: zeros, and nothing written to the places."""
    _, ids, sort = case(1, T, 2, 8, 16, "f32", first=100, local=4)
    x, y = randn(gen(2), T, 16), randn(gen(3), 2 * T, 16)
    to = torch.full((2 * T + 1, 16), 3.0, device="cuda")
    assert bool((R.reshard_permute(x, sort, out=to) == 3.0).all()) and not bool(R.reshard_permute(x, sort).any())
    w = torch.rand(T, 2, device="cuda")
    assert not bool(R.reshard_combine(y, sort, w).any()) and R.reshard_combine(y, sort, w).shape == (T, 16)
    dy, dw = R.reshard_combine_backward(x, y, sort, w)
    assert not bool(dy.any()) and not bool(dw.any()) and dy.shape == y.shape and dw.shape == w.shape


def test_infinities_stay_in_their_rows():
    T, k, H = 8, 2, 96
    _, ids, sort = case(4, T, k, 4, 1, "f32")
    position = sort[2].view(T, k)
    y, w = randn(gen(5), T * k, H), torch.rand(T, k, device="cuda") + 0.5
    y[position[3, 1].long(), 5] = float("inf")
    y[position[5, 0].long(), 7] = float("nan")
    out = R.reshard_combine(y, sort, w)
    assert float(out[3, 5]) == float("inf") and bool(torch.isnan(out[5, 7])) and int((~torch.isfinite(out)).sum()) == 2
    dw = R.reshard_combine_backward(torch.ones(T, H, device="cuda"), y, sort, w)[1]
    assert int((~torch.isfinite(dw)).sum()) == 2 and not bool(torch.isfinite(dw[3, 1])) and bool(torch.isnan(dw[5, 0]))


# --------------------------------------------------------------------------------------------------------- embedding

@pytest.mark.parametrize("T,rows,H", [(0, 5, 16), (1, 1, 1), (1, 50, 4096), (7, 13, 33), (33, 100, 1000), (500, 40, 2867), (130, 1000, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("how", ["dense", "pitch", "odd"])
@pytest.mark.parametrize("wide_ids", [False, True])
def test_embedding(T, rows, H, dtype, how, wide_ids):
    g = gen(T + rows)
    first = rows // 2
    ids = torch.randint(-3, 2 * rows + 3, (T,), generator=g, device="cuda", dtype=torch.int64 if wide_ids else torch.int32)
    table = laid(randn(g, rows, H).to(DT[dtype]), how)
    got = R.reshard_embedding(ids, table, first_row=first)
    assert got.dtype is table.dtype and torch.equal(got.to(F64), X.embedding(ids, table, 1.0, first))
    want = X.embedding(ids, table, 45.25, first)
    to = laid(torch.zeros(T, H, dtype=DT[dtype], device="cuda"), how)
    assert R.reshard_embedding(ids, table, scale=45.25, first_row=first, out=to) is to
    close(to, want, U * want.abs())
    assert torch.equal(R.reshard_embedding(ids, table, scale=45.25, first_row=first), to)


def test_embedding_ids_of_any_shape_and_value():
    g = gen(7)
    table = randn(g, 20, 48)
    ids = torch.randint(0, 20, (3, 4, 5), generator=g, device="cuda")
    assert torch.equal(R.reshard_embedding(ids, table), table[ids])
    assert torch.equal(R.reshard_embedding(ids.transpose(0, 2), table), table[ids.transpose(0, 2)])
    assert torch.equal(R.reshard_embedding(ids[:, :, 1:3], table), table[ids[:, :, 1:3]])
    far = torch.tensor([2 ** 62, -2 ** 62, 2 ** 32 + 3, -1, 19, 20], device="cuda")
    want = torch.zeros(6, 48, device="cuda")
    want[4] = table[19]
    assert torch.equal(R.reshard_embedding(far, table), want)
    got = R.reshard_embedding_backward(torch.ones(6, 48, device="cuda"), far, 20)
    assert float(got[19].sum()) == 48 and float(got.sum()) == 48
    # a shard whose rows lie beyond 32 bits
    got = R.reshard_embedding(far, table, first_row=2 ** 32)
    assert torch.equal(got[2], table[3]) and not bool(got[[0, 1, 3, 4, 5]].any())
    assert R.reshard_embedding(ids, table[:0]).shape == (3, 4, 5, 48) and not bool(R.reshard_embedding(ids, table[:0]).any())
    assert R.reshard_embedding(ids, table[:, :0]).shape == (3, 4, 5, 0)


def check_embedding_backward(grad, ids, rows, first=0, scale=1.0, **kw):
    got = R.reshard_embedding_backward(grad, ids, rows, scale=scale, first_row=first, **kw)
    want = X.embedding_backward(grad, ids, rows, scale, first)
    r = ids.long().reshape(-1) - first
    most = int(torch.bincount(r[(r >= 0) & (r < rows)], minlength=1).max()) if ids.numel() else 0
    # n additions and the scale's product
    close(got, want, (most + 2) * U * X.embedding_backward(grad, ids, rows, abs(scale), first, True))
    return got


@pytest.mark.parametrize("T,V,rows,H", [(0, 4, 4, 8), (1, 4, 4, 8), (1, 1, 1, 1), (15, 3, 3, 40), (16, 16, 16, 1024), (17, 30, 11, 33), (200, 7, 7, 2867), (255, 40, 30, 520), (256, 3, 3, 64), (257, 3, 3, 64), (1000, 5000, 1250, 64),
                                        (5000, 300, 300, 130), (40000, 70000, 70000, 24), (33000, 2000, 500, 256), (70000, 9, 9, 16)])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("skew", [False, True])
def test_embedding_backward(T, V, rows, H, types, skew):
    g = gen(T + V + H)
    first = (V - rows) // 2
    u = torch.rand(T, generator=g, device="cuda", dtype=F64)
    ids = ((torch.exp(u * torch.log(torch.tensor(V + 1.0, dtype=F64, device="cuda"))) - 1).long() if skew else (u * V).long()).clamp_max(V - 1)
    grad = randn(g, T, H).to(DT[types[0]])
    got = check_embedding_backward(grad, ids, rows, first, scale=1.0 if skew else 0.3, dtype=DT[types[1]])
    assert got.dtype is DT[types[1]] and got.shape == (rows, H)
    assert torch.equal(got, R.reshard_embedding_backward(grad, ids.int(), rows, first_row=first, scale=1.0 if skew else 0.3, dtype=DT[types[1]]))


@pytest.mark.parametrize("T", [1, 31, 32, 33, 255, 256, 257, 3000, 50000])
@pytest.mark.parametrize("how", ["dense", "pitch", "odd"])
def test_embedding_backward_one_row_takes_all(T, how):
    """All tokens of one id: the row's sum passes through every run and is joined from their pieces."""
    g = gen(T)
    grad = laid(randn(g, T, 72).bfloat16(), how)
    ids = torch.full((T,), 3, device="cuda")
    for rows, first in ((7, 0), (1, 3)):
        check_embedding_backward(grad, ids, rows, first, dtype=torch.float32)
    ids[T // 2] = 2                                   # and one token of another
    check_embedding_backward(grad, ids, 7, dtype=torch.float32)


@pytest.mark.parametrize("H", [64, 67])
@pytest.mark.parametrize("how", ["dense", "pitch", "odd"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_embedding_backward_accumulates(H, how, dtype):
    g = gen(H)
    ids = torch.randint(0, 40, (300,), generator=g, device="cuda") * 2       # odd rows have no token
    grad, base = randn(g, 300, H).bfloat16(), randn(g, 80, H).to(DT[dtype])
    base[1::2] = float("nan")
    main = laid(base, how)
    assert R.reshard_embedding_backward(grad, ids, 80, scale=0.5, out=main, accumulate=True) is main
    assert bool(torch.isnan(main[1::2]).all())
    want = X.embedding_backward(grad, ids, 80, 0.5)
    loose = 40 * U * X.embedding_backward(grad, ids, 80, 0.5, magnitudes=True) + U * base.to(F64).abs()
    close(main[::2], (want + base.to(F64))[::2], loose[::2])
    whole = laid(base, how)                            # written whole: what was there is gone, between the rows it stays
    R.reshard_embedding_backward(grad, ids, 80, scale=0.5, out=whole)
    assert not bool(whole[1::2].any()) and torch.equal(whole, R.reshard_embedding_backward(grad, ids, 80, scale=0.5, dtype=DT[dtype]))
    if how == "pitch":
        assert bool(torch.isnan(whole.as_strided((79, 16), (whole.stride(0), 1), whole.storage_offset() + whole.shape[1])).all())


def test_embedding_backward_keeps_its_order():
    """The same inputs give the same bits, and other tokens do not change a row's."""
    g = gen(9)
    ids = torch.randint(0, 50, (20000,), generator=g, device="cuda")
    grad = randn(g, 20000, 128)
    first = R.reshard_embedding_backward(grad, ids, 50)
    for _ in range(3):
        assert torch.equal(first, R.reshard_embedding_backward(grad, ids, 50))
    inf = grad.clone()
    inf[ids == 7] = float("inf")
    other = R.reshard_embedding_backward(inf, ids, 50)
    keep = torch.arange(50, device="cuda") != 7
    assert torch.equal(other[keep], first[keep]) and bool(torch.isinf(other[7]).all())


def test_rows_beyond_32_bits():
    """Rows 2^28 elements apart: the tenth begins beyond 2^31 elements."""
    step, H = 1 << 28, 40
    big = torch.empty(9 * step + H, dtype=torch.bfloat16, device="cuda").as_strided((10, H), (step, 1))
    big.copy_(randn(gen(3), 10, H))
    ids = torch.arange(10, device="cuda", dtype=torch.int32).view(10, 1)
    sort = R.reshard_dispatch(9 - ids, 10)
    y = R.reshard_permute(big, sort)
    assert torch.equal(y, big.flip(0))
    assert torch.equal(R.reshard_embedding(ids.view(-1), big), big.contiguous())
    one = torch.ones(10, 1, device="cuda")
    assert torch.equal(R.reshard_combine(big, sort, one), y)
    grad = big.contiguous()
    dy, dw = R.reshard_combine_backward(grad, big, sort, one)
    assert torch.equal(dy, y)
    close(dw, (grad.to(F64) * y.to(F64)).sum(1, keepdim=True), 40 * U * (grad.to(F64) * y.to(F64)).abs().sum(1, keepdim=True))
    small = grad.clone()
    R.reshard_permute(small, sort, out=big)
    assert torch.equal(big, small.flip(0))
    R.reshard_embedding_backward(small, ids.view(-1), 10, out=big)
    assert torch.equal(big, small)
    R.reshard_embedding_backward(big, ids.view(-1), 10, out=small, accumulate=True)
    assert torch.equal(small, big * 2)


# ------------------------------------------------------------------------------------ gradients, streams, graphs, refusals

@pytest.mark.parametrize("H", [48, 67])
def test_gradients_against_differences(H):
    """The calls are linear in each input: a difference over any step is the derivative, up to the roundings of both sides."""
    T, k = 5, 2
    g = gen(H)
    x, ids, sort = case(H, T, k, 4, H, "f32", first=1, local=3)
    position = sort[2]
    y, w, grad = randn(g, T * k, H), torch.rand(T, k, generator=g, device="cuda"), randn(g, T, H)
    dy, dw = R.reshard_combine_backward(grad, y, sort, w)
    loss = lambda yy, ww: float((R.reshard_combine(yy, sort, ww).to(F64) * grad.to(F64)).sum())      # noqa: E731
    bound = 4 * k * U * float((X.combine(y, position, w, k, True) * grad.abs().to(F64)).sum() + grad.abs().to(F64).sum() * 4)
    for s in range(T * k):
        h = torch.zeros_like(w)
        h.view(-1)[s] = 0.5
        assert abs(loss(y, w + h) - loss(y, w - h) - float(dw.view(-1)[s])) <= bound + abs(float(dw.view(-1)[s])) * H * U, s
        h = torch.zeros_like(y)
        h[s, s % H] = 0.5
        assert abs(loss(y + h, w) - loss(y - h, w) - float(dy[s, s % H])) <= bound, s
    place = randn(g, T * k, H)
    place[int(sort[0][-1]):] = 0
    dx = R.reshard_permute_backward(place, sort, k)
    zero = torch.zeros(T * k, H, device="cuda")
    loss = lambda xx: float((R.reshard_permute(xx, sort, out=zero.clone()).to(F64) * place.to(F64)).sum())      # noqa: E731
    for t in range(T):
        h = torch.zeros_like(x)
        h[t, 3] = 0.5
        assert abs(loss(x + h) - loss(x - h) - float(dx[t, 3])) <= 8 * k * U * float(place.abs().sum() * x.abs().max()), t
    table, tokens = randn(g, 9, H), torch.randint(0, 12, (30,), generator=g, device="cuda")
    out = randn(g, 30, H)
    dt = R.reshard_embedding_backward(out, tokens, 9, scale=2.0, first_row=2)
    loss = lambda tt: float((R.reshard_embedding(tokens, tt, scale=2.0, first_row=2).to(F64) * out.to(F64)).sum())      # noqa: E731
    for r in range(9):
        h = torch.zeros_like(table)
        h[r, 5] = 0.5
        assert abs(loss(table + h) - loss(table - h) - float(dt[r, 5])) <= 64 * U * float(out.abs().sum() * (table.abs().max() + 1)), r


def test_autograd_of_a_layer():
    """Embedding, routing, tokens to their experts, a product an expert, back with weights: the gradients of all leaves
    against the same layer in 64 bits. fp32 products of 64 columns and sums of 40 tokens: some 100 roundings a value on the way, so
    within 2^-14 of the largest gradient."""
    T, E, k, H, V = 40, 6, 2, 64, 30
    g = gen(11)
    tokens = torch.randint(0, V + 4, (T,), generator=g, device="cuda")
    leaves = [randn(g, V, H), randn(g, H, E) * H ** -0.5, randn(g, E, H, H) * H ** -0.5]
    pull = randn(g, T, H)

    def plain(table, router, experts):
        here = (tokens < V).to(table.dtype)
        x = table[tokens.clamp_max(V - 1)] * here[:, None] * 2.0
        p = torch.softmax(x @ router, 1)
        top = R.reshard_route(x.float() @ router.float(), k)[1].long()
        w = torch.gather(p, 1, top)
        w = w / w.sum(1, keepdim=True)
        y = torch.tanh(torch.einsum("th,tkhi->tki", x, experts[top]))
        return ((y * w[..., None]).sum(1) * pull.to(table.dtype)).sum()

    def ours(table, router, experts):
        x = R.reshard_embedding(tokens, table, scale=2.0)
        w, ids = R.reshard_route(x @ router, k)
        sort = R.reshard_dispatch(ids, E)
        rows = R.reshard_permute(x, sort)
        at = sort[0].tolist()
        y = torch.cat([torch.tanh(rows[at[e]:at[e + 1]] @ experts[e]) for e in range(E)])
        return (R.reshard_combine(y, sort, w) * pull).sum()

    a = [v.clone().requires_grad_() for v in leaves]
    b = [v.to(F64).requires_grad_() for v in leaves]
    ours(*a).backward()
    plain(*b).backward()
    for x, y in zip(a, b):
        assert float((x.grad.to(F64) - y.grad).abs().max()) <= 2.0 ** -14 * float(y.grad.abs().max())
    with torch.no_grad():
        assert not R.reshard_embedding(tokens, a[0]).requires_grad
    with pytest.raises(R.ReshardError, match="without out"):
        R.reshard_embedding(tokens, a[0], out=torch.empty(T, H, device="cuda"))


def test_gradients_that_come_broadcast_or_transposed():
    T, k, H = 12, 2, 32
    x, ids, sort = case(3, T, k, 4, H, "f32")
    for grad in (torch.ones(1, 1, device="cuda").expand(T * k, H), randn(gen(1), H, T * k).t(), randn(gen(1), 1, H).expand(T * k, H)):
        a = x.clone().requires_grad_()
        R.reshard_permute(a, sort).backward(grad)
        assert torch.equal(a.grad, R.reshard_permute_backward(grad.contiguous(), sort, k))
    y, w = randn(gen(2), T * k, H), torch.rand(T, k, device="cuda")
    for grad in (torch.ones(1, 1, device="cuda").expand(T, H), randn(gen(1), H, T).t()):
        a, b = y.clone().requires_grad_(), w.clone().requires_grad_()
        R.reshard_combine(a, sort, b).backward(grad)
        dy, dw = R.reshard_combine_backward(grad.contiguous(), y, sort, w)
        assert torch.equal(a.grad, dy) and torch.equal(b.grad, dw)
        a = y.clone().requires_grad_()
        R.reshard_combine(a, sort, w).backward(grad)
        assert torch.equal(a.grad, dy)
        b = w.clone().requires_grad_()
        R.reshard_combine(y, sort, b).backward(grad)
        assert torch.equal(b.grad, dw)
    tokens = torch.randint(0, 9, (4, 6), device="cuda")
    a = randn(gen(5), 9, H).requires_grad_()
    R.reshard_embedding(tokens, a).sum().backward()
    assert torch.equal(a.grad, torch.bincount(tokens.view(-1), minlength=9).float()[:, None].expand(9, H))


def step(x, sort, w, grad, tokens, table):
    y = R.reshard_permute(x, sort)
    out = R.reshard_combine(y, sort, w)
    dy, dw = R.reshard_combine_backward(grad, y, sort, w)
    dx = R.reshard_permute_backward(dy, sort, w.shape[1])
    e = R.reshard_embedding(tokens, table, scale=2.0)
    return [y, out, dy, dw, dx, e, R.reshard_embedding_backward(e, tokens, table.shape[0])]


@pytest.mark.parametrize("H", [64, 67])
def test_other_streams_and_graphs(H):
    """On another stream, captured and replayed with new data, and two graphs that share a pool replayed in turn."""
    T, k = 50, 2
    x, ids, sort = case(8, T, k, 8, H, "bf16")
    g = gen(8)
    w, grad, table = torch.rand(T, k, generator=g, device="cuda"), randn(g, T, H).bfloat16(), randn(g, 40, H).bfloat16()
    tokens = torch.randint(0, 40, (600,), generator=g, device="cuda")
    args = [x, sort, w, grad, tokens, table]
    want = step(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = R.reshard_permute(x, sort, stream=side)
    got = [y, R.reshard_combine(y, sort, w, stream=side.cuda_stream), *R.reshard_combine_backward(grad, y, sort, w, stream=side)]
    got += [R.reshard_permute_backward(got[2], sort, k, stream=side), R.reshard_embedding(tokens, table, scale=2.0, stream=side)]
    got += [R.reshard_embedding_backward(got[5], tokens, 40, stream=side.cuda_stream)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs, pool = [], [], None
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side, pool=pool):
            outs.append(step(*args))
        pool = graph.pool()
        graphs.append(graph)
    for i, scale in enumerate((1.0, 0.5, 2.0, 1.0)):
        x.mul_(scale)
        tokens.copy_((tokens + i) % 40)
        graphs[i % 2].replay()
        now = [v.clone() for v in outs[i % 2]]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(now, step(*args))), i


def test_stages_equal_the_expert_layer():
    """dispatch, permutation, quantization, grouped products and the weighted sum by hand give what the layer's own enqueue gives."""
    T, k, E, H, I = 200, 2, 4, 384, 256
    g = gen(5)
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    x, w = randn(g, T, H).bfloat16(), torch.softmax(randn(g, T, k), 1)
    w13, s13 = R.reshard_quantize_blocks(randn(g, E, 2 * I, H) * 0.02)
    w2, s2 = R.reshard_quantize_blocks(randn(g, E, H, I) * 0.02)
    out = R.reshard_experts_fp8(x, ids, w, w13, s13, w2, s2)
    sort = R.reshard_dispatch(ids, E)
    q, s = R.reshard_quantize_rows(R.reshard_permute(x, sort))
    gu = R.reshard_matmul_fp8(q, s, w13, s13, offsets=sort[0], out_dtype=torch.float32)
    hq, hs = R.reshard_quantize_rows(torch.nn.functional.silu(gu[:, :I]) * gu[:, I:])
    y = R.reshard_matmul_fp8(hq, hs, w2, s2, offsets=sort[0], out_dtype=torch.float32)
    want = R.reshard_combine(y, sort, w, out_dtype=torch.bfloat16)
    # the fused silu differs by some 2^-21: a share of about 1e-4 of h moves by an e4m3 step
    assert float((out.float() - want.float()).norm()) <= 4e-3 * float(want.float().norm())
    assert R.reshard_ops_status() == 0


def test_refusals_name_what_is_wrong():
    x, ids, sort = case(1, 4, 2, 4, 16, "f32")
    y, w = randn(gen(1), 8, 16), torch.rand(4, 2, device="cuda")
    table, tokens = randn(gen(2), 9, 16), torch.randint(0, 9, (5,), device="cuda")
    offsets, order, position = sort
    cases = [
        (lambda: R.reshard_permute(x[:3], sort), "does not fit 3 tokens"),
        (lambda: R.reshard_permute(x.double(), sort), "float32"),
        (lambda: R.reshard_permute(x.t(), sort), "contiguous rows"),
        (lambda: R.reshard_permute(x, (offsets, order.long(), position)), "order"),
        (lambda: R.reshard_permute(x, (offsets, order, position.cpu())), "position"),
        (lambda: R.reshard_permute(x, sort, out=torch.empty(8, 15, device="cuda")), "out"),
        (lambda: R.reshard_permute(x, sort, out=torch.empty(8, 16, device="cuda", dtype=torch.bfloat16)), "out"),
        (lambda: R.reshard_combine(y, sort), "k must be given"),
        (lambda: R.reshard_combine(y, sort, k=3), "divide"),
        (lambda: R.reshard_combine(y, sort, w, k=3), "columns"),
        (lambda: R.reshard_combine(y, sort, w[:3]), "do not fit"),
        (lambda: R.reshard_combine(y, sort, w.half()), "weights"),
        (lambda: R.reshard_combine(y, sort, w, out_dtype=torch.float64), "out"),
        (lambda: R.reshard_combine_backward(x, y[:, :15], sort, w), "does not fit"),
        (lambda: R.reshard_combine_backward(x, torch.zeros(9, 16, device="cuda"), sort, w), "places"),
        (lambda: R.reshard_embedding(tokens.float(), table), "ids"),
        (lambda: R.reshard_embedding(tokens.cpu(), table), "ids"),
        (lambda: R.reshard_embedding(tokens, table[0]), "dimensions"),
        (lambda: R.reshard_embedding(tokens, table, first_row=-1), "first_row"),
        (lambda: R.reshard_embedding(tokens, table, out=torch.empty(4, 16, device="cuda")), "out"),
        (lambda: R.reshard_embedding_backward(torch.zeros(4, 16, device="cuda"), tokens, 9), "does not fit"),
        (lambda: R.reshard_embedding_backward(torch.zeros(5, 16, device="cuda"), tokens, 9, accumulate=True), "needs out"),
        (lambda: R.reshard_embedding_backward(torch.zeros(5, 16, device="cuda"), tokens, -1), ">= 0"),
        (lambda: R.reshard_embedding_backward(torch.zeros(5, 16, device="cuda"), tokens, 9, out=torch.zeros(8, 16, device="cuda")), "out"),
    ]
    for i, (call, word) in enumerate(cases):
        with pytest.raises(R.ReshardError) as e:
            call()
        assert word in str(e.value), (i, word, str(e.value))
    host = torch.zeros(4, 16)
    rc = R.binding.LIB.reshard_permute(host.data_ptr(), 3, 4, 16, 16, order.data_ptr(), position.data_ptr(), 2, y.data_ptr(), 8, 16, 0, None)
    assert rc == R.RESHARD_ERR_INVALID_ARG and "pageable" in R.reshard_last_error()


# ------------------------------------------------------------------------- many rows: warps that stay, runs, several slices

@pytest.mark.parametrize("T,k,E,H", [(6000, 3, 16, 72), (700, 2, 8, 8200), (5000, 40, 48, 24), (9000, 2, 8, 1000)])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("share", [False, True])
def test_combine_of_many_tokens(T, k, E, H, types, share):
    """More spans than the GPU holds warps: each warp takes several."""
    g = gen(T + H)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].int().contiguous()
    sort = R.reshard_dispatch(ids, E // 4 if share else E, E // 4 if share else 0)
    position = sort[2]
    y, w = randn(g, T * k, H).to(DT[types[0]]), torch.rand(T, k, generator=g, device="cuda")
    out = R.reshard_combine(y, sort, w, out_dtype=DT[types[1]])
    close(out, X.combine(y, position, w, k), k * U * X.combine(y, position, w, k, True))
    grad = randn(g, T, H).to(DT[types[1]])
    dy, dw = R.reshard_combine_backward(grad, y, sort, w)
    wy, ww = X.combine_backward(grad, y, position, w, k)
    close(dy, wy, U * wy.abs())
    close(dw, ww, (H / 32 + 32) * U * X.combine_backward(grad, y, position, w, k, True)[1])
    x = randn(g, T, H).to(DT[types[0]])
    to = torch.zeros_like(y)
    assert torch.equal(R.reshard_permute(x, sort, out=to), X.permute(x, position, torch.zeros_like(y)))


@pytest.mark.parametrize("T,V,H", [(9000, 40, 4100), (20000, 3, 1032), (5000, 6000, 4096), (16385, 100, 8), (16384, 100, 9)])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")])
def test_embedding_backward_of_many_columns_and_runs(T, V, H, types):
    g = gen(T + H)
    ids = (torch.rand(T, generator=g, device="cuda") ** 3 * V).long().clamp_max(V - 1)
    check_embedding_backward(randn(g, T, H).to(DT[types[0]]), ids, V - V // 3, V // 3, dtype=DT[types[1]])


def test_two_calls_at_once():
    """Calls on two streams, workspaces of their own, give what they give alone."""
    g = gen(31)
    ids = [torch.randint(0, 300, (20000,), generator=g, device="cuda") for _ in range(2)]
    grads = [randn(g, 20000, 256) for _ in range(2)]
    want = [R.reshard_embedding_backward(a, i, 300) for a, i in zip(grads, ids)]
    norms = [R.reshard_grad_norm([a]) for a in grads]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for s in range(2):
            got[s].append((R.reshard_embedding_backward(grads[s], ids[s], 300, stream=streams[s]), R.reshard_grad_norm([grads[s]], stream=streams[s])))
    torch.cuda.synchronize()
    for s in range(2):
        assert all(torch.equal(a, want[s]) and torch.equal(n, norms[s]) for a, n in got[s])


def test_a_captured_training_step():
    """Forward and backward by autograd, captured once and replayed with other inputs; the eager step's graph is gone by then."""
    T, E, k, H, V = 64, 8, 2, 64, 50
    g = gen(41)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    table, router, experts = (randn(g, *s).requires_grad_() for s in ((V, H), (H, E), (E, H)))

    def step():
        x = R.reshard_embedding(tokens, table)
        w, ids = R.reshard_route(x @ router, k)
        sort = R.reshard_dispatch(ids, E)
        scale = experts[torch.searchsorted(sort[0][1:].contiguous(), torch.arange(T * k, device="cuda", dtype=torch.int32), right=True)]
        out = R.reshard_combine(R.reshard_permute(x, sort) * scale, sort, w)
        grads = torch.autograd.grad(out.square().sum(), [table, router, experts])
        R.reshard_clip_grads(list(grads), 1.0)
        return grads

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = step()
    for i in range(3):
        with torch.no_grad():
            tokens.copy_(torch.randint(0, V, (T,), generator=g, device="cuda"))
            table.mul_(0.9)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, step()):
            # torch's own indexing gradient adds in any order
            assert float((a - b).abs().max()) <= 1e-5 * float(b.abs().max())


# ------------------------------------------------------------------------------------------------------- no columns

@pytest.mark.parametrize("T", [0, 1, 5, 300])
@pytest.mark.parametrize("wide_ids", [False, True])
def test_rows_of_no_columns(T, wide_ids):
    """Tables and rows without columns: results and gradients of the right shape, through autograd too; a weight's gradient is 0."""
    ids = torch.arange(T, device="cuda", dtype=torch.int64 if wide_ids else torch.int32) % 9
    table = torch.zeros(9, 0, device="cuda", requires_grad=True)
    out = R.reshard_embedding(ids, table)
    out.sum().backward()
    assert out.shape == (T, 0) and table.grad.shape == (9, 0)
    grad = torch.zeros(T, 0, device="cuda")
    for accumulate in (False, True):
        main = torch.zeros(9, 0, device="cuda")
        assert R.reshard_embedding_backward(grad, ids, 9, out=main, accumulate=accumulate) is main
    sort = R.reshard_dispatch((ids % 4).int().view(T, 1), 4)
    x, w = torch.zeros(T, 0, device="cuda", requires_grad=True), torch.rand(T, 1, device="cuda", requires_grad=True)
    y = R.reshard_combine(R.reshard_permute(x, sort), sort, w)
    y.sum().backward()
    assert y.shape == x.grad.shape == (T, 0) and w.grad.shape == (T, 1) and not bool(w.grad.any())


# ------------------------------------------------------------------------------------------------------- derivatives

def test_tangents_are_refused():
    """A dual tensor that requires no gradient does not go past: its result would have no tangent."""
    x, ids, sort = case(1, 6, 2, 4, 16, "f32")
    y, w, table, tokens = randn(gen(1), 12, 16), torch.rand(6, 2, device="cuda"), randn(gen(2), 9, 16), torch.arange(5, device="cuda")
    logits = randn(gen(3), 6, 8)
    calls = [(logits, lambda t: R.reshard_route(t, 2)), (x, lambda t: R.reshard_permute(t, sort)), (y, lambda t: R.reshard_combine(t, sort, w)),
             (w, lambda t: R.reshard_combine(y, sort, t)), (table, lambda t: R.reshard_embedding(tokens, t)), (x, lambda t: R.reshard_combine_backward(t, y, sort, w))]
    for t, call in calls:
        with forward_ad.dual_level():
            want = call(t)
            with pytest.raises(R.ReshardError, match="forward mode"):
                call(forward_ad.make_dual(t, torch.ones_like(t)))
            with pytest.raises(R.ReshardError, match="forward mode"):
                call(forward_ad.make_dual(t.clone().requires_grad_(), torch.ones_like(t)))
        got = call(t)
        for a, b in zip(*((v if isinstance(v, tuple) else (v,)) for v in (got, want))):
            assert torch.equal(a, b)


def test_results_that_have_no_gradient_raise_when_it_is_asked_for():
    """The gradients' own calls: nothing is lost without a word, and under no_grad, or of inputs that require none, they are plain."""
    x, ids, sort = case(1, 6, 2, 4, 16, "f32")
    logits, dw = randn(gen(3), 6, 8), randn(gen(4), 6, 2)
    y, w, tokens = randn(gen(1), 12, 16), torch.rand(6, 2, device="cuda"), torch.arange(5, device="cuda") % 3
    routed = R.reshard_route(logits, 2)[1]
    calls = [([dw, logits], lambda a, b: R.reshard_route_backward(a, b, routed)),
             ([x, y, w], lambda a, b, c: R.reshard_combine_backward(a, b, sort, c)),
             ([randn(gen(5), 5, 16)], lambda a: R.reshard_embedding_backward(a, tokens, 4)),
             ([randn(gen(6), 5, 1, 16).transpose(0, 1)], lambda a: R.reshard_embedding_backward(a, tokens.view(1, 5), 4))]
    for inputs, call in calls:
        want = call(*inputs)
        want = want if isinstance(want, tuple) else (want,)
        assert not any(t.requires_grad for t in want)
        for i in range(len(inputs)):
            leaf = inputs[i].clone().requires_grad_()
            these = [*inputs[:i], leaf, *inputs[i + 1:]]
            with torch.no_grad():
                got = call(*these)
            assert not any(t.requires_grad for t in (got if isinstance(got, tuple) else (got,)))
            got = call(*these)
            for a, b in zip(got if isinstance(got, tuple) else (got,), want):
                assert torch.equal(a, b)
                with pytest.raises(R.ReshardError, match="has no gradient"):
                    torch.autograd.grad(a.sum(), leaf)


def test_the_permutations_gradient_is_differentiable():
    """It is linear in what comes in: its own gradient takes each token's row to its places."""
    x, ids, sort = case(1, 6, 2, 4, 16, "f32", 1, 2)
    dy = randn(gen(1), 12, 16).requires_grad_()
    pull = randn(gen(2), 6, 16)
    R.reshard_permute_backward(dy, sort, 2).backward(pull)
    assert torch.equal(dy.grad, R.reshard_permute(pull, sort))
    with pytest.raises(R.ReshardError, match="cannot be written to out"):
        R.reshard_permute_backward(dy, sort, 2, out=torch.empty(6, 16, device="cuda"))
    with torch.no_grad():
        to = torch.empty(6, 16, device="cuda")
        assert R.reshard_permute_backward(dy, sort, 2, out=to) is to


@pytest.mark.parametrize("H", [64, 67])
@pytest.mark.parametrize("more", [0, 1, 40])
@pytest.mark.parametrize("share", [False, True])
def test_autograd_of_padded_rows(H, more, share):
    """Experts' rows in a buffer that is longer than the sort: their weighted sum and its gradients are those of the places, rows
    behind them have gradient 0."""
    T, k = 9, 2
    g = gen(H + more)
    first, local = (1, 2) if share else (0, 4)
    _, ids, sort = case(5, T, k, 4, 1, "f32", first, local)
    y = randn(g, T * k + more, H)
    y[int(sort[0][-1]):] = float("nan")
    pull, w = randn(g, T, H), torch.softmax(randn(g, T, k), 1)
    for needs in ((True, True), (True, False), (False, True)):
        leaf, weights = y.clone().requires_grad_(needs[0]), w.clone().requires_grad_(needs[1])
        out = R.reshard_combine(leaf, sort, weights)
        assert torch.equal(out, R.reshard_combine(y[:T * k].contiguous(), sort, w))
        out.backward(pull)
        dy, dw = R.reshard_combine_backward(pull, y[:T * k], sort, w)
        if needs[0]:
            assert leaf.grad.shape == y.shape and torch.equal(leaf.grad[:T * k], dy) and not bool(leaf.grad[T * k:].any())
        if needs[1]:
            assert torch.equal(weights.grad, dw)
    leaf = y.clone().requires_grad_()
    R.reshard_combine(leaf, sort, k=k).backward(pull)
    assert torch.equal(leaf.grad[:T * k], R.reshard_combine_backward(pull, y[:T * k], sort, k=k)[0]) and not bool(leaf.grad[T * k:].any())


def test_the_weighted_sum_keeps_its_rows_only_for_the_weights():
    """The gradient to y does not read y: it may be written anew before the backward pass, and its memory is not held."""
    T, k, H = 64, 2, 4096
    _, ids, sort = case(5, T, k, 8, 1, "f32")
    w, pull = torch.softmax(randn(gen(1), T, k), 1), randn(gen(2), T, H)
    for weights in (w, None):
        source = randn(gen(3), T * k, H).requires_grad_()
        y = source * 2.0
        out = R.reshard_combine(y, sort, weights, k=k)
        with torch.no_grad():
            y.zero_()
        out.backward(pull)
        want = R.reshard_combine_backward(pull, y.detach(), sort, weights, k=k)[0]
        assert torch.equal(source.grad, 2.0 * want)
    source = randn(gen(3), T * k, H).requires_grad_()
    before = torch.cuda.memory_allocated()
    out = R.reshard_combine(source * 2.0, sort, w)
    assert torch.cuda.memory_allocated() - before < T * k * H * 4
    # of a weight that has a gradient y is kept, and a change of it is seen
    y, weights = source.detach().clone(), w.clone().requires_grad_()
    out = R.reshard_combine(y, sort, weights)
    y.zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward(pull)


# ------------------------------------------------------------------------------------------ one sum, several kernels

@pytest.mark.parametrize("T,k,E,H", [(1, 1, 4, 8), (3, 8, 16, 4), (5, 8, 8, 1003), (130, 8, 64, 520), (900, 8, 32, 2048), (40, 9, 16, 72), (700, 3, 8, 4100)])
@pytest.mark.parametrize("to", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("share", [False, True])
def test_the_sum_is_the_same_however_its_rows_lie(T, k, E, H, to, share):
    """Rows of whole pieces, few places or many, rows that start anywhere: fp32 terms added in the order of the choices."""
    g = gen(T + H)
    first, local = (E // 4, max(1, E // 2)) if share else (0, E)
    _, ids, sort = case(T + k, T, k, E, 1, "f32", first, local)
    y, w = randn(g, T * k, H), torch.softmax(randn(g, T, k), 1)
    position = sort[2].view(T, k)
    for weights in (w, None):
        want = torch.zeros(T, H, device="cuda", dtype=F64)
        for j in range(k):                            # a product of 24-bit numbers is exact in 64 bits, and so each sum rounds once but for 2^-53
            here = (position[:, j] >= 0)[:, None]
            term = y[position[:, j].clamp_min(0).long()].to(F64) * (w[:, j:j + 1] if weights is not None else 1.0)
            want = torch.where(here, (want + term).float().to(F64), want)
        close(R.reshard_combine(y, sort, weights, k=k, out_dtype=DT[to]), want, 2 * U * X.combine(y, position.reshape(-1), weights, k, True))
        outs = [R.reshard_combine(laid(y, how), sort, weights, k=k, out=laid(torch.zeros(T, H, device="cuda", dtype=DT[to]), how)) for how in ("dense", "pitch", "odd")]
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        many = torch.cat([w, torch.zeros(T, 9 - k, device="cuda")], 1) if k < 9 else w      # the same sum with nine choices
        padded = torch.cat([position, torch.full((T, max(0, 9 - k)), -1, dtype=torch.int32, device="cuda")], 1).contiguous().view(-1)
        if weights is not None:
            assert torch.equal(outs[0], R.reshard_combine(y, (sort[0], sort[1], padded), many.contiguous(), out_dtype=DT[to]))


# -------------------------------------------------------------------------------------------- the other pairs of types

@pytest.mark.parametrize("T,k,E,H", [(5, 2, 4, 7), (64, 4, 8, 1000), (33, 8, 8, 2867), (9, 12, 40, 8200)])
@pytest.mark.parametrize("types", [("bf16", "f16"), ("f16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("how", ["dense", "odd"])
def test_combine_and_its_gradients_of_other_types(T, k, E, H, types, how):
    g = gen(T * H + k)
    _, ids, sort = case(T + k, T, k, E, 1, "f32", E // 4, max(1, E // 2))
    offsets, order, position = sort
    held = int(offsets[-1])
    y, grad = laid(randn(g, T * k, H).to(DT[types[0]]), how), laid(randn(g, T, H).to(DT[types[1]]), how)
    w = torch.softmax(randn(g, T, k), 1)
    out = R.reshard_combine(y, sort, w, out_dtype=DT[types[1]])
    assert out.dtype is DT[types[1]]
    close(out, X.combine(y, position, w, k), k * U * X.combine(y, position, w, k, True))
    dy, dw = R.reshard_combine_backward(grad, y, sort, w)
    want_y, want_w = X.combine_backward(grad, y, position, w, k)
    assert dy.dtype is DT[types[0]] and not bool(dy[held:].any())
    close(dy, want_y, U * want_y.abs())
    close(dw, want_w, (H / 32 + 32) * U * X.combine_backward(grad, y, position, w, k, True)[1])


@pytest.mark.parametrize("T,rows,H", [(40, 30, 520), (200, 7, 33), (256, 9, 2867), (300, 40, 520), (3000, 50, 2867), (5000, 3000, 72)])
@pytest.mark.parametrize("types", [("f32", "bf16"), ("f32", "f16"), ("f16", "f32"), ("bf16", "f16"), ("f16", "bf16")])
@pytest.mark.parametrize("how", ["dense", "odd"])
def test_embedding_backward_of_other_types(T, rows, H, types, how):
    """Whole and accumulated, few tokens and many, the table's rows on 16 bytes or not."""
    g = gen(T + H)
    ids = torch.randint(0, 2 * rows, (T,), generator=g, device="cuda")
    grad = laid(randn(g, T, H).to(DT[types[0]]), how)
    whole = laid(torch.full((rows, H), 7.0, device="cuda", dtype=DT[types[1]]), how)
    want, size = X.embedding_backward(grad, ids, rows, 0.3, rows // 2), X.embedding_backward(grad, ids, rows, 0.3, rows // 2, True)
    most = int(torch.bincount(ids).max())
    R.reshard_embedding_backward(grad, ids, rows, scale=0.3, first_row=rows // 2, out=whole)
    close(whole, want, (most + 2) * U * size)
    base = randn(g, rows, H).to(DT[types[1]])
    main = laid(base, how)
    R.reshard_embedding_backward(grad, ids, rows, scale=0.3, first_row=rows // 2, out=main, accumulate=True)
    close(main, want + base.to(F64), (most + 2) * U * size + U * (want + base.to(F64)).abs())


def test_embedding_backward_when_other_tokens_change():
    """Runs are cut from all tokens of the shard: other tokens may regroup a row's sum, whose distance stays bounded; what does not
    change the ids changes no bit of it."""
    g = gen(19)
    ids = torch.randint(0, 50, (20000,), generator=g, device="cuda")
    grad = randn(g, 20000, 128)
    first = check_embedding_backward(grad, ids, 50)
    mine = ids == 49
    for change in (lambda i: torch.where(mine, i, i // 2), lambda i: torch.where(mine, i, 50), lambda i: torch.where(mine, i, i + 100)):
        other = check_embedding_backward(grad, change(ids.clone()), 50)
        want = X.embedding_backward(grad, ids, 50)[49]
        size = X.embedding_backward(grad, ids, 50, magnitudes=True)[49]
        close(other[49], want, (int(mine.sum()) + 2) * U * size)
    assert torch.equal(first, R.reshard_embedding_backward(grad, ids, 50))
