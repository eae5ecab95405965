"""The norm of many tensors and their clipping against the 64-bit oracle.

Tolerances (u = 2^-24): a thread's squares are summed over at most 8 of a chain and two more additions, each fused or added with
one rounding, and what follows carries its roundings along or has 64 bits; with the square's own that is 11 u of the sum, half
of it of the root, and the root's rounding to fp32: 7 u. The factor adds its rounding and takes over the norm's error, the
product its own: 9 u of the value, and half a step of the type that it is rounded to.
"""
import copy
import math
import pickle

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


def tensors(seed, sizes, kinds, skip=0, gap=0):
    """Normal tensors of these sizes, each from `skip` elements behind a 16-byte boundary on, values of `gap` behind each."""
    g, out = gen(seed), []
    for i, n in enumerate(sizes):
        dtype = DT[kinds[i % len(kinds)]]
        buf = torch.full((n + skip + gap + 8,), 7.0, dtype=dtype, device="cuda")
        t = buf[skip:skip + n]
        t.copy_(torch.randn(n, generator=g, device="cuda") * (0.01 + 0.1 * (i % 5)))
        out.append(t)
    return out


def around(t):
    """What lies before and behind a tensor of tensors()."""
    base = t._base if t._base is not None else t
    at = t.storage_offset()
    return torch.cat([base[:at], base[at + t.numel():]])


def check_norm(ts, n=None):
    n = R.reshard_grad_norm(ts) if n is None else n
    assert n.dtype is torch.float32 and n.shape == ()
    want = float(X.norm([t.cpu() for t in ts]))
    assert abs(float(n) - want) <= 7 * U * want, (float(n), want)
    return n


def check_clipped(got, ts, limit, n, types=None):
    want = X.clip([t.cpu() for t in ts], limit, n.cpu())
    for i, (a, b) in enumerate(zip(got, want)):
        info = torch.finfo(a.dtype)
        bad = (a.cpu().to(F64) - b).abs() - b.abs() * (9 * U + info.eps / 2 * (1 + 9 * U)) - info.smallest_normal * info.eps / 2
        assert bool((bad <= 0).all()), (i, a.dtype, float(bad.max()))


SIZES = [[1], [0, 5, 0], [7, 8, 9, 15, 16, 17], [2047, 2048, 2049, 2056, 1, 3], [100000, 3, 70001], [1] * 1025, [5, 600] * 1300, [3000001]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("kinds", [["bf16"], ["f32"], ["f16"], ["f32", "bf16", "f16"]], ids=lambda k: "-".join(k))
@pytest.mark.parametrize("skip", [0, 1, 5])
def test_norm_and_clip(sizes, kinds, skip):
    ts = tensors(len(sizes) + skip, sizes, kinds, skip)
    edges = [around(t).clone() for t in ts[:50]]
    n = check_norm(ts)
    for limit in (0.3 * float(n), 2.0 * float(n)):
        for to in (None, "bf16", "f32", "f16"):
            out = [torch.empty(t.numel() + 3, dtype=DT[to] if to else t.dtype, device="cuda")[(skip if to else 0) % 3:][:t.numel()] for t in ts]
            m = R.reshard_clip_grads(ts, limit, out=out)
            assert torch.equal(m, n)
            check_clipped(out, ts, limit, n)
    assert torch.equal(R.reshard_grad_norm(ts), n)
    # in place: the same values as into other tensors, and nothing beside them
    want = [torch.empty_like(t) for t in ts]
    R.reshard_clip_grads(ts, 0.3 * float(n), out=want)
    m = R.reshard_clip_grads(ts, 0.3 * float(n))
    assert torch.equal(m, n) and all(torch.equal(a, b) for a, b in zip(ts, want))
    assert all(torch.equal(around(t), e) for t, e in zip(ts, edges))
    # under the limit nothing changes
    R.reshard_clip_grads(ts, 1.01 * float(n))
    assert all(torch.equal(a, b) for a, b in zip(ts, want))


@pytest.mark.parametrize("count", [95, 96, 97, 1299, 1300, 1301, 1999, 2000, 2001, 4100])
def test_lists_of_as_many_tensors_as_a_launch_takes(count):
    kinds = ["bf16", "f32"] if count == 4100 else ["bf16"]
    ts = tensors(count, [3, 17, 0, 40] * (count // 4) + [9] * (count % 4), kinds)
    assert len(ts) == count
    n = check_norm(ts)
    out = [torch.zeros(t.shape, device="cuda") for t in ts]
    R.reshard_clip_grads(ts, 0.5 * float(n), out=out)
    check_clipped(out, ts, 0.5 * float(n), n)
    keep = [t.clone() for t in ts]
    R.reshard_clip_grads(ts, 0.5 * float(n))
    check_clipped(ts, keep, 0.5 * float(n), n)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_units_of_every_size(kind):
    """Totals for which a unit has 2,048, 4,096, 8,192 and 16,384 elements, tensors that end at its borders and beside them."""
    for unit, total in ((2048, 300000), (4096, 1500000), (8192, 3000000), (16384, 6000000)):
        ts = tensors(unit, [unit, unit - 1, unit + 1, 2 * unit + 7, 8, total], [kind], skip=1)
        n = check_norm(ts)
        out = [torch.zeros(t.shape, device="cuda") for t in ts]
        R.reshard_clip_grads(ts, 0.1, out=out)
        check_clipped(out, ts, 0.1, n)
        keep = [t.clone() for t in ts]
        R.reshard_clip_grads(ts, 0.1)
        check_clipped(ts, keep, 0.1, n)


def test_lists_made_once():
    ts = tensors(1, [300, 5000, 70000], ["bf16", "f32"])
    out = [torch.empty(t.shape, device="cuda") for t in ts]
    a, b = R.reshard_tensor_list(ts), R.reshard_tensor_list(out)
    assert len(a) == 3
    for scale in (1.0, 0.25, 8.0):
        for t in ts:
            t.mul_(scale)
        n = check_norm(ts, R.reshard_grad_norm(a))
        assert torch.equal(R.reshard_clip_grads(a, 0.5, out=b), n)
        check_clipped(out, ts, 0.5, n)
    # a norm over more than these tensors, as several ranks have it
    whole = torch.tensor(123.0, device="cuda")
    assert R.reshard_clip_grads(a, 2.0, norm=whole, out=b) is whole
    check_clipped(out, ts, 2.0, whole)
    for t, o in zip(ts, out):
        o.copy_(t)
    assert R.reshard_clip_grads(a, 124.0, norm=whole.view(1)).shape == (1,)
    assert all(torch.equal(t.float(), o) for t, o in zip(ts, out))
    # some in place, some not: those under the limit are copied
    mixed = [ts[0], torch.zeros_like(ts[1]), torch.zeros(ts[2].shape, device="cuda")]
    R.reshard_clip_grads(ts, float("inf"), out=mixed)
    assert all(torch.equal(t.float(), o.float()) for t, o in zip(ts, mixed))


def test_empty_lists():
    for ts in ([], [torch.empty(0, device="cuda")], [torch.empty(0, 5, device="cuda", dtype=torch.bfloat16)] * 3):
        assert float(R.reshard_grad_norm(ts)) == 0.0
        assert float(R.reshard_clip_grads(ts, 1.0)) == 0.0
        R.reshard_clip_grads(ts, 1.0, norm=torch.ones((), device="cuda"))


@pytest.mark.parametrize("kind,values", [("f32", [1e30, 3e30, -2e38]), ("bf16", [1e30, 3e38]), ("f32", [1e-30, 4e-38, 1e-44]), ("bf16", [1e-30, 1e-38]),
                                         ("f32", [1e-30, 1.0, 1e30]), ("f32", [2.0 ** 50, 2.0 ** -40]), ("f32", [0.0]), ("f16", [65504.0, 6e-8, 1.0])])
def test_norm_of_extreme_values(kind, values):
    """Squares beyond fp32's range, and below it, count for what they are; zeros are no such values."""
    for n in (1, 100, 40000):
        t = torch.zeros(n, dtype=DT[kind], device="cuda")
        for i, v in enumerate(values):
            t[i::max(1, min(n, 3000))] = v if n > 1 else values[-1]
        parts = list(t.split(max(1, n // 3)))
        want = float(X.norm([t]))
        got = float(R.reshard_grad_norm(parts))
        assert abs(got - want) <= 7 * U * want + 2.0 ** -150 or (want > 3.4028235e38 and got == math.inf), (n, got, want)


def test_norm_that_is_not_finite():
    for bad, kind in ((float("inf"), "f32"), (float("nan"), "bf16"), (float("-inf"), "f16")):
        ts = tensors(5, [40, 9000], [kind])
        ts[1][8001] = bad
        n = R.reshard_grad_norm(ts)
        assert bool(torch.isnan(n)) if math.isnan(bad) else float(n) == math.inf
        keep = [t.clone() for t in ts]
        R.reshard_clip_grads(ts, math.inf)                   # an infinite limit only measures
        assert all(torch.equal(a, b) or bool(torch.isnan(a).any()) for a, b in zip(ts, keep))
        assert torch.equal(ts[0], keep[0])
        R.reshard_clip_grads(ts, 1.0)
        if math.isnan(bad):
            assert all(bool(torch.isnan(t).all()) for t in ts)
        else:
            assert not bool(ts[0].any()) and int(torch.isnan(ts[1]).sum()) == 1 and not bool(torch.nan_to_num(ts[1]).any())
    ts = tensors(5, [40, 9000], ["f32"])
    R.reshard_clip_grads(ts, 0.0)
    assert not any(bool(t.any()) for t in ts)
    n = R.reshard_clip_grads(ts, 0.0)                        # zeros: 0 / 1e-6
    assert float(n) == 0.0 and not any(bool(t.any()) for t in ts)


def test_tensors_of_other_orders():
    """Dense in another order of dimensions is as good; a target has to have its source's."""
    g = gen(6)
    base = torch.randn(30, 20, 10, generator=g, device="cuda")
    ts = [base.permute(2, 0, 1), base.transpose(0, 1)[:, :1, :].contiguous()]
    n = check_norm(ts)
    out = [torch.empty(20 * 30 * 10, device="cuda").as_strided(t.shape, t.stride()) if t.dim() == 3 and not t.is_contiguous() else torch.empty_like(t) for t in ts]
    R.reshard_clip_grads(ts, 1.0, out=out)
    check_clipped(out, ts, 1.0, n)
    with pytest.raises(R.ReshardError, match="order of dimensions"):
        R.reshard_clip_grads(ts, 1.0, out=[torch.empty(t.shape, device="cuda") for t in ts])


def test_other_streams_and_graphs():
    ts = tensors(9, [1000, 40000, 7], ["bf16", "f32"])
    out = [torch.zeros(t.shape, device="cuda") for t in ts]
    n = R.reshard_grad_norm(ts)
    want = [torch.empty_like(o) for o in out]
    R.reshard_clip_grads(ts, 1.0, out=want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    m = R.reshard_clip_grads(ts, 1.0, out=out, stream=side)
    k = R.reshard_grad_norm(ts, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(m, n) and torch.equal(k, n) and all(torch.equal(a, b) for a, b in zip(out, want))
    # two graphs of one pool, of lists that are gone when they run, replayed in turn
    graphs, norms, pool = [], [], None
    for limit in (1.0, 5.0):
        a, b = R.reshard_tensor_list(ts), R.reshard_tensor_list(out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side, pool=pool):
            norms.append(R.reshard_clip_grads(a, limit, out=b))
        pool = graph.pool()
        graphs.append((graph, limit))
        del a, b
    for i in (0, 1, 1, 0):
        for t in ts:
            t.mul_(1.5)
        graphs[i][0].replay()
        torch.cuda.synchronize()
        check_norm(ts, norms[i])
        check_clipped(out, ts, graphs[i][1], norms[i])


def test_the_same_bits_every_time():
    ts = tensors(12, [100, 70000, 33, 500000] * 20, ["bf16", "f32", "f16"], skip=1)
    n = R.reshard_grad_norm(ts)
    for _ in range(5):
        assert torch.equal(R.reshard_grad_norm(ts), n)


def test_a_tensor_beyond_32_bits():
    t = torch.zeros((1 << 32) + 5, dtype=torch.bfloat16, device="cuda")
    t[-1], t[0], t[(1 << 31) + 1] = 3.0, 4.0, 12.0
    n = R.reshard_clip_grads([t], 6.5)
    assert float(n) == 13.0 and [float(t[i]) for i in (-1, 0, (1 << 31) + 1)] == [1.5, 2.0, 6.0]


def test_refusals_name_what_is_wrong():
    x, y = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    cases = [
        (lambda: R.reshard_grad_norm([x, x.cpu()]), "tensor 1 is on cpu"),
        (lambda: R.reshard_grad_norm([x.double()]), "float32"),
        (lambda: R.reshard_grad_norm([x.view(8, 8)[:, :4]]), "not dense"),
        (lambda: R.reshard_grad_norm([x[:1].expand(9)]), "not dense"),
        (lambda: R.reshard_grad_norm([x.to_sparse()]), "strided"),
        (lambda: R.reshard_clip_grads([x], -1.0), "limit"),
        (lambda: R.reshard_clip_grads([x], float("nan")), "limit"),
        (lambda: R.reshard_clip_grads([x], 1.0, norm=torch.ones(2, device="cuda")), "norm must"),
        (lambda: R.reshard_clip_grads([x], 1.0, norm=torch.ones(1)), "norm must"),
        (lambda: R.reshard_clip_grads([x], 1.0, norm=torch.ones(1, device="cuda", dtype=F64)), "norm must"),
        (lambda: R.reshard_clip_grads([x], 1.0, out=[y, y]), "out has 2"),
        (lambda: R.reshard_clip_grads([x], 1.0, out=[y[:63]]), "numbers of elements"),
        (lambda: R.reshard_clip_grads([x, x], 1.0), "must not overlap"),
        (lambda: R.reshard_clip_grads([x, x[32:]], 1.0), "must not overlap"),
        (lambda: R.reshard_clip_grads([x, x + 1], 1.0, out=[y, y]), "must not overlap"),
        (lambda: R.reshard_clip_grads([x[:32]], 1.0, out=[x[16:48]]), "overlaps one that is read"),
        (lambda: R.reshard_clip_grads([x, y], 1.0, out=[y, x]), "overlaps one that is read"),
        (lambda: R.reshard_clip_grads([x[:32], y[:32]], 1.0, out=[x[:32], x[32:]]), None),
    ]
    for i, (call, word) in enumerate(cases):
        if word is None:
            call()
            continue
        with pytest.raises(R.ReshardError) as e:
            call()
        assert word in str(e.value), (i, word, str(e.value))
    assert float(R.reshard_grad_norm([x + 1, x + 1])) == math.sqrt(128) or abs(float(R.reshard_grad_norm([x + 1, x + 1])) - math.sqrt(128)) < 1e-5


# ----------------------------------------------------------------------------------------------------- lists that are kept

@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle"])
def test_a_copied_list_outlives_its_source(how):
    ts = tensors(3, [300, 5000, 0, 7], ["bf16", "f32"])
    a = R.reshard_tensor_list(ts)
    n = check_norm(ts, R.reshard_grad_norm(a))
    b = {"copy": copy.copy, "deepcopy": copy.deepcopy, "pickle": lambda t: pickle.loads(pickle.dumps(t))}[how](a)
    assert len(b) == 4 and b.device == a.device and b._handle != a._handle
    assert [x.data_ptr() == y.data_ptr() for x, y in zip(a.tensors, b.tensors) if x.numel()] == [how == "copy"] * 3
    keep = [t.clone() for t in ts]
    del a
    assert torch.equal(R.reshard_clip_grads(b, 0.5 * float(n)), n)
    check_clipped(b.tensors, keep, 0.5 * float(n), n)
    if how != "copy":                                        # a deep copy's tensors are its own
        assert all(torch.equal(x, y) for x, y in zip(ts, keep))


def test_a_list_keeps_the_memory_that_it_was_made_of():
    """A tensor that is given other memory leaves its own to the list: calls do not write what belongs to others by then."""
    ts = [torch.randn(n, generator=gen(4), device="cuda") for n in (70000, 500)]
    t, at = ts[0], ts[0].data_ptr()
    a = R.reshard_tensor_list(ts)
    n = check_norm(ts, R.reshard_grad_norm(a))
    t.data = torch.zeros(70000, device="cuda")
    others = [torch.full((70000,), 7.0, device="cuda") for _ in range(20)]
    assert all(not o.data_ptr() <= at < o.data_ptr() + 4 * o.numel() for o in others)
    assert torch.equal(R.reshard_grad_norm(a), n)
    R.reshard_clip_grads(a, 0.5 * float(n))
    assert all(bool((o == 7.0).all()) for o in others) and not bool(t.any())


# ------------------------------------------------------------------------------------------------------- derivatives

def test_tangents_are_refused():
    ts = [torch.ones(8, device="cuda"), torch.ones(3, device="cuda")]
    a = R.reshard_tensor_list(ts)
    with forward_ad.dual_level():
        duals = [ts[0], forward_ad.make_dual(ts[1], torch.ones_like(ts[1]))]
        for call in (lambda: R.reshard_grad_norm(duals), lambda: R.reshard_clip_grads(duals, 1.0), lambda: R.reshard_clip_grads([t + 1.0 for t in ts], 1.0, out=duals),
                     lambda: R.reshard_clip_grads(ts, 1.0, norm=forward_ad.make_dual(torch.ones((), device="cuda"), torch.ones((), device="cuda")))):
            with pytest.raises(R.ReshardError, match="forward mode"):
                call()
        assert float(R.reshard_grad_norm(a)) == math.sqrt(11.0) or abs(float(R.reshard_grad_norm(a)) - math.sqrt(11.0)) <= 7 * U * 4
    assert all(bool((t == 1.0).all()) for t in ts)


def test_a_norm_has_no_gradient_and_says_so():
    ts = [torch.ones(n, device="cuda", requires_grad=i != 1) for i, n in enumerate((8, 3, 5))]
    for of in (ts, R.reshard_tensor_list(ts)):
        norm = R.reshard_grad_norm(of)
        assert float(norm.detach()) == 4.0
        for t in (ts[0], ts[2]):
            with pytest.raises(R.ReshardError, match="reshard_grad_norm has no gradient"):
                torch.autograd.grad(norm * 2.0 + t.sum(), t)
        with torch.no_grad():
            assert not R.reshard_grad_norm(of).requires_grad
    assert not R.reshard_grad_norm([t.detach() for t in ts]).requires_grad
    assert not R.reshard_clip_grads([t.detach() for t in ts], 1.0).requires_grad


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_an_infinite_limit_leaves_every_bit(bad, kind):
    """Whatever the norm is, NaN among it: in place nothing is written, other tensors get the values as they are."""
    ts = tensors(5, [40, 9000], [kind])
    ts[1][8001] = bad
    bits = {4: torch.int32, 2: torch.int16}[ts[0].element_size()]
    keep = [t.clone() for t in ts]
    out = [torch.empty_like(t) for t in ts]
    R.reshard_clip_grads(ts, math.inf)
    R.reshard_clip_grads(ts, math.inf, out=out)
    for t, o, k in zip(ts, out, keep):
        assert torch.equal(t.view(bits), k.view(bits))
        finite = torch.isfinite(k)
        assert torch.equal(o[finite], k[finite]) and torch.equal(torch.isnan(o), torch.isnan(k)) and torch.equal(torch.isinf(o), torch.isinf(k))
