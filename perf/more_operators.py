"""Operators of a training step around the expert layer that are timed and compared: rows moved by an index, with their
gradients (tokens to their experts and back, a sharded embedding), and the norm of many gradients with their clipping.

Each case runs in two forms on the same inputs: `own` False computes the definition with elementary torch operations in
32 bits, `own` True calls the library. `exact` computes the definition in 64 bits, on its own.

Definitions
  A sort (offsets, order, position) of the slots t * k + j (token t, choice j) by expert: place p holds slot order[p], slot s
  lies at position[s] (-1: its expert is another rank's). `held` = offsets[-1] places are taken.
  permute        y[position[t, j]] = x[t]; rows from `held` on stay as they were
  permute_grad   dx[t] = sum_j dy[position[t, j]]
  combine        out[t] = sum_j weights[t, j] * y[position[t, j]]
  combine_grad   dy[position[t, j]] = weights[t, j] * dout[t], rows from `held` on 0;  dweights[t, j] = <dout[t], y[position[t, j]]>
  embed          out[t] = scale * table[ids[t] - first], 0 where the id's row is another rank's
  embed_grad     dtable[r] = scale * sum of dout[t] over the t with ids[t] = first + r; the whole table's gradient
  norm           sqrt(sum over all tensors of x^2)
  clip           the same norm, and every tensor times min(1, limit / (norm + 1e-6)), in place or into tensors of another type
"""
import math

import torch

own = False

HID, FFN, EXP = 2048, 768, 128   # the expert layers of this repository's blockwise FP8 workload
EPS = 1e-6


def listed():
    return [
        # a small batch's decode step: rows to the experts, latency
        dict(name="permute_decode", op="permute", T=24, E=EXP, first=0, local=EXP, k=8, H=HID, dtype="bf16"),
        # a prompt or a training batch, all experts here
        dict(name="permute_prompt", op="permute", T=8192, E=EXP, first=0, local=EXP, k=8, H=HID, dtype="bf16"),
        # its gradient for an uneven shard of the hidden dimension: rows start at any element
        dict(name="permute_grad_uneven", op="permute_grad", T=8191, E=60, first=0, local=60, k=4, H=2867, dtype="f16"),
        # one rank's share of the experts, their outputs still in 32 bits
        dict(name="combine_share", op="combine", T=16383, E=EXP, first=32, local=16, k=8, H=4096, dtype="f32", to="bf16"),
        # a training step's gradients to the experts' outputs and to the routing weights
        dict(name="combine_grad_train", op="combine_grad", T=8192, E=EXP, first=0, local=EXP, k=8, H=HID, dtype="bf16", to="bf16"),
        # the tokens of a decode step; a training batch on one of four shards of a vocabulary
        dict(name="embed_decode", op="embed", T=33, V=32000, first=0, rows=32000, H=4096, dtype="bf16", scale=1.0, ids="i64"),
        dict(name="embed_batch", op="embed", T=32768, V=128000, first=32000, rows=32000, H=4096, dtype="bf16", scale=64.0, ids="i64"),
        # gradients: a few sequences into a ragged shard in 32 bits, a large batch into half of a vocabulary
        dict(name="embed_grad_ragged", op="embed_grad", T=4095, V=50001, first=12500, rows=12501, H=2048, dtype="f32", scale=1.0, ids="i32"),
        dict(name="embed_grad_batch", op="embed_grad", T=32768, V=128000, first=0, rows=64000, H=4096, dtype="bf16", scale=1.0, ids="i64"),
        # a few small gradients, clipped: latency
        dict(name="clip_few", op="clip", n=37, mean=4099, dtype="f32", to="same", limit=0.25, pad=4),
        # one of four shards of this repository's 10,000 small tensors, rows and columns of any number; under the limit in
        # place, as most steps are
        dict(name="clip_many", op="clip", n=10000, mean=150000, dtype="bf16", to="here", limit=4.0, pad=1),
        # an expert layer's gate, up and down gradients in 16 bits, clipped into the optimizer's 32
        dict(name="clip_experts", op="clip", n=3 * EXP, mean=FFN * HID, dtype="bf16", to="f32", limit=0.25, pad=8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["permute", "permute_grad", "combine", "combine_grad", "embed", "embed", "embed_grad", "embed_grad", "norm", "clip", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32", "f16"])
    if op in ("permute", "permute_grad", "combine", "combine_grad"):
        E = _log(rng, 4, 512)
        local = max(1, E // rng.choice([1, 1, 2, 8]))
        k = rng.randint(1, min(12, E))
        H = _log(rng, 64, 8192) if rng.random() < 0.3 else 16 * _log(rng, 4, 512)
        T = _log(rng, 1, min(32768, max(1, 8192 * 8 * HID // (k * H))))
        c = dict(op=op, T=T, E=E, first=rng.randint(0, E - local), local=local, k=k, H=H, dtype=dtype)
        if op.startswith("combine"):
            # experts' outputs in the activations' type, or still in 32 bits
            c["to"] = dtype if rng.random() < 0.6 else rng.choice(["bf16", "f16"])
            if c["to"] != dtype:
                c["dtype"] = "f32"
        return c
    if op in ("embed", "embed_grad"):
        V = _log(rng, 256, 262144)
        H = _log(rng, 64, 8192) if rng.random() < 0.3 else 16 * _log(rng, 4, 512)
        rows = max(1, V // rng.choice([1, 1, 2, 4, 8]))
        while rows * H > 64000 * 4096:
            rows = (rows + 1) // 2
        T = _log(rng, 1, min(65536, 32768 * 4096 // H))
        return dict(op=op, T=T, V=V, first=rng.randint(0, V - rows), rows=rows, H=H, dtype=dtype, scale=rng.choice([1.0, 1.0, 64.0]), ids=rng.choice(["i64", "i64", "i32"]))
    n = _log(rng, 1, 4000)
    mean = _log(rng, 16, min(4 << 20, 3 * EXP * FFN * HID // n))
    c = dict(op=op, n=n, mean=mean, dtype=rng.choice(["bf16", "f32", "f16", "mixed"]), pad=rng.choice([1, 8, 8]))
    if op == "clip":
        # clipped into tensors of their own; or in place under the limit, where most steps are and a pass changes nothing
        c["to"] = rng.choice(["same", "f32", "here"])
        c["limit"] = 4.0 if c["to"] == "here" else rng.choice([0.25, 0.25, 4.0])
    return c


DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _sizes(case):
    """The tensors' sizes, a model's own: between a 16th of the mean and twice as much."""
    import random
    m = case["mean"]
    rng = random.Random(case["n"] * 1000003 + m)
    return [rng.randint(max(1, m // 16), max(1, 2 * m - m // 16)) for _ in range(case["n"])]


def _buffers(sizes, pad, dtypes):
    """(tensors of these sizes and types, the zeroed buffers that hold those of a type side by side, each from a multiple of
    `pad` elements on)"""
    out, flat = [None] * len(sizes), []
    for dtype in dict.fromkeys(dtypes):
        mine = [i for i, d in enumerate(dtypes) if d is dtype]
        room = [-(-sizes[i] // pad) * pad for i in mine]
        flat.append(torch.zeros(sum(room), dtype=dtype, device="cuda"))
        for i, part in zip(mine, flat[-1].split(room)):
            out[i] = part[:sizes[i]]
    return out, flat


def prepare(case, seed):
    dev, op, c = "cuda", case["op"], dict(case)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": c}
    if op in ("norm", "clip"):
        sizes = _sizes(c)
        kinds = [torch.bfloat16, torch.float32, torch.float16] if c["dtype"] == "mixed" else [DT[c["dtype"]]]
        dtypes = [kinds[i % len(kinds)] for i in range(len(sizes))]
        grads, s["flat"] = _buffers(sizes, c["pad"], dtypes)
        std = (torch.rand(len(sizes), generator=g, device=dev) * 4 - 5).exp().tolist()     # layers differ: 0.007 to 0.37
        for x, v in zip(grads, std):
            x.normal_(0, v, generator=g)
        s["grads"] = grads
        if op == "clip":
            s["limit"] = c["limit"] * math.sqrt(sum(n * v * v for n, v in zip(sizes, std)))
            if c["to"] != "here":
                s["out"], s["flat"] = _buffers(sizes, c["pad"], dtypes if c["to"] == "same" else [DT[c["to"]]] * len(sizes))
        if own:
            import dtensor_resharding_gb300 as R
            s["list"] = R.reshard_tensor_list(grads)        # gradients stay where they are from step to step
            s["into"] = R.reshard_tensor_list(s["out"]) if "out" in s else None
        return s
    dt = DT[c["dtype"]]
    if op in ("embed", "embed_grad"):
        # tokens by frequency: the most frequent is some 6% of a text, spread over the vocabulary
        rank = (torch.rand(c["T"], generator=g, device=dev, dtype=torch.float64) * math.log(c["V"] + 1)).exp().long() - 1
        ids = (rank.clamp(0, c["V"] - 1) * 48271 + seed) % c["V"]
        s["ids"] = ids if c["ids"] == "i64" else ids.int()
        if op == "embed":
            s["table"] = (randn(c["rows"], c["H"]) * 0.02).to(dt)
        else:
            s["grad"] = (randn(c["T"], c["H"]) * 1e-2).to(dt)
        return s
    T, E, k, H = c["T"], c["E"], c["k"], c["H"]
    z = randn(T, E) + randn(E) * 0.5
    top = torch.sort(z, dim=1, descending=True)
    ids = top.indices[:, :k].reshape(-1)
    e = ids - c["first"]
    here = (e >= 0) & (e < c["local"])
    key = torch.where(here, e, c["local"])
    order = torch.sort(key, stable=True).indices
    held = int(here.sum())
    position = torch.full((T * k,), -1, dtype=torch.int32, device=dev)
    position[order[:held]] = torch.arange(held, device=dev, dtype=torch.int32)
    count = torch.bincount(key, minlength=c["local"] + 1)[:c["local"]]
    offsets = torch.zeros(c["local"] + 1, dtype=torch.int32, device=dev)
    offsets[1:] = torch.cumsum(count, 0)
    s["sort"] = (offsets, order.int(), position)
    s["weights"] = torch.softmax(top.values[:, :k], 1).contiguous()
    if op == "permute":
        s["x"] = randn(T, H).to(dt)
        s["out"] = torch.zeros(T * k, H, dtype=dt, device=dev)
    elif op == "permute_grad":
        s["grad"] = randn(T * k, H).to(dt)
    else:
        s["y"] = randn(T * k, H).to(dt)
        if op == "combine_grad":
            s["grad"] = randn(T, H).to(DT[c["to"]])
    return s


def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s, s["case"])


# ---------------------------------------------------------------------------------------------- the library's calls

def _own_permute(s, c):
    import dtensor_resharding_gb300 as R
    return R.reshard_permute(s["x"], s["sort"], out=s["out"])


def _own_permute_grad(s, c):
    import dtensor_resharding_gb300 as R
    return R.reshard_permute_backward(s["grad"], s["sort"], c["k"])


def _own_combine(s, c):
    import dtensor_resharding_gb300 as R
    return R.reshard_combine(s["y"], s["sort"], s["weights"], out_dtype=DT[c["to"]])


def _own_combine_grad(s, c):
    import dtensor_resharding_gb300 as R
    dy, dw = R.reshard_combine_backward(s["grad"], s["y"], s["sort"], s["weights"])
    return {"y": dy, "weights": dw}


def _own_embed(s, c):
    import dtensor_resharding_gb300 as R
    return R.reshard_embedding(s["ids"], s["table"], scale=c["scale"], first_row=c["first"])


def _own_embed_grad(s, c):
    import dtensor_resharding_gb300 as R
    return R.reshard_embedding_backward(s["grad"], s["ids"], c["rows"], scale=c["scale"], first_row=c["first"])


def _own_norm(s, c):
    import dtensor_resharding_gb300 as R
    return R.reshard_grad_norm(s["list"])


def _own_clip(s, c):
    import dtensor_resharding_gb300 as R
    norm = R.reshard_clip_grads(s["list"], s["limit"], out=s["into"])
    return {"norm": norm, "grads": s["flat"]}


# ------------------------------------------------------------------------------------- the plain form, in 32 bits

def _plain_permute(s, c):
    offsets, order, position = s["sort"]
    at = torch.nonzero(position >= 0).view(-1)
    s["out"][position[at].long()] = s["x"][at // c["k"]]
    return s["out"]


def _places(s, c):
    """(each slot's place, 0 where it has none; whether it has one, as 0 or 1)"""
    position = s["sort"][2].view(c["T"], c["k"])
    return position.clamp_min(0).long(), (position >= 0).float()


def _plain_permute_grad(s, c):
    at, here = _places(s, c)
    dx = torch.zeros(c["T"], c["H"], device=at.device)
    for j in range(c["k"]):
        dx += s["grad"][at[:, j]].float() * here[:, j:j + 1]
    return dx.to(s["grad"].dtype)


def _plain_combine(s, c):
    at, here = _places(s, c)
    out = torch.zeros(c["T"], c["H"], device=at.device)
    for j in range(c["k"]):
        out += s["y"][at[:, j]].float() * (s["weights"] * here)[:, j:j + 1]
    return out.to(DT[c["to"]])


def _plain_combine_grad(s, c):
    at, here = _places(s, c)
    dout = s["grad"].float()
    dy, dw = torch.zeros_like(s["y"]), torch.empty_like(s["weights"])
    for j in range(c["k"]):
        dw[:, j] = (dout * s["y"][at[:, j]].float()).sum(1) * here[:, j]
        t = torch.nonzero(here[:, j]).view(-1)
        dy[at[t, j]] = (dout[t] * s["weights"][t, j:j + 1]).to(dy.dtype)
    return {"y": dy, "weights": dw}


def _plain_embed(s, c):
    r = s["ids"].long() - c["first"]
    here = (r >= 0) & (r < c["rows"])
    x = s["table"][torch.where(here, r, 0)].float() * c["scale"]
    return torch.where(here.unsqueeze(1), x, 0.0).to(s["table"].dtype)


def _plain_embed_grad(s, c):
    r = s["ids"].long() - c["first"]
    t = torch.nonzero((r >= 0) & (r < c["rows"])).view(-1)
    d = torch.zeros(c["rows"], c["H"], device=r.device)
    d.index_add_(0, r[t], s["grad"][t].float())
    return (d * c["scale"]).to(s["grad"].dtype)


def _plain_norm(s, c):
    return torch.stack([x.float().square().sum() for x in s["grads"]]).double().sum().sqrt().float()


def _plain_clip(s, c):
    norm = _plain_norm(s, c)
    factor = (s["limit"] / (norm + EPS)).clamp_max(1.0)
    for x, y in zip(s["grads"], s.get("out", s["grads"])):
        y.copy_(x.float() * factor)
    return {"norm": norm, "grads": s["flat"]}


_own = {"permute": _own_permute, "permute_grad": _own_permute_grad, "combine": _own_combine, "combine_grad": _own_combine_grad,
        "embed": _own_embed, "embed_grad": _own_embed_grad, "norm": _own_norm, "clip": _own_clip}
_plain = {"permute": _plain_permute, "permute_grad": _plain_permute_grad, "combine": _plain_combine, "combine_grad": _plain_combine_grad,
          "embed": _plain_embed, "embed_grad": _plain_embed_grad, "norm": _plain_norm, "clip": _plain_clip}


# ------------------------------------------------------------------------------------------------ the work of a pass

ES = {"bf16": 2, "f16": 2, "f32": 4, "mixed": 8 / 3}


def work(case):
    c, op, es = case, case["op"], ES[case["dtype"]]
    if op in ("norm", "clip"):
        n = c["n"] * c["mean"]
        # under the limit in place nothing has to be written
        write = 0 if op == "norm" or c["to"] == "here" else ES[c["to"]] if c["to"] in ES else es
        return {"bytes": n * (es + write), "flops": n * (3 if write else 2)}
    if op == "embed":
        held, used = c["T"] * c["rows"] / c["V"], _used(c)
        return {"bytes": c["T"] * (int(c["ids"][1:]) // 8 + c["H"] * es) + used * c["H"] * es, "flops": held * c["H"]}
    if op == "embed_grad":
        held = c["T"] * c["rows"] / c["V"]
        return {"bytes": c["T"] * int(c["ids"][1:]) // 8 + (held + c["rows"]) * c["H"] * es, "flops": held * c["H"]}
    T, k, H = c["T"], c["k"], c["H"]
    held = T * k * c["local"] / c["E"]
    some = T * (1 - (1 - c["local"] / c["E"]) ** k)        # tokens with a choice here, about
    to = ES[c.get("to", c["dtype"])]
    if op == "permute":
        return {"bytes": (some + held) * H * es + 4 * T * k, "flops": 0}
    if op == "permute_grad":
        return {"bytes": (held + T) * H * es + 4 * T * k, "flops": held * H}
    if op == "combine":
        return {"bytes": held * H * es + T * H * to + 8 * T * k, "flops": 2 * held * H}
    return {"bytes": some * H * to + (held + T * k) * H * es + 12 * T * k, "flops": 3 * held * H}


def _used(c):
    """Rows of the table that some token reads, about: the r-th most frequent is 1 / (r log V) of the text."""
    lv, used, step = math.log(c["V"] + 1), 0.0, max(1, c["V"] // 4096)
    for r in range(0, c["V"], step):
        p = math.log((r + 2) / (r + 1)) / lv
        used += step * (1 - (1 - p) ** c["T"])
    return used * c["rows"] / c["V"]


# ------------------------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op in ("norm", "clip"):
        # one tensor at a time: the squares of a whole model in 64 bits would not fit beside it
        norm = sum(torch.dot(x.double(), x.double()) for x in s["grads"]).sqrt()
        if op == "norm":
            return norm
        factor = torch.minimum(torch.ones_like(norm), s["limit"] / (norm + EPS))
        flat = [torch.zeros(f.shape, dtype=torch.float64, device="cuda") for f in s["flat"]]
        for x, y in zip(s["grads"], s.get("out", s["grads"])):
            at = next(i for i, f in enumerate(s["flat"]) if f.dtype == y.dtype)
            flat[at][y.storage_offset():y.storage_offset() + y.numel()] = x.double() * factor
        return {"norm": norm, "grads": flat}
    if op == "embed":
        table = torch.cat([s["table"].double() * c["scale"], torch.zeros(1, c["H"], dtype=torch.float64, device="cuda")])
        r = s["ids"].long() - c["first"]
        r[(r < 0) | (r >= c["rows"])] = c["rows"]
        return table[r]
    if op == "embed_grad":
        r = s["ids"].long() - c["first"]
        r[(r < 0) | (r >= c["rows"])] = c["rows"]
        order = torch.argsort(r)
        d = torch.zeros(c["rows"] + 1, c["H"], dtype=torch.float64, device="cuda")
        for part in order.split(8192):
            d.index_add_(0, r[part], s["grad"][part].double())
        return d[:c["rows"]] * c["scale"]
    T, k, H = c["T"], c["k"], c["H"]
    offsets, order, _ = s["sort"]
    held = int(offsets[-1])
    slot = order[:held].long()
    t = slot // k
    if op == "permute":
        y = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        y[:held] = s["x"].double()[t]
        return y
    w = s["weights"].double().view(-1)[slot].unsqueeze(1)
    if op in ("permute_grad", "combine"):
        d = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        rows = s["grad"][:held].double() if op == "permute_grad" else s["y"][:held].double() * w
        return d.index_add_(0, t, rows)
    dy = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    dout = s["grad"].double()[t]
    dw[slot] = (dout * s["y"][:held].double()).sum(1)
    dy[:held] = dout * w
    return {"y": dy, "weights": dw.view(T, k)}
