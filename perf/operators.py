"""The expert-layer operators that are timed and compared: routing to experts and its gradient, quantization to
8-bit floating point in blocks of 128, the matrix product over such blocks, and the routed expert feed-forward.

Each case runs in two forms on the same inputs: `own` False computes the definition with elementary torch
operations in 32 bits, `own` True calls the library. `exact` computes the definition in 64 bits, on its own.

Definitions
  route     per row of logits z: score s = softmax(z) or sigmoid(z). Experts are ordered by s + bias (without a bias by
            z, which orders them alike), the lowest index first among equals. With groups, only the `kept` groups with
            the largest sum of their `group_top` best scores (+ bias) take part. The k first give ids and
            weights scale * s, divided by their sum where `renorm`. A logit of -inf or NaN is never chosen; where
            fewer than k are left, the id is -1 and the weight 0.
  quantize  per block: amax a = max |x| (at least 2^-100), scale a / 448, value e4m3(x * (448 / a)). Rows: blocks of
            1 x 128; weights: blocks of 128 x 128. A block that holds an infinity or NaN has scale and values NaN.
  linear    y = Q(x) W^T, where Q(x) is x quantized by rows and W the weights' values times their block scales.
  experts   y[t] = sum_j weight[t, j] * W2[e] Q(silu(g) * u), [g, u] = W13[e] Q(x[t]), e = ids[t, j]; only experts
            first .. first + local - 1 are held here, other ids (and -1) add nothing.
"""
import math

import torch

own = False

HID, FFN, EXP = 2048, 768, 128   # the expert layers of this repository's blockwise FP8 workload
TINY = 2.0 ** -100


def listed():
    return [
        # one decode step of a small batch: latency
        dict(name="route_decode", op="route", T=24, E=128, k=8, score="softmax", dtype="bf16", bias=False, groups=1, kept=1, group_top=1, renorm=True, scale=1.0, masked=False),
        # a prefill chunk under balanced sigmoid routing with group limits
        dict(name="route_groups", op="route", T=16384, E=256, k=8, score="sigmoid", dtype="f32", bias=True, groups=8, kept=4, group_top=2, renorm=True, scale=2.5, masked=False),
        # training steps: the routing gradient, whole softmax and renormalised sigmoid
        dict(name="route_grad_softmax", op="route_grad", T=8191, E=60, k=4, score="softmax", dtype="bf16", renorm=False, scale=1.0),
        dict(name="route_grad_sigmoid", op="route_grad", T=32768, E=128, k=8, score="sigmoid", dtype="f32", renorm=True, scale=2.5),
        # activations of a prefill chunk; an expert tensor on the receiving side of a refit
        dict(name="quantize_rows", op="quantize_rows", M=16384, K=4096, dtype="bf16"),
        dict(name="quantize_experts", op="quantize_blocks", E=EXP, N=FFN, K=HID, dtype="bf16"),
        # a dense FFN projection: one token, a ragged speculative batch on an uneven shard, a prefill chunk
        dict(name="linear_one_token", op="linear", M=1, N=14336, K=4096, dtype="bf16"),
        dict(name="linear_ragged", op="linear", M=77, N=2867, K=4096, dtype="bf16"),
        dict(name="linear_prefill", op="linear", M=8192, N=14336, K=4096, dtype="bf16"),
        # the expert feed-forward: a decode step, one rank's share of the experts, a prefill chunk
        dict(name="experts_decode", op="experts", T=16, E=EXP, first=0, local=EXP, k=8, H=HID, I=FFN, dtype="bf16"),
        dict(name="experts_share", op="experts", T=4095, E=EXP, first=32, local=16, k=8, H=4096, I=1536, dtype="bf16"),
        dict(name="experts_prefill", op="experts", T=8192, E=EXP, first=0, local=EXP, k=8, H=HID, I=FFN, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "quantize_rows", "quantize_blocks", "linear", "linear", "experts", "experts"])
    # activations that meet 8-bit weights come in 16-bit types; logits and what is quantized also in 32 bits
    dtype = rng.choice(["bf16", "bf16", "f16"] if op in ("linear", "experts") else ["bf16", "bf16", "f32", "f16"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 4, 512 // groups)
        kept = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1 if op == "route" else 2, min(12, kept * (E // groups)))   # one renormalised weight has no gradient
        T = _log(rng, 1, min(32768, 4194304 // E))
        score = rng.choice(["softmax", "sigmoid"])
        c = dict(op=op, T=T, E=E, k=k, score=score, dtype=dtype, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 1.0, 2.5]))
        if op == "route":
            # a softmax row's sum rounds by its order of summation, so a bias on top of it is drawn with sigmoid scores only
            c.update(bias=score == "sigmoid" and rng.random() < 0.6, groups=groups, kept=kept, group_top=min(rng.choice([1, 2]), E // groups), masked=rng.random() < 0.3)
        return c
    if op == "quantize_rows":
        K = _log(rng, 16, 16384)
        return dict(op=op, M=_log(rng, 1, 16384 * 4096 // max(K, 1024)), K=K, dtype=dtype)
    if op == "quantize_blocks":
        N, K = _log(rng, 64, 4096), _log(rng, 64, 4096)
        return dict(op=op, E=_log(rng, 1, min(EXP, max(1, EXP * FFN * HID // (N * K)))), N=N, K=K, dtype=dtype)
    if op == "linear":
        N, K = _log(rng, 32, 14336), _log(rng, 64, 14336)
        while N * K > 14336 * 4096:
            N, K = (N + 1) // 2, (K + 1) // 2
        return dict(op=op, M=_log(rng, 1, 8192), N=N, K=K, dtype=dtype)
    E = rng.choice([8, 16, 32, 64, 128])
    H, I = 16 * _log(rng, 8, 256), 128 * rng.randint(1, 12)
    while H * I > 4096 * 1536:
        H = 16 * max(8, H // 32)
    local = rng.choice([E, E, E // 2, E // 8 or 1])
    while local * H * I > EXP * HID * FFN:
        local = max(1, local // 2)
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, min(8192, max(1, 8192 * 8 * HID * FFN // (k * H * I) * E // local)))
    return dict(op=op, T=T, E=E, first=rng.randint(0, E - local), local=local, k=k, H=H, I=I, dtype=dtype)


DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _pitched(shape, dtype, dev):
    """A tensor whose rows start every multiple of 16 bytes, as the library's products read them."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.zeros(*shape[:-1], -(-shape[-1] // per) * per, dtype=dtype, device=dev)[..., :shape[-1]]


def _weights(g, E, N, K, dev):
    """Random weights (standard deviation 0.02, rows of varied size) as e4m3 values and 128 x 128 block scales."""
    nb, kb = -(-N // 128), -(-K // 128)
    q = _pitched((E, N, K), torch.float8_e4m3fn, dev)
    scale = torch.empty(E, nb, kb, device=dev).uniform_(0.5, 2.0, generator=g) * (0.08 / 448)
    for e in range(E):
        q[e].copy_((torch.randn(N, K, generator=g, device=dev) * 112).clamp_(-448, 448))
    return q, scale


def prepare(case, seed):
    dev, op = "cuda", case["op"]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c = dict(case)
    dt = DT[c["dtype"]]
    s = {"case": c}
    if op in ("route", "route_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        z = torch.randn(T, E, generator=g, device=dev) * 1.5 + torch.randn(E, generator=g, device=dev) * 0.7
        if c.get("masked"):
            z.masked_fill_(torch.rand(T, E, generator=g, device=dev) < 0.2, float("-inf"))
            z.masked_fill_(torch.rand(T, 1, generator=g, device=dev) < 0.05, float("-inf"))   # padding rows
        s["z"] = z.to(dt)
        if c.get("bias"):
            s["bias"] = torch.randn(E, generator=g, device=dev) * 0.1
        if op == "route_grad":
            s["ids"] = torch.sort(torch.rand(T, E, generator=g, device=dev) - z.float().sigmoid(), dim=1).indices[:, :k].int().contiguous()
            s["grad"] = torch.randn(T, k, generator=g, device=dev)
    elif op == "quantize_rows":
        s["x"] = _activations(g, c["M"], c["K"], dev).to(dt)
    elif op == "quantize_blocks":
        s["w"] = (torch.randn(c["E"], c["N"], c["K"], generator=g, device=dev) * 0.02).to(dt)
    elif op == "linear":
        s["x"] = _activations(g, c["M"], c["K"], dev).to(dt)
        q, w = _weights(g, 1, c["N"], c["K"], dev)
        s["w"], s["ws"] = q[0], w[0]
    else:
        T, E, H, I, n = c["T"], c["E"], c["H"], c["I"], c["local"]
        s["x"] = _activations(g, T, H, dev).to(dt)
        popular = torch.randn(E, generator=g, device=dev) * 0.5
        z = torch.randn(T, E, generator=g, device=dev) + popular
        top = torch.sort(z, dim=1, descending=True)
        s["ids"] = top.indices[:, :c["k"]].int().contiguous()
        s["weights"] = torch.softmax(top.values[:, :c["k"]], 1).contiguous()
        s["w13"], s["w13s"] = _weights(g, n, 2 * I, H, dev)
        s["w2"], s["w2s"] = _weights(g, n, H, I, dev)
    return s


def _activations(g, rows, cols, dev):
    """Normal values with a few channels ten times as large, as hidden states have them."""
    x = torch.randn(rows, cols, generator=g, device=dev)
    return x * torch.where(torch.rand(cols, generator=g, device=dev) < 0.01, 10.0, 1.0)


def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s, s["case"])


# ---------------------------------------------------------------------------------------------- the library's calls

def _own_route(s, c):
    import dtensor_resharding_gb300 as R
    w, ids = R.reshard_route(s["z"], c["k"], score=c["score"], bias=s.get("bias"), groups=c["groups"], groups_kept=c["kept"],
                             group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"])
    return {"weights": w, "ids": ids}


def _own_route_grad(s, c):
    import dtensor_resharding_gb300 as R
    return R.reshard_route_backward(s["grad"], s["z"], s["ids"], score=c["score"], renormalize=c["renorm"], scale=c["scale"])


def _own_quantize_rows(s, c):
    import dtensor_resharding_gb300 as R
    q, scale = R.reshard_quantize_rows(s["x"])
    return {"q": q, "scale": scale}


def _own_quantize_blocks(s, c):
    import dtensor_resharding_gb300 as R
    q, scale = R.reshard_quantize_blocks(s["w"])
    return {"q": q, "scale": scale}


def _own_linear(s, c):
    import dtensor_resharding_gb300 as R
    return R.reshard_linear_fp8(s["x"], s["w"], s["ws"])


def _own_experts(s, c):
    import dtensor_resharding_gb300 as R
    return R.reshard_experts_fp8(s["x"], s["ids"], s["weights"], s["w13"], s["w13s"], s["w2"], s["w2s"], first_expert=c["first"])


# ------------------------------------------------------------------------------------- the plain form, in 32 bits

def _plain_route(s, c):
    z = s["z"].float()
    T, E = z.shape
    none = float("-inf")
    z = torch.where(z.isnan(), none, z)
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
        rank = score
    else:
        top = z.amax(1, keepdim=True)
        rank = torch.exp(z - torch.where(top == none, 0.0, top))
        score = rank / rank.sum(1, keepdim=True)
    key = z if s.get("bias") is None else (score + s["bias"]).masked_fill(z == none, none)
    if c["groups"] > 1:
        part = (rank.masked_fill(z == none, none) if s.get("bias") is None else key).view(T, c["groups"], -1)
        best = torch.sort(part, dim=2, descending=True).values[:, :, :c["group_top"]]
        total = torch.where(best == none, 0.0, best).sum(2).masked_fill(best[:, :, 0] == none, none)
        order = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=z.device).scatter_(1, order, True)
        key = key.masked_fill(~keep.repeat_interleave(E // c["groups"], 1), none)
    first = torch.sort(key, dim=1, descending=True, stable=True)
    ids, dead = first.indices[:, :c["k"]], first.values[:, :c["k"]] == none
    if c["score"] == "softmax" and c["renorm"]:
        chosen = torch.gather(z, 1, ids).masked_fill(dead, none)
        top = chosen.amax(1, keepdim=True)
        w = torch.exp(chosen - torch.where(top == none, 0.0, top))
    else:
        w = torch.gather(score, 1, ids).masked_fill(dead, 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, 0.0, w / total)
    return {"weights": (w * c["scale"]).masked_fill(dead, 0.0), "ids": ids.masked_fill(dead, -1).int()}


def _plain_route_grad(s, c):
    z, g, ids = s["z"].float(), s["grad"] * c["scale"], s["ids"].long()
    if c["score"] == "softmax" and not c["renorm"]:
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        chosen = torch.gather(p, 1, ids)
        d = -p * (g * chosen).sum(1, keepdim=True)
        return d.scatter_add_(1, ids, g * chosen).to(s["z"].dtype)
    chosen = torch.gather(z, 1, ids)
    if c["score"] == "softmax":
        r = torch.exp(chosen - chosen.amax(1, keepdim=True))
        r = r / r.sum(1, keepdim=True)
        d = r * (g - (g * r).sum(1, keepdim=True))
    else:
        sg, co = 1.0 / (1.0 + torch.exp(-chosen)), 1.0 / (1.0 + torch.exp(chosen))
        if c["renorm"]:
            r = sg / sg.sum(1, keepdim=True)
            d = r * (g - (g * r).sum(1, keepdim=True)) * co
        else:
            d = g * sg * co
    return torch.zeros_like(z).scatter_(1, ids, d).to(s["z"].dtype)


def _pad(x, to):
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % to))


def _plain_rows(x):
    """(e4m3 values, scales) of x in blocks of 1 x 128."""
    M, K = x.shape
    b = _pad(x.float(), 128).view(M, -1, 128)
    a = b.abs().amax(2, keepdim=True).clamp_min(TINY)
    a = torch.where(a.isinf(), float("nan"), a)
    q = (b * (448.0 / a)).to(torch.float8_e4m3fn).view(M, -1)[:, :K]
    return q, (a / 448.0).view(M, -1)


def _plain_quantize_rows(s, c):
    q, scale = _plain_rows(s["x"])
    return {"q": q, "scale": scale}


def _plain_quantize_blocks(s, c):
    w = s["w"].float()
    E, N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    b = torch.nn.functional.pad(w, (0, kb * 128 - K, 0, nb * 128 - N)).view(E, nb, 128, kb, 128)
    a = b.abs().amax((2, 4), keepdim=True).clamp_min(TINY)
    a = torch.where(a.isinf(), float("nan"), a)
    q = (b * (448.0 / a)).to(torch.float8_e4m3fn).view(E, nb * 128, kb * 128)[:, :N, :K]
    return {"q": q, "scale": (a / 448.0).view(E, nb, kb)}


def _spread(scale, N, K):
    return scale.repeat_interleave(128, -2)[..., :N, :].repeat_interleave(128, -1)[..., :K]


def _plain_values(x):
    q, scale = _plain_rows(x)
    return q.float() * scale.repeat_interleave(128, 1)[:, :x.shape[1]]


def _plain_linear(s, c):
    w = s["w"].float() * _spread(s["ws"], c["N"], c["K"])
    return (_plain_values(s["x"]) @ w.t()).to(s["x"].dtype)


def _plain_experts(s, c):
    T, k, H, I, n = c["T"], c["k"], c["H"], c["I"], c["local"]
    e = s["ids"].long().view(-1) - c["first"]
    here = torch.nonzero((e >= 0) & (e < n)).view(-1)
    out = torch.zeros(T, H, device=e.device)
    if here.numel() == 0:
        return out.to(s["x"].dtype)
    here = here[torch.sort(e[here], stable=True).indices]           # slots by expert
    of = e[here]
    count = torch.bincount(of, minlength=n)
    at = torch.arange(here.numel(), device=e.device) - (torch.cumsum(count, 0) - count)[of]
    most = int(count.max())
    x = torch.zeros(n, most, H, device=e.device)
    x[of, at] = _plain_values(s["x"])[here // k]
    gu = torch.bmm(x, (s["w13"].float() * _spread(s["w13s"], 2 * I, H)).transpose(1, 2))
    gu = gu[of, at]
    g, u = gu[:, :I], gu[:, I:]
    h = _plain_values(g / (1.0 + torch.exp(-g)) * u)
    x = torch.zeros(n, most, I, device=e.device)
    x[of, at] = h
    y = torch.bmm(x, (s["w2"].float() * _spread(s["w2s"], H, I)).transpose(1, 2))[of, at]
    slots = torch.zeros(T * k, H, device=e.device)
    slots[here] = y * s["weights"].view(-1)[here].unsqueeze(1)
    return slots.view(T, k, H).sum(1).to(s["x"].dtype)


_own = {"route": _own_route, "route_grad": _own_route_grad, "quantize_rows": _own_quantize_rows, "quantize_blocks": _own_quantize_blocks,
        "linear": _own_linear, "experts": _own_experts}
_plain = {"route": _plain_route, "route_grad": _plain_route_grad, "quantize_rows": _plain_quantize_rows,
          "quantize_blocks": _plain_quantize_blocks, "linear": _plain_linear, "experts": _plain_experts}


# ------------------------------------------------------------------------------------------------ the work of a pass

def work(case):
    c, op = case, case["op"]
    es = 4 if c["dtype"] == "f32" else 2
    if op == "route":
        # logits in, weights and ids out; per expert an exponential, a sum and a comparison with each of the k best
        return {"bytes": c["T"] * (c["E"] * es + 8 * c["k"]) + 4 * c["E"] * bool(c["bias"]), "flops": c["T"] * c["E"] * 4}
    if op == "route_grad":
        # the whole softmax's gradient needs every logit, the others' the chosen ones
        every = c["score"] == "softmax" and not c["renorm"]
        return {"bytes": c["T"] * ((c["E"] if every else c["k"]) * es + c["E"] * es + 8 * c["k"]), "flops": c["T"] * (c["E"] * 4 * every + 10 * c["k"])}
    if op == "quantize_rows":
        return {"bytes": c["M"] * (c["K"] * (es + 1) + 4 * -(-c["K"] // 128)), "flops": 2 * c["M"] * c["K"]}
    if op == "quantize_blocks":
        return {"bytes": c["E"] * (c["N"] * c["K"] * (es + 1) + 4 * -(-c["N"] // 128) * -(-c["K"] // 128)), "flops": 2 * c["E"] * c["N"] * c["K"]}
    if op == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K * es + N * K + 4 * -(-N // 128) * -(-K // 128) + M * N * es, "flops": 2 * M * N * K}
    T, H, I, n, k = c["T"], c["H"], c["I"], c["local"], c["k"]
    slots = T * k * n / c["E"]
    used = n * (1 - (1 - k / c["E"]) ** T)       # experts that some token reaches, under even routing
    w = 3 * H * I * (1 + 4 / 16384)
    return {"bytes": used * w + T * H * es * 2 + T * k * 8, "flops": 6 * slots * H * I}


# ------------------------------------------------------------------------------------ the definition, in 64 bits

def _e4m3(v):
    """v (64 bits) rounded to the nearest e4m3 value, ties to even."""
    _, e = torch.frexp(v.abs())
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_rows(x):
    x = x.double()
    M, K = x.shape
    pad = torch.zeros(M, -K % 128, dtype=torch.float64, device=x.device)
    b = torch.cat([x, pad], 1).reshape(M, -1, 128)
    scale = b.abs().max(2).values.clamp_min(TINY) / 448
    return _e4m3(b / scale.unsqueeze(2)).reshape(M, -1)[:, :K], scale


def _exact_values(x):
    q, scale = _exact_rows(x)
    return q * scale[:, torch.arange(x.shape[1], device=x.device) // 128]


def _exact_weights(q, scale):
    r, c = (torch.arange(d, device=q.device) // 128 for d in q.shape)
    return q.double() * scale.double()[r][:, c]


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op == "route":
        z = s["z"].double()
        p = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
        key = (p + s["bias"].double()) if s.get("bias") is not None else z
        dead = z == float("-inf")
        if c["groups"] > 1:
            part = (key if s.get("bias") is not None else p).masked_fill(dead, float("-inf"))
            best = part.view(c["T"], c["groups"], -1).topk(c["group_top"], 2).values
            total = best.clamp_min(0).sum(2) if s.get("bias") is None else torch.where(best.isinf(), 0.0, best).sum(2)
            total = total.masked_fill(best[:, :, 0].isinf(), float("-inf"))
            rank = (total.unsqueeze(2) < total.unsqueeze(1)).sum(2) + torch.tril(total.unsqueeze(2) == total.unsqueeze(1), -1).sum(2)
            dead = dead | (rank >= c["kept"]).repeat_interleave(c["E"] // c["groups"], 1)
        key = key.masked_fill(dead, float("-inf"))
        ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["k"]]
        gone = torch.gather(dead, 1, ids)
        w = torch.gather(p, 1, ids).masked_fill(gone, 0.0)
        if c["renorm"]:
            w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
        return {"weights": w * c["scale"], "ids": None}
    if op == "route_grad":
        z = s["z"].double().requires_grad_()
        p = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
        w = torch.gather(p, 1, s["ids"].long())
        w = (w / w.sum(1, keepdim=True) if c["renorm"] else w) * c["scale"]
        (w * s["grad"].double()).sum().backward()
        return z.grad
    if op == "quantize_rows":
        q, scale = _exact_rows(s["x"])
        return {"q": q, "scale": scale}
    if op == "quantize_blocks":
        E, N, K = s["w"].shape
        r, k = (torch.arange(d, device=s["w"].device) // 128 for d in (N, K))
        q, scale = [], []
        for e in range(E):
            w = s["w"][e].double()
            a = torch.zeros(-(-N // 128), K, dtype=torch.float64, device=w.device).index_reduce_(0, r, w.abs(), "amax")
            a = torch.zeros(a.shape[0], -(-K // 128), dtype=torch.float64, device=w.device).index_reduce_(1, k, a, "amax").clamp_min(TINY) / 448
            q.append(_e4m3(w / a[r][:, k]))
            scale.append(a)
        return {"q": torch.stack(q), "scale": torch.stack(scale)}
    if op == "linear":
        return _exact_values(s["x"]) @ _exact_weights(s["w"], s["ws"]).t()
    x, I = _exact_values(s["x"]), c["I"]
    y = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=x.device)
    for e in range(c["local"]):
        t, j = torch.nonzero(s["ids"] == e + c["first"], as_tuple=True)
        if len(t) == 0:
            continue
        gu = x[t] @ _exact_weights(s["w13"][e], s["w13s"][e]).t()
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        out = _exact_values(h) @ _exact_weights(s["w2"][e], s["w2s"][e]).t()
        y.index_add_(0, t, out * s["weights"][t, j].double().unsqueeze(1))
    return y
