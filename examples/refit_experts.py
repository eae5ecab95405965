"""A refit of FP8 expert weights, and the expert layer that computes with them.

The training side holds a mixture-of-experts layer's gate, up and down projections, split over experts (EP). They are
quantized in blocks of 128 x 128 and moved to generation ranks that split the experts among fewer ranks and keep gate
and up fused ([gate; up] rows of one buffer), values and scales in one reshard. Each generation rank then routes the same
tokens and runs its own experts; the ranks' outputs sum to the whole layer's, which is checked against the layer run in
one piece. A step of the router's training then goes through the layer's stages, with gradients. All ranks are buffers on one GPU:

  python examples/refit_experts.py [--tokens 256] [--experts 32] [--hidden 1024] [--ffn 512] [--train 8] [--gen 2]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import dtensor_resharding_gb300 as R  # noqa: E402


def refit(train, experts, hidden, ffn, n_train, n_gen):
    """Moves every training rank's (values, scales) of gate, up and down to the generation ranks. Returns, for each of
    those, w13 [experts / n_gen, 2 ffn, hidden], its scale, w2 [experts / n_gen, hidden, ffn] and its scale."""
    per = experts // n_gen
    ranks = [dict(w13=torch.empty(per, 2 * ffn, hidden, dtype=torch.uint8, device="cuda"),
                  s13=torch.empty(per, 2 * ffn // 128, -(-hidden // 128), device="cuda"),
                  w2=torch.empty(per, hidden, ffn, dtype=torch.uint8, device="cuda"),
                  s2=torch.empty(per, -(-hidden // 128), ffn // 128, device="cuda")) for _ in range(n_gen)]
    specs, src, dst = [], [], []
    for name, fused, row in (("gate", True, 0), ("up", True, ffn), ("down", False, 0)):
        for part, code in ((0, "u8"), (1, "f32")):
            shards = [t[name][part] for t in train]
            into = [r[("w13" if fused else "w2") if part == 0 else ("s13" if fused else "s2")] for r in ranks]
            shape = (experts, *shards[0].shape[1:])
            at = (row if part == 0 else row // 128) * shape[2]      # the fused buffer's rows of this projection
            views = [R.View(at, (b.stride(0), b.stride(1), 1)) for b in into]
            specs.append(R.Spec(shape, code, (n_train,), ["S0"], (n_gen,), ["S0"], dst_views=views))
            src += shards
            dst += into
    plan = R.reshard_plan_batch(specs)
    R.reshard_execute(plan, src, dst, stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    R.reshard_plan_destroy(plan)
    return [(r["w13"], r["s13"], r["w2"], r["s2"]) for r in ranks]


@torch.no_grad()
def experts(rows, offsets, weights):
    """The experts' outputs, in 32 bits, for rows in the order of their experts."""
    w13, s13, w2, s2 = weights
    ffn = w13.shape[1] // 2
    gu = R.reshard_matmul_fp8(*R.reshard_quantize_rows(rows), w13, s13, offsets=offsets, out_dtype=torch.float32)
    h = torch.nn.functional.silu(gu[:, :ffn]) * gu[:, ffn:]
    return R.reshard_matmul_fp8(*R.reshard_quantize_rows(h), w2, s2, offsets=offsets, out_dtype=torch.float32)


def main(argv=None) -> float:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 256), ("experts", 32), ("hidden", 1024), ("ffn", 512), ("train", 8), ("gen", 2), ("k", 4)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    # training ranks: their experts' projections, quantized in blocks (values as the bytes that a reshard moves)
    per = a.experts // a.train
    train = []
    for _ in range(a.train):
        rank = {}
        for name, shape in (("gate", (per, a.ffn, a.hidden)), ("up", (per, a.ffn, a.hidden)), ("down", (per, a.hidden, a.ffn))):
            q, scale = R.reshard_quantize_blocks(randn(*shape, std=0.02))
            rank[name] = (q.view(torch.uint8), scale)
        train.append(rank)
    ranks = refit(train, a.experts, a.hidden, a.ffn, a.train, a.gen)

    # a step of the generation side: route, each rank's experts, the sum over ranks
    x, router = randn(a.tokens, a.hidden), randn(a.hidden, a.experts, std=a.hidden ** -0.5)
    weights, ids = R.reshard_route(x @ router, a.k)
    total = torch.zeros(a.tokens, a.hidden, device="cuda")
    for r, (w13, s13, w2, s2) in enumerate(ranks):
        total += R.reshard_experts_fp8(x, ids, weights, w13, s13, w2, s2, first_expert=r * (a.experts // a.gen))

    # the same layer in one piece, from the training side's shards
    cat = {n: [torch.cat([t[n][p] for t in train]) for p in (0, 1)] for n in ("gate", "up", "down")}
    whole = R.reshard_experts_fp8(x, ids, weights, torch.cat([cat["gate"][0], cat["up"][0]], 1), torch.cat([cat["gate"][1], cat["up"][1]], 1),
                                  *cat["down"])
    off = float((total - whole.float()).norm() / whole.float().norm())

    # a training step of the router through the same layer, its stages one by one: tokens to their experts' places, the experts
    # in FP8, back with the weights. The gradient reaches the weights, the logits and the router; it is clipped before the update.
    router = router.float().requires_grad_()
    weights, ids = R.reshard_route(x.float() @ router, a.k)
    sort = R.reshard_dispatch(ids, a.experts)
    y = experts(R.reshard_permute(x, sort), sort[0], [torch.cat([r[i] for r in ranks]) for i in range(4)])
    (R.reshard_combine(y, sort, weights, out_dtype=torch.bfloat16).float() - whole.float().roll(1, 0)).square().sum().backward()
    norm = R.reshard_clip_grads([router.grad], 1.0)
    assert float(norm) > 0 and abs(float(R.reshard_grad_norm([router.grad])) - min(1.0, float(norm))) < 1e-3 and R.reshard_ops_status() == 0
    print(f"{a.experts} experts from {a.train} training to {a.gen} generation ranks, {a.tokens} tokens: the ranks' sum is {off:.2e} from the whole layer")
    return off


if __name__ == "__main__":
    # each rank's output is rounded to bf16 before the sum, the whole layer's once: at most 2^-8 of each
    sys.exit(0 if main() < 2 ** -7 else 1)
