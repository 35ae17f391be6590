"""One step of reinforcement learning on a small mixture of experts, on the
GPU: the rollout engine routes tokens to NVFP4 experts, samples, and scores its
samples; the trainer takes the policy loss with an entropy bonus, its gradients
through the same routing, and an AdamW step with moments in 8 bits that writes
the router's new 16-bit weights straight into the arena; the refit brings the
engine the same bytes, so that both sides compute the same logits again, bit
for bit (build first: python -c "import __graft_entry__ as g; g.build()").
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch
import bit_exact_xor_gb300 as dcr

EXPERTS, CHOSEN, HIDDEN, FFN, VOCAB, TOKENS = 16, 4, 512, 256, 2048, 192
TEMPERATURE, ENTROPY_BONUS = 0.8, 0.01
SCALE = 0.05 * 6 / 2688      # of every NVFP4 matrix, set once, so that the bytes change sparsely


class Gather(torch.autograd.Function):
    """Tokens' rows in the experts' order."""

    @staticmethod
    def forward(ctx, x, route):
        ctx.route = route
        return dcr.experts_gather(x, route)

    @staticmethod
    def backward(ctx, grad):
        return dcr.experts_combine(grad.contiguous(), ctx.route, weighted=False), None


class Combine(torch.autograd.Function):
    """The experts' rows weighted and summed; the router's logits get their gradient through the weights."""

    @staticmethod
    def forward(ctx, y, logits, route):
        ctx.save_for_backward(y, logits)
        ctx.route = route
        return dcr.experts_combine(y, route)

    @staticmethod
    def backward(ctx, grad):
        y, logits = ctx.saved_tensors
        by_y, by_weights = dcr.experts_combine_grad(y, ctx.route, grad.contiguous())
        return by_y, dcr.route_experts_grad(logits, ctx.route, by_weights, scoring="sigmoid"), None


def trainer_logits(x, router, up, down, head, bias, keep):
    """The model in the trainer's precision: x [tokens, HIDDEN], router [EXPERTS, HIDDEN], up [EXPERTS, FFN, HIDDEN], down [EXPERTS,
    HIDDEN, FFN], head [VOCAB, HIDDEN].  Padding (keep is False) goes to no expert."""
    logits = x @ router.T
    route = dcr.route_experts(logits.detach(), CHOSEN, scoring="sigmoid", bias=bias, groups=4, group_top=2, mask=keep)
    rows, at = Gather.apply(x, route), route.offsets.tolist()
    out = [torch.nn.functional.silu(rows[a:b] @ up[e].T) @ down[e].T for e, (a, b) in enumerate(zip(at, at[1:]))]
    out.append(rows.new_zeros(len(rows) - at[-1], HIDDEN))      # rows that no expert has
    return (x + Combine.apply(torch.cat(out), logits, route)) @ head.T


def engine_logits(x, router, up, down, head, bias, keep):
    """The same from NVFP4 weights where the refit leaves them."""
    route = dcr.route_experts(x @ router.T, CHOSEN, scoring="sigmoid", bias=bias, groups=4, group_top=2, mask=keep)
    # rows that no expert has hold anything, and go nowhere
    rows = dcr.nvfp4_linear(dcr.experts_gather(x, route), up, offsets=route.offsets)
    rows = dcr.nvfp4_linear(torch.nn.functional.silu(rows), down, offsets=route.offsets)
    return dcr.nvfp4_linear(x + dcr.experts_combine(rows, route), head)


SHAPES = dict(up=(EXPERTS * FFN, HIDDEN), down=(EXPERTS * HIDDEN, FFN), head=(VOCAB, HIDDEN))


def make_plan():
    """The model's tensors one after another: a 16-bit router, then codes and scales of the NVFP4 matrices."""
    descs, at, where = [dcr.make_desc("router", 16, EXPERTS, HIDDEN, dcr.REPLICATED, 1, [0], 0)], EXPERTS * HIDDEN * 2, {}
    for name, (rows, cols) in SHAPES.items():
        for part, bits, n in (("codes", 4, rows * cols // 2), ("scales", 8, rows * cols // 16)):
            descs.append(dcr.make_desc("%s.%s" % (name, part), bits, rows, cols if bits == 4 else cols // 16, dcr.REPLICATED, 1, [at], at))
            where[name, part] = slice(at, at + n)
            at += n
    return dcr.Plan(descs), where


def views(arena, where, scale):
    """The model as it lies in an arena."""
    nvfp4 = {n: dcr.Nvfp4(arena[where[n, "codes"]].view(r, c // 2), arena[where[n, "scales"]].view(r, c // 16), scale)
             for n, (r, c) in SHAPES.items()}
    return arena[:EXPERTS * HIDDEN * 2].view(torch.bfloat16).view(EXPERTS, HIDDEN), nvfp4


def main():
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, device="cuda", generator=g) * std

    plan, where = make_plan()
    old, new = (torch.zeros(plan.info.shard_bytes[0], dtype=torch.uint8, device="cuda") for _ in range(2))
    scale = torch.tensor([SCALE], device="cuda")

    # masters in 32 bits, and version 0 of the arena
    masters = {"router": normal(EXPERTS, HIDDEN, std=0.05), **{n: normal(*s, std=0.02) for n, s in SHAPES.items()}}
    states = dict(zip(masters, dcr.adamw_states(masters.values(), bits=8)))
    for arena in (old, new):
        router, weights = views(arena, where, scale)
        router.copy_(masters["router"])
        for n in SHAPES:
            dcr.nvfp4_quantize(masters[n], scale=scale, out=weights[n])

    # the rollout engine at version 0
    target = torch.empty(plan.info.recv_bytes, dtype=torch.uint8, device="cuda")
    dcr.check(dcr.dense_refit(plan, [old], target))
    state = dcr.RecvState(plan, version=0)
    router, served = views(target, where, scale)
    bias = normal(EXPERTS, std=0.01)
    x, keep = normal(TOKENS, HIDDEN).bfloat16(), torch.arange(TOKENS, device="cuda") < TOKENS - 20

    # rollout: a token for each position, its log-probability, the row's entropy and the likeliest alternatives
    logits = engine_logits(x, router, bias=bias, keep=keep, **served)
    tokens = torch.multinomial(torch.softmax(logits.float() / TEMPERATURE, 1), 1, generator=g)[:, 0]
    tokens[~keep] = -1
    rollout = dcr.token_scores(logits, tokens, top=5, temperature=TEMPERATURE)

    # trainer: quantisation-aware, with the loss's gradient and the entropy's
    leaves = {}
    for n, m in masters.items():
        values = m.bfloat16() if n == "router" else dcr.nvfp4_quantize(m, scale=scale, values=torch.bfloat16)[1]
        leaves[n] = values.requires_grad_()
    z = trainer_logits(x, leaves["router"], leaves["up"].view(EXPERTS, FFN, HIDDEN), leaves["down"].view(EXPERTS, HIDDEN, FFN), leaves["head"],
                       bias, keep)
    weight = keep.float() / keep.sum()
    loss, logp, grad = dcr.policy_loss(z.detach(), tokens, rollout.logp, normal(TOKENS), weight, ref_logp=rollout.logp, kl_coef=0.02,
                                       temperature=TEMPERATURE)
    scores = dcr.token_scores(z.detach(), tokens, temperature=TEMPERATURE)
    grad += dcr.token_scores_grad(z.detach(), tokens, scores.stats, grad_entropy=-ENTROPY_BONUS * weight, temperature=TEMPERATURE)
    z.backward(grad)

    # the step: matrices, then the router, whose 16-bit weights go into the arena
    router, weights = views(new, where, scale)
    norm = dcr.grad_norm([v.grad for v in leaves.values()])
    step = dict(step=1, lr=2e-5, weight_decay=0.01, norm=norm, max_norm=1.0)
    dcr.adamw_step([masters[n] for n in SHAPES], [leaves[n].grad for n in SHAPES], [states[n] for n in SHAPES], **step)
    dcr.adamw_step([masters["router"]], [leaves["router"].grad], [states["router"]], copies=[router], **step)
    for n in SHAPES:
        dcr.nvfp4_quantize(masters[n], scale=scale, out=weights[n])

    # the refit
    payload = torch.empty(plan.window(0).payload_bound, dtype=torch.uint8, device="cuda")
    rc, size, changed = dcr.encode(plan, [old], [new], payload, base_version=0, target_version=1)
    dcr.check(rc)
    rc, result = dcr.apply(plan, state, payload, size, target)
    dcr.check(rc)
    assert state.version == 1
    router, served = views(target, where, scale)
    after = engine_logits(x, router, bias=bias, keep=keep, **served)
    router, weights = views(new, where, scale)
    assert torch.equal(after, engine_logits(x, router, bias=bias, keep=keep, **weights))
    dcr.ops_status()
    print("loss %.6f; entropy %.4f; gradient's norm %.6f; %d values changed; payload %d bytes; logits moved by at most %.4f" % (
        float(loss), float((scores.entropy * weight).sum()), float(norm), sum(changed), size, float((after.float() - logits.float()).abs().max())))


if __name__ == "__main__":
    main()
