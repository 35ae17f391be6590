"""One step of reinforcement learning around a refit, on the GPU: the rollout
engine's logits come from NVFP4 weights, the trainer takes the policy loss and
its gradient from logits, updates its bf16 weights, quantises them straight
into the arena that dcr_encode reads, and the refit brings the engine the same
bytes, so that both sides compute the same logits again, bit for bit (build
first: python -c "import __graft_entry__ as g; g.build()").
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch
import bit_exact_xor_gb300 as dcr

HIDDEN, VOCAB, TOKENS = 1024, 4096, 256
TEMPERATURE = 0.8

# one output projection, held as NVFP4: codes and scales are two tensors of the plan
n_codes, n_scales = VOCAB * HIDDEN // 2, VOCAB * HIDDEN // 16
plan = dcr.Plan([
    dcr.make_desc("head.codes", 4, VOCAB, HIDDEN, dcr.REPLICATED, 1, [0], 0),
    dcr.make_desc("head.scales", 8, VOCAB, HIDDEN // 16, dcr.REPLICATED, 1, [n_codes], n_codes),
])


def views(arena, scale):
    """The projection as it lies in an arena."""
    return dcr.Nvfp4(arena[:n_codes].view(VOCAB, HIDDEN // 2), arena[n_codes:n_codes + n_scales].view(VOCAB, HIDDEN // 16), scale)


g = torch.Generator(device="cuda").manual_seed(0)
weight = (torch.randn(VOCAB, HIDDEN, device="cuda", generator=g) * 0.02).bfloat16()
hidden = torch.randn(TOKENS, HIDDEN, device="cuda", generator=g).bfloat16()

# the trainer's arenas, version 0 and the one to come; the outer scale is set once, so that the bytes change sparsely
old, new = (torch.zeros(max(plan.info.shard_bytes[0], 16), dtype=torch.uint8, device="cuda") for _ in range(2))
scale = weight.float().abs().amax().reshape(1) * 1.25 / 2688
dcr.nvfp4_quantize(weight, scale=scale, out=views(old, scale))

# the rollout engine at version 0
target = torch.empty(plan.info.recv_bytes, dtype=torch.uint8, device="cuda")
dcr.check(dcr.dense_refit(plan, [old], target))
state = dcr.RecvState(plan, version=0)
served = views(target, scale)

# rollout: sample a token for each position, keep its log-probability
logits = dcr.nvfp4_linear(hidden, served)
tokens = torch.multinomial(torch.softmax(logits.float() / TEMPERATURE, 1), 1, generator=g)[:, 0]
old_logp = dcr.token_logprobs(logits, tokens, temperature=TEMPERATURE)

# trainer: loss and gradient by its own logits (quantisation-aware: computed from the values that the codes stand for)
_, values = dcr.nvfp4_quantize(weight, scale=scale, values=torch.bfloat16)
x = hidden.clone().requires_grad_()
w = values.clone().requires_grad_()
z = x @ w.T
advantages = torch.randn(TOKENS, device="cuda", generator=g)
weights = torch.full((TOKENS,), 1.0 / TOKENS, device="cuda")
weights[:32] = 0.0                                # the prompt
loss, logp, grad = dcr.policy_loss(z.detach(), tokens, old_logp, advantages, weights, ref_logp=old_logp, clip_low=0.2, clip_high=0.28,
                                   kl_coef=0.02, temperature=TEMPERATURE)
z.backward(grad)
weight = (weight.float() - 0.1 * w.grad.float()).bfloat16()

# sender: the new weights' bytes, then what changed of them
dcr.nvfp4_quantize(weight, scale=scale, out=views(new, scale))
payload = torch.empty(plan.window(0).payload_bound, dtype=torch.uint8, device="cuda")
rc, size, changed = dcr.encode(plan, [old], [new], payload, base_version=0, target_version=1)
dcr.check(rc)

# ... payload[:size] travels to the rollout engine ...
rc, result = dcr.apply(plan, state, payload, size, target)
dcr.check(rc)
assert state.version == 1
after, sender = dcr.nvfp4_linear(hidden, served), dcr.nvfp4_linear(hidden, views(new, scale))
assert torch.equal(after, sender)
dcr.ops_status()
print("loss %.6f; %d of %d values changed; payload %d bytes; logits moved by at most %.4f" % (
    float(loss), sum(changed), VOCAB * HIDDEN, size, float((after.float() - logits.float()).abs().max())))
