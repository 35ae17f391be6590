"""Cases, plain forms and 64-bit values of the operators that a step of reinforcement learning on a mixture of experts takes
next to the refit, the NVFP4 product and the policy loss:

scores    from logits, the log-probabilities of given tokens, the entropy of every row and its likeliest alternatives;
          with `train`, the gradient by the logits, too;
route     which experts a token goes to and with what weights, and the order of the rows by expert; with `train`, the
          gradient by the router's logits;
exchange  tokens' rows into the experts' order, and the weighted sum of the experts' rows back to the tokens; with
          `train`, the gradients of both;
update    an AdamW step over many tensors, moments in 32 or 8 bits; with `clip`, by the norm of all gradients.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
TEMPERATURE = 0.8
LR, BETA1, BETA2, EPS, DECAY, STEP, SEED = 1e-4, 0.9, 0.999, 1e-8, 0.1, 100, 20
BLOCK = 256                     # values that share a scale of an 8-bit moment
FLT_MAX = 3.4028234663852886e38


def listed():
    return [
        # One decode step of 8 sequences: what was sampled, and twenty alternatives for the user.
        dict(name="scores 8x128256", op="scores", t=8, v=128256, dtype="bf16", top=20, train=False),
        # An odd number of tokens over a vocabulary with a few tokens added: no row but the first is aligned.
        dict(name="scores 1021x32771", op="scores", t=1021, v=32771, dtype="f32", top=5, train=False),
        # A packed batch of a large vocabulary, alternatives kept for distillation.
        dict(name="scores 4096x128256", op="scores", t=4096, v=128256, dtype="bf16", top=20, train=False),
        # The trainer's pass over a batch with an entropy bonus: log-probabilities, entropies and the gradient.
        dict(name="scores train 4096x32768", op="scores", t=4096, v=32768, dtype="f32", top=0, train=True),
        # One decode step's routing over 64 experts.
        dict(name="route 64x64", op="route", t=64, e=64, k=8, dtype="f32", scoring="softmax", bias=False, groups=1, group_top=1,
             group_by=1, renormalise=True, masked=False, train=False),
        # A trainer's packed batch over 256 experts in 8 groups, a bias for balance, some of it padding.
        dict(name="route train 16381x256", op="route", t=16381, e=256, k=8, dtype="f32", scoring="sigmoid", bias=True, groups=8,
             group_top=4, group_by=2, renormalise=True, masked=True, train=True),
        # One decode step's rows to 8 of 64 experts and back.
        dict(name="exchange 64x6144", op="exchange", t=64, e=64, k=8, h=6144, dtype="bf16", out="bf16", masked=False, train=False),
        # A trainer's batch, the experts' outputs kept in 32 bits for the sum; padding at its end.
        dict(name="exchange train 8190x6144", op="exchange", t=8190, e=64, k=8, h=6144, dtype="bf16", out="f32", masked=True, train=True),
        # A small dense layer's matrix and norm.
        dict(name="update 1024x1024", op="update", model="layer", hidden=1024, ffn=0, layers=1, vocab=0, bits=32, weight="f32",
             grad="bf16", copy="bf16", clip=False, gap=0),
        # Half of a 24-layer dense transformer, clipped by the norm, the arena of the refit written along with the weights.
        dict(name="update 24 layers", op="update", model="dense", hidden=1024, ffn=2048, layers=24, vocab=16384, bits=32, weight="f32",
             grad="bf16", copy="bf16", clip=True, gap=0),
        # A wide layer's matrices with moments in 8 bits.
        dict(name="update 8 bits 4096", op="update", model="dense", hidden=4096, ffn=14336, layers=1, vocab=0, bits=8, weight="f32",
             grad="bf16", copy="bf16", clip=False, gap=0),
        # Many small odd tensors one behind another in a buffer, none of them aligned, without a copy in 32 bits.
        dict(name="update 8 bits odd", op="update", model="odd", hidden=301, ffn=117, layers=40, vocab=1001, bits=8, weight="bf16",
             grad="f32", copy="", clip=False, gap=3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scores", "scores", "route", "exchange", "update", "update"])
    if op == "scores":
        v = _log(rng, 2, 128256)
        t = _log(rng, 1, min(4096, max(1, 128 * 1048576 // v)))
        return dict(op=op, t=t, v=v, dtype=rng.choice(["f32", "bf16", "bf16", "f16"]), top=min(v, rng.choice([0, 1, 5, 20, 64])),
                    train=rng.random() < 0.4)
    if op == "route":
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        e = groups * _log(rng, 2, 512 // groups)
        group_top = rng.randint(1, groups)
        return dict(op=op, t=_log(rng, 1, 16384), e=e, k=min(e // groups * group_top, rng.choice([1, 2, 4, 6, 8])),
                    dtype=rng.choice(["f32", "f32", "bf16", "f16"]), scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    groups=groups, group_top=group_top, group_by=rng.choice([1, 2]), renormalise=rng.random() < 0.7,
                    masked=rng.random() < 0.3, train=rng.random() < 0.5)
    if op == "exchange":
        e = _log(rng, 2, 256)
        return dict(op=op, t=_log(rng, 1, 8192), e=e, k=min(e, rng.choice([1, 2, 4, 8])), h=_log(rng, 8, 6144),
                    dtype=rng.choice(["bf16", "f16", "f32"]), out=rng.choice(["bf16", "f16", "f32"]), masked=rng.random() < 0.3,
                    train=rng.random() < 0.5)
    model = rng.choice(["layer", "dense", "odd"])
    bits = rng.choice([32, 8])
    return dict(op=op, model=model, hidden=_log(rng, 16, 2048), ffn=_log(rng, 16, 4096), layers=_log(rng, 1, 16),
                vocab=_log(rng, 16, 16384), bits=bits, weight=rng.choice(["f32", "f32", "bf16", "f16"]),
                grad=rng.choice(["bf16", "f32", "f16"]), copy=rng.choice(["bf16", "f16", "f32", ""]),
                clip=bits == 32 and rng.random() < 0.4, gap=rng.choice([0, 0, 1, 8]))


def _shapes(case):
    """The sizes of a model's tensors, in the order of its buffer."""
    h, f, layers, v = case["hidden"], case["ffn"], case["layers"], case["vocab"]
    if case["model"] == "layer":
        return [h * h, h]
    if case["model"] == "dense":
        return ([v * h] if v else []) + layers * [h * h, h * h, h * h, h * h, f * h, h * f, h, h] + ([h, v * h] if v else [])
    return layers * [h * f, h, f * 3 + 1, 1] + [v, h * 5 + 2]


# ---- inputs -------------------------------------------------------------------------------------------------------


def _normal(g, shape, std):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g)


def _mask(g, case):
    """Padding: the last eighth of the batch, and a few tokens before it."""
    if not case["masked"]:
        return None
    t = case["t"]
    keep = torch.rand(t, device="cuda", generator=g) >= 0.02
    keep[t - t // 8:] = False
    return keep


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "scores":
        t, v = case["t"], case["v"]
        z = _normal(g, (t, v), 2.0)
        y = torch.randint(0, v, (t,), device="cuda", generator=g)
        z[torch.arange(t, device="cuda"), y] += 8.0
        s["logits"], s["tokens"] = z.to(DTYPES[case["dtype"]]), y
        # what the loss hands back: advantages over the tokens' number, and an entropy bonus
        s["grad_logp"] = _normal(g, (t,), 1.0) / t
        s["grad_entropy"] = torch.full((t,), -0.01 / t, device="cuda")
    elif case["op"] == "route":
        s["logits"] = _normal(g, (case["t"], case["e"]), 1.5).to(DTYPES[case["dtype"]])
        s["bias_values"] = _normal(g, (case["e"],), 0.05) if case["bias"] else None
        s["mask"] = _mask(g, case)
        s["grad_weights"] = _normal(g, (case["t"], case["k"]), 1.0)
    elif case["op"] == "exchange":
        t, e, k, h = case["t"], case["e"], case["k"], case["h"]
        s["x"] = _normal(g, (t, h), 1.0).to(DTYPES[case["dtype"]])
        # a router that prefers some experts
        logits = _normal(g, (t, e), 1.0) + _normal(g, (e,), 0.7)
        mask = _mask(g, case)
        experts = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]
        weights = torch.softmax(logits.gather(1, experts), 1)
        if mask is not None:
            experts, weights = torch.where(mask[:, None], experts, -1), torch.where(mask[:, None], weights, 0.0)
        s["route"] = (experts.to(torch.int32), weights) + _expert_order(experts, e)
        s["y"] = _normal(g, (t * k, h), 1.0).to(DTYPES[case["out"]])
        s["grad"] = _normal(g, (t, h), 1.0).to(DTYPES[case["dtype"]])
        s["grad_rows"] = _normal(g, (t * k, h), 1.0).to(DTYPES[case["dtype"]])
        # rows that no token goes to are left as they are
        s["rows"], s["grad_y"] = torch.zeros_like(s["grad_rows"]), torch.zeros_like(s["y"])
    else:
        sizes, gap, bits = _shapes(case), case["gap"], case["bits"]
        total = sum(sizes) + gap * len(sizes)
        at = [sum(sizes[:i]) + gap * (i + 1) for i in range(len(sizes))]
        blocks = [-(-n // BLOCK) for n in sizes]
        first = [sum(blocks[:i]) for i in range(len(blocks))]

        def views(flat):
            return [flat[a:a + n] for a, n in zip(at, sizes)]

        s["weights"] = _normal(g, (total,), 0.02).to(DTYPES[case["weight"]])
        # some parts of a model learn faster than others
        s["grads"] = _normal(g, (total,), 1e-3)
        for i, x in enumerate(views(s["grads"])):
            x.mul_(4.0 ** (i % 5 - 2))
        m, v = s["grads"] * 0.1, s["grads"].square()
        m += _normal(g, (total,), 1e-4)
        v.mul_(_normal(g, (total,), 1.0).exp_()).add_(1e-9)
        s["grads"] = s["grads"].to(DTYPES[case["grad"]])
        s["copies"] = torch.zeros(total, dtype=DTYPES[case["copy"]], device="cuda") if case["copy"] else None
        s["w"], s["g"] = views(s["weights"]), views(s["grads"])
        s["c"] = views(s["copies"]) if case["copy"] else None
        if bits == 32:
            s["m"], s["v"] = m, v
            s["state"] = list(zip(views(m), views(v)))
        else:
            s["m"], s["v"] = (torch.zeros(total, dtype=torch.uint8, device="cuda") for _ in range(2))
            s["m_scale"], s["v_scale"] = (torch.zeros(sum(blocks), device="cuda") for _ in range(2))
            s["state"] = [(a, x[f:f + b], c, y[f:f + b]) for a, c, f, b, x, y in
                          zip(views(s["m"]), views(s["v"]), first, blocks, [s["m_scale"]] * len(sizes), [s["v_scale"]] * len(sizes))]
            for (a, ms, c, vs), x, y in zip(s["state"], views(m), views(v)):
                half = torch.full_like(x, 0x8000, dtype=torch.int64)
                _to8(x, half, a, ms)
                _to8(y.sqrt(), half, c, vs)
    return s


# ---- plain forms --------------------------------------------------------------------------------------------------


def _top(z, n):
    """The n largest of each row, the lowest index first among equal ones: a key that holds both."""
    b = (z + 0.0).contiguous().view(torch.int32)
    key = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long() * 4294967296 - torch.arange(z.shape[1], device=z.device)
    at = torch.topk(key, n, 1)[1]
    return z.gather(1, at), at


def _scores(s):
    y, inv = s["tokens"], 1.0 / TEMPERATURE
    x = s["logits"].float()
    z = x * inv
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    entropy = log_total[:, 0] - (e * z).sum(1) / total[:, 0]
    out = dict(logp=z.gather(1, y[:, None])[:, 0] - log_total[:, 0], entropy=entropy)
    if s["top"]:
        out["tokens"] = _top(x, s["top"])[1]
        out["top"] = z.gather(1, out["tokens"]) - log_total
    if s["train"]:
        p = e / total
        a, b = s["grad_logp"][:, None], s["grad_entropy"][:, None]
        grad = -p * (a + b * (z - log_total + entropy[:, None]))
        grad.scatter_add_(1, y[:, None], a)
        out["grad"] = (grad * inv).to(s["logits"].dtype)
    return out


def _expert_order(experts, e):
    """Offsets of the experts' rows, the token's slot of each row, and the row of each slot."""
    t, k = experts.shape
    flat = torch.where(experts < 0, e, experts).reshape(-1).long()
    order = torch.sort(flat, stable=True)[1]
    counts = torch.bincount(flat, minlength=e + 1)[:e]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    row = torch.empty_like(order).scatter_(0, order, torch.arange(t * k, device=flat.device))
    there = torch.arange(t * k, device=flat.device) < offsets[-1]
    return (offsets.to(torch.int32), torch.where(there, order, -1).to(torch.int32),
            torch.where(flat < e, row, -1).reshape(t, k).to(torch.int32))


def _scored(x, scoring):
    return torch.sigmoid(x) if scoring == "sigmoid" else torch.softmax(x, 1)


def _route(s):
    t, e, k, groups = s["t"], s["e"], s["k"], s["groups"]
    x = s["logits"]
    # which experts are chosen is decided in 64 bits: two keys may be nearer to each other than 32 bits tell
    key = _scored(x.double(), s["scoring"])
    if s["bias"]:
        key = key + s["bias_values"].double()
    elif s["group_by"] == 1:
        key = x.double()        # the same order, without the rounding of scores near 1
    if groups > 1:
        each = key.reshape(t, groups, e // groups)
        best = torch.sort(each, dim=2, descending=True)[0][:, :, :s["group_by"]].sum(2)
        rank = torch.sort(torch.sort(best, dim=1, descending=True, stable=True)[1], dim=1)[1]
        key = torch.where((rank < s["group_top"])[:, :, None], each, -math.inf).reshape(t, e)
    experts = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
    score = _scored(x.float(), s["scoring"])
    w = score.gather(1, experts)
    total = w.sum(1, keepdim=True) if s["renormalise"] else torch.ones_like(w[:, :1])
    w = w / total * 2.5
    if s["mask"] is not None:
        experts, w = torch.where(s["mask"][:, None], experts, -1), torch.where(s["mask"][:, None], w, 0.0)
    offsets, order, positions = _expert_order(experts, e)
    out = dict(experts=experts.to(torch.int32), weights=w, offsets=offsets, order=order, positions=positions)
    if s["train"]:
        d = s["grad_weights"] * 2.5 / total
        chosen = experts.clamp(min=0)
        if s["renormalise"]:
            d = d - (d * w).sum(1, keepdim=True) / 2.5
        if s["mask"] is not None:
            d = torch.where(s["mask"][:, None], d, 0.0)
        by_score = torch.zeros_like(score).scatter_add_(1, chosen, d)
        if s["scoring"] == "sigmoid":
            grad = by_score * score * (1.0 - score)
        else:
            grad = score * (by_score - (by_score * score).sum(1, keepdim=True))
        out["grad"] = grad.to(x.dtype)
    return out


def _combined(y, positions, weights):
    """Each token's rows, weighted and summed in the order of its slots."""
    there = positions >= 0
    rows = y[positions.clamp(min=0).long()].float()
    rows = torch.where(there[:, :, None], rows, 0.0)
    return (rows if weights is None else rows * weights[:, :, None]).sum(1)


def _exchange(s):
    k = s["k"]
    experts, weights, offsets, order, positions = s["route"]
    there = order >= 0
    slot = order.clamp(min=0).long()
    token = slot // k
    s["rows"].copy_(torch.where(there[:, None], s["x"][token], s["rows"]))
    out = dict(rows=s["rows"], sum=_combined(s["y"], positions, weights).to(s["x"].dtype))
    if s["train"]:
        grad = s["grad"].float()[token]
        rows = torch.where(there, weights.reshape(-1)[slot], 0.0)
        s["grad_y"].copy_(torch.where(there[:, None], grad * rows[:, None], s["grad_y"].float()))
        dot = torch.where(there, (grad * s["y"].float()).sum(1), 0.0)
        out["grad_y"] = s["grad_y"]
        out["grad_weights"] = torch.where(positions >= 0, dot[positions.clamp(min=0).long()], 0.0)
        out["grad_x"] = _combined(s["grad_rows"], positions, None).to(s["x"].dtype)
    return out


def _pcg(x):
    """A permuted congruential generator's output for a state of 32 bits (O'Neill 2014), as 64-bit integers."""
    x = (x * 747796405 + 2891336453) & 0xFFFFFFFF
    x = (((x >> ((x >> 28) + 4)) ^ x) * 277803737) & 0xFFFFFFFF
    return (x >> 22) ^ x


def _random(first, n):
    """32 random bits for each of the elements `first` to `first + n` of a step's tensors."""
    key = _pcg((_pcg(SEED) + STEP) & 0xFFFFFFFF)
    i = torch.arange(first, first + n, device="cuda")
    return _pcg((i & 0xFFFFFFFF) ^ _pcg((key + (i >> 32)) & 0xFFFFFFFF))


def _from8(codes, scale):
    n = codes.numel()
    v = torch.nn.functional.pad(codes, (0, -n % BLOCK)).view(torch.float8_e4m3fn).float()
    return (v.reshape(-1, BLOCK) * scale[:, None]).reshape(-1)[:n]


def _to8(x, bits, codes, scale, keep=False):
    """x in e4m3 with a scale for every 256 values, rounded up with the probability of what is cut off, which 16 random
    bits decide; with `keep` nothing but 0 becomes 0."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % BLOCK)).reshape(-1, BLOCK)
    sc = b.abs().amax(1) * (1.0 / 448.0)
    r = torch.where(sc > 0, (1.0 / sc).clamp(max=FLT_MAX), torch.zeros_like(sc))
    y = (b.abs() * r[:, None]).clamp(max=448.0).reshape(-1)[:n]
    # a value of e4m3 is one of 32 bits whose exponent is 120 larger, with 3 bits of mantissa
    c = ((y * 2.0 ** -120).view(torch.int32).long() + bits * 16 + 8) >> 20
    if keep:
        c = torch.where((x != 0) & (c == 0), 1, c)
    codes.copy_(c + 128 * torch.signbit(x).long())
    scale.copy_(sc)


def _update_one(s, w, g, state, copy, coef, first):
    c1, c2 = 1.0 - BETA1 ** STEP, 1.0 - BETA2 ** STEP
    g = g.float() * coef
    if s["bits"] == 32:
        m, v = state
    else:
        m, v = _from8(state[0], state[1]), _from8(state[2], state[3]).square()
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g * g * (1.0 - BETA2)
    root = v.sqrt()
    new = w.float() * (1.0 - LR * DECAY) - m / (root * (1.0 / math.sqrt(c2)) + EPS) * (LR / c1)
    w.copy_(new)
    if copy is not None:
        copy.copy_(new)
    if s["bits"] == 32:
        state[0].copy_(m)
        state[1].copy_(v)
    else:
        bits = _random(first, w.numel())
        _to8(m, bits & 0xFFFF, state[0], state[1])
        _to8(root, bits >> 16, state[2], state[3], keep=True)


def _update(s):
    coef = 1.0
    if s["clip"]:
        norm = torch.stack([x.float().square().sum() for x in s["g"]]).sum().sqrt()
        coef = torch.where(norm > 1.0, 1.0 / norm, torch.ones_like(norm))
    n = [x.numel() for x in s["w"]]
    copies = s["c"] or [None] * len(n)
    for i, w in enumerate(s["w"]):
        _update_one(s, w, s["g"][i], s["state"][i], copies[i], coef, sum(n[:i]))
    return _updated(s, norm if s["clip"] else None)


def _updated(s, norm):
    """What a step has changed."""
    out = dict(weights=s["weights"], copies=s["copies"], norm=norm)
    if s["bits"] == 32:
        return dict(out, m=s["m"], v=s["v"])
    return dict(out, m=s["m"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn), m_scale=s["m_scale"], v_scale=s["v_scale"])


def run(s):
    if not own:
        return dict(scores=_scores, route=_route, exchange=_exchange, update=_update)[s["op"]](s)
    import bit_exact_xor_gb300 as dcr
    if s["op"] == "scores":
        r = dcr.token_scores(s["logits"], s["tokens"], top=s["top"], temperature=TEMPERATURE)
        out = dict(logp=r.logp, entropy=r.entropy)
        if s["top"]:
            out.update(top=r.top_logp, tokens=r.top_tokens)
        if s["train"]:
            out["grad"] = dcr.token_scores_grad(s["logits"], s["tokens"], r.stats, s["grad_logp"], s["grad_entropy"], temperature=TEMPERATURE)
        return out
    if s["op"] == "route":
        r = dcr.route_experts(s["logits"], s["k"], scoring=s["scoring"], bias=s["bias_values"], groups=s["groups"], group_top=s["group_top"],
                              group_by=s["group_by"], renormalise=s["renormalise"], scale=2.5, mask=s["mask"])
        out = r._asdict()
        if s["train"]:
            out["grad"] = dcr.route_experts_grad(s["logits"], r, s["grad_weights"], scoring=s["scoring"], renormalise=s["renormalise"], scale=2.5)
        return out
    if s["op"] == "exchange":
        r = dcr.Route(*s["route"])
        out = dict(rows=dcr.experts_gather(s["x"], r, out=s["rows"]), sum=dcr.experts_combine(s["y"], r, dtype=s["x"].dtype))
        if s["train"]:
            out["grad_y"], out["grad_weights"] = dcr.experts_combine_grad(s["y"], r, s["grad"], out=s["grad_y"])
            out["grad_x"] = dcr.experts_combine(s["grad_rows"], r, weighted=False)
        return out
    norm = dcr.grad_norm(s["g"]) if s["clip"] else None
    states = [dcr.AdamState32(*x) if s["bits"] == 32 else dcr.AdamState8(*x) for x in s["state"]]
    dcr.adamw_step(s["w"], s["g"], states, STEP, LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, copies=s["c"], norm=norm,
                   max_norm=1.0 if s["clip"] else None, seed=SEED)
    return _updated(s, norm)


def work(case):
    if case["op"] == "scores":
        n = case["t"] * case["v"]
        b = SIZE[case["dtype"]]
        return dict(bytes=n * b * (3 if case["train"] else 1) + case["t"] * (16 + 12 * case["top"]), flops=n * (14 if case["train"] else 6))
    if case["op"] == "route":
        t, e, k, b = case["t"], case["e"], case["k"], SIZE[case["dtype"]]
        return dict(bytes=t * e * b * (2 if case["train"] else 1) + t * k * (20 if case["train"] else 16) + 4 * e,
                    flops=t * e * (12 if case["train"] else 6))
    if case["op"] == "exchange":
        t, k, h, b, o = case["t"], case["k"], case["h"], SIZE[case["dtype"]], SIZE[case["out"]]
        n = t * h
        if not case["train"]:
            return dict(bytes=n * (b + k * b) + n * (k * o + b), flops=2 * n * k)
        return dict(bytes=n * (b + k * b) + n * (k * o + b) + n * (b + 2 * k * o) + n * (k * b + b), flops=6 * n * k)
    n = sum(_shapes(case))
    w, g, c = SIZE[case["weight"]], SIZE[case["grad"]], SIZE.get(case["copy"], 0)
    return dict(bytes=n * (2 * w + g * (2 if case["clip"] else 1) + c + case["bits"] // 2), flops=n * 16)


# ---- the same in 64 bits, from the definitions ---------------------------------------------------------------------


def _round8(x, u):
    """The e4m3 value below or above |x|, the upper one where what is cut off and the number u in (0, 1) pass 1."""
    a = x.abs()
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 1).clamp(min=-6) - 3)
    return torch.copysign((torch.floor(a / step + u) * step).clamp(max=448.0), x)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "scores":
        y, out = s["tokens"], {}
        parts = []
        for at in range(0, case["t"], 512):
            z = s["logits"][at:at + 512].double() / TEMPERATURE
            lse = torch.logsumexp(z, 1, keepdim=True)
            lp = z - lse
            p = torch.exp(lp)
            h = -(p * lp).sum(1)
            part = dict(logp=lp.gather(1, y[at:at + 512, None])[:, 0], entropy=h)
            if case["top"]:
                part["top"] = torch.topk(lp, case["top"], 1)[0]
            if case["train"]:
                d = torch.zeros_like(p).scatter_(1, y[at:at + 512, None], 1.0)
                part["grad"] = (s["grad_logp"][at:at + 512, None].double() * (d - p)
                                - s["grad_entropy"][at:at + 512, None].double() * p * (lp + h[:, None])) / TEMPERATURE
            parts.append(part)
        out = {n: torch.cat([p[n] for p in parts]) for n in parts[0]}
        if case["top"]:
            out["tokens"] = None
        return out
    if case["op"] == "route":
        r = _route(dict(s, train=False))        # which experts: whole numbers
        at = r["experts"].long().clamp(min=0)
        there = r["experts"] >= 0
        x = s["logits"].double()
        if case["scoring"] == "sigmoid":
            score, slope = 1 / (1 + torch.exp(-x)), 1 / ((1 + torch.exp(-x)) * (1 + torch.exp(x)))
        else:
            score = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
        w = score.gather(1, at)
        total = w.sum(1, keepdim=True) if case["renormalise"] else torch.ones_like(w)
        w = w / total
        out = dict(experts=None, weights=torch.where(there, 2.5 * w, 0.0), offsets=None, order=None, positions=None)
        if case["train"]:
            d = torch.where(there, s["grad_weights"].double() * 2.5, 0.0)
            if case["renormalise"]:
                d = (d - (d * w).sum(1, keepdim=True)) / total
            by = torch.zeros_like(score).scatter_add_(1, at, d)
            out["grad"] = by * slope if case["scoring"] == "sigmoid" else score * (by - (by * score).sum(1, keepdim=True))
        return out
    if case["op"] == "exchange":
        experts, weights, offsets, order, positions = s["route"]
        t, k = positions.shape
        total = int(offsets[-1])
        slot = order[:total].long()
        token = slot // k
        out = dict(rows=torch.zeros_like(s["rows"], dtype=torch.float64))
        out["rows"][:total] = s["x"][token].double()
        w = weights.reshape(-1)[slot].double()
        out["sum"] = torch.zeros_like(s["x"], dtype=torch.float64).index_add_(0, token, s["y"][:total].double() * w[:, None])
        if case["train"]:
            out["grad_y"] = torch.zeros_like(s["grad_y"], dtype=torch.float64)
            out["grad_y"][:total] = s["grad"].double()[token] * w[:, None]
            dot = (s["grad"].double()[token] * s["y"][:total].double()).sum(1)
            out["grad_weights"] = torch.zeros(t * k, dtype=torch.float64, device="cuda").index_copy_(0, slot, dot).reshape(t, k)
            out["grad_x"] = torch.zeros_like(s["x"], dtype=torch.float64).index_add_(0, token, s["grad_rows"][:total].double())
        return out
    out = {n: None if s.get(n) is None else s[n].double() for n in ("weights", "copies")}
    out["norm"] = torch.sqrt(sum(x.double().square().sum() for x in s["g"])) if case["clip"] else None
    coef = min(1.0, 1.0 / float(out["norm"])) if case["clip"] else 1.0
    m8 = case["bits"] == 8
    for n in ("m", "v"):
        out[n] = s[n].view(torch.float8_e4m3fn).double() if m8 else s[n].double()
        if m8:
            out[n + "_scale"] = s[n + "_scale"].double()
    sizes = _shapes(case)
    at, block, first = 0, 0, 0
    for i, n in enumerate(sizes):
        at += case["gap"]
        here, blocks = slice(at, at + n), -(-n // BLOCK)
        there = slice(block, block + blocks)
        g = s["g"][i].double() * coef
        m, v = out["m"][here], out["v"][here]
        if m8:
            m = m * out["m_scale"][there].repeat_interleave(BLOCK)[:n]
            v = (v * out["v_scale"][there].repeat_interleave(BLOCK)[:n]) ** 2
        m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g * g
        step = m / (1 - BETA1 ** STEP) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS)
        out["weights"][here] = out["weights"][here] * (1 - LR * DECAY) - LR * step
        if out["copies"] is not None:
            out["copies"][here] = out["weights"][here]
        if m8:
            bits = _random(first, n)
            for name, x, r in (("m", m, bits & 0xFFFF), ("v", torch.sqrt(v), bits >> 16)):
                sc = torch.nn.functional.pad(x.abs(), (0, -n % BLOCK)).reshape(-1, BLOCK).amax(1) / 448
                out[name + "_scale"][there] = sc
                y = x / sc.repeat_interleave(BLOCK)[:n].clamp(min=1e-300)
                y = _round8(y, (r.double() + 0.5) / 65536)
                out[name][here] = torch.where((x != 0) & (y == 0), 2.0 ** -9, y) if name == "v" else y
        else:
            out["m"][here], out["v"][here] = m, v
        at, block, first = at + n, block + blocks, first + n
    return out
