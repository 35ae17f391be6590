"""Plain forms of the operators of a trainer's and a rollout engine's step
(include/dcr_ops.h: token scores, routing, rows by expert, AdamW), on the CPU
and written from the formulas there: in 64 bits, except where every rounding
to 32 bits is part of the definition (AdamW and its 8-bit moments)."""
import math

import torch

EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # half a step, relative
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}  # half a step of the smallest, and more
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def scores(x, tokens, temp):
    """logp, entropy, p and (x - M) / T without a subtraction of near values."""
    z = x.double() / temp
    rows = torch.arange(len(z))
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    others = e.clone()
    others[rows, z.argmax(1)] = 0.0
    r = others.sum(1)
    mean = torch.where(e > 0, -z * e, torch.zeros_like(e)).sum(1) / (1 + r)
    y = tokens.clamp(0, z.shape[1] - 1)
    return z[rows, y] - torch.log1p(r), torch.log1p(r) + mean, e / (1 + r)[:, None], z, mean, r


def sum_error(x, temp):
    """A bound on the relative error of a sum of exponentials of a row: two multiply-adds round an exponent (in units of
    log 2) of at most A by 2^-24 of it each, the rest of log2(e) / T is another such part; at most 192 additions one after
    another, and a few more roundings."""
    z = x.double() / temp * 1.4426950408889634
    a = min(float((z.amax(1) - torch.where(torch.isfinite(z), z, z.amax(1, keepdim=True)).amin(1)).max()), 200.0)   # 0 beyond that
    return 2.0 ** -21 + (3 * a + 192) * 2.0 ** -24


def top(x, n):
    """Indexes of the n largest of each row: numbers before NaN, the lowest index first among equal ones."""
    z = x.double()
    rows = []
    for row in z.tolist():
        order = sorted(range(len(row)), key=lambda i: (math.isnan(row[i]), 0.0 if math.isnan(row[i]) else -row[i], i))
        rows.append(order[:n])
    return torch.tensor(rows)


def choose(x, k, scoring, bias, groups, group_top, group_by, mask):
    """Chosen experts [tokens, k], -1 where there is none, token by token."""
    out = []
    for t, row in enumerate(x.double().tolist()):
        picked = []
        if mask is None or bool(mask[t]):
            alive = [i for i, v in enumerate(row) if v > -math.inf]
            if scoring == "sigmoid":
                score = {i: 1 / (1 + math.exp(-row[i])) if row[i] >= 0 else math.exp(row[i]) / (1 + math.exp(row[i])) for i in alive}
            else:
                m = max((row[i] for i in alive), default=0.0)
                e = {i: 1.0 if row[i] == m else math.exp(row[i] - m) for i in alive}
                s = math.fsum(e.values())
                score = {i: v / s for i, v in e.items()}
            if bias is not None:
                key = {i: v + float(bias[i]) for i, v in score.items()}
                key = {i: v for i, v in key.items() if v > -math.inf}
            elif groups == 1 or group_by == 1:
                key = {i: row[i] for i in alive}
            else:
                key = score
            if groups > 1:
                size = len(row) // groups
                best = []
                for g in range(groups):
                    v = sorted((key[i] for i in range(g * size, (g + 1) * size) if i in key), reverse=True)[:group_by]
                    if v:
                        best.append((-sum(v), g))
                kept = {g for _, g in sorted(best)[:group_top]}
                key = {i: v for i, v in key.items() if i // size in kept}
            picked = sorted(key, key=lambda i: (-key[i], i))[:k]
        out.append(picked + [-1] * (k - len(picked)))
    return torch.tensor(out, dtype=torch.int64).reshape(len(out), k)


def weights(x, chosen, scoring, renormalise, scale):
    """The chosen experts' weights in 64 bits, differentiable by x."""
    x = torch.where(x > -math.inf, x, torch.full_like(x, -math.inf))     # NaN counts as -inf
    on = chosen >= 0
    z = torch.where(on, x.gather(1, chosen.clamp(min=0)), torch.full(chosen.shape, -math.inf, dtype=x.dtype))
    if scoring == "sigmoid":
        if renormalise:
            log_s = torch.where(on, torch.nn.functional.logsigmoid(torch.where(on, z, torch.zeros_like(z))), torch.full_like(z, -math.inf))
            w = torch.softmax(torch.where(on.any(1, keepdim=True), log_s, torch.zeros_like(z)), 1)
        else:
            w = torch.sigmoid(z)
    elif renormalise:
        w = torch.softmax(torch.where(on.any(1, keepdim=True), z, torch.zeros_like(z)), 1)
    else:
        # the difference from the maximum first: beside -3e38 a logarithm is lost in 64 bits, too
        w = torch.softmax(torch.where((x > -math.inf).any(1, keepdim=True), x, torch.zeros_like(x)), 1).gather(1, chosen.clamp(min=0))
    return torch.where(on, w * scale, torch.zeros_like(w))


def expert_order(chosen, experts):
    """offsets, order, positions of a counting sort that keeps the slots' order."""
    flat = chosen.reshape(-1).tolist()
    order = [s for _, s in sorted((c, i) for i, c in enumerate(flat) if c >= 0)]
    offsets = [0] * (experts + 1)
    for c in flat:
        if c >= 0:
            offsets[c + 1] += 1
    for e in range(experts):
        offsets[e + 1] += offsets[e]
    positions = [-1] * len(flat)
    for row, s in enumerate(order):
        positions[s] = row
    order += [-1] * (len(flat) - len(order))
    return torch.tensor(offsets), torch.tensor(order, dtype=torch.int64), torch.tensor(positions, dtype=torch.int64).reshape(chosen.shape)


def hash32(x):
    x = (x * 747796405 + 2891336453) & 0xFFFFFFFF
    x = (((x >> ((x >> 28) + 4)) ^ x) * 277803737) & 0xFFFFFFFF
    return (x >> 22) ^ x


def hash32_int(x):
    return int(hash32(torch.tensor(x)))


def random_bits(seed, step, first, n):
    key = hash32_int((hash32_int(seed & 0xFFFFFFFF) + step) & 0xFFFFFFFF)
    i = torch.arange(first, first + n)
    return hash32((i & 0xFFFFFFFF) ^ hash32((key + (i >> 32)) & 0xFFFFFFFF))


def e4m3_values():
    """What the 256 bytes of e4m3 stand for."""
    out = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out.append(float("nan") if b & 127 == 127 else -v if b >> 7 else v)
    return torch.tensor(out)


def from8(codes, scale):
    n = codes.numel()
    return e4m3_values()[codes.long()] * scale.repeat_interleave(256)[:n]


def to8(x, bits16, keep):
    """Codes and scales of x (float32), by the values of e4m3 and not by bits: the lower neighbour, and the upper one where the
    cut-off part and the random number pass one step."""
    n = x.numel()
    pad = torch.nn.functional.pad(x, (0, -n % 256)).reshape(-1, 256)
    scale = pad.abs().amax(1) * torch.tensor(1.0 / 448.0, dtype=torch.float32)
    inv = torch.where(scale > 0, (1.0 / scale).clamp(max=3.4028234663852886e38), torch.zeros_like(scale))
    y = (x.abs() * inv.repeat_interleave(256)[:n]).clamp(max=448.0).double()
    grid = e4m3_values()[:127].double()
    lo = (torch.searchsorted(grid, y.contiguous(), right=True) - 1).clamp(0, 126)
    hi = (lo + 1).clamp(max=126)
    step = torch.where(hi > lo, grid[hi] - grid[lo], torch.ones_like(y))
    # what is cut off is itself cut to 20 bits of the step, as 32 bits hold no more of it below the smallest normal number
    part = (y - grid[lo]) / step
    part = torch.where(y >= 2.0 ** -6, part, (y * 2.0 ** 29).round() / 2.0 ** 20 - lo.double())
    code = torch.where(part + (bits16.double() * 16 + 8) / 2 ** 20 >= 1, hi, lo)
    if keep:
        code = torch.where((x != 0) & (code == 0), torch.ones_like(code), code)
    return (code + 128 * torch.signbit(x).long()).to(torch.uint8), scale


def adamw(w, g, state, copy_dtype, step, lr, betas, eps, decay, coef=1.0, bits=None):
    """One step, every operation rounded to 32 bits; state: (m, v), or (m, m_scale, v, v_scale) with the random bits."""
    c1, c2 = 1.0 - betas[0] ** step, 1.0 - betas[1] ** step
    g = g.float() * coef
    eight = bits is not None
    if eight:
        m, v = from8(state[0], state[1]), from8(state[2], state[3])
        v = v * v
    else:
        m, v = state
    m = m * betas[0] + g * (1.0 - betas[0])
    v = v * betas[1] + (g * g) * (1.0 - betas[1])
    root = v.sqrt()
    new = w.float() * (1.0 - lr * decay) - m / (root * (1.0 / math.sqrt(c2)) + eps) * (lr / c1)
    copy = None if copy_dtype is None else new.to(copy_dtype)
    if not eight:
        return new.to(w.dtype), copy, (m, v)
    a, b = to8(m, bits & 0xFFFF, False), to8(root, bits >> 16, True)
    return new.to(w.dtype), copy, a + b
