"""Cases, plain forms and 64-bit values of the operators around a refit:

quantise   a weight or activation matrix to NVFP4 (e2m1 codes, an e4m3 scale per 16 values, a 32-bit scale per
           matrix or per row), with the values that the codes stand for;
linear     16- or 32-bit activations times NVFP4 weights, dense or per expert: the activations are quantised with
           a scale per row, then both 4-bit operands are multiplied;
loss       clipped policy loss with a KL term from logits: the loss, the tokens' log-probabilities and the
           gradient by the logits;
logprobs   the log-probabilities of sampled tokens alone.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
FLT_MAX = 3.4028234663852886e38
CLIP_LOW, CLIP_HIGH, KL, TEMPERATURE = 0.2, 0.28, 0.02, 0.8


def listed():
    return [
        # A small dense layer of a 32-bit master copy, on its way into the refit's arena.
        dict(name="quantise 1024x1024", op="quantise", rows=1024, cols=1024, dtype="f32", per_row=False, pad=0),
        # One decode step's activations, a scale per token, rows cut from a wider buffer; an odd number of tokens.
        dict(name="quantise rows 333x6144", op="quantise", rows=333, cols=6144, dtype="bf16", per_row=True, pad=64),
        # The gate matrices of all 64 experts of a layer.
        dict(name="quantise 131072x6144", op="quantise", rows=131072, cols=6144, dtype="bf16", per_row=False, pad=0),
        # One token through a down projection.
        dict(name="linear 1x6144x2048", op="linear", m=1, n=6144, k=2048, experts=0, dtype="bf16", out="bf16"),
        # A decode batch through the fused gate and up projections of a dense model; an odd batch.
        dict(name="linear 37x28672x4096", op="linear", m=37, n=28672, k=4096, experts=0, dtype="f16", out="f16"),
        # A prompt through the down projection of the same model.
        dict(name="linear 4096x4096x14336", op="linear", m=4096, n=4096, k=14336, experts=0, dtype="bf16", out="bf16"),
        # A decode batch of 64 sequences, 8 experts each, through fused gate and up projections of 64 experts.
        dict(name="experts 512x4096x6144", op="linear", m=512, n=4096, k=6144, experts=64, dtype="bf16", out="bf16"),
        # A prompt through the experts' down projections, kept in 32 bits for the sum over a token's experts.
        dict(name="experts 16384x6144x2048", op="linear", m=16384, n=6144, k=2048, experts=64, dtype="bf16", out="f32"),
        # Log-probabilities of one decode step's sampled tokens.
        dict(name="logprobs 8x128256", op="logprobs", t=8, v=128256, dtype="bf16"),
        # A short sequence in 32 bits over a small vocabulary.
        dict(name="loss 512x32768", op="loss", t=512, v=32768, dtype="f32"),
        # An odd number of tokens over a vocabulary with a few tokens added: no row but the first is aligned.
        dict(name="loss 1021x32771", op="loss", t=1021, v=32771, dtype="bf16"),
        # A packed batch of a large vocabulary.
        dict(name="loss 4096x128256", op="loss", t=4096, v=128256, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantise", "linear", "experts", "loss", "loss", "logprobs"])
    if op == "quantise":
        cols = 16 * _log(rng, 1, 896)
        rows = _log(rng, 1, min(131072, 131072 * 6144 // cols))
        dtype = rng.choice(["f32", "bf16", "f16"])
        if dtype == "f32":
            rows = min(rows, 65536)
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, per_row=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 24, 3]))
    if op == "linear":
        return dict(op="linear", m=_log(rng, 1, 4096), n=_log(rng, 8, 8192), k=32 * _log(rng, 1, 224), experts=0,
                    dtype=rng.choice(["bf16", "f16", "f32"]), out=rng.choice(["bf16", "f16", "f32"]))
    if op == "experts":
        return dict(op="linear", m=_log(rng, 1, 8192), n=_log(rng, 64, 4096), k=32 * _log(rng, 4, 96), experts=_log(rng, 2, 64),
                    dtype=rng.choice(["bf16", "f16"]), out=rng.choice(["bf16", "f16", "f32"]))
    v = _log(rng, 2, 128256)
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    t = _log(rng, 1, min(4096, max(1, 256 * 1048576 // v)))
    return dict(op=op, t=t, v=v, dtype=dtype)


# ---- inputs -------------------------------------------------------------------------------------------------------


def _normal(g, shape, dtype, std):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g).to(dtype)


def _activations(g, m, k, dtype):
    """Normal values with one channel in 64 ten times as large."""
    x = _normal(g, (m, k), torch.float32, 1.0)
    x[:, ::64] *= 10.0
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantise":
        rows, cols, pad = case["rows"], case["cols"], case["pad"]
        x = _normal(g, (rows, cols + pad), DTYPES[case["dtype"]], 0.02)
        s["x"] = x[:, :cols]
    elif case["op"] == "linear":
        m, n, k, e = case["m"], case["n"], case["k"], case["experts"]
        s["x"] = _activations(g, m, k, DTYPES[case["dtype"]])
        # weights as a refit leaves them: codes and scales row-major, all experts of a matrix one after another
        w = _normal(g, (max(e, 1) * n, k), torch.bfloat16, 0.02)
        parts, per = [], max(1, (1 << 28) // k)
        scale = _scale_of(w.abs().amax().float().reshape(1, 1), False)
        for at in range(0, w.shape[0], per):
            codes, scales, _ = _quantise(w[at:at + per].float(), scale)
            parts.append((_pack(codes), scales.to(torch.float8_e4m3fn).view(torch.uint8)))
        del w
        s["codes"], s["scales"] = (torch.cat(p) for p in zip(*parts))
        s["scale"] = scale
        s["offsets"], s["most"] = None, m
        if e:
            # a router that prefers some experts: a few get several times their share, some may get no token
            share = torch.empty(e, device="cuda").normal_(0.0, 0.7, generator=g).exp_()
            counts = torch.bincount(torch.multinomial(share, m, replacement=True, generator=g), minlength=e)
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
            s["most"] = int(counts.max())
    else:
        t, v = case["t"], case["v"]
        z = _normal(g, (t, v), torch.float32, 2.0)
        y = torch.randint(0, v, (t,), device="cuda", generator=g)
        z[torch.arange(t, device="cuda"), y] += 8.0
        z = z.to(DTYPES[case["dtype"]])
        s["logits"], s["tokens"] = z, y
        if case["op"] == "loss":
            lp = _logp(z, y, 1.0 / TEMPERATURE)[0]
            noise = torch.empty((3, t), device="cuda").normal_(0.0, 1.0, generator=g)
            s["old"], s["ref"], s["adv"] = lp + 0.15 * noise[0], lp + 0.3 * noise[1], noise[2]
            # a quarter of the rows belong to the prompt or are padding
            keep = torch.rand(t, device="cuda", generator=g) >= 0.25
            s["weights"] = keep.float() / max(1, t)
    return s


# ---- plain forms --------------------------------------------------------------------------------------------------


def _quantise(x, t):
    """e2m1 codes' values, e4m3 scales' values and the product of both scales, of a 32-bit matrix; t: [1] or [rows, 1]."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // 16, 16)
    t = t.reshape(-1, 1)
    s = (b.abs().amax(-1) / (t * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    st = s * t
    r = torch.where(st > 0, (1.0 / st).clamp(max=FLT_MAX), torch.zeros_like(st))
    y = b * r[..., None]
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0)
    return torch.copysign(q, y).reshape(rows, cols), s, st


def _pack(q):
    """Two e2m1 codes a byte, the first in the low four bits."""
    a = q.abs()
    c = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) + (torch.signbit(q).to(torch.uint8) << 3)
    return c[:, ::2] | (c[:, 1::2] << 4)


def _unpack(p):
    c = torch.stack([p & 15, p >> 4], -1).reshape(p.shape[0], -1)
    m, e = (c & 1).float(), ((c >> 1) & 3).float()
    a = torch.where(e == 0, m * 0.5, (1 + m * 0.5) * torch.exp2(e - 1))
    return torch.where(c >= 8, -a, a)


def _spread(q, st):
    return (q.reshape(st.shape[0], st.shape[1], 16) * st[..., None]).reshape(q.shape)


def _scale_of(x, per_row):
    a = x.abs().amax(1, keepdim=True) if per_row else x.abs().amax().reshape(1)
    return torch.where(a > 0, a * (1.0 / 2688.0), torch.ones_like(a))


def _logp(z, y, inv):
    z = z.float() * inv
    lse = torch.logsumexp(z, 1)
    return z.gather(1, y[:, None])[:, 0] - lse, z, lse


def _plain(s):
    if s["op"] == "quantise":
        x = s["x"].float()
        t = _scale_of(x, s["per_row"])
        q, scales, st = _quantise(x, t)
        return dict(values=_spread(q, st).to(torch.bfloat16), scales=scales.to(torch.float8_e4m3fn), scale=t.reshape(-1))
    if s["op"] == "linear":
        x = s["x"].float()
        m, k = x.shape
        tx = _scale_of(x, True)
        q, sx, _ = _quantise(x, tx)
        x = _spread(q, sx)
        w = _spread(_unpack(s["codes"]), s["scales"].view(torch.float8_e4m3fn).float())
        if s["offsets"] is None:
            y = x @ w.T
        else:
            # every expert's rows, padded to the most that one expert has
            e = s["experts"]
            lo, hi = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
            at = lo + torch.arange(s["most"], device=x.device)
            there = at < hi
            y = torch.bmm(x[at.clamp(max=m - 1)], w.reshape(e, -1, k).transpose(1, 2))[there]
        return (y * (tx * s["scale"])).to(DTYPES[s["out"]])
    z, y, inv = s["logits"], s["tokens"], 1.0 / TEMPERATURE
    lp, z, lse = _logp(z, y, inv)
    if s["op"] == "logprobs":
        return lp
    w = s["weights"]
    on = w != 0
    lp = torch.where(on, lp, 0.0)
    ratio = torch.exp(lp - s["old"])
    u, c = ratio * s["adv"], ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * s["adv"]
    k = s["ref"] - lp
    e = torch.exp(k)
    per = torch.where(c < u, -c, -u) + KL * (e - k - 1)
    loss = torch.where(on, w * per, 0.0).sum()
    d = torch.where(c < u, 0.0, -u) + KL * (1 - e)
    g = torch.where(on, w * d * inv, 0.0)
    grad = torch.exp(z - lse[:, None]) * -g[:, None]
    grad[torch.arange(len(y), device=y.device), y] += g
    return dict(loss=loss, logp=lp, grad=grad.to(s["logits"].dtype))


def run(s):
    if not own:
        return _plain(s)
    import bit_exact_xor_gb300 as dcr
    if s["op"] == "quantise":
        q, values = dcr.nvfp4_quantize(s["x"], per_row=s["per_row"], values=torch.bfloat16)
        return dict(values=values, scales=q.scales.view(torch.float8_e4m3fn), scale=q.scale)
    if s["op"] == "linear":
        return dcr.nvfp4_linear(s["x"], dcr.Nvfp4(s["codes"], s["scales"], s["scale"]), offsets=s["offsets"], dtype=DTYPES[s["out"]])
    if s["op"] == "logprobs":
        return dcr.token_logprobs(s["logits"], s["tokens"], temperature=TEMPERATURE)
    loss, lp, grad = dcr.policy_loss(s["logits"], s["tokens"], s["old"], s["adv"], s["weights"], ref_logp=s["ref"], clip_low=CLIP_LOW,
                                     clip_high=CLIP_HIGH, kl_coef=KL, temperature=TEMPERATURE)
    return dict(loss=loss, logp=lp, grad=grad)


def work(case):
    if case["op"] == "quantise":
        n = case["rows"] * case["cols"]
        return dict(bytes=n * (SIZE[case["dtype"]] + 2 + 0.5 + 1 / 16), flops=4 * n)
    if case["op"] == "linear":
        m, n, k, e = case["m"], case["n"], case["k"], case["experts"]
        # an expert without a row is not read; at most one expert a row is
        return dict(bytes=m * k * SIZE[case["dtype"]] + min(max(e, 1), m) * n * k * 0.5625 + m * n * SIZE[case["out"]], flops=2 * m * n * k)
    n = case["t"] * case["v"]
    both = 1 if case["op"] == "logprobs" else 2
    return dict(bytes=n * SIZE[case["dtype"]] * both, flops=4 * n * both)


# ---- the same in 64 bits, from the definitions ---------------------------------------------------------------------


def _e4m3_64(u):
    """The nearest e4m3 value (4 significant bits, exponents from -6, largest 448), ties to even."""
    _, e = torch.frexp(u)
    step = torch.ldexp(torch.ones_like(u), (e - 1).clamp(min=-6) - 3)
    return (torch.round(u / step) * step).clamp(max=448.0)


def _e2m1_64(v):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; a value halfway goes to the even code."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
    mid = (grid[1:] + grid[:-1]) / 2
    a = v.abs()
    right, left = torch.bucketize(a, mid, right=True), torch.bucketize(a, mid)
    return torch.sign(v) * grid[torch.where(right % 2 == 0, right, left)]


def _r32(v):
    """A 64-bit value rounded to 32 bits, where the definition of the format rounds."""
    return v.float().double()


def _scale_64(a):
    return torch.where(a > 0, _r32(a * float(torch.tensor(1 / 2688))), 1.0)


def _nvfp4_64(x, t):
    """Rows at a time (the matrix may be large): codes' values, e4m3 scales, and the product of both scales.  Which code a
    value gets is part of the format's definition, so the quotients that decide it are rounded to 32 bits here too."""
    b, t = x.double().reshape(x.shape[0], -1, 16), t.reshape(-1, 1)
    s = _e4m3_64(_r32(b.abs().amax(-1) / _r32(6 * t)))
    st = _r32(s * t)
    r = torch.where(st > 0, _r32(1 / st).clamp(max=FLT_MAX), 0.0)
    return _e2m1_64(_r32(b * r[..., None])), s, st


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        x = s["x"]
        a = x.abs().amax(1).double() if case["per_row"] else x.abs().amax().double().reshape(1)
        t = _scale_64(a)
        values, scales = torch.empty(x.shape, dtype=torch.float64, device="cuda"), []
        for at in range(0, x.shape[0], 8192):
            tt = t[at:at + 8192] if case["per_row"] else t
            q, sc, st = _nvfp4_64(x[at:at + 8192], tt)
            values[at:at + 8192] = (q * st[..., None]).flatten(1)
            scales.append(sc)
        return dict(values=values, scales=torch.cat(scales), scale=t)
    if case["op"] == "linear":
        x, n, e = s["x"], case["n"], max(case["experts"], 1)
        a = x.abs().amax(1).double()
        t = _scale_64(a)
        q, sx, _ = _nvfp4_64(x, t)
        xv = (q * sx[..., None]).flatten(1)
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
        at = [0, case["m"]] if s["offsets"] is None else s["offsets"].tolist()
        y = torch.empty((case["m"], n), dtype=torch.float64, device="cuda")
        for i in range(e):
            if at[i + 1] > at[i]:
                c = s["codes"][i * n:(i + 1) * n].long()
                w = torch.empty((n, case["k"]), dtype=torch.float64, device="cuda")
                w[:, ::2], w[:, 1::2] = table[c & 15], table[c >> 4]
                w *= s["scales"][i * n:(i + 1) * n].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
                y[at[i]:at[i + 1]] = xv[at[i]:at[i + 1]] @ w.T
        return y * t[:, None] * s["scale"].double()
    z = s["logits"].double() / TEMPERATURE
    rows = torch.arange(case["t"], device="cuda")
    top = z.amax(1, keepdim=True)
    ez = torch.exp(z - top)
    total = ez.sum(1, keepdim=True)
    lp = z[rows, s["tokens"]] - top[:, 0] - torch.log(total[:, 0])
    if case["op"] == "logprobs":
        return lp
    w, adv = s["weights"].double(), s["adv"].double()
    lp = torch.where(w != 0, lp, 0.0)
    ratio, ref = torch.exp(lp - s["old"].double()), torch.exp(s["ref"].double() - lp)
    clipped = torch.where(adv > 0, ratio > 1 + CLIP_HIGH, ratio < 1 - CLIP_LOW)
    kept = torch.where(clipped, torch.where(adv > 0, 1 + CLIP_HIGH, 1 - CLIP_LOW), ratio)
    loss = (w * (KL * (ref - (s["ref"].double() - lp) - 1) - kept * adv)).sum()
    slope = w * (KL * (1 - ref) - torch.where(clipped, 0.0, ratio * adv)) / TEMPERATURE
    grad = ez.div_(total).mul_(-slope[:, None])
    grad[rows, s["tokens"]] += slope
    return dict(loss=loss, logp=lp, grad=grad)
