"""Plain 64-bit forms of the operators of include/dcr_ops.h, written from the
formulas there.  Quotients that decide a code are rounded to 32 bits, as the
format defines them."""
import torch

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
F32_MAX = 3.4028234663852886e38


def r32(v):
    return v.float().double()


def e4m3_table():
    """Every finite non-negative e4m3 value, ascending: byte b stands for entry b."""
    out = []
    for b in range(127):
        e, m = b >> 3, b & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(out, dtype=torch.float64)


def nearest(v, table):
    """Index of the nearest entry of an ascending table, ties to the even index."""
    hi = torch.searchsorted(table, v.contiguous()).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    dh, dl = table[hi] - v, v - table[lo]
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.where(up, hi, lo)


def scale32(a):
    t = r32(a * float(torch.tensor(1 / 2688)))
    return torch.where(t > 0, t, torch.ones_like(t))


def quantize(x, t):
    """x [rows, cols] (any float type, cpu); t double [1] or [rows].  Returns
    codes (uint8 0..15, unpacked), scale bytes, values (double)."""
    rows, cols = x.shape
    x = x.double().reshape(rows, cols // 16, 16)
    t = t.reshape(-1, 1)
    nan = torch.isnan(x).any(-1)
    a = torch.where(torch.isnan(x), 0.0, x.abs()).amax(-1)
    tab = e4m3_table()
    u = r32(a / r32(6 * t)).clamp(max=448.0)
    u = torch.nan_to_num(u, nan=448.0, posinf=448.0)
    sb = nearest(u, tab)
    s = tab[sb]
    st = r32(s * t)
    r = torch.where(st > 0, r32(1 / st).clamp(max=F32_MAX), torch.zeros_like(st))
    v = r32(x * r[..., None])
    grid = torch.tensor(GRID, dtype=torch.float64)
    # inf * 0 (a block scale of 0) and NaN take the largest code, as the conversion of a NaN does
    mag = torch.nan_to_num(v.abs(), nan=6.0, posinf=6.0)
    q = nearest(mag, grid)
    neg = torch.signbit(v) & ~torch.isnan(v)
    values = torch.where(neg, -grid[q], grid[q]) * st[..., None]
    values = torch.where(nan[..., None], torch.full_like(values, float("nan")), values)
    codes = (q + 8 * neg.long()).to(torch.uint8).reshape(rows, cols)
    sb = torch.where(nan, torch.full_like(sb, 0x7F), sb).to(torch.uint8)
    return codes, sb, values.reshape(rows, cols)


def pack(codes):
    return codes[:, ::2] | (codes[:, 1::2] << 4)


def unpack(p):
    return torch.stack([p & 15, p >> 4], -1).reshape(p.shape[0], -1)


def spread(codes, scales):
    """c * s of packed codes and scale bytes (cpu)."""
    grid = torch.tensor(GRID + [-g for g in GRID], dtype=torch.float64)
    tab = torch.cat([e4m3_table(), torch.tensor([float("nan")], dtype=torch.float64)])
    return grid[unpack(codes).long()] * tab[scales.long()].repeat_interleave(16, 1)


def policy(z, tokens, old, adv, w, ref, lo, hi, kl, temp):
    """Loss, log-probabilities, gradient in double."""
    z = z.double() / temp
    rows, vocab = z.shape
    loss, lps, grad = torch.zeros((), dtype=torch.float64), torch.zeros(rows, dtype=torch.float64), torch.zeros_like(z)
    for i in range(rows):
        y = int(tokens[i])
        if float(w[i]) == 0.0 or not 0 <= y < vocab:
            continue
        lp = z[i, y] - torch.logsumexp(z[i], 0)
        lps[i] = lp
        ratio = torch.exp(lp - float(old[i]))
        a = float(adv[i])
        u, c = ratio * a, ratio.clamp(1 - lo, 1 + hi) * a
        per, slope = (-c, torch.zeros(())) if c < u else (-u, -u)
        if kl:
            k = float(ref[i]) - lp
            per = per + kl * (torch.exp(k) - k - 1)
            slope = slope + kl * (1 - torch.exp(k))
        loss = loss + float(w[i]) * per
        p = torch.softmax(z[i], 0)
        g = -p
        g[y] += 1
        grad[i] = float(w[i]) * slope / temp * g
    return loss, lps, grad
