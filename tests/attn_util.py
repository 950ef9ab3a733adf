"""Plain 64-bit statements of the drafter layer's operators, for the tests."""
import math

import torch

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def fields(cache, D):
    cut = (0, 8 * D, 16 * D, 17 * D, 18 * D)
    return [cache[..., a:b].unflatten(-1, (16, -1)) for a, b in zip(cut, cut[1:])]


def held(cache, D, slots):
    """fp64 keys and values [n, Hkv, D] that the cache stands for at ``slots``."""
    bs = 16 * cache.shape[2]
    rec = [f[slots // bs, :, slots % bs // 16, slots % 16] for f in fields(cache, D)]
    grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device=cache.device)
    out = []
    for codes, scales in ((rec[0], rec[2]), (rec[1], rec[3])):
        x = grid[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
        out.append((x.unflatten(-1, (-1, 16)) * scales.contiguous().view(torch.float8_e4m3fn).double().unsqueeze(-1)).flatten(-2))
    return out


def quantised(x):
    """fp64 values that bf16 rows [..., D] become in the cache."""
    y = x.double().unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1, keepdim=True).float() / 6).clamp(max=448).to(torch.float8_e4m3fn).double()
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    # saturation by hand: from far away every point of the grid is as near
    d = ((y.abs() / s).nan_to_num(0.0).clamp(max=6.0).unsqueeze(-1) - grid).abs()
    d += torch.arange(8, device=x.device) % 2 * 1e-9  # ties to the even code
    return (grid[d.argmin(-1)] * s * torch.where(torch.signbit(y), -1.0, 1.0)).flatten(-2)


def to_bf16(x):
    """fp64 to bf16 in one rounding (by way of fp32 there would be two)."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256.0), e - 8).to(torch.bfloat16)


def rotated(x, rope, pos, interleaved):
    """fp64 rotation of rows [T, H, D]; also the sum of its terms' magnitudes."""
    half = rope.shape[1] // 2
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = rope.double()[pos.long()][:, None].split(half, -1)
    y = x.double()
    z, mag = y.clone(), y.abs()
    z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    mag[..., a] = (y[..., a] * c).abs() + (y[..., b] * s).abs()
    mag[..., b] = (y[..., b] * c).abs() + (y[..., a] * s).abs()
    return z, mag


def random_cache(blocks, Hkv, bs, D, gen, std=0.3):
    """A cache of random codes with scales around ``std``."""
    c = torch.randint(0, 256, (blocks, Hkv, bs // 16, 18 * D), generator=gen, device="cuda").to(torch.uint8)
    s = (torch.rand(blocks, Hkv, bs // 16, 2 * D, generator=gen, device="cuda") + 0.5) * std
    c[..., 16 * D:] = s.to(torch.float8_e4m3fn).view(torch.uint8)
    return c


def attention(q, k, v, limit, scale, p_step=2.0 ** -8):
    """One request: q [m, Hq, D], k and v [L, Hkv, D] fp64, limit [m]; the fp64
    result and how far a bf16 result may be from it.

    The bound counts: the output's rounding (2^-8 of the value); the rounding
    of a weight to p_step of itself, and the error of its score (an fp32 sum of
    D products: D + 8 roundings of 2^-24 of the terms' magnitude, on a scale
    where it moves the weight by as much, and again in the weights' sum),
    each against sum p|v|; and 2^-18 for exp2 and the fp32 sums of weights."""
    m, Hq, D = q.shape
    L, Hkv = k.shape[:2]
    out = torch.zeros(m, Hq, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    if not L or not m:
        return out, tol
    for h in range(Hkv):
        G = Hq // Hkv
        qq = q[:, h * G:(h + 1) * G].double()
        hidden = torch.arange(L, device=q.device) >= limit[:, None, None]
        kk, vv = k[:, h], v[:, h]
        s = torch.einsum("mgd,ld->mgl", qq, kk) * scale
        mag = torch.einsum("mgd,ld->mgl", qq.abs(), kk.abs()) * abs(scale)
        s = s.masked_fill(hidden, -math.inf)
        p = torch.softmax(s, -1).nan_to_num(0.0)
        o = p @ vv
        off = 2 * (D + 8) * 2.0 ** -24 * mag.masked_fill(hidden, 0.0).amax(-1, keepdim=True)
        out[:, h * G:(h + 1) * G] = o
        tol[:, h * G:(h + 1) * G] = 2.0 ** -8 * o.abs() + (p_step + off + 2.0 ** -18) * (p @ vv.abs())
    return out, tol


def within(got, want, tol, what=""):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)  # a NaN is outside
    assert not bool(bad.any()), "%s: %d of %d outside; worst %.3g allowed %.3g" % (
        what, int(bad.sum()), bad.numel(), float(off[bad].max()), float(tol[bad].min()))
