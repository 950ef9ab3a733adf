"""Plain 64-bit statements of the filtered distributions, row by row, for the tests."""
import math

import torch


def probabilities(x, T=1.0, k=0, p=1.0, m=0.0):
    """fp64 probabilities of a row of logits under one request's filters (zeros: nothing to keep)."""
    x = x.detach().cpu().double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    T, p, m = (float(torch.tensor(v, dtype=torch.float32)) for v in (T, p, m))
    V = x.numel()
    top = float(x.max())
    out = torch.zeros(V, dtype=torch.float64)
    if top == -math.inf:
        return out
    w = (x == top).double() if math.isinf(top) else torch.exp((x - top) / T) if T else (x == top).double()
    xs, ws = x.tolist(), w.tolist()
    order = sorted(range(V), key=lambda c: (-xs[c], c))
    n = 1 if T == 0 else min(k, V) if k > 0 else V
    if p < 1:
        run, whole = 0.0, math.fsum(ws[c] for c in order[:n])
        keep = 0
        while keep < n and (keep == 0 or run < p * whole):
            run += ws[order[keep]]
            keep += 1
        n = keep
    keep = order[:n]
    if m > 0 and T:
        floor = top + T * math.log(min(m, 1.0)) if not math.isinf(top) else top
        keep = [c for c in keep if xs[c] >= floor]
    out[keep] = w[keep]
    return out / out.sum()


def draw(z, u):
    """The first column whose running sum exceeds u times the sum; and how far u is from the nearest
    border of that column (in probability)."""
    z = z / z.sum()
    run = torch.cumsum(z, 0)
    u = float(torch.tensor(u, dtype=torch.float32))
    c = int((run <= u).sum().clamp(max=z.numel() - 1))
    while float(z[c]) == 0:
        c -= 1
    return c, min(float(run[c]) - u, u - (float(run[c]) - float(z[c])) if c else 1.0)


def peaked(n, V, gen, dtype=torch.bfloat16, device="cuda"):
    """Rows like a language model's: a bulk, and some columns that stand out."""
    x = 2.0 * torch.randn(n, V, generator=gen, device=device)
    for i in range(min(V, 40)):
        x[torch.arange(n, device=device), torch.randint(0, V, (n,), generator=gen, device=device)] = 12.0 - 2.0 * math.log(i + 1.0)
    return x.to(dtype)


def pitched(x):
    """The same rows with a pitch of whole 16-byte vectors, the padding larger than any logit."""
    n, V = x.shape
    out = torch.full((n, -(-V // 8) * 8 + 8), 1e30, dtype=x.dtype, device=x.device)
    out[:, :V] = x
    return out[:, :V]
