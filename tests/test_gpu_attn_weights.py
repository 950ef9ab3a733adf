"""Softmax weights far below a row's largest: where the heaviest keys hold zeros
as values, the result is what the light ones carry.

Scores are set through element 0 of the keys, with a query of 1 there and 0
elsewhere, so that one product makes a score; levels are in powers of two
(scale = ln 2).  Tolerances: attn_util.attention, whose parts are all relative
to a row's own weights times values, as roundings of fp32 and bf16 are."""
import math

import pytest
import torch

import attn_util as u
from speculative_decoding_pe_gb300 import _native
from test_gpu_attn import BF, Cached, Prompt, dev

pytestmark = pytest.mark.gpu


def set_levels(c, level, Hq, D):
    """Every request of ``c`` (all of one length): the score of key t becomes
    level[t] (rounded to what the cache holds) in each head."""
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.scale = math.log(2.0)
    level = level.to("cuda")
    t = torch.arange(level.numel(), device="cuda")
    f = u.fields(c.cache, D)
    scale = (level.abs() / 4).to(torch.float8_e4m3fn).view(torch.uint8)
    code = torch.where(level < 0, 0x0e, 0x06).to(torch.uint8)  # -4, 4
    for b in range(len(c.limits)):
        slots = c.table[b].long()[t // c.bs] * c.bs + t % c.bs
        at = (slots // c.bs, slice(None), slots % c.bs // 16, slots % 16)
        f[0][(*at, 0)] = code[:, None]
        f[2][(*at, 0)] = scale[:, None]
    return f


def clear_values(c, f, keys):
    t = keys.nonzero().flatten().to("cuda")
    for b in range(len(c.limits)):
        slots = c.table[b].long()[t // c.bs] * c.bs + t % c.bs
        f[1][slots // c.bs, :, slots % c.bs // 16, slots % 16] = 0


def refresh(c, n, D):
    t = torch.arange(n, device="cuda")
    for b in range(len(c.limits)):
        c.kv[b] = u.held(c.cache, D, c.table[b].long()[t // c.bs] * c.bs + t % c.bs)


@pytest.mark.parametrize("Hq, Hkv, D, rows", [(8, 1, 64, 1), (32, 4, 128, 1), (16, 1, 64, 1), (16, 1, 128, 1), (8, 1, 64, 14),
                                              (8, 1, 128, 14)])
@pytest.mark.parametrize("gap", [24, 33, 50, 90, 108])
@pytest.mark.parametrize("where", ["first", "last"])
def test_the_heaviest_key_holds_zeros(Hq, Hkv, D, rows, gap, where):
    n = 600
    c = Cached([[n] * rows], Hq, Hkv, D, uniform=True, seed=3)
    g = torch.Generator().manual_seed(gap)
    level = -gap / 2 + 2.0 * torch.rand(n, generator=g)
    heavy = torch.zeros(n, dtype=torch.bool)
    heavy[[3, 200] if where == "first" else [590, 599]] = True
    level[heavy] = gap / 2
    f = set_levels(c, level, Hq, D)
    clear_values(c, f, heavy)
    refresh(c, n, D)
    c.check()
    assert bool((c.out != 0).any())


@pytest.mark.parametrize("rows", [1, 2, 14])
def test_peaked_rows(rows):
    """Weights over all of fp32's range, many draws.  Below 2^-126 of a maximum that
    may lie 2^8 under the largest an fp32 weight is no normal number and counts as 0:
    up to 2^-118 of each value on top of the relative bound."""
    for seed in range(30):
        c = Cached([[600 + i for i in range(rows)]], 16, 2, 64, uniform=True, q_std=30.0, seed=seed)
        out = c.run()
        k, v = c.kv[0]
        want, tol = u.attention(c.q, k, v, dev(c.limits[0], torch.int64), c.scale)
        u.within(out, want, tol + 2.0 ** -118 * v.abs().sum(0).repeat_interleave(8, 0), "seed %d" % seed)


@pytest.mark.parametrize("Hq, Hkv, D, rows, B, n", [
    (32, 4, 64, 14, 40, 900), (32, 4, 128, 14, 40, 900),       # whole items
    (8, 1, 64, 14, 1, 900), (8, 1, 128, 14, 1, 900),           # parts of one tile a stream
    (8, 1, 64, 14, 1, 100_000), (8, 1, 128, 14, 1, 100_000),   # parts of several
    (32, 4, 64, 1, 40, 900), (8, 1, 128, 1, 1, 100_000)])
@pytest.mark.parametrize("low, gap", [(40, 90), (60, 108), (90, 100), (99, 30), (120, 50)])
def test_scores_that_rise_in_steps(Hq, Hkv, D, rows, B, n, low, gap):
    """Keys at 0, then at ``low``, then a last few ``gap`` above them that hold zeros."""
    c = Cached([[n] * rows] * B, Hq, Hkv, D, uniform=True, seed=4)
    t = torch.arange(n)
    level = torch.where(t % 1024 < 512 if n > 1000 else t < 300, 0.0, float(low))
    last = t >= n - (100 if n < 1000 else 4000)
    level[last] = low + gap
    f = set_levels(c, level, Hq, D)
    clear_values(c, f, last)
    refresh(c, n, D)
    c.check()
    assert bool((c.out != 0).any())


class Levels(Prompt):
    """Prompts whose key t of each has the score level[t]."""

    def __init__(self, B, n, Hq, Hkv, D, level, seed=5):
        super().__init__([n] * B, Hq, Hkv, D, seed)
        self.q.zero_()
        self.q[..., 0] = 1.0
        self.k[..., 0] = level.repeat(B).to("cuda", BF)[:, None]

    def run(self, stream=None, out=None):
        out = self.out if out is None else out
        _native.attn_prompt(self.q, self.k, self.v, self.offsets, out, self.ws, self.err, scale=math.log(2.0), B=len(self.lens))
        return out

    def check_levels(self):
        out = self.run()
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        n = self.lens[0]
        lim = torch.arange(1, n + 1, device="cuda")
        for b in range(len(self.lens)):
            sl = slice(b * n, (b + 1) * n)
            want, tol = u.attention(self.q[sl], self.k[sl].double(), self.v[sl].double(), lim, math.log(2.0))
            u.within(out[sl], want, tol, "prompt %d" % b)
        return out


@pytest.mark.parametrize("B, Hq, Hkv, D", [(1, 8, 1, 64), (1, 8, 1, 128), (12, 64, 8, 64), (12, 32, 8, 128)])
@pytest.mark.parametrize("low, gap", [(7, 100), (40, 90), (60, 108), (99, 100)])
def test_prompts_whose_scores_rise_in_steps(B, Hq, Hkv, D, low, gap):
    n = 700
    t = torch.arange(n)
    level = torch.where(t < 200, 0.0, float(low))
    level[t >= 500] = low + gap
    p = Levels(B, n, Hq, Hkv, D, level)
    p.v.unflatten(0, (B, n))[:, 500:] = 0
    out = p.check_levels()
    assert bool((out.unflatten(0, (B, n))[:, 500:] != 0).any())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rise", [7, 60, 99, 150])
@pytest.mark.parametrize("size", [28, 60, 90])
def test_large_values_under_rising_scores(D, rise, size):
    """Values of 2^size: finite results stay finite."""
    n = 700
    level = torch.where(torch.arange(n) < 200, 0.0, float(rise))
    p = Levels(2, n, 16, 2, D, level)
    p.v.mul_(2.0 ** size)
    out = p.check_levels()
    assert bool(out.isfinite().all())
