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
from test_gpu_attn import Cached, dev

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
