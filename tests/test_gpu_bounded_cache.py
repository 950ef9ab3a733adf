"""Attention weights of cached keys and eviction by them, on the GPU, against
the formulas in 64 bits, and with the append and the attention around them.

Tolerance of a weight: its rows' scores are fp32 sums of D products (D + 8 roundings
of 2^-24 of the terms' magnitude, scaling included) that move a weight by as much of itself,
and again through its sum; 2^-20 more for exp2, log2 (each 2^-22 of itself or of a score of
magnitude up to 2 octaves; the log2-sum's fp32 rounding, 2^-24 of a score's octaves, counts
with the score) and the fp32 sums over rows and heads; and one fp32 rounding of the sum."""
import pytest
import torch

import attn_util as au
import speculative_decoding_pe_gb300 as pe
from speculative_decoding_pe_gb300 import _native

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def dev(x, dt=torch.int32):
    return torch.tensor(x, dtype=dt, device="cuda")


class Weigh:
    """Requests with given row limits over a shuffled cache whose unused slots
    hold bytes of all ones (every scale a NaN) and whose table ends in ids of no page."""

    def __init__(self, limits, Hq, Hkv, D, bs=16, seed=0, uniform=False, fresh=None, q_std=2.0, extra=2):
        g = gen(seed)
        self.limits, self.Hq, self.Hkv, self.D, self.bs = limits, Hq, Hkv, D, bs
        most = [max(r, default=0) for r in limits]
        need = [-(-n // bs) for n in most]
        blocks = sum(need) + 3
        perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(limits), max(need + [1]) + extra), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        live = au.random_cache(blocks, Hkv, bs, D, g)
        self.cache = torch.full_like(live, 255)
        self.mass = torch.rand(blocks, Hkv, bs, generator=g, device="cuda")
        self.slots, self.k = [], []
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
            t = torch.arange(most[b], device="cuda")
            slots = self.table[b].long()[t // bs] * bs + t % bs
            for dst, src in zip(au.fields(self.cache, D), au.fields(live, D)):
                dst[slots // bs, :, slots % bs // 16, slots % 16] = src[slots // bs, :, slots % bs // 16, slots % 16]
            self.slots.append(slots)
            self.k.append(au.held(live, D, slots)[0])
        flat = [n for r in limits for n in r]
        self.T = len(flat)
        self.q = (torch.randn(self.T, Hq, D, generator=g, device="cuda") * q_std).to(BF)
        self.rej = dev([n == 0 for n in flat], torch.uint8)
        self.pos = dev([n - 1 if n else 7 for n in flat])
        offs = [0]
        for r in limits:
            offs.append(offs[-1] + len(r))
        self.offsets = None if uniform else dev(offs)
        self.fresh = None if fresh is None else dev(fresh)
        self.ws = _native.new_weigh_workspace(self.T, Hq, self.table.shape[1], bs)
        self.ws.fill_(255)
        self.err = _native.new_error_word()

    def run(self, out, mass="own", stream=None):
        mass = self.mass if isinstance(mass, str) else mass
        _native.kv_weigh(self.q, self.cache, self.table, self.offsets, self.pos, self.rej, mass, out, self.ws, self.err,
                         fresh=self.fresh, stream=stream)

    def want(self, mass):
        """fp64 result and tolerance; what is not written is as in ``self.before``."""
        out, tol = self.before.double(), torch.zeros_like(self.before, dtype=torch.float64)
        at, G, scale = 0, self.Hq // self.Hkv, self.D ** -0.5
        for b, r in enumerate(self.limits):
            n = max(r, default=0)
            q = self.q[at:at + len(r)].double()
            at += len(r)
            if not n:
                continue
            lim = dev(r, torch.int64)
            j = torch.arange(n, device="cuda")
            sl = self.slots[b]
            for h in range(self.Hkv):
                qq, kk = q[:, h * G:(h + 1) * G], self.k[b][:, h]
                s = (torch.einsum("mgd,ld->mgl", qq, kk) * scale).masked_fill(j >= lim[:, None, None], -float("inf"))
                mag = (torch.einsum("mgd,ld->mgl", qq.abs(), kk.abs()) * scale).masked_fill(j >= lim[:, None, None], 0.0)
                p = torch.softmax(s, -1).nan_to_num(0.0)
                off = (self.D + 8) * 2.0 ** -24 * (mag + mag.amax(-1, keepdim=True)) + 2.0 ** -20
                old = torch.zeros(n, dtype=torch.float64, device="cuda")
                if mass is not None:
                    old = mass[sl // self.bs, h, sl % self.bs].double()
                    if self.fresh is not None:
                        old = torch.where(j < self.fresh[b], old, 0.0)
                new = p.sum((0, 1)) + old
                out[sl // self.bs, h, sl % self.bs] = new
                tol[sl // self.bs, h, sl % self.bs] = (p * off).sum((0, 1)) + 2.0 ** -23 * new
        return out, tol

    def check(self, mass="own", in_place=False):
        mass = self.mass if isinstance(mass, str) else mass
        old = None if mass is None else mass.clone()
        out = mass if in_place else torch.full_like(self.mass, -5.0)
        self.before = out.clone()
        self.run(out, mass)
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        want, tol = self.want(old)
        au.within(out, want, tol)
        return out


CASES = [([[1]], 8, 8, 64, 16), ([[17]], 64, 8, 64, 16), ([[4000]], 32, 4, 128, 16), ([[5, 6, 0, 7, 8]], 8, 1, 128, 32),
         ([[100] * 3, [0] * 3, [1, 2, 3], [33, 34, 35]], 12, 12, 64, 16),
         ([[2000 + i if i < 3 or i > 7 else 0 for i in range(14)], [i + 1 for i in range(14)]], 64, 8, 64, 64),
         ([[515] * 14, [129] * 14], 32, 4, 128, 16), ([list(range(1, 300))], 16, 2, 64, 16), ([[7], [300], [0], [4097]], 20, 4, 64, 32),
         ([[9, 9]], 256, 2, 64, 16)]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_weights(case):
    limits, Hq, Hkv, D, bs = CASES[case]
    same = len({len(r) for r in limits}) == 1
    for uniform in ([True, False] if same else [False]):
        Weigh(limits, Hq, Hkv, D, bs, seed=case, uniform=uniform).check()
    w = Weigh(limits, Hq, Hkv, D, bs, seed=case, fresh=[max(r, default=0) // 2 for r in limits])
    w.check(in_place=True)
    Weigh(limits, Hq, Hkv, D, bs, seed=case, fresh=[0] * len(limits)).check()
    Weigh(limits, Hq, Hkv, D, bs, seed=case).check(mass=None)


def test_weights_of_ragged_segments():
    Weigh([[40], [], [3, 4, 5, 6], [0, 0], [200, 0, 17]], 16, 2, 128).check()


def test_weights_over_many_requests():
    w = Weigh([[1 + (37 * b) % 900] for b in range(300)], 8, 2, 64, seed=5, uniform=True)
    w.check()


@pytest.mark.parametrize("limits, Hq, Hkv, D, extra", [
    ([[300, 0, 299, 17]], 8, 8, 128, 2600), ([[40 + i if i % 3 else 0 for i in range(14)]], 64, 8, 64, 2600),
    ([[500] * 3], 64, 8, 128, 2600), ([[5000], [70]], 8, 4, 64, 2600), ([[7] * 70 + [900] * 5], 4, 4, 64, 5200)])
def test_few_pairs_over_wide_tables(limits, Hq, Hkv, D, extra):
    # a table far wider than its requests: chunks of keys as blocks of their own, most without any
    w = Weigh(limits, Hq, Hkv, D, seed=11, extra=extra)
    w.check()
    v = Weigh(limits, Hq, Hkv, D, seed=11, extra=extra)
    v.offsets[-1] += 1
    out = torch.full_like(v.mass, -5.0)
    v.run(out, None)
    torch.cuda.synchronize()
    assert int(v.err.item()) == _native.ERR_OFFSETS and bool((out == -5.0).all())


@pytest.mark.parametrize("limits, Hq, Hkv, D", [([[60 + 31 * b + i if (b + i) % 4 else 0 for i in range(14)] for b in range(12)], 56, 8, 64),
                                                ([[9 + b] * 3 for b in range(30)], 24, 4, 128), ([[11] * 80, [400] * 70] * 10, 4, 4, 64)])
def test_many_pairs_of_many_columns(limits, Hq, Hkv, D):
    w = Weigh(limits, Hq, Hkv, D, seed=12, extra=1300)
    w.check()


def test_a_row_weighs_one():
    # every kept row's weights sum to one per head: within the tolerance's 2^-20 and the rows' scores
    w = Weigh([[3000, 2999, 0, 17]], 32, 4, 128, seed=3)
    out = w.check(mass=None)
    s = w.slots[0]
    total = out[s // 16, :, s % 16].double().sum(0)
    assert bool(((total - 3 * 8).abs() <= 3 * 8 * 2.0 ** -12).all())


def test_large_scores_and_far_keys():
    # one key takes everything; queries far from one
    for std in (2.0 ** -60, 40.0, 2.0 ** 60):
        w = Weigh([[700, 300]], 8, 2, 64, seed=4, q_std=std)
        out = torch.full_like(w.mass, -5.0)
        w.run(out, None)
        torch.cuda.synchronize()
        s = w.slots[0]
        total = out[s // 16, :, s % 16].double().sum(0)
        assert int(w.err.item()) == 0 and bool(((total - 2 * 4).abs() < 0.01).all())


def test_a_query_that_is_not_finite_is_its_heads_alone():
    w = Weigh([[50], [60]], 8, 2, 64, seed=6, uniform=True)
    w.q[0, 1, 3] = float("nan")  # request 0, key head 0
    out = torch.zeros_like(w.mass)
    w.run(out, None)
    torch.cuda.synchronize()
    a, b = w.slots
    assert bool(out[a // 16, 0, a % 16].isnan().all()) and bool(out[a // 16, 1, a % 16].isfinite().all())
    assert bool(out[b // 16, :, b % 16].isfinite().all())


def test_positions_pages_and_offsets_out_of_range():
    w = Weigh([[40, 33], [20, 21]], 8, 2, 64, seed=7, extra=0)
    out = torch.full_like(w.mass, -5.0)
    w.pos[1] = -3  # sees nothing
    w.run(out, None)
    torch.cuda.synchronize()
    assert int(w.err.item()) == _native.ERR_BLOCK_RANGE
    w = Weigh([[48, 33], [20, 21]], 8, 2, 64, seed=7, extra=0)
    w.pos[0] = 2 ** 31 - 1  # sees the table's keys
    w.before = out.fill_(-5.0)
    w.run(out, None)
    torch.cuda.synchronize()
    want, tol = w.want(None)
    assert int(w.err.item()) == _native.ERR_BLOCK_RANGE
    au.within(out, want, tol)
    # a page outside the cache is left out
    w = Weigh([[48, 47]], 8, 2, 64, seed=8)
    for bad in (-1, w.cache.shape[0], 2 ** 31 - 1):
        v = Weigh([[48, 47]], 8, 2, 64, seed=8)
        v.table[0, 1] = bad
        out = torch.full_like(v.mass, -5.0)
        v.run(out, None)
        torch.cuda.synchronize()
        assert int(v.err.item()) == _native.ERR_BLOCK_RANGE
        s = torch.cat((v.slots[0][:16], v.slots[0][32:]))
        total = out[s // 16, :, s % 16].double().sum(0)
        assert bool(((total - 2 * 4).abs() < 1e-3).all()) and int((out != -5.0).sum()) == 32 * 2
    # offsets that are no partition: nothing is written
    for offs in ([0, 3, 3], [1, 2, 4], [0, 5, 4], [0, -1, 4], [0, 2, 2 ** 31 - 1]):
        v = Weigh([[40, 33], [20, 21]], 8, 2, 64, seed=7)
        v.offsets = dev(offs)
        out = torch.full_like(v.mass, -5.0)
        v.run(out, None)
        torch.cuda.synchronize()
        assert int(v.err.item()) == _native.ERR_OFFSETS and bool((out == -5.0).all())


# ------------------------------------------------------------------- eviction
class Evict:
    def __init__(self, lens, keep, Hkv, D, bs=16, seed=0, sinks=0, recent=0, in_place=False, ties=False, max_keep=None):
        g = gen(seed)
        self.lens, self.keep, self.Hkv, self.D, self.bs = lens, keep, Hkv, D, bs
        self.sinks, self.recent = sinks, recent
        need = [-(-n // bs) for n in lens]
        room = [-(-min(n, k) // bs) for n, k in zip(lens, keep)]
        blocks = sum(need) + sum(room) + 2
        perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(lens), max(need + [1])), -9, dtype=torch.int32, device="cuda")
        self.dst = torch.full((len(lens), max(room + [1])), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        at = 0
        for b in range(len(lens)):
            self.table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            self.dst[b, :room[b]] = perm[at:at + room[b]]
            at += room[b]
        if in_place:
            self.dst = self.table
        self.cache = torch.randint(0, 256, (blocks, Hkv, bs // 16, 18 * D), generator=g, device="cuda").to(torch.uint8)
        self.mass = torch.rand(blocks, Hkv, bs, generator=g, device="cuda").pow(6)
        if ties:
            self.mass = (self.mass * 4).floor() / 4
        self.max_keep = max_keep or max(keep + [1])
        self.kept = torch.full((len(lens), Hkv, self.max_keep), -3, dtype=torch.int32, device="cuda")
        self.out = torch.full((len(lens),), -3, dtype=torch.int32, device="cuda")
        self.err = _native.new_error_word()

    def run(self, stream=None):
        _native.kv_evict(self.cache, self.mass, self.table, self.dst, dev(self.lens), dev(self.keep), self.kept, self.out,
                         self.err, sinks=self.sinks, recent=self.recent, stream=stream)

    def slots(self, table, b, j):
        t = table[b].long()[j // self.bs]
        return t, j % self.bs

    def want(self, skip=()):
        cache, mass, kept, out = self.cache.clone(), self.mass.clone(), self.kept.clone(), self.out.clone()
        for b, (n, k) in enumerate(zip(self.lens, self.keep)):
            if b in skip:
                out[b] = -1
                continue
            size = min(n, k)
            out[b] = size
            first = min(self.sinks, size)
            last = min(self.recent, size - first)
            j = torch.arange(n, device="cuda")
            blk, off = self.slots(self.table, b, j)
            for h in range(self.Hkv):
                m = self.mass[blk, h, off].tolist()
                key = lambda i: (-(float("-inf") if m[i] != m[i] else m[i]), m[i] != m[i], i)  # noqa: E731
                inner = sorted(range(first, n - last), key=key)
                keep = sorted(list(range(first)) + inner[:size - first - last] + list(range(n - last, n)))[:size]
                keep = dev(keep, torch.int64)
                kept[b, h, :size] = keep.int()
                sb, so = self.slots(self.table, b, keep)
                db, do = self.slots(self.dst, b, torch.arange(size, device="cuda"))
                mass[db, h, do] = self.mass[sb, h, so]
                for dst, src in zip(au.fields(cache, self.D), au.fields(self.cache, self.D)):
                    dst[db, h, do // 16, do % 16] = src[sb, h, so // 16, so % 16]
        return cache, mass, kept, out

    def check(self, skip=(), want_err=0):
        want = self.want(skip)
        self.run()
        torch.cuda.synchronize()
        assert int(self.err.item()) == want_err
        got = self.cache, self.mass.view(torch.int32), self.kept, self.out
        want = want[0], want[1].view(torch.int32), want[2], want[3]
        for name, a, b in zip(("cache", "mass", "kept", "lengths"), got, want):
            assert torch.equal(a, b), name


EVICTS = [dict(lens=[1], keep=[1]), dict(lens=[2], keep=[1]), dict(lens=[0, 5], keep=[3, 0]), dict(lens=[17, 16, 15], keep=[16, 16, 16]),
          dict(lens=[1000, 40, 300], keep=[100, 100, 299], sinks=4, recent=32), dict(lens=[5000], keep=[1024], sinks=4, recent=64),
          dict(lens=[777, 778], keep=[500, 1], sinks=3, recent=10), dict(lens=[100], keep=[60], sinks=80), dict(lens=[100], keep=[60], recent=80),
          dict(lens=[100], keep=[60], sinks=30, recent=30), dict(lens=[20000], keep=[9000], recent=5),
          dict(lens=[65 * b % 700 for b in range(90)], keep=[50 + b for b in range(90)], sinks=2, recent=8)]


@pytest.mark.parametrize("case", range(len(EVICTS)))
@pytest.mark.parametrize("Hkv, D, bs", [(2, 64, 16), (3, 128, 32)])
def test_evict(case, Hkv, D, bs):
    for in_place in (False, True):
        Evict(Hkv=Hkv, D=D, bs=bs, seed=case, in_place=in_place, **EVICTS[case]).check()
    Evict(Hkv=Hkv, D=D, bs=bs, seed=case, in_place=True, ties=True, **EVICTS[case]).check()


def test_evict_many_pairs():
    # more pairs of request and head than CTAs at once
    Evict([50 + b % 77 for b in range(200)], [40] * 200, 16, 64, seed=1, in_place=True, recent=3).check()


def test_evict_more_keys_than_shared_memory_holds():
    for in_place in (False, True):
        Evict([800000], [3001], 1, 64, bs=64, seed=6, sinks=4, recent=50, in_place=in_place, ties=in_place).check()


def test_evict_special_weights():
    e = Evict([600, 600], [300, 300], 2, 64, seed=2, sinks=1, recent=1)
    blk, off = e.slots(e.table, 0, torch.arange(600, device="cuda"))
    nan, inf = float("nan"), float("inf")
    e.mass[blk[:400], 0, off[:400]] = nan        # the numbers first, then the first NaNs
    e.mass[blk[::3], 1, off[::3]] = inf
    e.mass[blk[1::3], 1, off[1::3]] = -inf
    blk, off = e.slots(e.table, 1, torch.arange(600, device="cuda"))
    e.mass[blk, 0, off] = 0.0                    # all alike, zeros of both signs: the first ones
    e.mass[blk[::2], 0, off[::2]] = -0.0
    e.mass[blk, 1, off] = torch.linspace(-1e-45, 3e38, 600, device="cuda")
    e.check()


def test_evict_part_in_place():
    # the first pages stay where they are, the others go to new ones
    e = Evict([400], [200], 2, 64, seed=3)
    e.dst[0, :5] = e.table[0, :5]
    e.check()


def test_evict_refuses_sizes_and_pages():
    base = dict(lens=[100, 100, 100, 100, 100, 100], keep=[50] * 6, Hkv=2, D=64)
    e = Evict(seed=4, **base)
    e.lens = [100, -1, 100, 10 ** 6, 100, 100]
    e.keep = [50, 50, -2, 50, 50, 50]
    e.check(skip=(1, 2, 3), want_err=_native.ERR_PARAM)
    e = Evict(seed=4, **base)
    e.table[1, 6] = -1
    e.table[2, 0] = e.cache.shape[0]
    e.dst[4, 3] = 2 ** 31 - 1
    e.check(skip=(1, 2, 4), want_err=_native.ERR_BLOCK_RANGE)
    e = Evict(seed=4, max_keep=49, **base)  # more than kept has room for
    e.check(skip=tuple(range(6)), want_err=_native.ERR_PARAM)


# ------------------------------------------------------------------- together
def chain(seed, graph=False):
    """Append, attend, weigh, evict in place, append at the new lengths, attend: as a decode loop does."""
    g = gen(seed)
    B, Hq, Hkv, D, bs, n, keep = 3, 16, 2, 64, 16, 200, 96
    cache = pe.new_kv_cache(B * 20, bs, Hkv, D)
    mass = pe.new_kv_mass(cache)
    table = torch.randperm(B * 20, generator=g, device="cuda").to(torch.int32).view(B, 20)
    rope = pe.rope_table(n + 8, D)
    err, aws = pe.new_error_word(), pe.new_attn_workspace(D)
    wws = pe.new_weigh_workspace(B * n, Hq, 20, bs)
    state = dict(cache=cache, mass=mass, table=table, err=err)
    q, k, v = (torch.randn(B * n, h, D, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B)
    req = torch.arange(B, device="cuda").repeat_interleave(n)
    slots = table[req, pos.long() // bs].long() * bs + pos % bs
    out = torch.empty_like(q)
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    size = torch.empty(B, dtype=torch.int32, device="cuda")
    lens, budget = dev([n] * B), dev([keep] * B)
    q1, k1, v1 = (torch.randn(B, h, D, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    true_pos, out1, zero = dev([n] * B), torch.empty(B, Hq, D, dtype=BF, device="cuda"), dev([0] * B)
    r1 = torch.empty_like(q1)
    qr = torch.empty_like(q)

    def steps():
        pe.kv_append(q, k, v, pos, slots, rope, cache, qr, err)
        pe.attn_cached(qr, cache, table, None, pos, None, out, aws, err)
        pe.kv_weigh(qr, cache, table, None, pos, None, mass, mass, wws, err, fresh=zero)
        pe.kv_evict(cache, mass, table, table, lens, budget, kept, size, err, sinks=2, recent=16)
        at = table.gather(1, (size // bs).long()[:, None])[:, 0].long() * bs + size % bs
        pe.kv_append(q1, k1, v1, true_pos, at, rope, cache, r1, err)
        pe.attn_cached(r1, cache, table, None, size, None, out1, aws, err)
        pe.kv_weigh(r1, cache, table, None, size, None, mass, mass, wws, err, fresh=size)

    if graph:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            steps()
        torch.cuda.current_stream().wait_stream(s)
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            steps()
        kept.fill_(-1), out1.zero_(), mass.fill_(7.0)
        cg.replay()
    else:
        steps()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return dict(state, kept=kept, size=size, out=out, out1=out1, r1=r1, q=qr, pos=pos, req=req, slots=slots, k=k, v=v, rope=rope,
                D=D, bs=bs, n=n, keep=keep, Hkv=Hkv, Hq=Hq, B=B, pages=table)


def test_chain():
    c = chain(1)
    D, bs, n, keep, Hkv, B = c["D"], c["bs"], c["n"], c["keep"], c["Hkv"], c["B"]
    assert c["size"].tolist() == [keep] * B
    kr = au.to_bf16(au.rotated(c["k"], c["rope"], c["pos"], False)[0])
    kq, vq = au.quantised(kr), au.quantised(c["v"])
    for b in range(B):
        r = slice(b * n, (b + 1) * n)
        G = c["Hq"] // Hkv
        t = torch.arange(keep + 1, device="cuda")
        slots = c["pages"][b].long()[t // bs] * bs + t % bs
        hk, hv = au.held(c["cache"], D, slots)
        for h in range(Hkv):
            s = torch.einsum("mgd,ld->mgl", c["q"][r, h * G:(h + 1) * G].double(), kq[r, h]) * D ** -0.5
            s = s.masked_fill(t.new_tensor(range(n)) > torch.arange(n, device="cuda")[:, None, None], -float("inf"))
            w = torch.softmax(s, -1).sum((0, 1))
            got = c["kept"][b, h].long()
            # the first two and the last sixteen; of the others no evicted key is heavier than a kept one by more than
            # the weights' own error (1e-4 of themselves: as in the weights' tests, for scores of magnitude up to 40)
            assert got[:2].tolist() == [0, 1] and got[-16:].tolist() == list(range(n - 16, n))
            gone = torch.ones(n, dtype=torch.bool, device="cuda")
            gone[got] = False
            assert float(w[gone].max()) <= float(w[got[2:-16]].min()) * (1 + 1e-4)
            # what is held is what was appended, bit for bit
            assert torch.equal(hk[:keep, h], kq[r, h][got]) and torch.equal(hv[:keep, h], vq[r, h][got])
        # attention of the next token over the kept keys and its own
        want, tol = au.attention(c["r1"][b:b + 1], hk, hv, dev([keep + 1], torch.int64), D ** -0.5)
        au.within(c["out1"][b:b + 1], want, tol)


def test_chain_in_a_graph():
    a, b = chain(2), chain(2, graph=True)
    for name in ("cache", "kept", "size", "out", "out1"):
        assert torch.equal(a[name], b[name]), name
    live = [a["pages"][i, :7] for i in range(a["B"])]
    for p in live:  # slots of the kept keys and the new one
        assert torch.equal(a["mass"][p.long()].flatten(2)[:6], b["mass"][p.long()].flatten(2)[:6])


def test_another_stream():
    s = torch.cuda.Stream()
    e, f = (Evict([500, 60], [100, 100], 2, 64, seed=9, recent=7) for _ in range(2))
    w, x = (Weigh([[500, 499], [60, 0]], 8, 2, 64, seed=9) for _ in range(2))
    o, r = torch.zeros_like(w.mass), torch.zeros_like(w.mass)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        e.run(stream=s)
        w.run(o, stream=s)
    s.synchronize()
    f.run()
    x.run(r)
    torch.cuda.synchronize()
    assert torch.equal(e.kept, f.kept) and torch.equal(e.cache, f.cache) and torch.equal(o, r)


def test_two_calls_at_once():
    # (many columns in one launch beside a single token's chunks, each with a workspace of its own)
    both = [Weigh([[3000 + 7 * i, 2999] for i in range(9)], 16, 2, 64, seed=41),
            Weigh([[9000 + 13 * i] for i in range(50)], 8, 4, 128, seed=42)]
    want = [torch.zeros_like(w.mass) for w in both]
    got = [torch.zeros_like(w.mass) for w in both]
    for w, o in zip(both, want):
        w.run(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(8):
        for w, o, s in zip(both, got, streams):
            w.run(o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
