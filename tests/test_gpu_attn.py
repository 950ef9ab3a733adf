"""Attention over the 4-bit paged cache and over packed prompts, on the GPU,
against the formulas in 64 bits (tolerances: attn_util.attention)."""
import pytest
import torch

import attn_util as u
from speculative_decoding_pe_gb300 import _native

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def dev(x, dt=torch.int32):
    return torch.tensor(x, dtype=dt, device="cuda")


class Cached:
    """Requests with given row limits over a shuffled cache whose unused slots
    hold bytes of all ones (every scale a NaN) and whose table ends in ids of no
    page."""

    def __init__(self, limits, Hq, Hkv, D, bs=16, seed=0, q_std=2.0, uniform=False, extra=2):
        g = gen(seed)
        self.limits, self.D, self.bs = limits, D, bs
        T = sum(map(len, limits))
        width = max([max(r, default=0) for r in limits] + [1]) // bs + 1 + extra
        most = [max(r, default=0) for r in limits]
        need = [-(-n // bs) for n in most]
        blocks = sum(need) + 3
        perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(limits), width), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        live = u.random_cache(blocks, Hkv, bs, D, g)
        self.cache = torch.full_like(live, 255)
        at = 0
        self.kv = []
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
            t = torch.arange(most[b], device="cuda")
            slots = self.table[b].long()[t // bs] * bs + t % bs
            for dst, src in zip(u.fields(self.cache, D), u.fields(live, D)):
                dst[slots // bs, :, slots % bs // 16, slots % 16] = src[slots // bs, :, slots % bs // 16, slots % 16]
            self.kv.append(u.held(live, D, slots))
        self.q = (torch.randn(T, Hq, D, generator=g, device="cuda") * q_std).to(BF)
        flat = [n for r in limits for n in r]
        self.rej = dev([n == 0 for n in flat], torch.uint8)
        self.pos = dev([n - 1 if n else 7 for n in flat])
        offs = [0]
        for r in limits:
            offs.append(offs[-1] + len(r))
        self.offsets = None if uniform else dev(offs)
        self.scale = D ** -0.5
        self.ws = _native.new_attn_workspace(D)
        self.err = _native.new_error_word()
        self.out = torch.full((T, Hq, D), float("nan"), dtype=BF, device="cuda")

    def run(self, stream=None, out=None):
        out = self.out if out is None else out
        _native.attn_cached(self.q, self.cache, self.table, self.offsets, self.pos, self.rej, out, self.ws,
                            self.err, scale=self.scale, stream=stream)
        return out

    def check(self):
        out = self.run().clone()
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        at = 0
        for b, r in enumerate(self.limits):
            k, v = self.kv[b]
            sl = slice(at, at + len(r))
            at += len(r)
            want, tol = u.attention(self.q[sl], k, v, dev(r, torch.int64), self.scale)
            u.within(out[sl], want, tol, "request %d" % b)
            dead = [i for i, n in enumerate(r) if not n]
            assert not out[sl][dead].any()
        assert torch.equal(self.run(out=torch.empty_like(out)).view(torch.int16), out.view(torch.int16))


def draft(p, a, Kp=7, K=7):
    """Row limits of a draft batch: first position p, accepted length a."""
    return [p + k + 1 if k <= a else 0 for k in range(Kp + 1)] + [p + a + i + 1 for i in range(1, K)]


HEADS = [(64, 8, 64), (32, 4, 128), (32, 8, 128), (12, 12, 64), (20, 4, 64), (8, 1, 128), (3, 1, 64), (14, 2, 128),
         (128, 1, 64), (5, 5, 128)]


@pytest.mark.parametrize("Hq, Hkv, D", HEADS)
@pytest.mark.parametrize("bs", [16, 48])
def test_single_tokens(Hq, Hkv, D, bs):
    Cached([[n] for n in (1, 2, 15, 16, 17, 0, 63, 64, 65, 127, 128, 129, 1000)], Hq, Hkv, D, bs, 1, uniform=True).check()


@pytest.mark.parametrize("Hq, Hkv, D", HEADS)
@pytest.mark.parametrize("bs", [16, 32])
def test_draft_rows(Hq, Hkv, D, bs):
    Cached([draft(p, a) for p, a in ((0, 0), (1, 7), (120, 3), (500, 2), (127, 0), (128, 7))], Hq, Hkv, D, bs, 2,
           uniform=True).check()


@pytest.mark.parametrize("Hq, Hkv, D", HEADS[:6])
def test_ragged_segments(Hq, Hkv, D):
    lim = [[], [5], draft(300, 4), [0, 0, 0], list(range(1, 70)), [], [1000, 1, 700], [0] * 20 + [129], list(range(250, 600)), []]
    Cached(lim, Hq, Hkv, D, 16, 3).check()


@pytest.mark.parametrize("rows", [1, 2, 3, 14])
@pytest.mark.parametrize("Hq, Hkv, D", [(64, 8, 64), (32, 4, 128)])
def test_long_context_of_one_request(Hq, Hkv, D, rows):
    n = 40_000 + rows
    Cached([[n - rows + i + 1 for i in range(rows)]], Hq, Hkv, D, 16, 4, uniform=True).check()


@pytest.mark.parametrize("Hq, Hkv, D", [(64, 8, 64), (8, 1, 128)])
@pytest.mark.parametrize("one", [False, True])
def test_many_requests(Hq, Hkv, D, one):
    g = torch.Generator().manual_seed(5)
    p = torch.randint(0, 900, (300,), generator=g).tolist()
    Cached([[n] if one else draft(n, n % 8) for n in p], Hq, Hkv, D, 16, 6, uniform=True).check()


def test_all_rows_rejected():
    c = Cached([[0] * 5, [0] * 5], 8, 2, 64, uniform=True)
    c.check()
    assert not c.out.any()


@pytest.mark.parametrize("uniform", [False, True])
def test_without_flags_and_default_scale(uniform):
    c = Cached([[100], [37]], 8, 2, 64, uniform=uniform)
    c.rej, c.scale = None, None
    out = c.run()
    for b in range(2):
        k, v = c.kv[b]
        want, tol = u.attention(c.q[b:b + 1], k, v, dev([c.limits[b][0]], torch.int64), 0.125)
        u.within(out[b:b + 1], want, tol)


@pytest.mark.parametrize("std", [1e-4, 30.0, 1e5])
@pytest.mark.parametrize("rows", [1, 14])
def test_small_and_large_queries(std, rows):
    """bf16 reaches past every 16-bit format's range; peaked and flat weights."""
    c = Cached([[600 + i for i in range(rows)]], 16, 2, 64, uniform=True, q_std=std)
    c.scale = 0.125 * min(1.0, 30.0 / std)
    c.check()


@pytest.mark.parametrize("rows", [1, 14])
def test_queries_of_very_different_elements(rows):
    c = Cached([[600 + i for i in range(rows)]], 16, 2, 64, uniform=True)
    g = gen(9)
    c.q *= (10.0 ** torch.randint(-12, 3, c.q.shape, generator=g, device="cuda")).to(BF)
    c.scale = 1e-3
    c.check()


@pytest.mark.parametrize("rows", [1, 14])
def test_rising_and_falling_scores(rows):
    """Scores that climb along the context by more than any kept maximum, and ones that fall."""
    for sign in (1.0, -1.0):
        c = Cached([[900] * rows], 8, 1, 64, uniform=True, q_std=0.0)
        c.q[..., 0] = sign * 8.0
        t = torch.arange(900, device="cuda")
        slots = c.table[0].long()[t // 16] * 16 + t % 16
        f = u.fields(c.cache, 64)
        f[0][slots // 16, :, 0, slots % 16, 0] = 0x06  # element 0: code 4.0
        sc = (t.float() / 900 * 20 + 0.02).to(torch.float8_e4m3fn).view(torch.uint8)
        f[2][slots // 16, :, 0, slots % 16, 0] = sc[:, None]
        c.kv[0] = u.held(c.cache, 64, slots)
        c.scale = 1.0
        c.check()


@pytest.mark.parametrize("rows", [1, 14])
@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_pages_outside_the_cache_are_left_out(rows, bad):
    n = 500
    c = Cached([[n] * rows, [n - 3] * rows], 16, 2, 64, uniform=True)
    for b, page in ((0, 0), (0, 7), (1, 31), (1, 13)):
        c.table[b, page] = bad
        k, v = c.kv[b]
        keep = torch.arange(k.shape[0], device="cuda") // 16 != page
        c.kv[b] = [k.masked_fill(~keep[:, None, None], float("nan")), v]
    out = c.run()
    torch.cuda.synchronize()
    assert int(c.err.item()) == _native.ERR_BLOCK_RANGE
    for b in range(2):
        k, v = c.kv[b]
        keep = ~k[:, 0, 0].isnan()
        keep[c.limits[b][0]:] = False
        want, tol = u.attention(c.q[b * rows:(b + 1) * rows], k[keep], v[keep], dev([int(keep.sum())] * rows, torch.int64), c.scale)
        u.within(out[b * rows:(b + 1) * rows], want, tol)


@pytest.mark.parametrize("rows", [1, 14])
def test_positions_outside_the_table(rows):
    c = Cached([[33] * rows, [64] * rows], 16, 2, 64, uniform=True, extra=0)
    assert c.table.shape[1] == 5
    c.table = c.table[:, :4].contiguous()
    c.pos[rows:] = 90        # sees the 64 keys of the table
    c.pos[0] = -5            # sees nothing
    out = c.run()
    torch.cuda.synchronize()
    assert int(c.err.item()) == _native.ERR_BLOCK_RANGE
    assert not out[0].any()
    k, v = c.kv[1]
    want, tol = u.attention(c.q[rows:], k, v, dev([64] * rows, torch.int64), c.scale)
    u.within(out[rows:], want, tol)


@pytest.mark.parametrize("offs", [[1, 3, 6], [0, 7, 6], [0, 3, 5], [0, 3, 7], [0, -1, 6]])
def test_offsets_that_are_no_partition(offs):
    c = Cached([[30] * 3, [40] * 3], 8, 2, 64)
    c.offsets = dev(offs)
    out = c.run()
    torch.cuda.synchronize()
    assert int(c.err.item()) == _native.ERR_OFFSETS and bool(out.isnan().all())
    p = Prompt([3, 3], 8, 2, 64)
    p.offsets = dev(offs)
    out = p.run()
    torch.cuda.synchronize()
    assert int(p.err.item()) == _native.ERR_OFFSETS and bool(out.isnan().all())


class Prompt:
    def __init__(self, lens, Hq, Hkv, D, seed=0, fused=True, std=1.5, uniform=False):
        g = gen(seed)
        T = sum(lens)
        self.lens, self.D = lens, D
        if fused:
            w = (torch.randn(T, (Hq + 2 * Hkv) * D + 16, generator=g, device="cuda") * std).to(BF)
            self.q = w[:, :Hq * D].unflatten(1, (Hq, D))
            self.k = w[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
            self.v = w[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].unflatten(1, (Hkv, D))
        else:  # heads outside rows: [H, T, D] seen as [T, H, D]
            self.q, self.k, self.v = ((torch.randn(h, T, D, generator=g, device="cuda") * std).to(BF).transpose(0, 1)
                                      for h in (Hq, Hkv, Hkv))
        offs = [0]
        for n in lens:
            offs.append(offs[-1] + n)
        self.offsets = None if uniform else dev(offs)
        self.ws, self.err = _native.new_attn_workspace(D), _native.new_error_word()
        self.out = torch.full((T, Hq, D), float("nan"), dtype=BF, device="cuda")

    def run(self, stream=None, out=None):
        out = self.out if out is None else out
        _native.attn_prompt(self.q, self.k, self.v, self.offsets, out, self.ws, self.err, B=len(self.lens), stream=stream)
        return out

    def check(self, rows=None):
        out = self.run().clone()
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        at = 0
        for b, n in enumerate(self.lens):
            sl = slice(at, at + n)
            at += n
            lim = torch.arange(1, n + 1, device="cuda")
            pick = lim - 1 if n <= 1500 else torch.cat((lim[:200], lim[n // 2:n // 2 + 200], lim[-300:])) - 1
            want, tol = u.attention(self.q[sl][pick], self.k[sl].double(), self.v[sl].double(), lim[pick], self.D ** -0.5)
            u.within(out[sl][pick], want, tol, "prompt %d" % b)
        assert torch.equal(self.run(out=torch.empty_like(out)).view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("Hq, Hkv, D", HEADS)
@pytest.mark.parametrize("fused", [True, False])
def test_prompts(Hq, Hkv, D, fused):
    Prompt([1, 0, 2, 31, 32, 33, 127, 128, 129, 0, 255, 256, 257, 700, 0], Hq, Hkv, D, 1, fused).check()


@pytest.mark.parametrize("Hq, Hkv, D", [(64, 8, 64), (32, 4, 128), (2, 2, 64)])
def test_long_prompts(Hq, Hkv, D):
    Prompt([5001, 9, 3333], Hq, Hkv, D, 2).check()


@pytest.mark.parametrize("lens", [[1], [0, 1], [1] * 400, [7] * 100, [0, 0, 40]])
def test_short_prompts(lens):
    Prompt(lens, 16, 2, 64, 3, uniform=len(set(lens)) == 1).check()


def test_large_scores():
    Prompt([300, 500], 8, 2, 64, 4, std=12.0).check()
    Prompt([300, 500], 8, 2, 128, 4, std=1e-3).check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_masked_places_may_hold_anything(D, what):
    """A key or value that a row does not see does not touch it: not the next
    request's, not a later one of its own."""
    lens = [70, 200, 300]
    p = Prompt(lens, 8, 2, D, 5)
    want = p.run().clone()
    for t in (70, 70 + 150, 270 + 17, 270 + 299):  # rows from here on, of the same request, see it
        p = Prompt(lens, 8, 2, D, 5)
        p.k[t], p.v[t, :, 3:50:7] = what, what
        got = p.run()
        torch.cuda.synchronize()
        end = 270 if t < 270 else 570
        clean = torch.ones(570, dtype=torch.bool, device="cuda")
        clean[t:end] = False
        assert torch.equal(got[clean].view(torch.int16), want[clean].view(torch.int16)), t


def test_values_that_are_not_finite_reach_the_rows_that_see_them():
    for t in (5, 290):
        p = Prompt([300], 4, 2, 64, 6)
        p.v[t, 0, 9] = float("inf")
        p.v[t, 1, 11] = float("nan")
        got = p.run()
        torch.cuda.synchronize()
        assert bool((got[t:, :2, 9] == float("inf")).all()) and bool(got[t:, 2:, 11].isnan().all())
        got[t:, :2, 9], got[t:, 2:, 11] = 0, 0
        assert bool(got.isfinite().all())


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("kind", ["token", "draft", "prompt"])
def test_a_query_that_is_not_finite_keeps_to_its_row(kind, what):
    """Its row is NaN, whole or put together from parts of a long context; the others are as they were."""
    make = lambda: (Prompt([3000, 40], 8, 2, 64, 7) if kind == "prompt" else  # noqa: E731
                    Cached([[9000], [33]] if kind == "token" else [draft(9000, 3), draft(33, 7)], 8, 2, 64, seed=7, uniform=True))
    want = make().run().clone()
    c = make()
    rows = (2990, 3000) if kind == "prompt" else (0, 1) if kind == "token" else (1, 15)
    for t in rows:
        c.q[t, 5, 7] = what
    got = c.run()
    torch.cuda.synchronize()
    for t in rows:
        assert bool(got[t, 5].isnan().all())
        got[t, 5] = want[t, 5]
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("kind", ["token", "draft", "prompt"])
def test_streams_graphs_and_a_reused_workspace(kind):
    """One workspace through calls of changing size, on another stream, and in
    a captured graph whose inputs change between replays."""
    ws = _native.new_attn_workspace(128)

    def make(seed, big):
        if kind == "prompt":
            return Prompt([500, 20, 900] if big else [5, 33], 8, 2, 64, seed)
        rows = [[1500 + 31 * i] if kind == "token" else draft(700 + 40 * i, i % 8) for i in range(9 if big else 2)]
        return Cached(rows, 8, 2, 64, seed=seed, uniform=True)

    for seed, big in ((1, True), (2, False), (3, True)):
        c = make(seed, big)
        c.ws = ws
        c.check()
    want = c.run().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.out.fill_(float("nan"))
    torch.cuda.synchronize()
    c.run(stream=s)
    s.synchronize()
    assert torch.equal(c.out.view(torch.int16), want.view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    other = make(4, True)
    w2 = other.run().clone()
    c.q.copy_(other.q)
    if kind == "prompt":
        c.k.copy_(other.k), c.v.copy_(other.v)
    else:
        c.cache.copy_(other.cache), c.table.copy_(other.table)
    for _ in range(2):
        c.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out.view(torch.int16), w2.view(torch.int16))


def test_binding_refusals():
    c = Cached([[30], [40]], 8, 2, 64, uniform=True)
    good = dict(q=c.q, cache=c.cache, block_table=c.table, offsets=None, positions=c.pos, is_rejected=c.rej, out=c.out,
                workspace=c.ws, err=c.err)
    for name, bad, kind in (("q", c.q.float(), TypeError), ("q", c.q[:, :, :32], ValueError), ("out", c.out[:1], ValueError),
                            ("positions", c.pos[:1], ValueError), ("positions", c.pos.long(), TypeError),
                            ("cache", c.cache.int(), ValueError), ("workspace", c.ws[:64], ValueError),
                            ("offsets", dev([0, 2]), ValueError), ("is_rejected", c.rej[:1], ValueError),
                            ("block_table", c.table[0], ValueError), ("scale", float("nan"), _native.PEError)):
        with pytest.raises(kind):
            _native.attn_cached(**{**good, name: bad})
