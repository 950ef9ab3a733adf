"""Sampling from filtered rows and its verification, on the GPU, against the
definitions in 64 bits.

Tolerances: the kernels' weights and sums carry some 32 bits (2^-31 is the
largest rounding of a weight, and sums are exact beside it), so a running sum is
within 2^-30 of the exact one; a draw whose u is within 2^-29 of a border between
columns is not compared.  A probability is rounded to fp32: half a step, 2^-24, and
2^-29 for the quotient of two sums."""
import pytest
import torch

import filter_util as f
from speculative_decoding_pe_gb300 import _native

pytestmark = pytest.mark.gpu
NEAR = 2.0 ** -29
BF, FP = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def vec(v, dt=FP):
    return torch.tensor(v, dtype=dt, device="cuda")


ASKS = [(1.0, 0, 1.0, 0.0), (0.7, 20, 0.8, 0.0), (0.0, 0, 1.0, 0.0), (0.8, 0, 0.95, 0.0), (1.3, 0, 1.0, 0.05),
        (0.9, 300, 0.9, 0.02), (1.0, 1, 1.0, 0.0), (2.0, 0, 0.999, 0.0), (1.0, 3, 0.0, 0.0), (1.0, 0, 1.0, 1.0),
        (0.5, 257, 1.0, 0.0), (1.0, 0, 0.3, 0.5), (1.4, 30, 0.97, 0.3), (3.0, 250, 0.9, 0.5), (3.0, 600, 0.95, 0.4), (1e-6, 0, 1.0, 0.0), (1e6, 0, 0.5, 0.0), (1.0, 256, 2.0, -1.0)]


def asked(rows):
    t, k, p, m = zip(*rows)
    return dict(temperature=vec(t), top_k=vec(k, torch.int32), top_p=vec(p), min_p=vec(m))


def sample(x, rows, u, stream=None, sample_idx=None, want_err=0):
    n = u.numel()
    tok = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((n,), 9.0, device="cuda")
    err = _native.new_error_word()
    _native.draft_sample(x, u, tok, err, out_prob=prob, sample_idx=sample_idx, stream=stream, **asked(rows))
    torch.cuda.synchronize()
    assert int(err.item()) == want_err
    return tok.tolist(), prob.tolist()


def check(x, rows, u, tok, prob, idx=None):
    per = len(tok) // len(rows)
    compared = 0
    for i, c in enumerate(tok):
        z = f.probabilities(x[idx[i] if idx else i], *rows[i // per])
        want, gap = f.draw(z, u[i])
        if gap < NEAR:
            continue
        compared += 1
        assert c == want, "row %d: column %d, not %d" % (i, c, want)
        assert abs(prob[i] - float(z[c])) <= (2.0 ** -24 + 2.0 ** -29) * float(z[c]), "row %d" % i
    return compared


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 100, 257, 1000, 4099, 20011])
def test_rows_of_any_width(V, dtype):
    g = gen(V)
    n = 2 * len(ASKS)
    x = f.pitched(f.peaked(n, V, g, dtype))
    u = torch.rand(n, generator=g, device="cuda")
    u[:2] = vec([0.0, 1.0 - 2.0 ** -24])
    tok, prob = sample(x, ASKS, u)
    assert check(x, ASKS, u.tolist(), tok, prob) >= n - 2


@pytest.mark.parametrize("V, dtype, n", [(151936, BF, 15), (201088, BF, 15), (201088, FP, 15), (262144, FP, 1),
                                         (262144, BF, 3), (151936, BF, 300)])
def test_wide_rows(V, dtype, n):
    g = gen(V + n)
    x = f.peaked(n, V, g, dtype)
    u = torch.rand(n, generator=g, device="cuda")
    rows = (ASKS * 20)[:n]
    tok, prob = sample(x, rows, u)
    few = list(range(n)) if n < 20 else [0, 3, 4, 7, 150, 299]  # (the statement is slow)
    for i in few:
        check(x[i:i + 1], [rows[i]], [float(u[i])], [tok[i]], [prob[i]])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_ties_go_to_the_lowest_columns(dtype):
    # every column alike; two values; the cut's value at many columns
    V = 5003
    x = torch.zeros(6, V, device="cuda")
    x[1, ::3] = 1.0
    x[2, :] = -4.0
    x[3, 100:4000] = 2.0
    x[4] = torch.arange(V, device="cuda") % 7
    x[5] = -(torch.arange(V, device="cuda") % 5).float() * 0.0  # zeros of both signs
    x = f.pitched(x.to(dtype))
    rows = [(1.0, 50, 1.0, 0.0), (1.0, 2000, 1.0, 0.0), (1.0, 0, 0.37, 0.0), (1.0, 300, 0.5, 0.0), (1.0, 1000, 0.9, 0.1),
            (1.0, 1500, 0.2, 0.0)]
    for u in (0.0, 0.25, 0.8, 0.99999):
        tok, prob = sample(x, rows, vec([u] * 6))
        # u * n lies on a border between equal columns for some of these: those are within NEAR
        check(x, rows, [u] * 6, tok, prob)
    tok, _ = sample(x, [(1.0, 2000, 1.0, 0.0)] * 6, vec([1.0 - 2.0 ** -24] * 6))
    assert tok[0] == 1999 and tok[2] == 1999 and tok[5] == 1999


def test_flat_rows_with_every_column_kept():
    g = gen(3)
    V, n = 151936, 12
    x = torch.randn(n, V, generator=g, device="cuda").to(BF)
    u = torch.rand(n, generator=g, device="cuda")
    rows = [(1.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 0.99, 0.01), (1.0, 70000, 0.8, 0.0)] * 3
    tok, prob = sample(x, rows, u)
    assert check(x, rows, u.tolist(), tok, prob) >= n - 1


@pytest.mark.parametrize("dtype", [BF, FP])
def test_wide_cuts(dtype):
    # cuts among thousands of columns, and lists longer than the kernel's
    g = gen(7)
    rows = [(1.0, 2000, 1.0, 0.0), (3.0, 0, 0.9, 0.0), (3.0, 0, 0.5, 0.2), (2.0, 30000, 0.8, 0.01), (1.0, 1000, 0.95, 0.0),
            (1.0, 0, 0.9999, 0.0), (1.0, 0, 0.9999999, 0.0), (1.0, 50304, 0.999, 0.0), (50.0, 0, 1e-6, 0.0), (1.0, 1, 0.5, 0.0),
            (0.01, 0, 0.99, 0.0), (1.0, 256, 0.999, 0.0), (1.0, 255, 1.0, 0.9)]
    x = f.peaked(len(rows), 50304, g, dtype)
    x[5, :40000] = 3.0  # a tie of most columns
    u = torch.rand(len(rows), generator=g, device="cuda")
    tok, prob = sample(x, rows, u)
    assert check(x, rows, u.tolist(), tok, prob) >= len(rows) - 1


def test_masked_infinite_and_nan_logits():
    V = 3001
    inf, nan = float("inf"), float("nan")
    x = f.pitched(torch.full((9, V), -inf, device="cuda"))
    x[0, 17] = -1e30                         # one column left
    x[1, 5:40] = torch.linspace(-2, 2, 35)   # a window
    x[2, :] = 0.0
    x[2, 100:] = torch.finfo(FP).min         # the type's lowest value
    x[3, 7], x[3, 9], x[3, 2000] = inf, 3.0, inf
    x[4, :50] = 1.0
    x[4, 3:20] = nan
    x[5, :] = nan                            # nothing
    x[7, 1000:1010] = 5.0
    x[8, :3] = torch.tensor([-inf, nan, 0.5])
    for rows in ([(1.0, 0, 1.0, 0.0)] * 9, [(0.5, 40, 0.9, 0.0)] * 9, [(0.5, 1000, 0.9, 0.1)] * 9, [(0.0, 0, 1.0, 0.0)] * 9):
        for u in (0.0, 0.3, 0.9):
            tok, prob = sample(x[:5], rows[:5], vec([u] * 5))
            check(x[:5], rows[:5], [u] * 5, tok, prob)
            tok, prob = sample(x, rows, vec([u] * 9), want_err=_native.ERR_EMPTY_ROW)
            assert tok[5] == -1 and tok[6] == -1 and prob[5] == 0 and prob[6] == 0
            assert tok[8] == 2 and prob[8] == 1.0 and 1000 <= tok[7] < 1010


def test_parameters_that_are_not_usable():
    nan, inf = float("nan"), float("inf")
    x = f.pitched(f.peaked(10, 100, gen(1)))
    rows = [(nan, 0, 1.0, 0.0), (-1.0, 0, 1.0, 0.0), (inf, 0, 1.0, 0.0), (1e-12, 0, 1.0, 0.0), (1.0, 0, nan, 0.0),
            (1.0, 0, 1.0, nan), (1.0, 5, 1.0, 0.0), (1.0, 5, 1.0, 0.0), (1.0, 5, 1.0, 0.0), (1.0, -3, 1.0, 0.0)]
    tok, prob = sample(x, rows, vec([0.5] * 6 + [nan, 1.0, -0.25, 0.5]), want_err=_native.ERR_PARAM)
    assert tok[:9] == [-1] * 9 and prob[:9] == [0.0] * 9 and tok[9] >= 0


def test_row_indices_defaults_and_shared_parameters():
    g = gen(8)
    x = f.pitched(f.peaked(9, 999, g))
    u = torch.rand(6, generator=g, device="cuda")
    idx = [8, 0, 3, 3, 7, 1]
    rows = [(0.7, 20, 0.8, 0.0), (1.0, 0, 1.0, 0.0)]
    tok, prob = sample(x, rows, u, sample_idx=vec(idx, torch.int32))
    assert check(x, rows, u.tolist(), tok, prob, idx) == 6
    tok, _ = sample(x, rows, u, sample_idx=vec([8, 9, -1, 3, 2 ** 31 - 1, 1], torch.int32), want_err=_native.ERR_ROW_RANGE)
    assert [t < 0 for t in tok] == [False, True, True, False, True, False]
    # no parameters at all: the plain distribution; no probabilities
    out, err = torch.empty(9, dtype=torch.int32, device="cuda"), _native.new_error_word()
    u = torch.rand(9, generator=g, device="cuda")
    _native.draft_sample(x, u, out, err)
    assert out.tolist() == [f.draw(f.probabilities(r), v)[0] for r, v in zip(x, u.tolist())]
    _native.draft_sample(x[:0], u[:0], out[:0], err)  # nothing to do


def test_shares_of_draws():
    # evenly spaced u: every column gets its share, to one draw
    x = f.peaked(1, 500, gen(2))
    n = 4096
    u = (torch.arange(n, device="cuda") + 0.5) / n
    tok = torch.empty(n, dtype=torch.int32, device="cuda")
    err = _native.new_error_word()
    idx = torch.zeros(n, dtype=torch.int32, device="cuda")
    _native.draft_sample(x, u, tok, err, top_k=vec([30], torch.int32), sample_idx=idx)
    share = torch.bincount(tok.long().cpu(), minlength=500).double()
    z = f.probabilities(x[0], k=30)
    assert float((share - n * z).abs().max()) <= 1.0 + 1e-6
    assert bool((tok[1:] >= tok[:-1]).all())


# ------------------------------------------------------------------ verification
class Verify:
    def __init__(self, B, Kp, V, rows, seed, dtype=BF, noise=0.7):
        g = gen(seed)
        self.B, self.Kp, self.V, self.rows = B, Kp, V, rows
        self.target = f.pitched(f.peaked(B * (Kp + 1), V, g, dtype))
        d = self.target.view_as(self.target).float()
        keep = torch.arange(B * (Kp + 1), device="cuda") % (Kp + 1) < Kp
        d = d[keep] + noise * torch.randn(B * Kp, V, generator=g, device="cuda")
        self.draft = f.pitched(d.to(dtype))
        self.tokens = torch.zeros(B, Kp + 1, dtype=torch.int32, device="cuda")
        if Kp:
            t = torch.empty(B * Kp, dtype=torch.int32, device="cuda")
            err = _native.new_error_word()
            _native.draft_sample(self.draft, torch.rand(B * Kp, generator=g, device="cuda"), t, err, **asked(rows))
            assert int(err.item()) == 0
            self.tokens[:, 1:] = t.view(B, Kp)
        self.coins = torch.rand(B * Kp, generator=g, device="cuda")
        self.u = torch.rand(B, generator=g, device="cuda")
        self.acc = torch.full((B,), -7, dtype=torch.int32, device="cuda")
        self.bonus = torch.full((B,), -7, dtype=torch.int32, device="cuda")
        self.chance = torch.full((B * Kp,), 9.0, device="cuda")
        self.ws = _native.new_filtered_workspace(B, Kp)
        self.ws.fill_(255)  # its content does not matter
        self.err = _native.new_error_word()

    def run(self, stream=None):
        _native.verify_filtered(self.target, self.draft, self.Kp, self.tokens, self.coins, self.u, self.acc, self.bonus,
                                self.ws, self.err, accept_prob=self.chance, stream=stream, **asked(self.rows))

    def check(self, want_err=0):
        self.run()
        torch.cuda.synchronize()
        assert int(self.err.item()) == want_err
        Kp, compared, rejected = self.Kp, 0, 0
        for b in range(self.B):
            a, near = Kp, False
            for j in range(Kp):
                x = int(self.tokens[b, j + 1])
                p = f.probabilities(self.target[b * (Kp + 1) + j], *self.rows[b])
                q = f.probabilities(self.draft[b * Kp + j], *self.rows[b])
                px, qx = (float(z[x]) if 0 <= x < self.V else 0.0 for z in (p, q))
                want = px / qx if px < qx else float(px > 0)
                assert abs(float(self.chance[b * Kp + j]) - want) <= (2.0 ** -24 + 2.0 ** -28) * want
                c = float(self.coins[b * Kp + j])
                if a == Kp:
                    near |= abs(c * qx - px) < 2.0 ** -28 * (px + qx)
                    if not c * qx < px:
                        a, rest, whole = j, (p - q).clamp(min=0), p
            if a == Kp:
                rest = whole = f.probabilities(self.target[b * (Kp + 1) + Kp], *self.rows[b])
            if near:
                continue
            assert int(self.acc[b]) == a, "request %d" % b
            rejected += a < Kp
            # p - q is off by at most 2^-30 of p + q, and so are its sums: against the rest's whole weight
            total = float(rest.sum())
            if float(whole.sum()) == 0:
                assert int(self.bonus[b]) == -1
                continue
            if total == 0:
                rest, total = whole, 1.0
            elif total < 1e-9:
                continue
            col, gap = f.draw(rest, float(self.u[b]))
            if gap * total < 2.0 ** -28:
                continue
            compared += 1
            assert int(self.bonus[b]) == col, "request %d" % b
        return compared, rejected


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B, Kp, V", [(15, 3, 1000), (30, 1, 97), (15, 7, 4099), (4, 0, 511), (2, 40, 203), (1, 7, 20011)])
def test_verify(B, Kp, V, dtype):
    v = Verify(B, Kp, V, (ASKS * 2)[:B], B + V, dtype)
    compared, rejected = v.check()
    assert compared >= B - 2 and (Kp < 3 or B < 10 or rejected > 0)


@pytest.mark.parametrize("V, dtype", [(151936, BF), (201088, FP)])
def test_verify_wide(V, dtype):
    v = Verify(5, 2, V, [ASKS[i] for i in (0, 1, 3, 4, 5)], 5, dtype, noise=1.0)
    compared, _ = v.check()
    assert compared >= 4


def test_verify_the_same_rows_accepts_everything():
    v = Verify(15, 4, 600, ASKS[:15], 9, noise=0.0)
    v.run()
    torch.cuda.synchronize()
    assert v.acc.tolist() == [4] * 15 and bool((v.chance == 1.0).all())
    # a coin at the top of its range still accepts p = q; a token that q cannot give and p does not keep is rejected,
    # and p - q of equal rows is zero everywhere: the bonus token comes from p
    v.tokens[:, 2] = torch.stack([v.target[5 * b + 1].argmin() for b in range(15)])
    v.coins.fill_(1.0 - 2.0 ** -24)
    v.rows = [(0.7, 20, 0.8, 0.0)] * 15
    compared, rejected = v.check()
    assert rejected == 15 and compared >= 14


def test_verify_from_rows_of_different_support():
    # target and draft keep disjoint columns: always rejected, and the bonus comes from p alone
    v = Verify(6, 2, 400, [(1.0, 5, 1.0, 0.0)] * 6, 11)
    v.draft[:, :200] = -50.0
    v.target[:, 200:] = -50.0
    v.tokens[:, 1:] = 300
    compared, rejected = v.check()
    assert rejected == 6 and compared >= 5 and bool((v.bonus < 200).all())


def test_verify_empty_rows_and_bad_tokens():
    v = Verify(6, 3, 300, [(0.9, 10, 0.9, 0.0)] * 6, 13)
    v.target[0 * 4 + 1] = float("-inf")  # an empty target row: its draft is rejected, no token
    v.draft[1 * 3 + 0] = float("nan")    # an empty draft row: q = 0
    v.tokens[2, 1] = 300                 # outside the vocabulary
    v.tokens[3, 2] = -1
    v.target[4 * 4 + 3] = float("-inf")  # an empty bonus row
    v.coins.fill_(0.0)                   # accepts wherever p(x) > 0
    v.check(want_err=_native.ERR_EMPTY_ROW)
    assert int(v.acc[0]) <= 1 and int(v.acc[2]) == 0 and int(v.acc[3]) <= 1
    assert int(v.bonus[0]) == -1 or int(v.acc[0]) == 0
    assert int(v.chance[2 * 3]) == 0


def test_verify_parameters_that_are_not_usable():
    rows = [(0.9, 10, 0.9, 0.0)] * 5
    v = Verify(5, 3, 300, rows, 17)
    v.rows = [(-1.0, 10, 0.9, 0.0)] + rows[1:]
    v.u[2] = 1.0
    v.run()
    torch.cuda.synchronize()
    assert int(v.err.item()) == _native.ERR_PARAM
    for b in (0, 2):
        assert int(v.acc[b]) == 0 and int(v.bonus[b]) == -1 and not bool(v.chance[3 * b:3 * b + 3].any())
    good = Verify(5, 3, 300, rows, 17)
    good.run()
    for b in (1, 3, 4):
        assert int(v.acc[b]) == int(good.acc[b]) and int(v.bonus[b]) == int(good.bonus[b])


def test_verify_keeps_the_target_distribution():
    # drafts by draft_sample and the verification's first token together: the target's filtered distribution
    V, n = 40, 1 << 14
    g = gen(21)
    t, d = f.peaked(1, V, g), f.peaked(1, V, g)
    u = torch.rand(n, generator=g, device="cuda")
    tok = torch.zeros(n, 2, dtype=torch.int32, device="cuda")
    first = torch.empty(n, dtype=torch.int32, device="cuda")
    err = _native.new_error_word()
    par = dict(top_k=torch.full((n,), 12, dtype=torch.int32, device="cuda"))
    D = d.expand(n, V).contiguous()
    _native.draft_sample(D, u, first, err, **par)
    tok[:, 1] = first
    acc, bonus = torch.empty_like(first), torch.empty_like(first)
    _native.verify_filtered(t.expand(2 * n, V).contiguous(), D, 1, tok, torch.rand(n, generator=g, device="cuda"),
                            torch.rand(n, generator=g, device="cuda"), acc, bonus, _native.new_filtered_workspace(n, 1), err,
                            **par)
    out = torch.where(acc > 0, first, bonus)
    share = torch.bincount(out.long(), minlength=V).cpu().double() / n
    z = f.probabilities(t[0], k=12)
    # six standard deviations of a share of n independent draws
    assert bool(((share - z).abs() <= 6 * (z * (1 - z) / n).sqrt()).all()) and int(err.item()) == 0


# -------------------------------------------------------------- streams, graphs
def test_another_stream_and_graph_replay():
    v = Verify(15, 3, 4099, ASKS[:15], 23)
    v.run()
    torch.cuda.synchronize()
    want = v.acc.clone(), v.bonus.clone(), v.chance.clone()
    s = torch.cuda.Stream()
    v.acc.fill_(-7), v.bonus.fill_(-7)
    s.wait_stream(torch.cuda.current_stream())
    v.run(stream=s)
    s.synchronize()
    assert torch.equal(v.acc, want[0]) and torch.equal(v.bonus, want[1])
    par, err = asked(ASKS[:15]), _native.new_error_word()
    tok = torch.empty(15 * 3, dtype=torch.int32, device="cuda")
    u = torch.rand(45, generator=gen(1), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _native.draft_sample(v.draft, u, tok, err, **par)
        _native.verify_filtered(v.target, v.draft, 3, v.tokens, v.coins, v.u, v.acc, v.bonus, v.ws, v.err,
                                accept_prob=v.chance, **par)
    for seed in (1, 2):  # other inputs at the same addresses
        u.copy_(torch.rand(45, generator=gen(seed), device="cuda"))
        tok.fill_(-7), v.acc.fill_(-7), v.bonus.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        plain = torch.empty_like(tok)
        _native.draft_sample(v.draft, u, plain, err, **par)
        assert torch.equal(tok, plain) and torch.equal(v.acc, want[0]) and torch.equal(v.bonus, want[1])
        assert torch.equal(v.chance, want[2])
    assert int(err.item()) == 0


def test_the_same_result_every_time():
    g = gen(31)
    x = f.peaked(60, 50001 // 8 * 8, g)
    u = torch.rand(60, generator=g, device="cuda")
    rows = (ASKS * 4)[:60]
    first = sample(x, rows, u)
    for _ in range(5):
        assert sample(x, rows, u) == first


def test_two_calls_at_once():
    both = [Verify(40, 5, 20011, [ASKS[(i + at) % len(ASKS)] for i in range(40)], 31 + at) for at in range(2)]
    want = []
    for v in both:
        v.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (v.acc, v.bonus, v.chance)])
    streams = [torch.cuda.Stream() for _ in both]
    for v in both:
        v.acc.fill_(-7), v.bonus.fill_(-7), v.chance.fill_(-7)
    torch.cuda.synchronize()
    # The parameters' arrays live until both streams are done: dropped earlier, their memory would go
    # to the other call's parameters, made on the current stream, while a kernel still reads it.
    held = [asked(v.rows) for v in both]
    torch.cuda.synchronize()
    for _ in range(8):  # each has a workspace of its own
        for v, s, par in zip(both, streams, held):
            _native.verify_filtered(v.target, v.draft, v.Kp, v.tokens, v.coins, v.u, v.acc, v.bonus, v.ws, v.err,
                                    accept_prob=v.chance, stream=s, **par)
    torch.cuda.synchronize()
    for v, w in zip(both, want):
        assert all(torch.equal(a, b) for a, b in zip((v.acc, v.bonus, v.chance), w))
