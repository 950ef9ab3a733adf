"""Filtered sampling where roundings decide: rows whose tail holds much of the weight or next to none of
it, tokens that no row can give, rows alike, and what an earlier call left in a workspace.

Tolerances as in test_gpu_filtered.py unless a test derives its own."""
import math

import pytest
import torch

import filter_util as f
from speculative_decoding_pe_gb300 import _native
from test_gpu_filtered import BF, FP, NEAR, Verify, asked, gen, sample, vec

pytestmark = pytest.mark.gpu
LN2 = math.log(2.0)


# ------------------------------------------------- shares that round to nothing
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("octaves", [44, 46, 47, 48, 49, 50, 51, 52, 60])
def test_a_peak_over_a_bulk_next_to_nothing(octaves, dtype):
    # A lane's columns add up to some units of the sums' last bit, a vector's or a part's to none of them.
    V = 151936
    x = torch.full((4, V), 1.0 - octaves * LN2, device="cuda").to(dtype)
    for i, c in enumerate((140003, 5, 75000, V - 1)):
        x[i, c] = 1.0
    u = [0.0, 2.0 ** -40, 2.0 ** -33, 0.5]
    for k in (0, 100000):  # every column; a cut
        for v in u:
            tok, prob = sample(x, [(1.0, k, 1.0, 0.0)] * 4, vec([v] * 4))
            for i, c in enumerate(tok):
                z = torch.exp((x[i].double() - 1.0))
                if k:
                    z[torch.argsort(-z, stable=True)[k:]] = 0.0
                z /= z.sum()
                run = z.cumsum(0)
                assert 0 <= c < V and float(z[c]) > 0
                assert float(run[c] - z[c]) <= v + NEAR and float(run[c]) >= v - NEAR
                assert abs(prob[i] - float(z[c])) <= (2.0 ** -24 + 2.0 ** -29) * float(z[c])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("octaves", [20, 40, 50, 56, 58, 60, 62])
def test_a_rest_next_to_nothing(octaves, dtype):
    # The target's rows have a bulk that the draft's lack, and the rest p - q is that bulk alone: equal weights,
    # whose roundings are alike too (2^-20 of u covers the sums'; from 2^-50 on units of 2^-60 decide).
    V, B, peak = 50000, 8, 40001
    v = Verify(B, 1, V, [(1.0, 0, 1.0, 0.0)] * B, 3, dtype)
    v.target[:] = 1.0 - octaves * LN2
    v.target[:, peak] = 1.0
    v.draft[:] = float("-inf")
    v.draft[:, peak] = 1.0
    v.draft[0::2, 7] = 1.0 - (octaves - 3) * LN2  # eight times what the target gives: rejected
    v.tokens[0::2, 1] = 7
    v.tokens[1::2, 1] = peak                      # accepted: the bonus row's own draw
    v.coins.fill_(0.5)
    v.u.copy_(vec([0.0, 0.0, 2.0 ** -45, 2.0 ** -45, 0.75, 0.75, 1.0 - 2.0 ** -24, 1.0 - 2.0 ** -24]))
    v.run()
    torch.cuda.synchronize()
    assert int(v.err.item()) == 0 and v.acc.tolist() == [0, 1] * 4
    for b in range(B):
        c, u = int(v.bonus[b]), float(v.u[b])
        z = torch.exp(v.target[2 * b + b % 2].double() - 1.0)
        if b % 2 == 0:
            z[peak] = z[7] = 0.0
        run = z.cumsum(0) / z.sum()
        assert 0 <= c < V and float(z[c]) > 0
        if b % 2 or octaves <= 50:
            near = NEAR if b % 2 else 2.0 ** -20
            assert float(run[c] - z[c] / z.sum()) <= u + near and float(run[c]) >= u - near


# ------------------------------------------------- tokens that no row can give
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("flat_target", [True, False])
@pytest.mark.parametrize("ask", [(2.0, 0, 1.0, 0.0), (2.0, 20, 1.0, 0.0), (2.0, 0, 0.9, 0.0), (2.0, 600, 1.0, 0.0), (1.0, 0, 1.0, 1e-3)])
def test_tokens_outside_the_vocabulary_are_rejected(ask, flat_target, dtype):
    # whatever the coins and the two rows' sums of weights
    B, Kp, V = 12, 3, 1000
    v = Verify(B, Kp, V, [ask] * B, 41, dtype)
    v.target.mul_(0.3 if flat_target else 2.0)
    v.draft.mul_(2.0 if flat_target else 0.3)
    bad = torch.tensor([-1, V, 2 ** 31 - 1, -2 ** 31, V + 8, -2], dtype=torch.int32, device="cuda")
    at = torch.arange(B, device="cuda") % Kp
    v.tokens[torch.arange(B, device="cuda"), 1 + at] = bad[torch.arange(B, device="cuda") % 6]
    for coins in (0.0, 0.5, 1.0 - 2.0 ** -24, None):
        if coins is None:
            v.coins.copy_(torch.rand(B * Kp, generator=gen(42), device="cuda"))
        else:
            v.coins.fill_(coins)
        v.check()
        assert bool((v.acc <= at).all())
        assert not bool(v.chance.view(B, Kp).gather(1, at[:, None]).any())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_a_draft_that_could_not_be_drawn_is_rejected(dtype):
    # draft_sample writes -1 where its number is not usable; the draft's row itself is sound
    B, V = 16, 900
    v = Verify(B, 1, V, [(1.5, 0, 1.0, 0.0)] * B, 43, dtype)
    v.target.mul_(0.2)
    tok, _ = sample(v.draft, v.rows, vec([float("nan")] * B), want_err=_native.ERR_PARAM)
    assert tok == [-1] * B
    v.tokens[:, 1] = -1
    v.coins.fill_(0.99)
    compared, rejected = v.check()
    assert rejected == B and compared >= B - 2


# ------------------------------------------------- rows alike
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("ask", [(1.0, 20, 1.0, 0.0), (0.7, 30, 0.9999, 0.0), (1.0, 0, 1.0, 1e-12), (1.0, 300, 1.0, 0.0), (1.0, 0, 1.0, 0.0)])
def test_rows_alike_leave_no_rest(ask, dtype):
    # p - q is zero everywhere, for weights of every size: the bonus token comes from p
    B, V = 10, 700
    v = Verify(B, 1, V, [ask] * B, 44, dtype)
    rows = -0.75 * torch.arange(V, device="cuda").float() + 0.1 * torch.randn(B, V, generator=gen(45), device="cuda")
    rows = rows[:, torch.randperm(V, generator=gen(46), device="cuda")]
    rows[:, 3] = float("-inf")
    v.target[0::2], v.target[1::2], v.draft[:] = rows.to(dtype), 0.0, rows.to(dtype)
    v.tokens[:, 1] = 3  # neither gives it
    v.u.copy_((torch.arange(B, device="cuda") + 0.5) / B)
    compared, rejected = v.check()
    assert rejected == B and compared >= B - 1


# ------------------------------------------------- what the workspace held
@pytest.mark.parametrize("dtype", [BF, FP])
def test_an_empty_draft_row_hides_what_the_workspace_held(dtype):
    B, V = 96, 100000
    v = Verify(B, 1, V, [(1.0, 0, 1.0, 0.0)] * B, 47, dtype)
    v.target[:] = (-0.7 * torch.arange(B * 2, device="cuda")[:, None] / B - 12.0 +
                   0.5 * torch.randn(B * 2, V, generator=gen(48), device="cuda")).to(dtype)
    v.target[:, 50000], v.target[:, 9] = 1.0, float("-inf")
    v.draft[:] = float("nan")
    v.tokens[:, 1] = 9
    for b in range(B):  # numbers next to borders of the weights below 2^-16
        run = torch.exp(v.target[2 * b].double() - 1.0).cumsum(0)
        v.u[b] = (run[30 + 1000 * b] / run[-1]).float()
    got = []
    for words in ([-1] * 12, [0] * 12, [0, 2 ** 31 - 1, -8388608] + [0] * 9, [-2, 5, 0x7f800000] + [1065353216] * 9):
        held = torch.tensor(words, dtype=torch.int32, device="cuda")
        n = v.ws.numel() // 48
        v.ws[:48 * n].view(torch.int32).view(n, 12).copy_(held.expand(n, 12))
        v.bonus.fill_(-7)
        v.run()
        torch.cuda.synchronize()
        assert int(v.err.item()) == _native.ERR_EMPTY_ROW and not bool(v.acc.any())
        got.append(v.bonus.tolist())
    assert got[1:] == got[:1] * 3


# ------------------------------------------------- outputs over inputs
def test_verify_refuses_outputs_over_its_numbers():
    # (refused on the host, before any launch)
    v = Verify(4, 3, 200, [(1.0, 0, 1.0, 0.0)] * 4, 49)
    v.run()
    torch.cuda.synchronize()
    want = v.chance.clone()
    room = torch.rand(28, device="cuda")
    room[:12], room[12:16] = v.coins, v.u
    coins, u, chance = v.coins, v.u, v.chance
    for at in (0, 11, 12, 15):
        v.coins, v.u, v.chance = room[:12], room[12:16], room[at:at + 12]
        with pytest.raises(_native.PEError):
            v.run()
    v.chance = room[16:28]  # next to them
    v.run()
    torch.cuda.synchronize()
    assert int(v.err.item()) == 0 and torch.equal(room[16:28], want) and torch.equal(room[:12], coins) and torch.equal(room[12:16], u)


# ------------------------------------------------- tails of small weights
# Weights below 2^-16 of the largest go through the hardware's exponential, which is off by 1.4e-7 at most after its mean
# of -5.1e-8 has been put back.  For one value, 2^-19: bf16 rows round the exponent (half of its last bit, 2^-19 from
# 16 to 32: 6.6e-7 of the weight), fp32 rows the difference (2^-24 of it: 2^-24 * 32 * ln 2 = 1.3e-6).  Over the values
# of a row: measured for T from 0.3 to 2 at -5.0e-8 to -5.4e-8 in fp32, within 2^-27 of the weight after the correction,
# and at -3.2e-8 to -7.9e-8 over bf16's some hundred values, within 2^-25.  A border moves by that times the tail's
# share at most.
ANY = 2.0 ** -19
MEAN = {FP: 2.0 ** -27, BF: 2.0 ** -25}


def tail_row(V, T, dtype, seed, least=16.5, most=19.5, at=4.0):
    """One column of weight 1, the others of 2^-least to 2^-most: a third of the sum for 100,000 columns."""
    x = at - T * LN2 * (least + (most - least) * torch.rand(1, V, generator=gen(seed), device="cuda"))
    x[0, V // 3] = at
    return x.to(dtype)


def borders(x, T, keep=None):
    """64-bit running sums and the whole, the tail's share."""
    T = float(torch.tensor(T, dtype=FP))
    w = torch.exp((x[0].double() - x[0].double().max()) / T).nan_to_num(0.0)
    small = float(w[w < 2.0 ** -16].sum() / w.sum())
    return w.cumsum(0), float(w.sum()), small


def compare_draws(tok, u, run, whole, near, least):
    u = u.double() * whole
    want = torch.searchsorted(run, u, right=True)
    before = torch.cat((run.new_zeros(1), run))[want]
    clear = (torch.minimum(u - before, run[want] - u) > near * whole) | ((want == 0) & (run[want] - u > near * whole))
    assert int(clear.sum()) >= least * u.numel()
    wrong = clear & (tok.long() != want)
    assert int(wrong.sum()) == 0, "%d of %d draws" % (int(wrong.sum()), int(clear.sum()))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T", [0.8, 1.0, 1.1, 1.3])
@pytest.mark.parametrize("V", [100000, 30000])
def test_draws_from_a_tail(T, V, dtype):
    x = f.pitched(tail_row(V, T, dtype, 61))
    n = 100000 if V > 50000 else 30000
    u = torch.rand(n, generator=gen(62), device="cuda")
    tok, prob, err = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda"), _native.new_error_word()
    idx = torch.zeros(n, dtype=torch.int32, device="cuda")
    _native.draft_sample(x, u, tok, err, temperature=vec([T]), out_prob=prob, sample_idx=idx)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    run, whole, share = borders(x, T)
    assert share > 0.1
    compare_draws(tok, u, run, whole, MEAN[dtype] * share + NEAR, 0.95)
    z = torch.diff(run, prepend=run.new_zeros(1))[tok.long()] / whole
    assert bool(((prob.double() - z).abs() <= z * (2.0 ** -24 + 2.0 ** -29 + MEAN[dtype] * share)).all())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T", [0.7, 1.0, 1.3])
@pytest.mark.parametrize("octaves", [16.3, 17.1, 18.9])
def test_draws_from_equal_small_weights(octaves, T, dtype):
    # one value only
    V, n = 60000, 4096
    x = torch.full((1, V), 3.0 - T * LN2 * octaves, device="cuda").to(dtype)
    x[0, 20000] = 3.0
    u = torch.rand(n, generator=gen(63), device="cuda")
    tok, err = torch.empty(n, dtype=torch.int32, device="cuda"), _native.new_error_word()
    _native.draft_sample(x, u, tok, err, temperature=vec([T]), sample_idx=torch.zeros(n, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    run, whole, share = borders(x, T)
    compare_draws(tok, u, run, whole, ANY * share + NEAR, 0.8)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T", [0.8, 1.0, 1.3])
def test_a_rest_of_a_tail(T, dtype):
    # The target has a tail and a second large column at the end, the draft neither: the rest is both.
    V, B = 100000, 600
    v = Verify(B, 1, V, [(T, 0, 1.0, 0.0)] * B, 64, dtype)
    row = tail_row(V, T, dtype, 65)
    row[0, V - 1] = 4.0 - T
    v.target[0::2], v.target[1::2] = row, 0.0
    v.draft[:] = float("-inf")
    v.draft[:, V // 3] = 4.0
    v.draft[:, 7] = 4.0 - 12.0 * T
    v.tokens[:, 1] = 7  # some 1 of 6 times what the target gives it, to be rejected by its coin
    v.coins.fill_(0.999)
    v.u.copy_(torch.rand(B, generator=gen(66), device="cuda"))
    p = torch.exp((row[0].double() - 4.0) / float(torch.tensor(T, dtype=FP)))
    q = torch.exp((v.draft[0].double() - 4.0) / float(torch.tensor(T, dtype=FP)))
    p, q = p / p.sum(), q / q.sum()
    if float(p[7]) >= 0.999 * float(q[7]):  # (a bf16 value may be the larger one)
        v.draft[:, 7] = 4.0 - 10.0 * T
        q = torch.exp((v.draft[0].double() - 4.0) / float(torch.tensor(T, dtype=FP)))
        q = q / q.sum()
    v.run()
    torch.cuda.synchronize()
    assert int(v.err.item()) == 0 and not bool(v.acc.any())
    rest = (p - q).clamp(min=0)
    # the tail's weights over the rest's whole
    near = MEAN[dtype] * float(rest[rest < 2.0 ** -16].sum() / rest.sum()) + NEAR / float(rest.sum())
    compare_draws(v.bonus, v.u, rest.cumsum(0), float(rest.sum()), near, 0.9)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_masked_columns_in_a_tail(dtype):
    # NaN and -infinity among small weights, alone in a vector or all of it; largest logits of any size
    inf, nan = float("inf"), float("nan")
    V, n = 40000, 20000
    x = tail_row(V, 1.0, dtype, 67)
    x[0, 100:9000], x[0, 20001::7], x[0, 5::11], x[0, 30000:30064] = -inf, nan, -inf, nan
    x[0, V // 3] = 4.0
    u = torch.rand(n, generator=gen(68), device="cuda")
    idx = torch.zeros(n, dtype=torch.int32, device="cuda")
    tok, err = torch.empty(n, dtype=torch.int32, device="cuda"), _native.new_error_word()
    _native.draft_sample(x, u, tok, err, sample_idx=idx)
    run, whole, share = borders(torch.where(x.isnan(), -inf, x.float()), 1.0)
    compare_draws(tok, u, run, whole, MEAN[dtype] * share + NEAR, 0.95)
    low = torch.finfo(dtype).min
    for T in (2.0 ** -30, 1e-3, 1.0, 100.0, 2.0 ** 30):
        for top, rest in ((low, -inf), (-3.0e38, low), (3.0e38, low), (3.0e38, -inf), (1e-30, -inf), (-17.0, low), (0.0, nan)):
            y = torch.full((1, 5000), rest, device="cuda").to(dtype)
            y[0, 17::1000] = top
            m = 512
            u = (torch.arange(m, device="cuda") + 0.5) / m
            tok = torch.empty(m, dtype=torch.int32, device="cuda")
            prob = torch.empty(m, device="cuda")
            _native.draft_sample(y, u, tok, err, temperature=vec([T]), sample_idx=idx[:m], out_prob=prob)
            torch.cuda.synchronize()
            assert tok.tolist() == [17 + 1000 * int(5 * (i + 0.5) / m) for i in range(m)], (T, top, rest)
            assert bool((prob - 0.2).abs().max() <= 2.0 ** -26)
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("p", [0.7, 0.9, 0.9999])
def test_a_share_of_a_tail(p, dtype):
    # top-p ends within the tail: its whole weight decides where
    V, n, T = 100000, 20000, 1.1
    x = tail_row(V, T, dtype, 69)
    u = torch.rand(n, generator=gen(70), device="cuda")
    tok, err = torch.empty(n, dtype=torch.int32, device="cuda"), _native.new_error_word()
    _native.draft_sample(x, u, tok, err, temperature=vec([T]), top_p=vec([p]), sample_idx=torch.zeros(n, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    run, whole, share = borders(x, T)
    w = torch.diff(run, prepend=run.new_zeros(1))
    order = torch.argsort(x[0].float(), descending=True, stable=True)
    sums = w[order].cumsum(0)
    p = float(torch.tensor(p, dtype=FP))
    kept = int((sums - w[order] < p * whole).sum())
    gap = min(abs(float(sums[kept - 1]) / whole - p), abs(float(sums[kept - 1] - w[order[kept - 1]]) / whole - p))
    off = MEAN[dtype] * share + NEAR
    w[order[kept:]] = 0.0
    run = w.cumsum(0)
    # one column more or less in the prefix, where the share falls next to a border, moves borders by its weight
    compare_draws(tok, u, run, float(run[-1]), off + (0.0 if gap > off else 2.0 ** -16), 0.9 if gap > off else 0.0)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("ask", [(1.1, 90000, 1.0, 0.0), (0.9, 60000, 1.0, 0.0), (1.1, 0, 1.0, 1e-6)])
@pytest.mark.parametrize("values", [1, 5])
def test_sums_of_equal_weights(values, ask, dtype):
    # Behind a cut every weight is taken in full: sums of equal ones, whose roundings go one way, hold to NEAR too.
    V, n, (T, k, _, m) = 100000, 60000, ask
    x = torch.full((1, V), 4.0, device="cuda") - T * (11.5 + (torch.arange(V, device="cuda") % values) * 0.25)
    x[0, V // 3] = 4.0
    x = x.to(dtype)
    u = torch.rand(n, generator=gen(71), device="cuda")
    tok, err = torch.empty(n, dtype=torch.int32, device="cuda"), _native.new_error_word()
    _native.draft_sample(x, u, tok, err, sample_idx=torch.zeros(n, dtype=torch.int32, device="cuda"), **asked([ask]))
    torch.cuda.synchronize()
    run, whole, share = borders(x, T)
    w = torch.diff(run, prepend=run.new_zeros(1))
    order = torch.argsort(x[0].float(), descending=True, stable=True)
    if k:
        w[order[k:]] = 0.0
    if m:
        w[w < float(torch.tensor(m, dtype=FP))] = 0.0
    run = w.cumsum(0)
    compare_draws(tok, u, run, float(run[-1]), NEAR, 0.9)


def test_a_rest_of_equal_weights():
    # p - q of a row without a draft's tail, behind a cut: as above, in units of p
    V, B, T = 100000, 3000, 1.0
    v = Verify(B, 1, 64, [(T, 0, 1.0, 0.0)] * B, 72, FP)
    v.V, v.rows = V, [(T, 99999, 1.0, 0.0)] * B
    row = torch.full((V,), 4.0 - 11.5, device="cuda")
    row[V // 3], row[V - 2], row[V - 1] = 4.0, 3.0, -90.0
    v.target = row.to(BF).expand(2 * B, V).contiguous()
    v.draft = torch.full((B, V), float("-inf"), dtype=BF, device="cuda")
    v.draft[:, V // 3], v.draft[:, 7] = 4.0, 0.0
    v.tokens[:, 1] = 7
    v.coins.fill_(0.5)
    v.run()
    torch.cuda.synchronize()
    assert int(v.err.item()) == 0 and not bool(v.acc.any())
    p, q = (torch.exp(r.double() - 4.0) for r in (v.target[0], v.draft[0]))
    p[V - 1] = 0.0
    rest = (p / p.sum() - q / q.sum()).clamp(min=0)
    compare_draws(v.bonus, v.u, rest.cumsum(0), float(rest.sum()), 2.0 ** -28 / float(rest.sum()), 0.9)


# ------------------------------------------------- a share that a list cannot hold
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("V", [40003, 90000, 151936])
def test_min_p_leaves_less_than_the_share(V, dtype):
    # Flat rows of a weight of thousands of their largest, of which min-p leaves some hundreds of columns: top-p keeps
    # tens of thousands, so that min-p alone decides.  Shares just above whole multiples of 2^12 of the largest weight.
    n = 24
    x = -3.0 * torch.rand(n, V, generator=gen(80), device="cuda")
    x[:, torch.randperm(V, generator=gen(81), device="cuda")[:3000]] += 0.9
    x = f.pitched(x.to(dtype))
    w = torch.exp(x.double() - x.double().max(1, keepdim=True)[0])
    whole = w.sum(1).tolist()
    asks = [(1.0, 0, (4096 * (1 + i % int(whole[i] / 4096)) + 100) / whole[i], 0.55) for i in range(n)]
    u = torch.rand(n, generator=gen(82), device="cuda")
    tok, prob = sample(x, asks, u)
    counted = 0
    for i, c in enumerate(tok):
        floor = float(x[i].double().max()) + math.log(float(torch.tensor(0.55, dtype=FP)))
        kept = x[i].double() >= floor
        assert 200 < int(kept.sum()) < asks[i][2] * V / 10
        z = torch.where(kept, w[i], 0.0)
        z /= z.sum()
        run = z.cumsum(0)
        want = int((run <= float(u[i])).sum())
        if min(abs(float(run[want]) - float(u[i])), abs(float(u[i] - (run[want] - z[want])))) < NEAR:
            continue
        counted += 1
        assert c == want and abs(prob[i] - float(z[c])) <= (2.0 ** -24 + 2.0 ** -29) * float(z[c])
    assert counted >= n - 2


# ------------------------------------------------- probabilities of next to nothing
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("k, V", [(40, 300), (600, 4000), (0, 4000)])
def test_probabilities_of_tiny_weights(k, V, dtype):
    # columns of 2^-1 to 2^-44 of the largest, kept in a short list, a long one, or without any
    B = 40
    v = Verify(B, 1, V, [(1.0, k, 1.0, 0.0)] * B, 90, dtype)
    fall = torch.arange(40, device="cuda").float() * (44 * LN2 / 40)
    for i, rows in enumerate((v.target, v.draft)):
        rows[:] = -60.0
        x = 8.0 - fall - 0.3 * torch.rand(rows.shape[0], 40, generator=gen(91 + i), device="cuda")
        rows[:, 17:17 + 40 * 5:5] = x.flip(1).to(dtype)  # the lightest first
    v.tokens[:, 1] = 17 + 5 * torch.arange(B, device="cuda") % 200
    v.run()
    # u = 0 draws the first kept column that weighs anything; here it may be any of the lightest
    tok, prob = sample(v.target, [v.rows[0]] * (2 * B), vec([0.0] * (2 * B)))
    torch.cuda.synchronize()
    assert int(v.err.item()) == 0
    for b in range(B):
        p, q = (f.probabilities(r[b], 1.0, k) for r in (v.target[0::2], v.draft))
        x = int(v.tokens[b, 1])
        want = min(1.0, float(p[x]) / float(q[x]))
        assert abs(float(v.chance[b]) - want) <= (2.0 ** -24 + 2.0 ** -28) * want, b
        c = tok[2 * b]
        assert 0 <= c <= 17 + 200 and float(p[c]) > 0 and abs(prob[2 * b] - float(p[c])) <= (2.0 ** -24 + 2.0 ** -29) * float(p[c])
