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
