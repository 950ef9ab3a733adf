"""Attention weights of cached keys where queries are not finite (tolerances as in test_gpu_bounded_cache.py), and
outputs of an eviction that lie over its inputs."""
import pytest
import torch

import attn_util as au
import speculative_decoding_pe_gb300 as pe
from speculative_decoding_pe_gb300 import _native
from test_gpu_bounded_cache import Evict, Weigh

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("limits, Hq, Hkv, D, extra", [
    ([[70 if i % 3 else 0 for i in range(100)]], 8, 2, 64, 2), ([[70 if i % 3 else 0 for i in range(100)]], 8, 2, 64, 5200),
    ([[300 + i if i % 3 else 0 for i in range(100)] + [17] * 5] * 12, 32, 4, 128, 300), ([[40, 0, 39, 41]], 16, 2, 128, 2),
    ([[5, 0, 7]] * 4 + [[900] * 100, [0] * 70], 8, 8, 64, 2)])
def test_rejected_rows_that_are_not_finite_give_nothing(limits, Hq, Hkv, D, extra, value):
    w = Weigh(limits, Hq, Hkv, D, seed=21, extra=extra)
    w.q[w.rej.bool()] = value
    w.q[w.rej.bool(), :, ::3] = 0.0
    w.check()


@pytest.mark.parametrize("D, many", [(64, False), (64, True), (128, False), (128, True)])
def test_rows_out_of_the_table_that_are_not_finite_give_nothing(D, many):
    w = Weigh([[60, 0, 59] + [58] * (70 * many)], 8, 2, D, seed=22)
    w.rej.zero_()
    w.pos[1] = -4
    w.q[1] = float("nan")
    out = torch.full_like(w.mass, -5.0)
    w.before = out.clone()
    w.run(out, None)
    torch.cuda.synchronize()
    assert int(w.err.item()) == _native.ERR_BLOCK_RANGE
    au.within(out, *w.want(None))


@pytest.mark.parametrize("limits", [[[1], [2]], [[1] * 12, [3]], [[1] * 80, [3] * 80], [[20], [1]]])
@pytest.mark.parametrize("Hq, Hkv, D", [(8, 2, 64), (4, 4, 128)])
def test_a_query_with_an_infinity(limits, Hq, Hkv, D):
    # whichever sign, and wherever the keys' signs make every score -infinity
    G = Hq // Hkv
    for at in range(0, D, 5):
        for sign in (1.0, -1.0):
            w = Weigh(limits, Hq, Hkv, D, seed=23)
            w.q[0, G, at] = sign * float("inf")  # request 0, key head 1
            out = torch.zeros_like(w.mass)
            w.run(out, None)
            torch.cuda.synchronize()
            a, b = w.slots
            assert int(w.err.item()) == 0
            assert bool(out[a // 16, 1, a % 16].isnan().all()) and bool(out[b // 16, :, b % 16].isfinite().all())
            rest = [h for h in range(Hkv) if h != 1]
            assert bool(out[a // 16][:, rest][torch.arange(len(a)), :, a % 16].isfinite().all())


def test_evict_refuses_outputs_over_its_sizes():
    # (refused on the host, before any launch)
    n, out = torch.full((4,), 40, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    e = Evict([40, 40], [20, 20], 2, 64, seed=24)
    for lengths, keep, size in ((n[:2], n[2:], n[:2]), (n[:2], n[2:], n[2:]), (n[:2], n[2:], n[1:3])):
        with pytest.raises(_native.PEError):
            _native.kv_evict(e.cache, e.mass, e.table, e.dst, lengths, keep, e.kept, size, e.err)
    both = torch.tensor([40, 40, -1, -1, 20, 20], dtype=torch.int32, device="cuda")  # next to each other
    _native.kv_evict(e.cache, e.mass, e.table, e.dst, both[:2], both[4:], e.kept, both[2:4], e.err)
    _native.kv_evict(e.cache, e.mass, e.table, e.dst, both[:2], both[4:], e.kept, out, e.err)
    assert int(e.err.item()) == 0 and both.tolist() == [40, 40, 20, 20, 20, 20] and out.tolist() == [20, 20]


@pytest.mark.parametrize("Hq, Hkv, D, bs", [(16, 2, 64, 16), (8, 4, 128, 32)])
def test_a_draft_batch_after_an_eviction(Hq, Hkv, D, bs):
    # Verified rows (some rejected) and MASK rows of a step, appended behind what an eviction left: rotation by the true
    # positions, slots, limits and weights by the cached ones.
    g = torch.Generator(device="cuda")
    g.manual_seed(25)
    B, n, keep, Kp, K, width = 4, 300, [96, 97, 111, 300], 7, 5, 24
    m, G = Kp + K, Hq // Hkv
    accepted = [0, 3, 7, 5]
    cache = au.random_cache(B * width, Hkv, bs, D, g)
    mass = torch.rand(B * width, Hkv, bs, generator=g, device="cuda")
    table = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width)
    err, i32 = pe.new_error_word(), torch.int32
    dev = lambda x, dt=i32: torch.tensor(x, dtype=dt, device="cuda")  # noqa: E731
    kept, size = torch.full((B, Hkv, 300), -1, dtype=i32, device="cuda"), torch.empty(B, dtype=i32, device="cuda")
    before = [au.held(cache, D, table[b].long()[torch.arange(n, device="cuda") // bs] * bs + torch.arange(n, device="cuda") % bs)
              for b in range(B)]
    old = [mass[table[b].long()[torch.arange(n, device="cuda") // bs], :, torch.arange(n, device="cuda") % bs] for b in range(B)]
    pe.kv_evict(cache, mass, table, table, dev([n] * B), dev(keep), kept, size, err, sinks=2, recent=20)
    assert size.tolist() == keep
    step = [[(k, k <= a) for k in range(Kp + 1)] + [(a + i, True) for i in range(1, K)] for a in accepted]
    rel, live = dev([[p for p, _ in r] for r in step]), dev([[k for _, k in r] for r in step], torch.bool)
    cached = size[:, None] + rel
    slots = torch.where(live, table.gather(1, (cached // bs).long()).long() * bs + cached % bs, -1)
    rope = pe.rope_table(n + 32, D)
    q, k, v = (torch.randn(B * m, h, D, generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    qr, out = torch.empty_like(q), torch.empty_like(q)
    k[~live.flatten()] = float("nan")
    rejected = (~live).flatten().to(torch.uint8)
    pe.kv_append(q, k, v, (n + rel).flatten(), slots.flatten(), rope, cache, qr, err)
    qr[~live.flatten()] = float("nan")
    pe.attn_cached(qr, cache, table, None, cached.flatten(), rejected, out, pe.new_attn_workspace(D), err)
    ws = pe.new_weigh_workspace(B * m, Hq, width, bs)
    pe.kv_weigh(qr, cache, table, None, cached.flatten(), rejected, mass, mass, ws, err, fresh=size)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    key = au.quantised(au.to_bf16(au.rotated(k, rope, (n + rel).flatten(), False)[0]))
    for b in range(B):
        L = keep[b] + accepted[b] + K
        j = torch.arange(L, device="cuda")
        hk, hv = au.held(cache, D, table[b].long()[j // bs] * bs + j % bs)
        rows = slice(b * m, (b + 1) * m)
        limit = torch.where(live[b], cached[b] + 1, 0).long()
        for h in range(Hkv):  # what was kept, and the step's rows behind it
            at = kept[b, h, :keep[b]].long()
            assert torch.equal(hk[:keep[b], h], before[b][0][at, h]) and torch.equal(hv[:keep[b], h], before[b][1][at, h])
            assert torch.equal(hk[cached[b][live[b]].long(), h], key[rows][live[b]][:, h])
            qq = qr[rows][live[b]][:, h * G:(h + 1) * G].double()
            hidden = j >= limit[live[b]][:, None, None]
            s = (torch.einsum("mgd,ld->mgl", qq, hk[:, h]) * D ** -0.5).masked_fill(hidden, -float("inf"))
            mag = (torch.einsum("mgd,ld->mgl", qq.abs(), hk[:, h].abs()) * D ** -0.5).masked_fill(hidden, 0.0)
            p = torch.softmax(s, -1)
            # (as in the weights' own tests)
            off = (D + 8) * 2.0 ** -24 * (mag + mag.amax(-1, keepdim=True)) + 2.0 ** -20
            want = p.sum((0, 1))
            want[:keep[b]] += old[b][at, h].double()
            got = mass[table[b].long()[j // bs], h, j % bs]
            au.within(got, want, (p * off).sum((0, 1)) + 2.0 ** -23 * want)
        w, tol = au.attention(qr[rows].nan_to_num(0.0), hk, hv, limit, D ** -0.5)
        au.within(out[rows], w, tol)
