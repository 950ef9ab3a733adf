"""Attention weights of cached keys where queries are not finite (tolerances as in test_gpu_bounded_cache.py), and
outputs of an eviction that lie over its inputs."""
import pytest
import torch

import attn_util as au
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
