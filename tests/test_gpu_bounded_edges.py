"""Attention weights of cached keys where queries are not finite; tolerances as in test_gpu_bounded_cache.py."""
import pytest
import torch

import attn_util as au
from speculative_decoding_pe_gb300 import _native
from test_gpu_bounded_cache import Weigh

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
