"""Rotated append of keys that are not finite, or whose rotation is not."""
import pytest
import torch

import attn_util as u
from speculative_decoding_pe_gb300 import _native

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
INF, NAN, MAX = float("inf"), float("nan"), 3.3895313892515355e38  # the largest bf16


@pytest.mark.parametrize("D, rot, interleaved", [(64, 64, False), (128, 128, False), (64, 32, True), (128, 64, True)])
def test_infinities_and_overflow_of_the_rotation(D, rot, interleaved):
    """A key rotates as fp64 arithmetic says: an infinity times a cosine is an
    infinity, and a finite pair may turn past the largest bf16."""
    pairs = [(INF, 1.0), (-INF, 2.0), (0.5, INF), (INF, INF), (INF, -INF), (NAN, 1.0), (1.0, NAN), (MAX, MAX), (MAX, -MAX),
             (-MAX, -MAX), (MAX, 0.0), (1.0, 2.0)]
    T = len(pairs) * 4
    x = torch.ones(T, 1, D, dtype=BF, device="cuda")
    half = rot // 2
    i = 3  # the third pair
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    for t in range(T):
        x[t, 0, a], x[t, 0, b] = pairs[t % len(pairs)]
    pos = torch.arange(T, device="cuda", dtype=torch.int32) // len(pairs) * 7  # 0: turns by nothing
    rope = _native.rope_table(64, rot)
    cache = _native.new_kv_cache(T // 16 + 1, 16, 1, D)
    slots = torch.arange(T, device="cuda")
    err = _native.new_error_word()
    q_out, k_out = torch.empty_like(x), torch.empty_like(x)
    _native.kv_append(x, x, x, pos, slots, rope, cache, q_out, err, k_out=k_out, interleaved=interleaved)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    z, _ = u.rotated(x, rope, pos, interleaved)
    finite = z.isfinite()
    # 2^128 (1 - 2^-9) and above round to infinity
    want = torch.where(finite & (z.abs() < 2.0 ** 128 * (1 - 2.0 ** -9)), u.to_bf16(z.nan_to_num(0.0, 0.0, 0.0).clamp(-MAX, MAX)).double(),
                       torch.where(finite, torch.copysign(torch.full_like(z, INF), z), z))
    assert torch.equal(k_out.isnan(), want.isnan())
    assert torch.equal(k_out.double().nan_to_num(7.0, INF, -INF), want.nan_to_num(7.0, INF, -INF))
    # the cache holds groups with an infinity saturated; of groups with a NaN it holds finite codes
    hk, hv = u.held(cache, D, slots)
    assert bool(hk.isfinite().all()) and bool(hv.isfinite().all())
    for got, src in ((hk, k_out), (hv, x)):
        groups = ~src.isnan().unflatten(-1, (-1, 16)).any(-1)
        same = (got == u.quantised(src.nan_to_num(0.0, INF, -INF))).unflatten(-1, (-1, 16)).all(-1)
        assert bool(same[groups].all())
