"""Rotated append to the 4-bit paged cache, and its read-back, on the GPU."""
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


def make(T, Hq, Hkv, D, seed, blocks=None, bs=16, dense=False, rejected=0.3):
    g = gen(seed)
    if dense:
        q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    else:  # slices of one projection, with a few columns between the rows
        w = torch.randn(T, (Hq + 2 * Hkv) * D + 8, generator=g, device="cuda").to(BF)
        q = w[:, :Hq * D].unflatten(1, (Hq, D))
        k = w[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        v = w[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].unflatten(1, (Hkv, D))
    blocks = blocks or T // bs + 3
    cache = torch.randint(0, 256, (blocks, Hkv, bs // 16, 18 * D), generator=g, device="cuda").to(torch.uint8)
    pos = torch.randint(0, 9000, (T,), generator=g, device="cuda").to(torch.int32)
    slots = torch.randperm(blocks * bs, generator=g, device="cuda")[:T]
    slots = torch.where(torch.rand(T, generator=g, device="cuda") < rejected, -1, slots)
    return q, k, v, pos, slots, cache


def append(q, k, v, pos, slots, rope, cache, interleaved=False, q_out=None, k_out=None, with_k=True):
    err = _native.new_error_word()
    q_out = torch.empty(q.shape, dtype=BF, device="cuda") if q_out is None else q_out
    if k_out is None and with_k:
        k_out = torch.empty(k.shape, dtype=BF, device="cuda")
    _native.kv_append(q, k, v, pos, slots, rope, cache, q_out, err, k_out=k_out, interleaved=interleaved)
    torch.cuda.synchronize()
    return q_out, k_out, int(err.item())


@pytest.mark.parametrize("T, Hq, Hkv, D, rot, inter, bs", [
    (1, 64, 8, 64, 64, False, 16), (14, 64, 8, 64, 64, False, 16), (257, 32, 4, 128, 128, False, 16),
    (100, 20, 4, 64, 32, False, 32), (77, 12, 12, 64, 64, True, 64), (63, 32, 8, 128, 64, True, 48),
    (1000, 8, 1, 128, 96, False, 16), (33, 1, 1, 64, 32, True, 16), (5000, 64, 8, 64, 64, False, 16),
    (9, 3, 3, 128, 128, False, 128)])
def test_append_matches_the_definition(T, Hq, Hkv, D, rot, inter, bs):
    q, k, v, pos, slots, cache = make(T, Hq, Hkv, D, T, bs=bs)
    rope = _native.rope_table(9000, rot)
    before = cache.clone()
    q_out, k_out, err = append(q, k, v, pos, slots, rope, cache, inter)
    assert err == 0
    want, mag = u.rotated(q, rope, pos, inter)
    # fp32: a product and a fused product, two roundings of the terms; then bf16's half step
    u.within(q_out, want, 2.0 ** -8 * want.abs() + 2 * 2.0 ** -24 * 1.01 * mag, "q")
    k_exact = u.to_bf16(u.rotated(k, rope, pos, inter)[0])
    assert torch.equal(k_out, k_exact)
    live = slots >= 0
    hk, hv = u.held(cache, D, slots[live])
    assert torch.equal(hk, u.quantised(k_exact[live])) and torch.equal(hv, u.quantised(v[live]))
    # every byte that no slot names is as it was
    for f in u.fields(before, D):
        at = slots[live]
        f[at // bs, :, at % bs // 16, at % 16] = 0
    after = cache.clone()
    for f in u.fields(after, D):
        f[at // bs, :, at % bs // 16, at % 16] = 0
    assert torch.equal(before, after)
    # and the read-back returns what is held, zeros for -1
    err = _native.new_error_word()
    ko, vo = torch.empty_like(k_out), torch.empty_like(k_out)
    _native.kv_read(cache, slots, ko, vo, err)
    assert torch.equal(ko[live].double(), hk) and torch.equal(vo[live].double(), hv)
    assert not ko[~live].any() and not vo[~live].any() and int(err.item()) == 0


def test_append_in_place_and_without_keys_out():
    q, k, v, pos, slots, cache = make(50, 8, 2, 64, 3, dense=True)
    rope = _native.rope_table(9000, 64)
    c2 = cache.clone()
    q1, k1, _ = append(q, k, v, pos, slots, rope, cache)
    append(q, k, v, pos, slots, rope, c2, with_k=False)
    assert torch.equal(cache, c2)
    append(q, k, v, pos, slots, rope, c2, q_out=q, k_out=k)
    assert torch.equal(q, q1) and torch.equal(k, k1) and torch.equal(cache, c2)


def test_codes_at_borders_and_extremes():
    D, g = 64, gen(5)
    rows = []
    for s in (2.0 ** -9, 3 * 2.0 ** -9, 2.0 ** -6, 0.0625, 0.4375, 1.0, 15.0, 448.0):
        x = torch.tensor(u.GRID + [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0]) * s  # every code and every border
        rows += [x, -x, x.flip(0) * (1 + 2.0 ** -7), x * (1 - 2.0 ** -8)]
    rows += [torch.zeros(16), torch.full((16,), 2.0 ** -14), torch.full((16,), -1e30),
             torch.tensor([3e38, -3e38] + [1.0] * 14), torch.tensor([1e-38] * 16), -torch.zeros(16)]
    for _ in range(2):
        rows += list((torch.randn(15, 16, generator=g, device="cuda") * 10.0 ** torch.randint(-4, 4, (15, 1), generator=g, device="cuda")).cpu())
    x = torch.cat(rows).to("cuda").to(BF)
    x = x[:x.numel() // D * D].view(-1, 1, D)
    T = x.shape[0]
    cache = _native.new_kv_cache(T // 16 + 1, 16, 1, D)
    slots = torch.arange(T, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")  # position 0 turns by nothing
    append(x, x, x, pos, slots, _native.rope_table(1, D), cache)
    hk, hv = u.held(cache, D, slots)
    want = u.quantised(x)
    assert torch.equal(hk, want) and torch.equal(hv, want)


def test_an_infinity_saturates_its_group_only():
    x = torch.ones(1, 1, 64, device="cuda", dtype=BF)
    x[0, 0, 17] = -float("inf")
    cache = _native.new_kv_cache(1, 16, 1, 64)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    append(torch.ones_like(x), torch.ones_like(x), x, z, z.long(), _native.rope_table(1, 64), cache)
    _, v = u.held(cache, 64, z.long())
    assert float(v[0, 0, 17]) == -6 * 448 and not v[0, 0, 16] and bool((v[0, 0, :16] == 1.03125).all())  # 6 * e4m3(1/6)
    assert bool(v.isfinite().all())


def test_bad_positions_and_slots():
    q, k, v, pos, slots, cache = make(40, 8, 2, 64, 7, rejected=0)
    rope = _native.rope_table(9000, 64)
    pos[3], pos[5], slots[7], slots[9] = -1, 9000, cache.shape[0] * 16, -2
    before = cache.clone()
    q_out, k_out, err = append(q, k, v, pos, slots, rope, cache)
    assert err == _native.ERR_POS_RANGE | _native.ERR_BLOCK_RANGE
    assert torch.equal(q_out[[3, 5]], q[[3, 5]]) and torch.equal(k_out[[3, 5]], k[[3, 5]])
    used = slots.clone()
    used[[7, 9]] = slots[0]
    hk, _ = u.held(cache, 64, used)
    good = torch.ones(40, dtype=torch.bool, device="cuda")
    good[[7, 9]] = False
    assert torch.equal(hk[good], u.quantised(k_out)[good])
    for f, b in zip(u.fields(cache, 64), u.fields(before, 64)):
        f[used // 16, :, 0, used % 16] = b[used // 16, :, 0, used % 16]
    assert torch.equal(cache, before)
    err = _native.new_error_word()
    ko = torch.ones_like(k_out)
    _native.kv_read(cache, slots, ko, None, err)
    assert int(err.item()) == _native.ERR_BLOCK_RANGE and not ko[[7, 9]].any()


def test_cache_past_32_bits():
    """Slots whose bytes lie past 4 GB."""
    D, Hkv, blocks = 128, 4, 500_000
    cache = torch.empty(blocks, Hkv, 1, 18 * D, dtype=torch.uint8, device="cuda")
    q, k, v, pos, _, _ = make(64, 4, Hkv, D, 11)
    slots = blocks * 16 - 1 - torch.arange(64, device="cuda") * 5
    _, k_out, err = append(q, k, v, pos, slots, _native.rope_table(9000, D), cache)
    hk, hv = u.held(cache[-64:], D, slots - (blocks - 64) * 16)
    assert err == 0 and torch.equal(hk, u.quantised(k_out)) and torch.equal(hv, u.quantised(v))


def test_empty_and_streams():
    q, k, v, pos, slots, cache = make(40, 8, 2, 64, 8)
    rope = _native.rope_table(9000, 64)
    before = cache.clone()
    _, _, err = append(q[:0], k[:0], v[:0], pos[:0], slots[:0], rope, cache)
    assert err == 0 and torch.equal(cache, before)
    q1, k1, _ = append(q, k, v, pos, slots, rope, cache)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    e, q2 = _native.new_error_word(), torch.empty_like(q1)
    torch.cuda.synchronize()
    _native.kv_append(q, k, v, pos, slots, rope, before, q2, e, stream=s)
    s.synchronize()
    assert torch.equal(q1, q2) and torch.equal(before, cache)
