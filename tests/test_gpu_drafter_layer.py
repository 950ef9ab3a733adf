"""The step, the rotated append and both attentions together, as the example uses them."""
import os
import sys

import pytest
import torch

import attn_util as u

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq, Hkv, D", [(16, 2, 64), (8, 2, 128)])
def test_prefill_then_decode(Hq, Hkv, D):
    import drafter_layer as ex
    import speculative_decoding_pe_gb300 as pe

    outs, layer = ex.run(requests=5, prompt=(20, 300), steps=3, H=128, V=1008, Hq=Hq, Hkv=Hkv, D=D)
    for i, (step, w, out) in enumerate(outs):
        assert bool(out.isfinite().all())
        rejected = step.is_rejected != 0
        assert not out[rejected].any() and bool((step.slot_mapping[rejected] == -1).all())
        if i:
            assert int(rejected.sum()) > 0
    # the last step's attention from what the cache holds, request by request
    step, w, out = outs[-1]
    qkv = step.X @ layer.w
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    pos = step.out_positions
    q = u.to_bf16(u.rotated(q, layer.rope, pos, False)[0])  # (within a step of the kernel's own rounding)
    for b in range(w.B):
        r = slice(int(step.out_offsets[b]), int(step.out_offsets[b + 1]))
        limit = torch.where(step.is_rejected[r] != 0, 0, pos[r].long() + 1)
        n = int(limit.max())
        t = torch.arange(n, device="cuda")
        slots = w.block_table[b].long()[t // 16] * 16 + t % 16
        k, v = u.held(layer.cache, D, slots)
        ko = torch.empty(n, Hkv, D, dtype=torch.bfloat16, device="cuda")
        vo = torch.empty_like(ko)
        pe.kv_read(layer.cache, slots, ko, vo, layer.err)
        assert torch.equal(ko.double(), k) and torch.equal(vo.double(), v)
        want, tol = u.attention(q[r], k, v, limit, D ** -0.5)
        # a query half a bf16 step off (2^-8) moves a score by at most 2^-8 of its terms' magnitude, and the
        # weights, and their sum, by as much
        s = torch.einsum("mhgd,lhd->mhgl", q[r].double().abs().unflatten(1, (Hkv, -1)), k.abs()).amax(-1).flatten(1)
        a = torch.zeros_like(want)
        for h in range(Hq):
            kk, vv = k[:, h * Hkv // Hq], v[:, h * Hkv // Hq]
            z = (q[r][:, h].double() @ kk.T * D ** -0.5).masked_fill(t >= limit[:, None], -float("inf"))
            a[:, h] = torch.softmax(z, -1).nan_to_num(0.0) @ vv.abs()
        u.within(out[r], want, tol + 2 * 2.0 ** -8 * D ** -0.5 * s.unsqueeze(-1) * a, "request %d" % b)
