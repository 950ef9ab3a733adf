"""One drafter layer's attention around the drafting step, prefill then decode.

    python examples/drafter_layer.py [--requests 8 --prompt 1024 8192 --steps 3]

For each prompt batch the fused step builds the drafter's rows, a projection
gives queries, keys and values, kv_append rotates them and writes keys and
values into the 4-bit paged cache at the step's slot mapping, and attn_prompt
attends over the prompts.  Every decode step then verifies the drafts, builds
the next rows and attends over the cache; rejected rows have slot -1, leave the
cache alone and get zeros.  Weights and logits are random.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_pe_gb300 as pe  # noqa: E402
from speculative_decoding_pe_gb300 import harness  # noqa: E402
from speculative_decoding_pe_gb300 import workloads as wl  # noqa: E402


class Layer:
    """Projection weights, rotation table and cache of one layer."""

    def __init__(self, H, Hq, Hkv, D, blocks, block_size, max_pos, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(1)
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.w = (torch.randn(2 * H, (Hq + 2 * Hkv) * D, generator=g, device=device) * (2 * H) ** -0.5).bfloat16()
        self.rope = pe.rope_table(max_pos, D, device=device)
        self.cache = pe.new_kv_cache(blocks, block_size, Hkv, D, device)
        self.workspace = pe.new_attn_workspace(D, device)
        self.err = pe.new_error_word(device)

    def rows(self, step: pe.StepOutputs):
        """Rotated queries and keys, and values, of a step's rows; the cache takes
        the keys and values."""
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        qkv = step.X @ self.w
        q, k, v = qkv.split((Hq * D, Hkv * D, Hkv * D), 1)
        q, k, v = q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        pe.kv_append(q, k, v, step.out_positions, step.slot_mapping, self.rope, self.cache, q_out, self.err,
                     k_out=k_out)
        return q_out, k_out, v

    def prefill(self, step):
        q, k, v = self.rows(step)
        out = torch.empty_like(q)
        pe.attn_prompt(q, k, v, step.out_offsets, out, self.workspace, self.err)
        return out

    def decode(self, step, block_table):
        q, _, _ = self.rows(step)
        out = torch.empty_like(q)
        pe.attn_cached(q, self.cache, block_table, step.out_offsets, step.out_positions, step.is_rejected, out,
                       self.workspace, self.err)
        return out


def decode_workload(w, lengths, Kp, seed):
    """A decode batch that continues workload ``w``'s requests at ``lengths``."""
    d = wl.make_workload(w.spec.with_(Kp=Kp, accept_p=0.3, start_lo=0, start_hi=1), seed, device=w.emb.device)
    step = torch.arange(Kp + 1, dtype=torch.int32, device=w.emb.device)
    d.in_positions = (lengths[:, None] + step).flatten().contiguous()
    d.emb, d.h_shared, d.block_table = w.emb, w.h_shared, w.block_table
    return d


def run(requests=8, prompt=(1024, 8192), steps=3, H=2880, V=201088, Hq=64, Hkv=8, D=64, seed=3, device="cuda"):
    """Attention outputs of the prefill and of each decode step, and the layer."""
    Kp = 7
    reach = prompt[1] + (steps + 2) * (Kp + 1)
    spec = wl.SPECS["prefill_b8"].with_(B=requests, prompt_lo=prompt[0], prompt_hi=prompt[1], H=H, V=V,
                                        bt_width=reach // 16 + 1)
    w = wl.make_workload(spec, seed, device=device)
    blocks = int(w.block_table.max()) + 1
    layer = Layer(H, Hq, Hkv, D, blocks, w.block_size, reach + 16, device)
    step, ws, err = harness.allocate(w, device)
    harness.run(w, step, ws, err)
    outs = [(step, w, layer.prefill(step))]
    lengths = (w.in_offsets[1:] - w.in_offsets[:-1]).to(torch.int32)
    for i in range(steps):
        d = decode_workload(w, lengths, Kp, seed + 1 + i)
        step, ws, err = harness.allocate(d, device)
        harness.run(d, step, ws, err)
        outs.append((step, d, layer.decode(step, w.block_table)))
        lengths = lengths + step.accepted_len + 1  # the bonus token's predecessor is the last one kept
    torch.cuda.synchronize()
    if int(layer.err.item()):
        raise RuntimeError("error word %d" % int(layer.err.item()))
    return outs, layer


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, nargs=2, default=(1024, 8192), metavar=("SHORTEST", "LONGEST"))
    ap.add_argument("--steps", type=int, default=3)
    a = ap.parse_args()
    outs, layer = run(a.requests, tuple(a.prompt), a.steps)
    for i, (step, w, out) in enumerate(outs):
        kept = int((step.is_rejected == 0).sum())
        print("%s: %d rows, %d kept, output rms %.4f" % ("prefill" if i == 0 else "decode %d" % i, out.shape[0], kept,
                                                         float(out.float().square().mean().sqrt())))
    print("cache: %.1f MB" % (layer.cache.numel() / 1e6))


if __name__ == "__main__":
    main()
