"""GB300-native per-step data path of P-EAGLE parallel drafting.

Greedy verification, the fused draft-batch rebuild and the drafter input
assembly run in hand-written CUDA kernels for sm_103a behind the C ABI of
``libpe.so`` (``include/pe_api.h``).  This package holds the ctypes binding
(``_native``), the in-tree build (``build``), seeded synthetic workloads
(``workloads``) and the glue the tests and the benchmark share (``harness``).
"""
from ._native import (DraftBatch, PEError, StepArgs, StepOutputs,  # noqa: F401
                      assemble_draft_inputs, attn_cached, attn_prompt, build_draft_batch,
                      draft_readout, draft_sample, get_tuning, kv_append, kv_evict, kv_read, kv_weigh,
                      load, make_step_args, new_attn_workspace, new_error_word, new_filtered_workspace,
                      new_kv_cache, new_kv_mass, new_weigh_workspace, new_workspace, rope_table,
                      set_tuning, step, step_packed, verify_filtered, verify_greedy, workspace_bytes,
                      workspace_bytes_attn, workspace_bytes_filtered, workspace_bytes_weigh)
