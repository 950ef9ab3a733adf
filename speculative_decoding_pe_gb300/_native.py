"""ctypes binding of libpe.so (argument marshalling only).

Every function takes torch CUDA tensors, checks their dtype / device /
layout, and passes raw pointers plus the current CUDA stream to the C ABI
declared in ``include/pe_api.h``.  All work runs in the library's kernels;
there is no fallback of any kind: if the library is missing or a call is
rejected, an exception is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libpe.so")
# the same ABI compiled with PE_CHECKED (NaN logits and internal invariants
# raise ERR_NAN / ERR_INTERNAL; slower, for debugging)
CHECKED_LIB_PATH = os.path.join(_HERE, "_build", "libpe_checked.so")

PE_F32, PE_BF16 = 0, 1
ERR_TOKEN_RANGE = 1
ERR_BLOCK_RANGE = 2
ERR_SLOT_RANGE = 4
ERR_OFFSETS = 8
ERR_MAP_RANGE = 16
ERR_TIMEOUT = 32
ERR_ROW_RANGE = 64
ERR_NAN = 128
ERR_INTERNAL = 256
ERR_WORKSPACE = 512
ERR_POS_RANGE = 1024
ERR_PARAM = 2048
ERR_EMPTY_ROW = 4096
MAX_KP, MAX_K = 255, 256

# every function the C header declares
EXPORTS = ("pe_workspace_bytes", "pe_verify_greedy", "pe_draft_readout",
           "pe_workspace_bytes_sampled", "pe_verify_sampled",
           "pe_build_draft_batch",
           "pe_assemble_draft_inputs", "pe_step", "pe_step_early_exit", "pe_step_noalloc",
           "pe_get_tuning",
           "pe_set_tuning", "pe_latency_floor", "pe_status_str",
           "pe_kv_append", "pe_kv_read", "pe_workspace_bytes_attn", "pe_attn_cached",
           "pe_attn_prompt", "pe_draft_sample", "pe_workspace_bytes_filtered",
           "pe_verify_filtered", "pe_workspace_bytes_weigh", "pe_kv_weigh", "pe_kv_evict")


class PEError(RuntimeError):
    def __init__(self, status: int, what: str, lib=None):
        name = lib.pe_status_str(status).decode() if lib is not None else str(status)
        super().__init__("%s failed: %s" % (what, name))
        self.status = status


P = ctypes.c_void_p
i32, i64 = ctypes.c_int32, ctypes.c_int64


class StepArgs(ctypes.Structure):
    """Mirror of pe_step_args."""
    _fields_ = [("B", i32), ("Kp", i32), ("K", i32), ("V", i32), ("H", i32), ("R", i32),
                ("mask_id", i32), ("bt_width", i32), ("block_size", i32),
                ("logits_dtype", i32), ("x_dtype", i32),
                ("logits_row_stride", i64),
                ("logits", P), ("in_offsets", P), ("in_tokens", P), ("in_positions", P),
                ("block_table", P), ("emb", P), ("target_hidden", P), ("h_shared", P),
                ("accepted_len", P), ("bonus_token", P), ("target_argmax", P),
                ("out_offsets", P), ("out_tokens", P), ("out_positions", P),
                ("is_rejected", P), ("is_masked", P), ("hidden_map", P),
                ("slot_mapping", P), ("sample_idx", P), ("X", P),
                ("workspace", P), ("err", P)]


class Tuning(ctypes.Structure):
    """Mirror of pe_tuning."""
    _fields_ = [("ctas_per_sm", i32), ("chunk_batches", i32), ("rows_per_unit", i32),
                ("variant", i32), ("queue_order", i32), ("early_full_read_mb", i32),
                ("single_pass", i32)]


class KvAppendArgs(ctypes.Structure):
    """Mirror of pe_kv_append_args."""
    _fields_ = ([(n, i32) for n in ("T", "Hq", "Hkv", "D", "block_size", "rot_dim", "interleaved",
                                    "max_pos")] +
                [(n, i64) for n in ("num_blocks", "q_row", "q_head", "k_row", "k_head", "v_row",
                                    "v_head")] +
                [(n, P) for n in ("q", "k", "v", "positions", "slots", "rope", "cache", "q_out",
                                  "k_out", "err")])


class AttnCachedArgs(ctypes.Structure):
    """Mirror of pe_attn_cached_args."""
    _fields_ = ([(n, i32) for n in ("T", "B", "Hq", "Hkv", "D", "block_size", "bt_width")] +
                [("scale", ctypes.c_float), ("num_blocks", i64)] +
                [(n, P) for n in ("q", "cache", "block_table", "offsets", "positions",
                                  "is_rejected", "out", "workspace", "err")])


class AttnPromptArgs(ctypes.Structure):
    """Mirror of pe_attn_prompt_args."""
    _fields_ = ([(n, i32) for n in ("T", "B", "Hq", "Hkv", "D")] + [("scale", ctypes.c_float)] +
                [(n, i64) for n in ("q_row", "q_head", "k_row", "k_head", "v_row", "v_head")] +
                [(n, P) for n in ("q", "k", "v", "offsets", "out", "workspace", "err")])


class DraftSampleArgs(ctypes.Structure):
    """Mirror of pe_draft_sample_args (its pe_filter's fields in place)."""
    _fields_ = ([(n, i32) for n in ("n", "requests", "rows", "V", "dtype")] + [("row_stride", i64)] +
                [(n, P) for n in ("logits", "sample_idx", "temperature", "top_k", "top_p", "min_p",
                                  "u", "out_tokens", "out_prob", "err")])


class VerifyFilteredArgs(ctypes.Structure):
    """Mirror of pe_verify_filtered_args (its pe_filter's fields in place)."""
    _fields_ = ([(n, i32) for n in ("B", "Kp", "V", "dtype")] +
                [(n, i64) for n in ("target_stride", "draft_stride")] +
                [(n, P) for n in ("target_logits", "draft_logits", "in_tokens", "u_accept", "u_draw",
                                  "temperature", "top_k", "top_p", "min_p", "accepted_len",
                                  "bonus_token", "accept_prob", "workspace", "err")])


class KvWeighArgs(ctypes.Structure):
    """Mirror of pe_kv_weigh_args."""
    _fields_ = ([(n, i32) for n in ("T", "B", "Hq", "Hkv", "D", "block_size", "bt_width")] +
                [("scale", ctypes.c_float), ("num_blocks", i64)] +
                [(n, P) for n in ("q", "cache", "block_table", "offsets", "positions",
                                  "is_rejected", "mass", "out", "fresh", "workspace", "err")])


class KvEvictArgs(ctypes.Structure):
    """Mirror of pe_kv_evict_args."""
    _fields_ = ([(n, i32) for n in ("B", "Hkv", "D", "block_size", "bt_width", "dst_width", "max_keep",
                                    "sinks", "recent")] + [("num_blocks", i64)] +
                [(n, P) for n in ("cache", "mass", "block_table", "dst_table", "lengths", "keep", "kept",
                                  "out_lengths", "err")])


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return LIB_PATH


def load():
    """Load libpe.so; raise if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            _lib = _open(LIB_PATH)
        return _lib


_checked = None


def load_checked():
    """Load libpe_checked.so (same entry points, PE_CHECKED); raise if absent."""
    global _checked
    with _lock:
        if _checked is None:
            _checked = _open(CHECKED_LIB_PATH)
        return _checked


def _open(path: str):
    if not os.path.exists(path):
        raise RuntimeError(
            "%s is not built; run speculative_decoding_pe_gb300.build.build() first -- "
            "there is no fallback path" % path)
    lib = ctypes.CDLL(path)
    lib.pe_workspace_bytes.argtypes = [i32, i32]
    lib.pe_workspace_bytes.restype = ctypes.c_size_t
    lib.pe_verify_greedy.argtypes = [P, ctypes.c_int, i64, i32, i32, i32, P, P, P,
                                     P, P, P, P]
    lib.pe_draft_readout.argtypes = [P, ctypes.c_int, i64, i32, i32, P, i32, P, P, P, P]
    lib.pe_draft_readout.restype = ctypes.c_int
    lib.pe_workspace_bytes_sampled.argtypes = [i32, i32]
    lib.pe_workspace_bytes_sampled.restype = ctypes.c_size_t
    lib.pe_verify_sampled.argtypes = [P, P, ctypes.c_int, i64, i64, i32, i32, i32, P, P,
                                      ctypes.c_float, ctypes.c_uint64, P, P, P, P, P]
    lib.pe_verify_sampled.restype = ctypes.c_int
    lib.pe_build_draft_batch.argtypes = ([i32, i32, i32, i32, i32, P, P, P, P, P, P,
                                          i32, i32] + [P] * 10)
    lib.pe_assemble_draft_inputs.argtypes = [ctypes.c_int, i32, i32, i32, i32] + [P] * 9
    lib.pe_step.argtypes = [ctypes.POINTER(StepArgs), P]
    lib.pe_step_early_exit.argtypes = [ctypes.POINTER(StepArgs), P]
    lib.pe_step_early_exit.restype = ctypes.c_int
    lib.pe_step_noalloc.argtypes = [ctypes.POINTER(StepArgs), P]
    lib.pe_step_noalloc.restype = ctypes.c_int
    lib.pe_get_tuning.argtypes = [ctypes.POINTER(Tuning)]
    lib.pe_set_tuning.argtypes = [ctypes.POINTER(Tuning)]
    lib.pe_latency_floor.argtypes = [i32, i32, P, i32, P, P]
    lib.pe_latency_floor.restype = ctypes.c_int
    lib.pe_kv_append.argtypes = [ctypes.POINTER(KvAppendArgs), P]
    lib.pe_kv_read.argtypes = [P, i64, i32, i32, i32, P, i32, P, P, P, P]
    lib.pe_workspace_bytes_attn.argtypes = [i32]
    lib.pe_workspace_bytes_attn.restype = ctypes.c_size_t
    lib.pe_attn_cached.argtypes = [ctypes.POINTER(AttnCachedArgs), P]
    lib.pe_attn_prompt.argtypes = [ctypes.POINTER(AttnPromptArgs), P]
    lib.pe_draft_sample.argtypes = [ctypes.POINTER(DraftSampleArgs), P]
    lib.pe_workspace_bytes_filtered.argtypes = [i32, i32]
    lib.pe_workspace_bytes_filtered.restype = ctypes.c_size_t
    lib.pe_verify_filtered.argtypes = [ctypes.POINTER(VerifyFilteredArgs), P]
    lib.pe_workspace_bytes_weigh.argtypes = [i32, i32, i32, i32]
    lib.pe_workspace_bytes_weigh.restype = ctypes.c_size_t
    lib.pe_kv_weigh.argtypes = [ctypes.POINTER(KvWeighArgs), P]
    lib.pe_kv_evict.argtypes = [ctypes.POINTER(KvEvictArgs), P]
    for f in ("pe_kv_append", "pe_kv_read", "pe_attn_cached", "pe_attn_prompt", "pe_draft_sample",
              "pe_verify_filtered", "pe_kv_weigh", "pe_kv_evict"):
        getattr(lib, f).restype = ctypes.c_int
    lib.pe_status_str.argtypes = [ctypes.c_int]
    lib.pe_status_str.restype = ctypes.c_char_p
    for f in ("pe_verify_greedy", "pe_build_draft_batch", "pe_assemble_draft_inputs",
              "pe_step", "pe_get_tuning", "pe_set_tuning"):
        getattr(lib, f).restype = ctypes.c_int
    return lib


# ------------------------------------------------------------------ helpers

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return PE_F32
    if t.dtype == torch.bfloat16:
        return PE_BF16
    raise TypeError("expected float32 or bfloat16, got %s" % t.dtype)


def _dev(t: torch.Tensor | None, name: str, dtype=None, numel=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if numel is not None and t.numel() < numel:
        raise ValueError("%s holds %d elements, needs %d" % (name, t.numel(), numel))
    return ctypes.c_void_p(t.data_ptr())


def _logits(t: torch.Tensor):
    if not t.is_cuda or t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("logits must be a 2-D CUDA tensor with unit column stride")
    return ctypes.c_void_p(t.data_ptr()), _dtype_code(t), t.stride(0)


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(lib, rc: int, what: str):
    if rc != 0:
        raise PEError(rc, what, lib)


# ---------------------------------------------------------------- public API

def workspace_bytes(logits_rows: int, B: int) -> int:
    return int(load().pe_workspace_bytes(logits_rows, B))


def new_workspace(logits_rows: int, B: int, device="cuda") -> torch.Tensor:
    """Zero-filled scratch for verify_greedy / step (reusable across calls)."""
    return torch.zeros(workspace_bytes(logits_rows, B), dtype=torch.uint8, device=device)


def new_error_word(device="cuda") -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def verify_greedy(logits, Kp, in_tokens, accepted_len, bonus_token, workspace, err,
                  target_argmax=None, stream=None):
    """Greedy verification of B requests (rows B*(Kp+1) of ``logits``)."""
    lib = load()
    lp, dt, stride = _logits(logits)
    rows = logits.shape[0]
    if rows % (Kp + 1):
        raise ValueError("logits rows must be a multiple of Kp+1")
    B = rows // (Kp + 1)
    rc = lib.pe_verify_greedy(
        lp, dt, stride, B, Kp, logits.shape[1],
        _dev(in_tokens, "in_tokens", torch.int32, rows if Kp else None),
        _dev(accepted_len, "accepted_len", torch.int32, B),
        _dev(bonus_token, "bonus_token", torch.int32, B),
        _dev(target_argmax, "target_argmax", torch.int32, rows),
        _dev(workspace, "workspace", torch.uint8, workspace_bytes(rows, B)),
        _dev(err, "err", torch.int32, 1), _stream(stream))
    _check(lib, rc, "pe_verify_greedy")


def workspace_bytes_sampled(B: int, Kp: int) -> int:
    return int(load().pe_workspace_bytes_sampled(B, Kp))


def verify_sampled(target_logits, draft_logits, Kp, in_tokens, u_accept, temperature, seed,
                   accepted_len, bonus_token, workspace, err, stream=None):
    """Rejection-sampling verification of B requests: target rows B*(Kp+1),
    draft rows B*Kp, accept coins u_accept[B*Kp], Philox seed for the draws."""
    lib = load()
    tp, dt, tstride = _logits(target_logits)
    rows, V = target_logits.shape
    if rows % (Kp + 1):
        raise ValueError("target_logits rows must be a multiple of Kp+1")
    B = rows // (Kp + 1)
    if Kp:
        dp, ddt, dstride = _logits(draft_logits)
        if ddt != dt or draft_logits.shape[1] != V or draft_logits.shape[0] < B * Kp:
            raise ValueError("draft_logits must be [B*Kp, V] of the target's dtype")
    else:
        dp, dstride = None, 0
    rc = lib.pe_verify_sampled(
        tp, dp, dt, tstride, dstride, B, Kp, V,
        _dev(in_tokens, "in_tokens", torch.int32, rows if Kp else None),
        _dev(u_accept, "u_accept", torch.float32, B * Kp if Kp else None),
        float(temperature), int(seed) & 0xFFFFFFFFFFFFFFFF,
        _dev(accepted_len, "accepted_len", torch.int32, B),
        _dev(bonus_token, "bonus_token", torch.int32, B),
        _dev(workspace, "workspace", torch.uint8, workspace_bytes_sampled(B, Kp)),
        _dev(err, "err", torch.int32, 1), _stream(stream))
    _check(lib, rc, "pe_verify_sampled")


def draft_readout(logits, out_tokens, workspace, err, sample_idx=None, stream=None):
    """Greedy draft tokens: argmax of logits row sample_idx[i] (row i when
    sample_idx is None) into out_tokens[i]."""
    lib = load()
    lp, dt, stride = _logits(logits)
    rows, V = logits.shape
    n = sample_idx.numel() if sample_idx is not None else out_tokens.numel()
    rc = lib.pe_draft_readout(
        lp, dt, stride, rows, V, _dev(sample_idx, "sample_idx", torch.int32, n), n,
        _dev(out_tokens, "out_tokens", torch.int32, n),
        _dev(workspace, "workspace", torch.uint8, workspace_bytes(n, n)),
        _dev(err, "err", torch.int32, 1), _stream(stream))
    _check(lib, rc, "pe_draft_readout")


@dataclass
class DraftBatch:
    """Outputs of the rebuild (and of the fused step)."""
    out_offsets: torch.Tensor
    out_tokens: torch.Tensor
    out_positions: torch.Tensor
    is_rejected: torch.Tensor
    is_masked: torch.Tensor
    hidden_map: torch.Tensor
    slot_mapping: torch.Tensor
    sample_idx: torch.Tensor | None

    @staticmethod
    def empty(B, K, R, device="cuda", sample_idx=True):
        T = R + B * (K - 1)
        e = lambda n, dt: torch.empty(n, dtype=dt, device=device)
        return DraftBatch(e(B + 1, torch.int32), e(T, torch.int32), e(T, torch.int32),
                          e(T, torch.uint8), e(T, torch.uint8), e(R, torch.int32),
                          e(T, torch.int64), e(B * K, torch.int32) if sample_idx else None)


def build_draft_batch(B, Kp, K, mask_id, R, in_offsets, in_tokens, in_positions,
                      accepted_len, bonus_token, block_table, block_size, out: DraftBatch,
                      err, stream=None):
    lib = load()
    T = R + B * (K - 1)
    if block_table.dim() != 2 or block_table.shape[0] < B:
        raise ValueError("block_table must be [B, width]")
    rc = lib.pe_build_draft_batch(
        B, Kp, K, mask_id, R, _dev(in_offsets, "in_offsets", torch.int32, B + 1),
        _dev(in_tokens, "in_tokens", torch.int32, R),
        _dev(in_positions, "in_positions", torch.int32, R),
        _dev(accepted_len, "accepted_len", torch.int32, B),
        _dev(bonus_token, "bonus_token", torch.int32, B),
        _dev(block_table, "block_table", torch.int32), block_table.shape[1], block_size,
        _dev(out.out_offsets, "out_offsets", torch.int32, B + 1),
        _dev(out.out_tokens, "out_tokens", torch.int32, T),
        _dev(out.out_positions, "out_positions", torch.int32, T),
        _dev(out.is_rejected, "is_rejected", torch.uint8, T),
        _dev(out.is_masked, "is_masked", torch.uint8, T),
        _dev(out.hidden_map, "hidden_map", torch.int32, R),
        _dev(out.slot_mapping, "slot_mapping", torch.int64, T),
        _dev(out.sample_idx, "sample_idx", torch.int32, B * K),
        _dev(err, "err", torch.int32, 1), _stream(stream))
    _check(lib, rc, "pe_build_draft_batch")


def assemble_draft_inputs(emb, target_hidden, h_shared, out_tokens, hidden_map,
                          is_masked, X, err, stream=None):
    lib = load()
    V, H = emb.shape
    T, R = out_tokens.numel(), hidden_map.numel()
    dt = _dtype_code(emb)
    for name, t in (("target_hidden", target_hidden), ("h_shared", h_shared), ("X", X)):
        if t.dtype != emb.dtype:
            raise TypeError("%s must match the embedding dtype" % name)
    rc = lib.pe_assemble_draft_inputs(
        dt, H, V, T, R, _dev(emb, "emb"), _dev(target_hidden, "target_hidden", None, R * H),
        _dev(h_shared, "h_shared", None, H), _dev(out_tokens, "out_tokens", torch.int32),
        _dev(hidden_map, "hidden_map", torch.int32), _dev(is_masked, "is_masked", torch.uint8, T),
        _dev(X, "X", None, T * 2 * H), _dev(err, "err", torch.int32, 1), _stream(stream))
    _check(lib, rc, "pe_assemble_draft_inputs")


@dataclass
class StepOutputs(DraftBatch):
    accepted_len: torch.Tensor = None
    bonus_token: torch.Tensor = None
    target_argmax: torch.Tensor | None = None
    X: torch.Tensor = None

    @staticmethod
    def empty(B, Kp, K, R, H, dtype, device="cuda", sample_idx=True, target_argmax=True):
        d = DraftBatch.empty(B, K, R, device, sample_idx)
        T = R + B * (K - 1)
        return StepOutputs(**d.__dict__,
                           accepted_len=torch.empty(B, dtype=torch.int32, device=device),
                           bonus_token=torch.empty(B, dtype=torch.int32, device=device),
                           target_argmax=(torch.empty(B * (Kp + 1), dtype=torch.int32,
                                                      device=device) if target_argmax else None),
                           X=torch.empty(T, 2 * H, dtype=dtype, device=device))


def make_step_args(*, logits, Kp, K, mask_id, in_offsets, in_tokens, in_positions,
                   block_table, block_size, emb, target_hidden, h_shared,
                   out: StepOutputs, workspace, err) -> StepArgs:
    """Check the tensors once and pack a pe_step_args (reusable while the
    same tensors stay alive)."""
    lp, ldt, stride = _logits(logits)
    V, H = emb.shape
    if logits.shape[1] != V:
        raise ValueError("logits width must equal the vocabulary size")
    rows = logits.shape[0]
    if rows % (Kp + 1):
        raise ValueError("logits rows must be a multiple of Kp+1")
    B = rows // (Kp + 1)
    R = in_tokens.numel()
    T = R + B * (K - 1)
    a = StepArgs()
    a.B, a.Kp, a.K, a.V, a.H, a.R = B, Kp, K, V, H, R
    a.mask_id, a.bt_width, a.block_size = mask_id, block_table.shape[1], block_size
    a.logits_dtype, a.x_dtype = ldt, _dtype_code(emb)
    a.logits_row_stride = stride
    a.logits = lp
    a.in_offsets = _dev(in_offsets, "in_offsets", torch.int32, B + 1)
    a.in_tokens = _dev(in_tokens, "in_tokens", torch.int32, R)
    a.in_positions = _dev(in_positions, "in_positions", torch.int32, R)
    a.block_table = _dev(block_table, "block_table", torch.int32)
    a.emb = _dev(emb, "emb")
    a.target_hidden = _dev(target_hidden, "target_hidden", emb.dtype, R * H)
    a.h_shared = _dev(h_shared, "h_shared", emb.dtype, H)
    a.accepted_len = _dev(out.accepted_len, "accepted_len", torch.int32, B)
    a.bonus_token = _dev(out.bonus_token, "bonus_token", torch.int32, B)
    a.target_argmax = _dev(out.target_argmax, "target_argmax", torch.int32, rows)
    a.out_offsets = _dev(out.out_offsets, "out_offsets", torch.int32, B + 1)
    a.out_tokens = _dev(out.out_tokens, "out_tokens", torch.int32, T)
    a.out_positions = _dev(out.out_positions, "out_positions", torch.int32, T)
    a.is_rejected = _dev(out.is_rejected, "is_rejected", torch.uint8, T)
    a.is_masked = _dev(out.is_masked, "is_masked", torch.uint8, T)
    a.hidden_map = _dev(out.hidden_map, "hidden_map", torch.int32, R)
    a.slot_mapping = _dev(out.slot_mapping, "slot_mapping", torch.int64, T)
    a.sample_idx = _dev(out.sample_idx, "sample_idx", torch.int32, B * K)
    a.X = _dev(out.X, "X", emb.dtype, T * 2 * H)
    a.workspace = _dev(workspace, "workspace", torch.uint8, workspace_bytes(rows, B))
    a.err = _dev(err, "err", torch.int32, 1)
    return a


def step_packed(args: StepArgs, stream=None):
    """Launch the fused step from a packed argument block."""
    lib = load()
    _check(lib, lib.pe_step(ctypes.byref(args), _stream(stream)), "pe_step")


def step_early_exit_packed(args: StepArgs, stream=None):
    """The fused step with early exit (rows after each request's first
    mismatch are not read; target_argmax holds -1 for them)."""
    lib = load()
    _check(lib, lib.pe_step_early_exit(ctypes.byref(args), _stream(stream)),
           "pe_step_early_exit")


def step(**kw):
    """The whole step (verify, rebuild, assemble) in one launch; see
    make_step_args for the arguments and an optional ``stream``."""
    stream = kw.pop("stream", None)
    step_packed(make_step_args(**kw), stream)


def latency_floor(ctas: int, hops: int = 0, chain=None, out=None, stream=None):
    """An empty launch of ``ctas`` CTAs, plus ``hops`` dependent loads through
    ``chain`` (int32, entry i = index of the next) ending in ``out[0]``."""
    lib = load()
    n = chain.numel() if chain is not None else 0
    rc = lib.pe_latency_floor(ctas, hops, _dev(chain, "chain", torch.int32), n,
                              _dev(out, "out", torch.int32, 1), _stream(stream))
    _check(lib, rc, "pe_latency_floor")


# ------------------------------------------------ the drafter layer's attention

# These calls are short next to what Python spends on checking their arguments,
# so each check reads a tensor's properties once.

_BF16 = torch.bfloat16


def _raw_stream(stream, t: torch.Tensor) -> int:
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(t.device.index)


_here = contextlib.nullcontext()


def _on(t: torch.Tensor, *others):
    """The device that all the tensors lie on, as the current one during the call."""
    dev = t.device
    for x in others:
        if x is not None and x.device != dev:
            raise ValueError("all tensors must be on one device, got %s and %s" % (dev, x.device))
    return _here if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _rows(t: torch.Tensor, name: str, shape):
    """Pointer and strides of bf16 rows [T, heads, D] with dense elements."""
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype is not _BF16:
        raise TypeError("%s must be bfloat16, got %s" % (name, t.dtype))
    row, head, elt = t.stride()
    if elt != 1 and shape[2] > 1:
        raise ValueError("%s must have unit element stride" % name)
    # the stride of an axis of one element is never used
    return t.data_ptr(), row if shape[0] > 1 else 0, head if shape[1] > 1 else 0


def _heads(t: torch.Tensor, name: str):
    if t.dim() != 3:
        raise ValueError("%s must be [T, heads, D]" % name)
    return t.shape


def _dense(t: torch.Tensor | None, name: str, shape):
    """Pointer of a contiguous bf16 tensor of the given shape."""
    if t is None:
        return None
    if t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor %s" % (name, list(shape)))
    if t.dtype is not _BF16:
        raise TypeError("%s must be bfloat16, got %s" % (name, t.dtype))
    return t.data_ptr()


def _cache(t: torch.Tensor):
    """Pointer, blocks, block size, heads and head size of a 4-bit cache."""
    if not t.is_cuda or t.dim() != 4 or t.dtype is not torch.uint8 or not t.is_contiguous():
        raise ValueError("cache must be a contiguous uint8 CUDA tensor "
                         "[num_blocks, Hkv, block_size/16, 18*D]")
    blocks, Hkv, sub, rec = t.shape
    if rec % 18:
        raise ValueError("cache of shape %s does not hold records of 18*D bytes" % list(t.shape))
    return t.data_ptr(), blocks, 16 * sub, Hkv, rec // 18


def _vector(t: torch.Tensor | None, name: str, dtype, n: int):
    """Pointer of a contiguous tensor of exactly n elements."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor of %d elements" % (name, n))
    return t.data_ptr()


def _scratch(workspace, err, D: int):
    if not workspace.is_cuda or workspace.dtype is not torch.uint8 or \
            not workspace.is_contiguous() or workspace.numel() < workspace_bytes_attn(D):
        raise ValueError("workspace must be what new_attn_workspace(%d) gives" % D)
    return workspace.data_ptr(), _vector(err, "err", torch.int32, 1)


def new_kv_cache(num_blocks: int, block_size: int, Hkv: int, D: int, device="cuda") -> torch.Tensor:
    """A zeroed 4-bit paged KV cache (see include/pe_api.h for the layout):
    1.125 bytes per element pair of key and value."""
    if num_blocks < 1 or Hkv < 1 or D not in (64, 128) or block_size < 16 or block_size % 16:
        raise ValueError("need num_blocks >= 1, Hkv >= 1, D 64 or 128, block_size a multiple of 16")
    return torch.zeros(num_blocks, Hkv, block_size // 16, 18 * D, dtype=torch.uint8, device=device)


def rope_table(max_pos: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """fp32 [max_pos, rot_dim]: cos then sin of pos * base^(-2i/rot_dim), the
    angles in fp64 so that far positions keep their digits."""
    inv = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float()


def kv_append(q, k, v, positions, slots, rope, cache, q_out, err, k_out=None, interleaved=False,
              stream=None):
    """Rotate q and k by position; write k and v into ``cache`` at ``slots``
    (slot_mapping of the draft batch: -1 writes nothing); q_out (and k_out)
    take the rotated rows."""
    lib = _lib or load()
    cp, blocks, bs, Hkv, D = _cache(cache)
    T, Hq, _ = _heads(q, "q")
    qs, ks = (T, Hq, D), (T, Hkv, D)
    qp, q_row, q_head = _rows(q, "q", qs)
    kp, k_row, k_head = _rows(k, "k", ks)
    vp, v_row, v_head = _rows(v, "v", ks)
    if rope.dim() != 2:
        raise ValueError("rope must be [max_pos, rot_dim]")
    max_pos, rot = rope.shape
    a = KvAppendArgs(T, Hq, Hkv, D, bs, rot, 1 if interleaved else 0, max_pos, blocks, q_row, q_head,
                     k_row, k_head, v_row, v_head, qp, kp, vp,
                     _vector(positions, "positions", torch.int32, T),
                     _vector(slots, "slots", torch.int64, T),
                     _vector(rope, "rope", torch.float32, max_pos * rot), cp,
                     _dense(q_out, "q_out", qs), _dense(k_out, "k_out", ks),
                     _vector(err, "err", torch.int32, 1))
    _check(lib, lib.pe_kv_append(ctypes.byref(a), _raw_stream(stream, q)), "pe_kv_append")


def kv_read(cache, slots, k_out, v_out, err, stream=None):
    """The values that ``cache`` holds at ``slots``, as bf16 rows [n, Hkv, D]
    (zeros for slot -1); either output may be None."""
    lib = _lib or load()
    cp, nb, bs, Hkv, D = _cache(cache)
    n = slots.numel()
    rc = lib.pe_kv_read(cp, nb, bs, Hkv, D, _vector(slots, "slots", torch.int64, n), n,
                        _dense(k_out, "k_out", (n, Hkv, D)), _dense(v_out, "v_out", (n, Hkv, D)),
                        _vector(err, "err", torch.int32, 1), _raw_stream(stream, cache))
    _check(lib, rc, "pe_kv_read")


_attn_bytes = {}  # by head size: constants of the library


def workspace_bytes_attn(D: int) -> int:
    if D not in _attn_bytes:
        _attn_bytes[D] = int(load().pe_workspace_bytes_attn(D))
    return _attn_bytes[D]


def new_attn_workspace(D: int, device="cuda") -> torch.Tensor:
    """Zero-filled scratch for attn_cached / attn_prompt (reusable)."""
    return torch.zeros(workspace_bytes_attn(D), dtype=torch.uint8, device=device)


def attn_cached(q, cache, block_table, offsets, positions, is_rejected, out, workspace, err,
                scale=None, stream=None):
    """Attention of the packed rows over their requests' cached keys
    (0..positions[t]; rejected rows give zeros).  offsets [B+1], or None for
    equal segments; scale defaults to D**-0.5."""
    lib = _lib or load()
    cp, blocks, bs, Hkv, D = _cache(cache)
    T, Hq, _ = _heads(q, "q")
    shape = (T, Hq, D)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, width]")
    B, width = block_table.shape
    ws, ep = _scratch(workspace, err, D)
    a = AttnCachedArgs(T, B, Hq, Hkv, D, bs, width, D ** -0.5 if scale is None else scale, blocks,
                       _dense(q, "q", shape), cp,
                       _vector(block_table, "block_table", torch.int32, B * width),
                       _vector(offsets, "offsets", torch.int32, B + 1),
                       _vector(positions, "positions", torch.int32, T),
                       _vector(is_rejected, "is_rejected", torch.uint8, T),
                       _dense(out, "out", shape), ws, ep)
    _check(lib, lib.pe_attn_cached(ctypes.byref(a), _raw_stream(stream, q)), "pe_attn_cached")


def attn_prompt(q, k, v, offsets, out, workspace, err, scale=None, B=None, stream=None):
    """Causal attention over packed prompts.  offsets [B+1], or None for B
    equal segments; scale defaults to D**-0.5."""
    lib = _lib or load()
    shape = _heads(q, "q")
    T, Hq, D = shape
    Hkv = _heads(k, "k")[1]
    qp, q_row, q_head = _rows(q, "q", shape)
    kp, k_row, k_head = _rows(k, "k", (T, Hkv, D))
    vp, v_row, v_head = _rows(v, "v", (T, Hkv, D))
    if offsets is not None:
        B = offsets.numel() - 1
    elif B is None:
        raise ValueError("offsets or B is needed")
    ws, ep = _scratch(workspace, err, D)
    a = AttnPromptArgs(T, B, Hq, Hkv, D, D ** -0.5 if scale is None else scale, q_row, q_head,
                       k_row, k_head, v_row, v_head, qp, kp, vp,
                       _vector(offsets, "offsets", torch.int32, B + 1),
                       _dense(out, "out", shape), ws, ep)
    _check(lib, lib.pe_attn_prompt(ctypes.byref(a), _raw_stream(stream, q)), "pe_attn_prompt")


# ------------------------------------------------------------- a bounded cache

def new_kv_mass(cache: torch.Tensor) -> torch.Tensor:
    """Zeroed attention weights [num_blocks, Hkv, block_size] of a cache's keys."""
    blocks, Hkv, sub, _ = cache.shape
    return torch.zeros(blocks, Hkv, 16 * sub, dtype=torch.float32, device=cache.device)


def workspace_bytes_weigh(T: int, Hq: int, bt_width: int, block_size: int) -> int:
    return int(load().pe_workspace_bytes_weigh(T, Hq, bt_width, block_size))


def new_weigh_workspace(T: int, Hq: int, bt_width: int, block_size: int, device="cuda") -> torch.Tensor:
    """Scratch for kv_weigh of up to T rows of Hq heads over tables of bt_width pages (reusable)."""
    return torch.empty(workspace_bytes_weigh(T, Hq, bt_width, block_size), dtype=torch.uint8, device=device)


def kv_weigh(q, cache, block_table, offsets, positions, is_rejected, mass, out, workspace, err,
             fresh=None, scale=None, stream=None):
    """Add the attention weight that the packed rows give to every cached key they
    see to ``mass`` (new_kv_mass; None: nothing yet), into ``out`` (it may be
    mass); keys from fresh[b] on start from nothing.  Rows as in attn_cached."""
    lib = _lib or load()
    cp, blocks, bs, Hkv, D = _cache(cache)
    T, Hq, _ = _heads(q, "q")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, width]")
    B, width = block_table.shape
    n = blocks * Hkv * bs
    if not workspace.is_cuda or workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or \
            workspace.numel() < lib.pe_workspace_bytes_weigh(T, Hq, width, bs):
        raise ValueError("workspace must be what new_weigh_workspace(%d, %d, %d, %d) gives" % (T, Hq, width, bs))
    a = KvWeighArgs(T, B, Hq, Hkv, D, bs, width, D ** -0.5 if scale is None else scale, blocks,
                    _dense(q, "q", (T, Hq, D)), cp,
                    _vector(block_table, "block_table", torch.int32, B * width),
                    _vector(offsets, "offsets", torch.int32, B + 1),
                    _vector(positions, "positions", torch.int32, T),
                    _vector(is_rejected, "is_rejected", torch.uint8, T),
                    _vector(mass, "mass", torch.float32, n), _vector(out, "out", torch.float32, n),
                    _vector(fresh, "fresh", torch.int32, B), workspace.data_ptr(),
                    _vector(err, "err", torch.int32, 1))
    with _on(q, cache, block_table, offsets, positions, is_rejected, mass, out, workspace, fresh, err):
        _check(lib, lib.pe_kv_weigh(ctypes.byref(a), _raw_stream(stream, q)), "pe_kv_weigh")


def kv_evict(cache, mass, block_table, dst_table, lengths, keep, kept, out_lengths, err, sinks=0, recent=0,
             stream=None):
    """Per request and key head, keep the first ``sinks``, the last ``recent`` and
    the heaviest of the others of the lengths[b] cached keys, keep[b] in all: in
    ascending order at the front of dst_table's pages (block_table itself: in
    place), their weights too, their indices in kept [B, Hkv, max_keep], how many
    in out_lengths."""
    lib = _lib or load()
    cp, blocks, bs, Hkv, D = _cache(cache)
    if block_table.dim() != 2 or dst_table.dim() != 2 or dst_table.shape[0] != block_table.shape[0]:
        raise ValueError("block_table must be [B, width], dst_table [B, dst_width]")
    B, width = block_table.shape
    if kept.dim() != 3 or kept.shape[:2] != (B, Hkv):
        raise ValueError("kept must be [B, Hkv, max_keep]")
    a = KvEvictArgs(B, Hkv, D, bs, width, dst_table.shape[1], kept.shape[2], sinks, recent, blocks, cp,
                    _vector(mass, "mass", torch.float32, blocks * Hkv * bs),
                    _vector(block_table, "block_table", torch.int32, B * width),
                    _vector(dst_table, "dst_table", torch.int32, dst_table.numel()),
                    _vector(lengths, "lengths", torch.int32, B), _vector(keep, "keep", torch.int32, B),
                    _vector(kept, "kept", torch.int32, kept.numel()),
                    _vector(out_lengths, "out_lengths", torch.int32, B), _vector(err, "err", torch.int32, 1))
    with _on(cache, mass, block_table, dst_table, lengths, keep, kept, out_lengths, err):
        _check(lib, lib.pe_kv_evict(ctypes.byref(a), _raw_stream(stream, cache)), "pe_kv_evict")


# ------------------------------------------------------------ filtered sampling

def _columns(t: torch.Tensor, name: str):
    """Pointer, element type and row stride of logits rows [rows, V]."""
    if not t.is_cuda or t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError("%s must be a 2-D CUDA tensor with unit column stride" % name)
    rows, V = t.shape
    # the stride of one row is never used
    return t.data_ptr(), _dtype_code(t), t.stride(0) if rows > 1 else -(-V // 8) * 8


def _filter(temperature, top_k, top_p, min_p, n: int):
    """Pointers of the parameter arrays of n requests."""
    return (_vector(temperature, "temperature", torch.float32, n), _vector(top_k, "top_k", torch.int32, n),
            _vector(top_p, "top_p", torch.float32, n), _vector(min_p, "min_p", torch.float32, n))


def draft_sample(logits, u, out_tokens, err, temperature=None, top_k=None, top_p=None, min_p=None,
                 out_prob=None, sample_idx=None, stream=None):
    """Sampled draft tokens: out_tokens[i] is drawn by u[i] from the distribution
    of logits row sample_idx[i] (row i when None) under temperature, top-k, top-p
    and min-p: arrays of one entry per request, rows request after request, or
    None (1, off, off, off).  out_prob takes the tokens' probabilities."""
    lib = _lib or load()
    lp, dt, stride = _columns(logits, "logits")
    rows, V = logits.shape
    n = u.numel()
    counts = {t.numel() for t in (temperature, top_k, top_p, min_p) if t is not None} or {1}
    requests = counts.pop()
    if counts or n and (not requests or n % requests):
        raise ValueError("the parameters must have one entry per request, and %d rows share them evenly" % n)
    a = DraftSampleArgs(n, requests, rows, V, dt, stride, lp, _vector(sample_idx, "sample_idx", torch.int32, n),
                        *_filter(temperature, top_k, top_p, min_p, requests),
                        _vector(u, "u", torch.float32, n), _vector(out_tokens, "out_tokens", torch.int32, n),
                        _vector(out_prob, "out_prob", torch.float32, n), _vector(err, "err", torch.int32, 1))
    with _on(logits, u, out_tokens, err, temperature, top_k, top_p, min_p, out_prob, sample_idx):
        _check(lib, lib.pe_draft_sample(ctypes.byref(a), _raw_stream(stream, logits)), "pe_draft_sample")


def workspace_bytes_filtered(B: int, Kp: int) -> int:
    return int(load().pe_workspace_bytes_filtered(B, Kp))


def new_filtered_workspace(B: int, Kp: int, device="cuda") -> torch.Tensor:
    """Scratch for verify_filtered of up to B requests of depth Kp (reusable)."""
    return torch.empty(workspace_bytes_filtered(B, Kp), dtype=torch.uint8, device=device)


def verify_filtered(target_logits, draft_logits, Kp, in_tokens, u_accept, u_draw, accepted_len, bonus_token,
                    workspace, err, temperature=None, top_k=None, top_p=None, min_p=None, accept_prob=None,
                    stream=None):
    """Rejection sampling of B requests' drafts against the filtered
    distributions that draft_sample draws from: target rows B*(Kp+1), draft rows
    B*Kp, accept coins u_accept[B*Kp], u_draw[B] for the bonus tokens; parameters
    of one entry per request, or None.  accept_prob takes min(1, p/q) of every
    draft."""
    lib = _lib or load()
    tp, dt, t_stride = _columns(target_logits, "target_logits")
    rows, V = target_logits.shape
    if Kp < 0 or rows % (Kp + 1):
        raise ValueError("target_logits rows must be a multiple of Kp+1")
    B = rows // (Kp + 1)
    dp, d_stride = None, 0
    if Kp:
        dp, ddt, d_stride = _columns(draft_logits, "draft_logits")
        if ddt != dt or draft_logits.shape != (B * Kp, V):
            raise ValueError("draft_logits must be [B*Kp, V] of the target's dtype")
    need = lib.pe_workspace_bytes_filtered(B, Kp)
    if not workspace.is_cuda or workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or \
            workspace.numel() < need:
        raise ValueError("workspace must be what new_filtered_workspace(%d, %d) gives" % (B, Kp))
    a = VerifyFilteredArgs(B, Kp, V, dt, t_stride, d_stride, tp, dp,
                           _vector(in_tokens, "in_tokens", torch.int32, rows) if Kp else None,
                           _vector(u_accept, "u_accept", torch.float32, B * Kp) if Kp else None,
                           _vector(u_draw, "u_draw", torch.float32, B),
                           *_filter(temperature, top_k, top_p, min_p, B),
                           _vector(accepted_len, "accepted_len", torch.int32, B),
                           _vector(bonus_token, "bonus_token", torch.int32, B),
                           _vector(accept_prob, "accept_prob", torch.float32, B * Kp),
                           workspace.data_ptr(), _vector(err, "err", torch.int32, 1))
    with _on(target_logits, draft_logits if Kp else None, in_tokens if Kp else None, u_accept if Kp else None, u_draw,
             accepted_len, bonus_token, workspace, err, temperature, top_k, top_p, min_p, accept_prob):
        _check(lib, lib.pe_verify_filtered(ctypes.byref(a), _raw_stream(stream, target_logits)), "pe_verify_filtered")


def get_tuning() -> dict:
    lib = load()
    t = Tuning()
    _check(lib, lib.pe_get_tuning(ctypes.byref(t)), "pe_get_tuning")
    return {f: getattr(t, f) for f, _ in Tuning._fields_}


def set_tuning(**kw):
    lib = load()
    t = Tuning(**{f: int(kw.get(f, 0)) for f, _ in Tuning._fields_})
    _check(lib, lib.pe_set_tuning(ctypes.byref(t)), "pe_set_tuning")
