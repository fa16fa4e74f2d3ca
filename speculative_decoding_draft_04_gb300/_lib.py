"""ctypes binding of libspec.so: the C ABI of include/spec.h, same names.

Argument marshalling only -- every step of the path runs in the library's
CUDA kernels.  Tensors are torch CUDA tensors (torch is used for device
memory and streams); pointers, sizes and the stream handle are passed as
plain integers.  There is no CPU fallback: if the library is missing or a
call fails, a SpecError is raised.
"""
from __future__ import annotations

import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libspec.so")

SPEC_F32, SPEC_BF16 = 0, 1
SPEC_OPT_EPS_SCALE, SPEC_OPT_FORCE_SIMT, SPEC_OPT_BIAS_PATH, SPEC_OPT_TRACE = 1, 2, 3, 5
SPEC_OPT_PERTURB = 6
SPEC_OPT_TEST_STALL = 7
SPEC_OPT_DRAFT_KERNEL = 8
SPEC_OPT_VERIFY_KERNEL = 9
DEV_BITS = {1: "BAD_TOKEN", 2: "BAD_LEN", 4: "BAD_TEMP", 8: "TIMEOUT", 16: "REFINED",
            32: "OVERFLOW", 64: "BAD_CONF", 128: "BAD_TREE", 256: "NO_PAGES", 512: "BAD_SLOT",
            1024: "BAD_LOGIT", 2048: "BAD_KV", 4096: "BAD_FILTER", 8192: "BAD_POSITION"}

EXPORTED = ("spec_workspace_bytes", "spec_markov_draft", "spec_markov_draft_static",
            "spec_verify", "spec_status_string",
            "spec_set_option", "spec_profile_enable", "spec_profile_read", "spec_stage_name",
            "spec_num_stages", "spec_operating_point", "spec_acceptance_stats",
            "spec_confidence", "spec_schedule_workspace_bytes", "spec_prefix_schedule",
            "spec_rnn_draft", "spec_tree_select", "spec_tree_draft", "spec_tree_verify",
            "spec_tree_workspace_bytes", "spec_cycle_host", "spec_cache_bytes",
            "spec_block_tables", "spec_cache_append", "spec_cache_attention_workspace_bytes",
            "spec_cache_attention", "spec_logprobs_workspace_bytes", "spec_logprobs",
            "spec_rotary_append", "spec_prefix_attention_workspace_bytes", "spec_prefix_attention",
            "spec_sample")


class SpecError(RuntimeError):
    pass


_i32, _vp, _sz = ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
_i64, _f32 = ctypes.c_int64, ctypes.c_float


class DraftArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("gamma", _i32), ("V", _i32), ("r", _i32), ("dtype", _i32),
                ("U", _vp), ("W1", _vp), ("W2", _vp), ("anchor", _vp), ("temperature", _vp),
                ("u_draft", _vp), ("draft_tokens", _vp), ("q_tok", _vp), ("lse_q", _vp),
                ("dev_status", _vp), ("diag", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class VerifyArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("gamma", _i32), ("V", _i32), ("r", _i32), ("dtype", _i32),
                ("target", _vp), ("U", _vp), ("W1", _vp), ("W2", _vp), ("anchor", _vp),
                ("temperature", _vp), ("draft_tokens", _vp), ("q_tok", _vp), ("lse_q", _vp),
                ("verify_len", _vp), ("u_accept", _vp), ("u_final", _vp), ("accept_len", _vp),
                ("out_tokens", _vp), ("alpha", _vp), ("p_tok", _vp), ("dev_status", _vp),
                ("a_rows", _vp), ("diag", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class CycleHostArgs(ctypes.Structure):
    _fields_ = [("draft", DraftArgs), ("verify", VerifyArgs), ("h_U", _vp), ("h_target", _vp),
                ("h_anchor", _vp), ("h_temperature", _vp), ("h_u_draft", _vp),
                ("h_verify_len", _vp), ("h_u_accept", _vp), ("h_u_final", _vp),
                ("h_accept_len", _vp), ("h_out_tokens", _vp), ("h_draft_tokens", _vp),
                ("h_alpha", _vp), ("copy_stream", _vp)]


class RnnDraftArgs(ctypes.Structure):
    _fields_ = [("draft", DraftArgs), ("Wr", _vp), ("hproj", _vp), ("a_rows", _vp)]


_LIB = None


class OpArgs(ctypes.Structure):
    _fields_ = [("alpha", ctypes.c_double), ("c", ctypes.c_double), ("c_hat", ctypes.c_double),
                ("gamma", ctypes.c_int32), ("gamma_max", ctypes.c_int32)]


class OpResult(ctypes.Structure):
    _fields_ = [("expected_tau", ctypes.c_double), ("speedup", ctypes.c_double),
                ("speedup_gamma1", ctypes.c_double), ("bound", ctypes.c_double),
                ("gamma_continuous", ctypes.c_double), ("speedup_star", ctypes.c_double),
                ("compute_ratio", ctypes.c_double), ("gamma_star", ctypes.c_int32),
                ("gains", ctypes.c_int32)]


class ConfidenceArgs(ctypes.Structure):
    _fields_ = [("R", _i32), ("gamma", _i32), ("d", _i32), ("V", _i32), ("r", _i32),
                ("dtype", _i32), ("hidden", _vp), ("W1", _vp), ("w", _vp), ("anchor", _vp),
                ("draft_tokens", _vp), ("conf", _vp), ("dev_status", _vp)]


class ScheduleArgs(ctypes.Structure):
    _fields_ = [("R", _i32), ("gamma", _i32), ("conf", _vp), ("sps", _vp), ("sps_len", _i32),
                ("survival", _vp), ("verify_len", _vp), ("totals", _vp), ("theta", _vp),
                ("dev_status", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class TreeDraftArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("N", _i32), ("gamma", _i32), ("V", _i32), ("r", _i32),
                ("dtype", _i32), ("U", _vp), ("W1", _vp), ("W2", _vp), ("anchor", _vp),
                ("temperature", _vp), ("parent", _vp), ("mask", _vp), ("u_draft", _vp),
                ("tokens", _vp), ("q_tok", _vp), ("dev_status", _vp), ("workspace", _vp),
                ("workspace_bytes", _sz)]


class TreeVerifyArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("N", _i32), ("gamma", _i32), ("V", _i32), ("r", _i32),
                ("dtype", _i32), ("target", _vp), ("U", _vp), ("W1", _vp), ("W2", _vp),
                ("anchor", _vp), ("temperature", _vp), ("parent", _vp), ("mask", _vp),
                ("tokens", _vp), ("u_accept", _vp), ("u_final", _vp), ("accept_len", _vp),
                ("out_tokens", _vp), ("path", _vp), ("dev_status", _vp), ("workspace", _vp),
                ("workspace_bytes", _sz)]


class BlockTablesArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("page_size", _i32), ("num_pages", _i32), ("table_stride", _i32),
                ("max_rows", _i32), ("seq_len", _vp), ("accept_len", _vp), ("new_len", _vp),
                ("num_blocks", _vp), ("ring_pos", _vp), ("free_ring", _vp), ("block_table", _vp),
                ("seq_len_out", _vp), ("kv_len", _vp), ("num_blocks_out", _vp),
                ("ring_pos_out", _vp), ("row_ptr", _vp), ("slots", _vp), ("positions", _vp),
                ("dev_status", _vp)]


class CacheAppendArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("Hkv", _i32), ("D", _i32), ("dtype", _i32), ("page_size", _i32),
                ("num_pages", _i32), ("k", _vp), ("v", _vp), ("k_row_stride", _i64),
                ("k_head_stride", _i64), ("v_row_stride", _i64), ("v_head_stride", _i64),
                ("slots", _vp), ("k_scale", _f32), ("v_scale", _f32), ("cache", _vp),
                ("k_stored", _vp), ("v_stored", _vp), ("dev_status", _vp)]


class CacheAttentionArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("Hq", _i32), ("Hkv", _i32), ("D", _i32),
                ("dtype", _i32), ("page_size", _i32), ("num_pages", _i32), ("table_stride", _i32),
                ("mask_words", _i32), ("q", _vp), ("q_row_stride", _i64), ("q_head_stride", _i64),
                ("cache", _vp), ("block_table", _vp), ("kv_len", _vp), ("row_ptr", _vp),
                ("tree_mask", _vp), ("softmax_scale", _f32), ("k_scale", _f32), ("v_scale", _f32),
                ("out", _vp), ("lse", _vp), ("dev_status", _vp), ("workspace", _vp),
                ("workspace_bytes", _sz)]


class PrefixAttentionArgs(ctypes.Structure):
    _fields_ = [("own", CacheAttentionArgs), ("groups", _i32), ("prefix_stride", _i32),
                ("prefix_table", _vp), ("prefix_len", _vp), ("group_ptr", _vp)]


class RotaryAppendArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("Hq", _i32), ("Hkv", _i32), ("D", _i32), ("R", _i32), ("dtype", _i32),
                ("page_size", _i32), ("num_pages", _i32), ("rope_rows", _i32), ("interleaved", _i32),
                ("q", _vp), ("k", _vp), ("v", _vp), ("q_row_stride", _i64), ("q_head_stride", _i64),
                ("k_row_stride", _i64), ("k_head_stride", _i64), ("v_row_stride", _i64),
                ("v_head_stride", _i64), ("q_weight", _vp), ("k_weight", _vp), ("positions", _vp),
                ("slots", _vp), ("rope", _vp), ("eps", _f32), ("k_scale", _f32), ("v_scale", _f32),
                ("q_out", _vp), ("q_out_row_stride", _i64), ("q_out_head_stride", _i64),
                ("cache", _vp), ("k_stored", _vp), ("v_stored", _vp), ("dev_status", _vp)]


class SampleArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("n", _i32), ("V", _i32), ("dtype", _i32), ("logits", _vp),
                ("b_stride", _i64), ("row_stride", _i64), ("u", _vp), ("temperature", _vp),
                ("top_k", _vp), ("top_p", _vp), ("min_p", _vp), ("tokens", _vp), ("logprob", _vp),
                ("kept", _vp), ("dev_status", _vp)]


class LogprobsArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("n", _i32), ("V", _i32), ("K", _i32), ("dtype", _i32),
                ("logits", _vp), ("b_stride", _i64), ("row_stride", _i64), ("tokens", _vp),
                ("temperature", _vp), ("logprob", _vp), ("entropy", _vp), ("top_ids", _vp),
                ("top_logprobs", _vp), ("dev_status", _vp), ("workspace", _vp),
                ("workspace_bytes", _sz)]


def lib(path: str | None = None) -> ctypes.CDLL:
    """Load libspec.so (built in-tree by build.build())."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise SpecError(f"{p} is missing: build it with speculative_decoding_draft_04_gb300."
                        "build.build() (there is no CPU fallback)")
    L = ctypes.CDLL(p)
    L.spec_workspace_bytes.restype = _sz
    L.spec_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32]
    L.spec_markov_draft.restype = _i32
    L.spec_markov_draft.argtypes = [ctypes.POINTER(DraftArgs), _vp]
    L.spec_markov_draft_static.restype = _i32
    L.spec_markov_draft_static.argtypes = [ctypes.POINTER(DraftArgs), _vp]
    L.spec_cycle_host.restype = _i32
    L.spec_cycle_host.argtypes = [ctypes.POINTER(CycleHostArgs), _vp]
    L.spec_verify.restype = _i32
    L.spec_verify.argtypes = [ctypes.POINTER(VerifyArgs), _vp]
    L.spec_status_string.restype = ctypes.c_char_p
    L.spec_status_string.argtypes = [_i32]
    L.spec_set_option.restype = _i32
    L.spec_set_option.argtypes = [_i32, ctypes.c_double]
    L.spec_profile_enable.restype = _i32
    L.spec_profile_enable.argtypes = [_i32]
    L.spec_profile_read.restype = _i32
    L.spec_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_i32), _i32]
    L.spec_stage_name.restype = ctypes.c_char_p
    L.spec_stage_name.argtypes = [_i32]
    L.spec_num_stages.restype = _i32
    L.spec_num_stages.argtypes = []
    L.spec_operating_point.restype = _i32
    L.spec_operating_point.argtypes = [ctypes.POINTER(OpArgs), ctypes.POINTER(OpResult)]
    L.spec_acceptance_stats.restype = _i32
    L.spec_acceptance_stats.argtypes = [_i32, _i32, _vp, _vp, _vp, _vp, _vp]
    L.spec_tree_select.restype = _i32
    L.spec_tree_select.argtypes = [_i32, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp]
    L.spec_tree_draft.restype = _i32
    L.spec_tree_draft.argtypes = [ctypes.POINTER(TreeDraftArgs), _vp]
    L.spec_tree_verify.restype = _i32
    L.spec_tree_verify.argtypes = [ctypes.POINTER(TreeVerifyArgs), _vp]
    L.spec_tree_workspace_bytes.restype = _sz
    L.spec_tree_workspace_bytes.argtypes = [_i32, _i32, _i32]
    L.spec_rnn_draft.restype = _i32
    L.spec_rnn_draft.argtypes = [ctypes.POINTER(RnnDraftArgs), _vp]
    L.spec_confidence.restype = _i32
    L.spec_confidence.argtypes = [ctypes.POINTER(ConfidenceArgs), _vp]
    L.spec_schedule_workspace_bytes.restype = _sz
    L.spec_schedule_workspace_bytes.argtypes = [_i32, _i32]
    L.spec_prefix_schedule.restype = _i32
    L.spec_prefix_schedule.argtypes = [ctypes.POINTER(ScheduleArgs), _vp]
    L.spec_cache_bytes.restype = _sz
    L.spec_cache_bytes.argtypes = [_i32, _i32, _i32, _i32]
    L.spec_block_tables.restype = _i32
    L.spec_block_tables.argtypes = [_vp, _vp]
    L.spec_cache_append.restype = _i32
    L.spec_cache_append.argtypes = [_vp, _vp]
    L.spec_cache_attention_workspace_bytes.restype = _sz
    L.spec_cache_attention_workspace_bytes.argtypes = [_i32, _i32, _i32]
    L.spec_cache_attention.restype = _i32
    L.spec_cache_attention.argtypes = [_vp, _vp]
    L.spec_logprobs_workspace_bytes.restype = _sz
    L.spec_logprobs_workspace_bytes.argtypes = [_i32, _i32, _i32]
    L.spec_logprobs.restype = _i32
    L.spec_logprobs.argtypes = [_vp, _vp]
    L.spec_rotary_append.restype = _i32
    L.spec_rotary_append.argtypes = [_vp, _vp]
    L.spec_prefix_attention_workspace_bytes.restype = _sz
    L.spec_prefix_attention_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32]
    L.spec_prefix_attention.restype = _i32
    L.spec_prefix_attention.argtypes = [_vp, _vp]
    L.spec_sample.restype = _i32
    L.spec_sample.argtypes = [_vp, _vp]
    if path is None:
        _LIB = L
    return L


def _check(rc: int, what: str) -> None:
    if rc != 0:
        msg = lib().spec_status_string(rc).decode()
        raise SpecError(f"{what} failed: {rc} ({msg})")


def _hptr(t) -> int | None:
    """Address of a contiguous host (CPU) tensor."""
    if t is None:
        return None
    if t.is_cuda:
        raise SpecError("host buffers must be CPU tensors")
    if not t.is_contiguous():
        raise SpecError("tensors must be contiguous")
    return t.data_ptr()


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise SpecError("tensors must be CUDA tensors")
    if not t.is_contiguous():
        raise SpecError("tensors must be contiguous")
    return t.data_ptr()


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise SpecError(f"unsupported logits dtype {t.dtype}")


def _stream(stream) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def spec_workspace_bytes(B: int, gamma: int, V: int, r: int, dtype: int) -> int:
    return int(lib().spec_workspace_bytes(B, gamma, V, r, dtype))


def spec_status_string(status: int) -> str:
    return lib().spec_status_string(status).decode()


def spec_set_option(key: int, value: float) -> None:
    _check(lib().spec_set_option(key, float(value)), "spec_set_option")


def spec_markov_draft(U, W1, W2, anchor, temperature, u_draft, draft_tokens, q_tok, lse_q,
                      dev_status, workspace, diag=None, stream=None) -> None:
    """Enqueue the Markov-head draft (shapes as in include/spec.h)."""
    B, gamma, V = U.shape
    a = DraftArgs(B, gamma, V, W1.shape[1], _dtype_code(U), _ptr(U), _ptr(W1), _ptr(W2),
                  _ptr(anchor), _ptr(temperature), _ptr(u_draft), _ptr(draft_tokens),
                  _ptr(q_tok), _ptr(lse_q), _ptr(dev_status), _ptr(diag), _ptr(workspace),
                  workspace.numel() * workspace.element_size())
    _check(lib().spec_markov_draft(ctypes.byref(a), _stream(stream)), "spec_markov_draft")


def spec_markov_draft_static(U, W1, W2, anchor, temperature, u_draft, draft_tokens, q_tok,
                             lse_q, dev_status, diag=None, stream=None) -> None:
    """The draft with the library's built-in scratch area instead of a caller
    workspace, for callers that cannot allocate device memory (see spec.h)."""
    B, gamma, V = U.shape
    a = DraftArgs(B, gamma, V, W1.shape[1], _dtype_code(U), _ptr(U), _ptr(W1), _ptr(W2),
                  _ptr(anchor), _ptr(temperature), _ptr(u_draft), _ptr(draft_tokens),
                  _ptr(q_tok), _ptr(lse_q), _ptr(dev_status), _ptr(diag), None, 0)
    _check(lib().spec_markov_draft_static(ctypes.byref(a), _stream(stream)),
           "spec_markov_draft_static")


def spec_verify(target, U, W1, W2, anchor, temperature, draft_tokens, q_tok, lse_q, verify_len,
                u_accept, u_final, accept_len, out_tokens, alpha, dev_status, workspace,
                p_tok=None, diag=None, stream=None, a_rows=None) -> None:
    """Enqueue the verification (shapes as in include/spec.h); ``a_rows`` are
    the RNN head's factor rows (None: the Markov head)."""
    B, gamma, V = U.shape
    a = VerifyArgs(B, gamma, V, W1.shape[1], _dtype_code(U), _ptr(target), _ptr(U), _ptr(W1),
                   _ptr(W2), _ptr(anchor), _ptr(temperature), _ptr(draft_tokens), _ptr(q_tok),
                   _ptr(lse_q), _ptr(verify_len), _ptr(u_accept), _ptr(u_final),
                   _ptr(accept_len), _ptr(out_tokens), _ptr(alpha), _ptr(p_tok),
                   _ptr(dev_status), _ptr(a_rows), _ptr(diag), _ptr(workspace),
                   workspace.numel() * workspace.element_size())
    _check(lib().spec_verify(ctypes.byref(a), _stream(stream)), "spec_verify")


def spec_cycle_host(draft: DraftArgs, verify: VerifyArgs, h_U, h_target, h_anchor,
                    h_temperature, h_u_draft, h_verify_len, h_u_accept, h_u_final, h_accept_len,
                    h_out_tokens, h_draft_tokens=None, h_alpha=None, stream=None,
                    copy_stream=None) -> None:
    """Enqueue one cycle whose inputs and results live in host memory (CPU
    tensors, page-locked for asynchronous copies); ``draft`` / ``verify``
    name the device buffers (see include/spec.h)."""
    a = CycleHostArgs(draft, verify, _hptr(h_U), _hptr(h_target), _hptr(h_anchor),
                      _hptr(h_temperature), _hptr(h_u_draft), _hptr(h_verify_len),
                      _hptr(h_u_accept), _hptr(h_u_final), _hptr(h_accept_len),
                      _hptr(h_out_tokens), _hptr(h_draft_tokens), _hptr(h_alpha),
                      None if copy_stream is None else int(copy_stream.cuda_stream))
    _check(lib().spec_cycle_host(ctypes.byref(a), _stream(stream)), "spec_cycle_host")


def draft_args(U, W1, W2, anchor, temperature, u_draft, draft_tokens, q_tok, lse_q, dev_status,
               workspace, diag=None) -> DraftArgs:
    """The spec_draft_args of these device tensors."""
    B, gamma, V = U.shape
    return DraftArgs(B, gamma, V, W1.shape[1], _dtype_code(U), _ptr(U), _ptr(W1), _ptr(W2),
                     _ptr(anchor), _ptr(temperature), _ptr(u_draft), _ptr(draft_tokens),
                     _ptr(q_tok), _ptr(lse_q), _ptr(dev_status), _ptr(diag), _ptr(workspace),
                     workspace.numel() * workspace.element_size())


def verify_args(target, U, W1, W2, anchor, temperature, draft_tokens, q_tok, lse_q, verify_len,
                u_accept, u_final, accept_len, out_tokens, alpha, dev_status, workspace,
                p_tok=None, diag=None, a_rows=None) -> VerifyArgs:
    """The spec_verify_args of these device tensors."""
    B, gamma, V = U.shape
    return VerifyArgs(B, gamma, V, W1.shape[1], _dtype_code(U), _ptr(target), _ptr(U), _ptr(W1),
                      _ptr(W2), _ptr(anchor), _ptr(temperature), _ptr(draft_tokens),
                      _ptr(q_tok), _ptr(lse_q), _ptr(verify_len), _ptr(u_accept),
                      _ptr(u_final), _ptr(accept_len), _ptr(out_tokens), _ptr(alpha),
                      _ptr(p_tok), _ptr(dev_status), _ptr(a_rows), _ptr(diag), _ptr(workspace),
                      workspace.numel() * workspace.element_size())


def spec_profile_enable(on: bool) -> None:
    _check(lib().spec_profile_enable(1 if on else 0), "spec_profile_enable")


def spec_profile_read() -> dict[str, tuple[float, int]]:
    """{stage name: (total ms, launches)} since the previous read."""
    L = lib()
    n = L.spec_num_stages()
    ms = (ctypes.c_double * n)()
    cnt = (_i32 * n)()
    _check(L.spec_profile_read(ms, cnt, n), "spec_profile_read")
    return {L.spec_stage_name(i).decode(): (ms[i], cnt[i]) for i in range(n)}


def spec_operating_point(alpha: float, c: float, gamma: int, gamma_max: int = 256,
                         c_hat: float = 0.0) -> dict:
    """The analytic operating point (host computation, no GPU work)."""
    out = OpResult()
    _check(lib().spec_operating_point(ctypes.byref(OpArgs(alpha, c, c_hat, gamma, gamma_max)),
                                      ctypes.byref(out)), "spec_operating_point")
    return {f: getattr(out, f) for f, _ in OpResult._fields_}


def spec_acceptance_stats(alpha, verify_len, accept_len, out, stream=None) -> None:
    """Device sums (alpha over j < L_b, positions, tau, requests) into out (float64[4])."""
    B, gamma = alpha.shape
    _check(lib().spec_acceptance_stats(B, gamma, _ptr(alpha), _ptr(verify_len), _ptr(accept_len),
                                       _ptr(out), _stream(stream)), "spec_acceptance_stats")


def spec_confidence(hidden, W1, w, anchor, draft_tokens, conf, dev_status, stream=None) -> None:
    """Enqueue the confidence head: conf[r, k] = sigmoid(w . [h; W1[x_k]])."""
    R, gamma, d = hidden.shape
    V, r = W1.shape
    a = ConfidenceArgs(R, gamma, d, V, r, _dtype_code(hidden), _ptr(hidden), _ptr(W1), _ptr(w),
                       _ptr(anchor), _ptr(draft_tokens), _ptr(conf), _ptr(dev_status))
    _check(lib().spec_confidence(ctypes.byref(a), _stream(stream)), "spec_confidence")


def spec_schedule_workspace_bytes(R: int, gamma: int) -> int:
    return int(lib().spec_schedule_workspace_bytes(R, gamma))


def spec_prefix_schedule(conf, sps, survival, verify_len, totals, theta, dev_status, workspace,
                         stream=None) -> None:
    """Enqueue the hardware-aware prefix scheduler (verify lengths from conf)."""
    R, gamma = conf.shape
    a = ScheduleArgs(R, gamma, _ptr(conf), _ptr(sps), sps.numel(), _ptr(survival),
                     _ptr(verify_len), _ptr(totals), _ptr(theta), _ptr(dev_status),
                     _ptr(workspace), workspace.numel() * workspace.element_size())
    _check(lib().spec_prefix_schedule(ctypes.byref(a), _stream(stream)), "spec_prefix_schedule")


def spec_rnn_draft(U, W1, W2, Wr, hproj, anchor, temperature, u_draft, draft_tokens, q_tok,
                   lse_q, a_rows, dev_status, workspace, diag=None, stream=None) -> None:
    """Enqueue the RNN head draft (shapes as in include/spec.h)."""
    B, gamma, V = U.shape
    d = DraftArgs(B, gamma, V, W1.shape[1], _dtype_code(U), _ptr(U), _ptr(W1), _ptr(W2),
                  _ptr(anchor), _ptr(temperature), _ptr(u_draft), _ptr(draft_tokens),
                  _ptr(q_tok), _ptr(lse_q), _ptr(dev_status), _ptr(diag), _ptr(workspace),
                  workspace.numel() * workspace.element_size())
    a = RnnDraftArgs(d, _ptr(Wr), _ptr(hproj), _ptr(a_rows))
    _check(lib().spec_rnn_draft(ctypes.byref(a), _stream(stream)), "spec_rnn_draft")


def spec_tree_workspace_bytes(B: int, N: int, V: int) -> int:
    return int(lib().spec_tree_workspace_bytes(B, N, V))


def spec_tree_select(parent, conf, n, survival, mask, dev_status, gamma, expected=None,
                     stream=None) -> None:
    """Top-n slots of each request's candidate tree by survival."""
    B, N = parent.shape
    _check(lib().spec_tree_select(B, N, gamma, _ptr(parent), _ptr(conf), n, _ptr(survival),
                                  _ptr(mask), _ptr(expected), _ptr(dev_status), _stream(stream)),
           "spec_tree_select")


def spec_tree_draft(U, W1, W2, anchor, temperature, parent, mask, u_draft, tokens, q_tok,
                    dev_status, workspace, stream=None) -> None:
    B, gamma, V = U.shape
    a = TreeDraftArgs(B, parent.shape[1], gamma, V, W1.shape[1], _dtype_code(U), _ptr(U),
                      _ptr(W1), _ptr(W2), _ptr(anchor), _ptr(temperature), _ptr(parent),
                      _ptr(mask), _ptr(u_draft), _ptr(tokens), _ptr(q_tok), _ptr(dev_status),
                      _ptr(workspace), workspace.numel() * workspace.element_size())
    _check(lib().spec_tree_draft(ctypes.byref(a), _stream(stream)), "spec_tree_draft")


def spec_tree_verify(target, U, W1, W2, anchor, temperature, parent, mask, tokens, u_accept,
                     u_final, accept_len, out_tokens, path, dev_status, workspace,
                     stream=None) -> None:
    B, gamma, V = U.shape
    a = TreeVerifyArgs(B, parent.shape[1], gamma, V, W1.shape[1], _dtype_code(U), _ptr(target),
                       _ptr(U), _ptr(W1), _ptr(W2), _ptr(anchor), _ptr(temperature), _ptr(parent),
                       _ptr(mask), _ptr(tokens), _ptr(u_accept), _ptr(u_final), _ptr(accept_len),
                       _ptr(out_tokens), _ptr(path), _ptr(dev_status), _ptr(workspace),
                       workspace.numel() * workspace.element_size())
    _check(lib().spec_tree_verify(ctypes.byref(a), _stream(stream)), "spec_tree_verify")


# ------------------------------------------------------- target side of a cycle
# These calls are made every step of a server, some of them for microseconds of
# GPU work: their tensors are checked by the compiled module _args, and their
# arguments packed into the C structs' bytes in one go (the formats follow the
# structures above field by field).

def _format(py) -> struct.Struct:
    """struct format of a mirror, native alignment."""
    return struct.Struct("@" + _codes(py) + "0P")


def _codes(py) -> str:
    codes = {_i32: "i", _vp: "P", _i64: "q", _f32: "f", _sz: "N"}
    # a structure within it ends on a pointer's boundary
    return "".join(codes[t] if t in codes else _codes(t) + "0P" for _, t in py._fields_)


_TABLES, _APPEND = _format(BlockTablesArgs), _format(CacheAppendArgs)
_ATTENTION, _LOGPROBS = _format(CacheAttentionArgs), _format(LogprobsArgs)
_PREFIX, _ROTARY, _SAMPLE = _format(PrefixAttentionArgs), _format(RotaryAppendArgs), _format(SampleArgs)


def _pack(fmt: struct.Struct, *values) -> bytes:
    try:
        return fmt.pack(*values)
    except struct.error as e:
        raise SpecError(f"an argument does not fit its C type: {e}") from e


_torch = _args = None
_device = None              # the current device: launches go to it, so every tensor and the stream have to be on it


def _types():
    """torch, imported at the first call that needs it, with the module that
    checks tensors."""
    global _torch, _args, _device
    if _torch is None:
        import torch
        try:
            from . import _args as checks
        except ImportError as e:
            raise SpecError(f"the compiled checks are missing ({e}): build them with "
                            "speculative_decoding_draft_04_gb300.build.build()") from e
        from .build import built_for
        if checks.built_for != built_for():              # before it reads any of this torch's objects
            raise SpecError(f"the compiled checks were built for {checks.built_for}, this is {built_for()}: build "
                            "them again with speculative_decoding_draft_04_gb300.build.build()")
        checks.use(SpecError)
        _device = torch._C._cuda_getDevice if torch.cuda.is_available() else lambda: -1
        _torch, _args = torch, checks
    return _torch


def _raw_stream(device: int, stream) -> int:
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise SpecError(f"the stream is on cuda:{stream.device_index}, the call on cuda:{device}")
    return stream.cuda_stream


def _cache_shape(cache, D: int) -> tuple:
    """(num_pages, Hkv, page_size) of a 4-bit cache [num_pages][Hkv][page_size / 16][18 D]."""
    s = cache.shape
    if len(s) != 4 or s[3] != 18 * D or cache.dtype is not _torch.uint8:
        raise SpecError(f"cache must be torch.uint8 [num_pages, Hkv, page_size / 16, {18 * D}], not "
                        f"{cache.dtype} {list(s)}")
    return s[0], s[1], s[2] * 16


def _storage(t) -> int:
    if t.dtype is _torch.bfloat16:
        return SPEC_BF16
    if t.dtype is _torch.float32:
        return SPEC_F32
    raise SpecError(f"unsupported type {t.dtype}")


def spec_cache_bytes(num_pages: int, Hkv: int, page_size: int, D: int) -> int:
    return int(lib().spec_cache_bytes(num_pages, Hkv, page_size, D))


def spec_block_tables(seq_len, accept_len, new_len, num_blocks, ring_pos, free_ring, block_table,
                      seq_len_out, kv_len, num_blocks_out, ring_pos_out, row_ptr, slots, positions,
                      dev_status, page_size: int, stream=None) -> None:
    """Block tables, slots and positions of every request's next tokens
    (accept_len None: the lengths are final)."""
    T = _types()
    i32, i64 = T.int32, T.int64
    b = tuple(seq_len.shape)
    table, rows, ring = tuple(block_table.shape), tuple(slots.shape), tuple(free_ring.shape)
    if len(b) != 1 or len(table) != 2 or len(rows) != 1 or len(ring) != 1 or table[0] != b[0]:
        raise SpecError("seq_len, slots and free_ring must be vectors, block_table [B, pages]")
    B = b[0]
    dev = _device()
    a = _pack(_TABLES, B, page_size, ring[0], table[1], rows[0], *_args.addresses(
        dev, "seq_len", seq_len, i32, b, "accept_len?", accept_len, i32, b, "new_len", new_len, i32, b,
        "num_blocks", num_blocks, i32, b, "ring_pos", ring_pos, i64, (2,), "free_ring", free_ring, i32, ring,
        "block_table", block_table, i32, table, "seq_len_out", seq_len_out, i32, b, "kv_len", kv_len, i32, b,
        "num_blocks_out", num_blocks_out, i32, b, "ring_pos_out", ring_pos_out, i64, (2,),
        "row_ptr", row_ptr, i32, (B + 1,), "slots", slots, i32, rows, "positions", positions, i32, rows,
        "dev_status", dev_status, i32, (4,)))
    rc = lib().spec_block_tables(a, _raw_stream(dev, stream))
    if rc:
        _check(rc, "spec_block_tables")


def spec_cache_append(k, v, slots, cache, dev_status, k_scale: float = 1.0, v_scale: float = 1.0,
                      k_stored=None, v_stored=None, stream=None) -> None:
    """Round keys and values [T][Hkv][D] to 4 bits into the cache at their
    slots; k_stored / v_stored receive the values as stored."""
    T = _types()
    shape = tuple(k.shape)
    if len(shape) != 3:
        raise SpecError(f"k must be [T, Hkv, D], not {list(shape)}")
    rows, H, D = shape
    pages, Hkv, P = _cache_shape(cache, D)
    if Hkv != H or v.dtype is not k.dtype:
        raise SpecError(f"k, v and cache disagree: {H} and {Hkv} heads, {k.dtype} and {v.dtype}")
    dev = _device()
    kp, kr, kh, vp, vr, vh, sp, cp, ks, vs, st = _args.addresses(
        dev, "k", k, None, shape, "v", v, None, shape, "slots", slots, T.int32, (rows,),
        "cache", cache, T.uint8, (pages, H, P // 16, 18 * D), "k_stored?", k_stored, k.dtype, shape,
        "v_stored?", v_stored, k.dtype, shape, "dev_status", dev_status, T.int32, (4,))
    a = _pack(_APPEND, rows, H, D, _storage(k), P, pages, kp, vp, kr, kh, vr, vh, sp, k_scale, v_scale, cp,
              ks, vs, st)
    rc = lib().spec_cache_append(a, _raw_stream(dev, stream))
    if rc:
        _check(rc, "spec_cache_append")


def spec_cache_attention_workspace_bytes(Hq: int, Hkv: int, D: int) -> int:
    return int(lib().spec_cache_attention_workspace_bytes(Hq, Hkv, D))


def _attention_values(dev, q, cache, block_table, kv_len, row_ptr, out, dev_status, workspace,
                      softmax_scale, k_scale, v_scale, tree_mask, lse) -> tuple:
    """The fields of spec_cache_attention_args."""
    T = _torch
    i32 = T.int32
    shape, table = tuple(q.shape), tuple(block_table.shape)
    if len(shape) != 3 or len(table) != 2:
        raise SpecError(f"q must be [T, Hq, D] and block_table [B, pages], not {list(shape)}, {list(table)}")
    rows, Hq, D = shape
    B = table[0]
    pages, Hkv, P = _cache_shape(cache, D)
    if tree_mask is not None and tree_mask.dim() != 2:
        raise SpecError(f"tree_mask must be [T, words], not {list(tree_mask.shape)}")
    words = 0 if tree_mask is None else tree_mask.shape[1]
    qp, qr, qh, cp, tp, lp, rp, mp, op, ep, st, wp, wn = _args.addresses(
        dev, "q", q, None, shape, "cache", cache, T.uint8, (pages, Hkv, P // 16, 18 * D),
        "block_table", block_table, i32, table, "kv_len", kv_len, i32, (B,), "row_ptr", row_ptr, i32, (B + 1,),
        "tree_mask?", tree_mask, i32, (rows, words), "out", out, q.dtype, shape, "lse?", lse, T.float32, (rows, Hq),
        "dev_status", dev_status, i32, (4,), "workspace", workspace, None, None)
    return (B, rows, Hq, Hkv, D, _storage(q), P, pages, table[1], words, qp, qr, qh, cp, tp, lp, rp, mp,
            softmax_scale, k_scale, v_scale, op, ep, st, wp, wn)


def spec_cache_attention(q, cache, block_table, kv_len, row_ptr, out, dev_status, workspace,
                         softmax_scale: float, k_scale: float = 1.0, v_scale: float = 1.0,
                         tree_mask=None, lse=None, stream=None) -> None:
    """Attention of the packed rows q [T][Hq][D] of every request over its
    cached tokens; tree_mask [T][words] (int32 bit words) replaces the causal
    order among a request's new tokens."""
    _types()
    dev = _device()
    a = _pack(_ATTENTION, *_attention_values(dev, q, cache, block_table, kv_len, row_ptr, out, dev_status, workspace,
                                             softmax_scale, k_scale, v_scale, tree_mask, lse))
    rc = lib().spec_cache_attention(a, _raw_stream(dev, stream))
    if rc:
        _check(rc, "spec_cache_attention")


def spec_prefix_attention_workspace_bytes(T: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().spec_prefix_attention_workspace_bytes(T, Hq, Hkv, D))


def spec_prefix_attention(q, cache, block_table, kv_len, row_ptr, prefix_table, prefix_len, group_ptr, out,
                          dev_status, workspace, softmax_scale: float, k_scale: float = 1.0,
                          v_scale: float = 1.0, tree_mask=None, lse=None, stream=None) -> None:
    """spec_cache_attention with prefixes that groups of requests share: requests
    group_ptr[g] .. group_ptr[g + 1] - 1 see the first prefix_len[g] tokens of
    prefix_table[g] before their own, which block_table and kv_len describe."""
    T = _types()
    dev = _device()
    own = _attention_values(dev, q, cache, block_table, kv_len, row_ptr, out, dev_status, workspace,
                            softmax_scale, k_scale, v_scale, tree_mask, lse)
    table = tuple(prefix_table.shape)
    if len(table) != 2:
        raise SpecError(f"prefix_table must be [groups, pages], not {list(table)}")
    a = _pack(_PREFIX, *own, *table, *_args.addresses(
        dev, "prefix_table", prefix_table, T.int32, table, "prefix_len", prefix_len, T.int32, (table[0],),
        "group_ptr", group_ptr, T.int32, (table[0] + 1,)))
    rc = lib().spec_prefix_attention(a, _raw_stream(dev, stream))
    if rc:
        _check(rc, "spec_prefix_attention")


def spec_rotary_append(q, k, v, positions, slots, rope, q_out, cache, dev_status, k_scale: float = 1.0,
                       v_scale: float = 1.0, q_weight=None, k_weight=None, eps: float = 1e-6,
                       interleaved: bool = False, k_stored=None, v_stored=None, stream=None) -> None:
    """Norm queries and keys per head (with a weight), rotate them by rope
    [rows][R / 2][2] (cosine, sine) at each row's position, write the queries to
    q_out and the keys and values into the cache at their slots."""
    T = _types()
    qs, shape, rs = tuple(q.shape), tuple(k.shape), tuple(rope.shape)
    if len(qs) != 3 or len(shape) != 3 or len(rs) != 3 or rs[2] != 2:
        raise SpecError(f"q must be [T, Hq, D], k [T, Hkv, D] and rope [rows, R / 2, 2], not {list(qs)}, "
                        f"{list(shape)}, {list(rs)}")
    rows, H, D = shape
    pages, Hkv, P = _cache_shape(cache, D)
    dt = q.dtype
    if qs[0] != rows or qs[2] != D or Hkv != H or k.dtype is not dt or v.dtype is not dt or q_out.dtype is not dt:
        raise SpecError(f"q, k, v, q_out and cache disagree: q {list(qs)} {dt}, k {list(shape)} {k.dtype}, "
                        f"v {v.dtype}, q_out {q_out.dtype}, cache of {Hkv} heads")
    i32 = T.int32
    dev = _device()
    qp, qr, qh, kp, kr, kh, vp, vr, vh, wq, wk, pp, sp, rp, op, orow, ohead, cp, ks, vs, st = _args.addresses(
        dev, "q", q, None, qs, "k", k, None, shape, "v", v, None, shape, "q_weight?", q_weight, dt, (D,),
        "k_weight?", k_weight, dt, (D,), "positions", positions, i32, (rows,), "slots", slots, i32, (rows,),
        "rope", rope, T.float32, rs, "q_out", q_out, None, qs, "cache", cache, T.uint8, (pages, H, P // 16, 18 * D),
        "k_stored?", k_stored, dt, shape, "v_stored?", v_stored, dt, shape, "dev_status", dev_status, i32, (4,))
    a = _pack(_ROTARY, rows, qs[1], H, D, 2 * rs[1], _storage(q), P, pages, rs[0], 1 if interleaved else 0, qp, kp, vp,
              qr, qh, kr, kh, vr, vh, wq, wk, pp, sp, rp, eps, k_scale, v_scale, op, orow, ohead, cp, ks, vs, st)
    rc = lib().spec_rotary_append(a, _raw_stream(dev, stream))
    if rc:
        _check(rc, "spec_rotary_append")


def spec_sample(logits, u, tokens, dev_status, temperature=None, top_k=None, top_p=None, min_p=None,
                logprob=None, kept=None, stream=None) -> None:
    """Draw a token of each row of logits [B][n][V] with the uniform numbers u
    [B][n], after temperature, top_k, top_p and min_p ([B] each)."""
    T = _types()
    f32, i32 = T.float32, T.int32
    shape = tuple(logits.shape)
    if len(shape) != 3:
        raise SpecError(f"logits must be [B, n, V], not {list(shape)}")
    B, n, V = shape
    b, bn = (B,), (B, n)
    dev = _device()
    xp, xb, xr, *rest = _args.addresses(
        dev, "logits", logits, None, shape, "u", u, f32, bn, "temperature?", temperature, f32, b,
        "top_k?", top_k, i32, b, "top_p?", top_p, f32, b, "min_p?", min_p, f32, b, "tokens", tokens, i32, bn,
        "logprob?", logprob, f32, bn, "kept?", kept, i32, bn, "dev_status", dev_status, i32, (4,))
    a = _pack(_SAMPLE, B, n, V, _storage(logits), xp, xb, xr, *rest)
    rc = lib().spec_sample(a, _raw_stream(dev, stream))
    if rc:
        _check(rc, "spec_sample")


def spec_logprobs_workspace_bytes(rows: int, V: int, K: int) -> int:
    return int(lib().spec_logprobs_workspace_bytes(rows, V, K))


def spec_logprobs(logits, tokens, logprob, entropy, dev_status, workspace, temperature=None,
                  top_ids=None, top_logprobs=None, stream=None) -> None:
    """Log probabilities of tokens [B][n] under logits [B][n][V], the entropies,
    and the K = top_ids.shape[2] largest entries of each row."""
    T = _types()
    f32, i32 = T.float32, T.int32
    shape = tuple(logits.shape)
    if len(shape) != 3:
        raise SpecError(f"logits must be [B, n, V], not {list(shape)}")
    if (top_ids is None) != (top_logprobs is None):
        raise SpecError("top_ids and top_logprobs go together")
    B, n, V = shape
    if top_ids is not None and top_ids.dim() != 3:
        raise SpecError(f"top_ids must be [B, n, K], not {list(top_ids.shape)}")
    K = 0 if top_ids is None else top_ids.shape[2]
    dev = _device()
    xp, xb, xr, tp, Tp, lp, ep, ip, kp, st, wp, wn = _args.addresses(
        dev, "logits", logits, None, shape, "tokens", tokens, i32, (B, n), "temperature?", temperature, f32, (B,),
        "logprob", logprob, f32, (B, n), "entropy", entropy, f32, (B, n), "top_ids?", top_ids, i32, (B, n, K),
        "top_logprobs?", top_logprobs, f32, (B, n, K), "dev_status", dev_status, i32, (4,),
        "workspace", workspace, None, None)
    a = _pack(_LOGPROBS, B, n, V, K, _storage(logits), xp, xb, xr, tp, Tp, lp, ep, ip if K else 0,
              kp if K else 0, st, wp, wn)
    rc = lib().spec_logprobs(a, _raw_stream(dev, stream))
    if rc:
        _check(rc, "spec_logprobs")
