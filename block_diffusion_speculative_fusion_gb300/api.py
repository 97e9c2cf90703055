"""Thin Python binding of libdflash (ctypes): argument marshalling only.

Every function takes torch CUDA tensors, checks their dtype, shape and
contiguity, and passes raw device pointers plus the current CUDA stream to the
C ABI declared in ``include/dflash.h``. All arithmetic runs in the library's
kernels; there is no fallback path. Workspaces are zero-initialised device
buffers cached per device and stream-ordered like every other tensor.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, List, Optional, Sequence, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdflash.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA = 0, 1, 2, 3, 4
F32, BF16 = 0, 1
FLAG_ACCEPT_BOUNDARY, FLAG_CDF_BOUNDARY, FLAG_DEGENERATE, FLAG_INVALID = 1, 2, 4, 8
FLAG_GATE_BOUNDARY = 1
WS_COUNTER_BYTES = 16384
WS_ERROR_WORD_OFFSET = WS_COUNTER_BYTES - 4
DEVERR_BAD_PAGE = 100
DEVERR_BAD_N_DRAFT = 101
# recorded only by the debug library (select_library(debug=True))
DEVERR_BAD_CTX_LEN, DEVERR_BAD_COMMIT_LEN, DEVERR_BAD_POSITION = 102, 103, 104


class DflashError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"dflash error {code}: {msg}")
        self.code = code


c_i32 = ctypes.c_int32
c_p = ctypes.c_void_p


class CtxKvDims(ctypes.Structure):
    _fields_ = [(n, c_i32) for n in ("B", "rows_max", "m", "d", "L", "Hkv", "D", "page_size",
                                     "max_pages", "num_pages", "dtype")]


class AttnDims(ctypes.Structure):
    _fields_ = [(n, c_i32) for n in ("B", "n_q", "n_kv_blk", "Hq", "Hkv", "D", "page_size",
                                     "max_pages", "num_pages", "max_ctx", "dtype", "causal")]


class VerifyDims(ctypes.Structure):
    _fields_ = [(n, c_i32) for n in ("B", "n_max", "V", "dtype")]


class GateDims(ctypes.Structure):
    _fields_ = [(n, c_i32) for n in ("B", "k", "V", "dtype")]


class TreeDims(ctypes.Structure):
    _fields_ = [(n, c_i32) for n in ("B", "n", "V", "dtype", "K", "budget")]


class RulesDims(ctypes.Structure):
    _fields_ = [(n, c_i32) for n in ("B", "n_rows", "V", "dtype", "hist_max", "n_bias")]


class PagesDims(ctypes.Structure):
    _fields_ = [(n, c_i32) for n in ("B", "page_size", "max_pages", "num_pages")]


class Fp8QuantDims(ctypes.Structure):
    _fields_ = [(n, c_i32) for n in ("T", "K", "dtype", "block_rows")]


class Fp8GemmDims(ctypes.Structure):
    _fields_ = [(n, c_i32) for n in ("T", "N", "K", "out_dtype")]


_SIGS = {
    "dflash_last_error": (ctypes.c_char_p, []),
    "dflash_last_launch_count": (ctypes.c_int, []),
    "dflash_set_wait_limit_ns": (ctypes.c_int, [ctypes.c_uint64]),
    "dflash_wait_limit_ns": (ctypes.c_uint64, []),
    "dflash_verify_greedy_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(VerifyDims)]),
    "dflash_verify_greedy": (ctypes.c_int, [ctypes.POINTER(VerifyDims), c_p, c_p, c_p, c_p, c_p, c_p,
                                            c_p, c_p, c_p, ctypes.c_size_t, c_p]),
    "dflash_verify_greedy_noalloc": (ctypes.c_int, [ctypes.POINTER(VerifyDims), c_p, c_p, c_p, c_p, c_p,
                                                    c_p, c_p, c_p, c_p]),
    "dflash_verify_sample_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(VerifyDims)]),
    "dflash_verify_sample": (ctypes.c_int, [ctypes.POINTER(VerifyDims), ctypes.c_float, c_p, c_p, c_p,
                                            c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_p,
                                            ctypes.c_size_t, c_p]),
    "dflash_gate_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(GateDims)]),
    "dflash_gate": (ctypes.c_int, [ctypes.POINTER(GateDims), ctypes.c_float, ctypes.c_float, c_p, c_p,
                                   c_p, c_p, c_p, c_p, c_p, c_p, ctypes.c_size_t, c_p]),
    # dims, stage, n_max, T, g, draft_logits, cand, active, c_s, cont, row_lse, flags, n_verify, ws, bytes, stream
    "dflash_gate_stage": (ctypes.c_int, [ctypes.POINTER(GateDims), ctypes.c_int32, ctypes.c_int32, ctypes.c_float,
                                         ctypes.c_float] + [c_p] * 9 + [ctypes.c_size_t, c_p]),
    # dims, T, target, draft, draft_row_lse, cand, n_draft, u_accept, u_final, accept_len, bonus,
    # commit_len, out_tokens, flags, probs, workspace, ws_bytes, stream
    "dflash_verify_sample_lse": (ctypes.c_int, [ctypes.POINTER(VerifyDims), ctypes.c_float] + [c_p] * 14 +
                                 [ctypes.c_size_t, c_p]),
    "dflash_ddtree_topk": (ctypes.c_int, [ctypes.POINTER(TreeDims), ctypes.c_float, c_p, c_p, c_p, c_p]),
    "dflash_ddtree_build": (ctypes.c_int, [ctypes.POINTER(TreeDims)] + [c_p] * 9),
    "dflash_ddtree_verify_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(TreeDims)]),
    "dflash_ddtree_verify_greedy": (ctypes.c_int, [ctypes.POINTER(TreeDims)] + [c_p] * 10 + [ctypes.c_size_t, c_p]),
    "dflash_draft_select_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(VerifyDims)]),
    "dflash_draft_select": (ctypes.c_int, [ctypes.POINTER(VerifyDims), ctypes.c_float, c_p, c_p, c_p, c_p, c_p,
                                           c_p, c_p, c_p, c_p, ctypes.c_size_t, c_p]),
    # dims, logits, cand, n_draft, hist, hist_len, prompt_len, repetition, presence, frequency, bias_tok,
    # bias_val, mask, mask_on, out, stream
    "dflash_logits_rules": (ctypes.c_int, [ctypes.POINTER(RulesDims)] + [c_p] * 15),
    "dflash_pages_resize": (ctypes.c_int, [ctypes.POINTER(PagesDims)] + [c_p] * 9),
    "dflash_slot_map": (ctypes.c_int, [ctypes.POINTER(PagesDims), c_i32] + [c_p] * 8),
    "dflash_fp8_quant": (ctypes.c_int, [ctypes.POINTER(Fp8QuantDims)] + [c_p] * 4),
    "dflash_fp8_gemm_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(Fp8GemmDims)]),
    "dflash_fp8_gemm": (ctypes.c_int, [ctypes.POINTER(Fp8GemmDims)] + [c_p] * 7 + [ctypes.c_size_t, c_p]),
    "dflash_materialize_fp8_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(CtxKvDims)]),
    # dims, hidden, commit_len, start_pos, W_f, W_f_scale, b_f, W_kv, W_kv_scale, k_norm_w, eps, theta, k_pools,
    # v_pools, page_table, new_len, workspace, ws_bytes, stream
    "dflash_materialize_ctx_kv_fp8": (ctypes.c_int, [ctypes.POINTER(CtxKvDims)] + [c_p] * 9 +
                                      [ctypes.c_float, ctypes.c_float] + [c_p] * 5 + [ctypes.c_size_t, c_p]),
    "dflash_block_attn_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(AttnDims)]),
    "dflash_block_attn": (ctypes.c_int, [ctypes.POINTER(AttnDims), c_p, c_p, c_p, c_p, c_p, c_p, c_p,
                                         ctypes.c_float, c_p, c_p, ctypes.c_size_t, c_p]),
    "dflash_block_attn_active": (ctypes.c_int, [ctypes.POINTER(AttnDims), c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_p,
                                                ctypes.c_float, c_p, c_p, ctypes.c_size_t, c_p]),
    "dflash_materialize_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(CtxKvDims)]),
    "dflash_materialize_ctx_kv": (ctypes.c_int, [ctypes.POINTER(CtxKvDims), c_p, c_p, c_p, c_p, c_p,
                                                 c_p, c_p, ctypes.c_float, ctypes.c_float, c_p, c_p,
                                                 c_p, c_p, c_p, ctypes.c_size_t, c_p]),
}

_lib = None
LIB_DEBUG_PATH = os.path.join(_HERE, "libdflash_debug.so")


def select_library(debug: bool = False) -> str:
    """Use libdflash.so, or libdflash_debug.so (built by ``build.build(debug=True)``,
    whose kernels also record clamped inputs in the error word), for every later
    call; returns its path."""
    global _lib, LIB_PATH
    LIB_PATH = LIB_DEBUG_PATH if debug else os.path.join(_HERE, "libdflash.so")
    _lib = None
    return LIB_PATH


def lib() -> ctypes.CDLL:
    """Load libdflash.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "block_diffusion_speculative_fusion_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name, None)
            if fn is None:
                continue
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def last_error() -> str:
    return lib().dflash_last_error().decode()


def last_launch_count() -> int:
    return int(lib().dflash_last_launch_count())


def set_wait_limit_ns(ns: int) -> None:
    """Limit of the tensor-core kernels' bounded waits (``dflash_set_wait_limit_ns``);
    0 restores the 2 s default."""
    _check(lib().dflash_set_wait_limit_ns(int(ns)))


def wait_limit_ns() -> int:
    return int(lib().dflash_wait_limit_ns())


def _check(rc: int):
    if rc != OK:
        raise DflashError(rc, last_error())


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
_DT = {torch.float32: F32, torch.bfloat16: BF16}


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")
    return _DT[t.dtype]


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _opt(t: Optional[torch.Tensor], name: str, dtype=None, shape=None):
    return None if t is None else _dev(t, name, dtype, shape)


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _arg(t: Optional[torch.Tensor], name: str, dev: int, dtype: torch.dtype, shape: Tuple[int, ...]):
    """Device pointer of a contiguous tensor of this dtype and shape on CUDA
    device ``dev`` (None stays None); raises what ``_dev`` raises otherwise.
    The checks of a small call cost more host time than its launch, so the
    valid case takes the fewest attribute reads."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev \
            and t.is_contiguous():
        return t.data_ptr()
    _dev(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")


def _out(o: dict, name: str, like: torch.Tensor, dev: int, dtype: torch.dtype, shape: Tuple[int, ...]) -> int:
    """Device pointer of output ``name``: the caller's tensor, checked, or a new
    one on the device of ``like``."""
    t = o.get(name)
    if t is not None:
        return _arg(t, name, dev, dtype, shape)
    t = o[name] = torch.empty(shape, dtype=dtype, device=like.device)
    return t.data_ptr()


# the stream handle without a Stream object, where this torch has the call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _launch(dev: int, fn, *args) -> None:
    """``fn(*args, stream)`` with CUDA device ``dev`` current, on its current stream."""
    if dev == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev))
    if rc != OK:
        raise DflashError(rc, last_error())


_WS: Dict[Tuple[int, int], torch.Tensor] = {}
_WS_OUTGROWN: List[Tuple[Tuple[int, int], torch.Tensor]] = []


def workspace(device: torch.device, nbytes: int, slot: int = 0) -> torch.Tensor:
    """A zero-initialised device workspace of at least ``nbytes`` (cached per
    device and slot; calls on one stream may share a slot). One that a larger
    call outgrows is kept until ``reset_workspaces``: a captured graph may still
    replay with it. The one that takes its place is at least twice as large, so
    that all those kept take no more than it does."""
    idx = torch.device(device).index
    if idx is None:
        idx = torch.cuda.current_device()
    key = (idx, slot)
    ws = _WS.get(key)
    if ws is None or ws.numel() < nbytes:
        if ws is not None:
            _WS_OUTGROWN.append((key, ws))
            nbytes = max(nbytes, 2 * ws.numel())
        ws = torch.zeros(max(nbytes, WS_COUNTER_BYTES), dtype=torch.uint8, device=f"cuda:{idx}")
        _WS[key] = ws
    return ws


def reset_workspaces():
    _WS.clear()
    _WS_OUTGROWN.clear()


def cached_workspaces() -> List[Tuple[Tuple[int, int], torch.Tensor]]:
    """((device, slot), tensor) of every cached workspace, those that a larger
    call has outgrown included."""
    return _WS_OUTGROWN + list(_WS.items())


# ---------------------------------------------------------------------------
# (c) verify
# ---------------------------------------------------------------------------
def verify_greedy(target_logits: torch.Tensor, cand: torch.Tensor, n_draft: Optional[torch.Tensor] = None,
                  want_target_pred: bool = False, out: Optional[dict] = None, ws: Optional[torch.Tensor] = None):
    """Greedy accept rule (``dflash_verify_greedy``). Returns a dict of device
    tensors: accept_len, bonus, commit_len, out_tokens[, target_pred]."""
    _dev(target_logits, "target_logits")
    B, R, V = target_logits.shape
    n_max = R - 1
    dev = target_logits.device
    dims = VerifyDims(B, n_max, V, _dtype_code(target_logits))
    o = out if out is not None else {}
    o.setdefault("accept_len", torch.empty(B, dtype=torch.int32, device=dev))
    o.setdefault("bonus", torch.empty(B, dtype=torch.int64, device=dev))
    o.setdefault("commit_len", torch.empty(B, dtype=torch.int32, device=dev))
    o.setdefault("out_tokens", torch.empty((B, R), dtype=torch.int64, device=dev))
    if want_target_pred:
        o.setdefault("target_pred", torch.empty((B, R), dtype=torch.int64, device=dev))
    need = lib().dflash_verify_greedy_workspace_size(ctypes.byref(dims))
    if need == 0:
        raise DflashError(ERR_INVALID_ARG, last_error())
    w = ws if ws is not None else workspace(dev, need)
    rc = lib().dflash_verify_greedy(
        ctypes.byref(dims), _dev(target_logits, "target_logits"), _dev(cand, "cand", torch.int64, (B, R)),
        _opt(n_draft, "n_draft", torch.int32, (B,)),
        _dev(o["accept_len"], "accept_len", torch.int32), _dev(o["bonus"], "bonus", torch.int64),
        _dev(o["commit_len"], "commit_len", torch.int32), _opt(o.get("out_tokens"), "out_tokens", torch.int64),
        _opt(o.get("target_pred"), "target_pred", torch.int64), w.data_ptr(), w.numel(), _stream(dev))
    _check(rc)
    return o


def verify_greedy_noalloc(target_logits: torch.Tensor, cand: torch.Tensor, n_draft: Optional[torch.Tensor] = None,
                          want_target_pred: bool = False, out: Optional[dict] = None):
    """Greedy accept rule on the library's fixed scratch
    (``dflash_verify_greedy_noalloc``). Outputs are caller tensors (``out``),
    created here only when not given; the C call itself allocates nothing."""
    _dev(target_logits, "target_logits")
    B, R, V = target_logits.shape
    dev = target_logits.device
    dims = VerifyDims(B, R - 1, V, _dtype_code(target_logits))
    o = out if out is not None else {}
    o.setdefault("accept_len", torch.empty(B, dtype=torch.int32, device=dev))
    o.setdefault("bonus", torch.empty(B, dtype=torch.int64, device=dev))
    o.setdefault("commit_len", torch.empty(B, dtype=torch.int32, device=dev))
    o.setdefault("out_tokens", torch.empty((B, R), dtype=torch.int64, device=dev))
    if want_target_pred:
        o.setdefault("target_pred", torch.empty((B, R), dtype=torch.int64, device=dev))
    rc = lib().dflash_verify_greedy_noalloc(
        ctypes.byref(dims), _dev(target_logits, "target_logits"), _dev(cand, "cand", torch.int64, (B, R)),
        _opt(n_draft, "n_draft", torch.int32, (B,)),
        _dev(o["accept_len"], "accept_len", torch.int32), _dev(o["bonus"], "bonus", torch.int64),
        _dev(o["commit_len"], "commit_len", torch.int32), _opt(o.get("out_tokens"), "out_tokens", torch.int64),
        _opt(o.get("target_pred"), "target_pred", torch.int64), _stream(dev))
    _check(rc)
    return o


def verify_sample(target_logits: torch.Tensor, draft_logits: torch.Tensor, cand: torch.Tensor,
                  u_accept: torch.Tensor, u_final: torch.Tensor, temperature: float = 1.0,
                  n_draft: Optional[torch.Tensor] = None, want_probs: bool = False,
                  out: Optional[dict] = None, ws: Optional[torch.Tensor] = None,
                  draft_row_lse: Optional[torch.Tensor] = None):
    """Sampled accept rule with residual resample (``dflash_verify_sample``).
    With ``draft_row_lse`` [B, n_max] (LSE(draft row / T), e.g. the DLoop
    gates' row_lse) the draft rows are not streamed
    (``dflash_verify_sample_lse``). Returns accept_len, bonus, commit_len,
    out_tokens, flags[, probs]."""
    _dev(target_logits, "target_logits")
    B, R, V = target_logits.shape
    n_max = R - 1
    dev = target_logits.device
    dt = _dtype_code(target_logits)
    if draft_logits.dtype != target_logits.dtype:
        raise TypeError("draft_logits and target_logits must share a dtype")
    dims = VerifyDims(B, n_max, V, dt)
    o = out if out is not None else {}
    o.setdefault("accept_len", torch.empty(B, dtype=torch.int32, device=dev))
    o.setdefault("bonus", torch.empty(B, dtype=torch.int64, device=dev))
    o.setdefault("commit_len", torch.empty(B, dtype=torch.int32, device=dev))
    o.setdefault("out_tokens", torch.empty((B, R), dtype=torch.int64, device=dev))
    o.setdefault("flags", torch.empty(B, dtype=torch.uint8, device=dev))
    if want_probs:
        o.setdefault("probs", torch.empty((B, 2 * n_max + 1), dtype=torch.float32, device=dev))
    need = lib().dflash_verify_sample_workspace_size(ctypes.byref(dims))
    if need == 0:
        raise DflashError(ERR_INVALID_ARG, last_error())
    w = ws if ws is not None else workspace(dev, need)
    head = [ctypes.byref(dims), ctypes.c_float(temperature), _dev(target_logits, "target_logits"),
            _dev(draft_logits, "draft_logits", None, (B, n_max, V))]
    if draft_row_lse is not None:
        fn = lib().dflash_verify_sample_lse
        head.append(_dev(draft_row_lse, "draft_row_lse", torch.float32, (B, n_max)))
    else:
        fn = lib().dflash_verify_sample
    rc = fn(
        *head, _dev(cand, "cand", torch.int64, (B, R)),
        _opt(n_draft, "n_draft", torch.int32, (B,)), _dev(u_accept, "u_accept", torch.float32, (B, n_max)),
        _dev(u_final, "u_final", torch.float32, (B,)),
        _dev(o["accept_len"], "accept_len", torch.int32), _dev(o["bonus"], "bonus", torch.int64),
        _dev(o["commit_len"], "commit_len", torch.int32), _opt(o.get("out_tokens"), "out_tokens", torch.int64),
        _opt(o.get("flags"), "flags", torch.uint8), _opt(o.get("probs"), "probs", torch.float32),
        w.data_ptr(), w.numel(), _stream(dev))
    _check(rc)
    return o


# ---------------------------------------------------------------------------
# DLoop gate
# ---------------------------------------------------------------------------
def gate(draft_logits: torch.Tensor, tokens: torch.Tensor, temperature: float = 1.0, g: float = -0.5,
         active: Optional[torch.Tensor] = None, want_row_lse: bool = False,
         out: Optional[dict] = None, ws: Optional[torch.Tensor] = None):
    """DLoop block gate (``dflash_gate``). Returns c, cont, flags[, row_lse]."""
    _dev(draft_logits, "draft_logits")
    B, k, V = draft_logits.shape
    dev = draft_logits.device
    dims = GateDims(B, k, V, _dtype_code(draft_logits))
    o = out if out is not None else {}
    o.setdefault("c", torch.empty(B, dtype=torch.float32, device=dev))
    o.setdefault("cont", torch.empty(B, dtype=torch.uint8, device=dev))
    o.setdefault("flags", torch.empty(B, dtype=torch.uint8, device=dev))
    if want_row_lse:
        o.setdefault("row_lse", torch.empty((B, k), dtype=torch.float32, device=dev))
    need = lib().dflash_gate_workspace_size(ctypes.byref(dims))
    if need == 0:
        raise DflashError(ERR_INVALID_ARG, last_error())
    w = ws if ws is not None else workspace(dev, need)
    rc = lib().dflash_gate(
        ctypes.byref(dims), ctypes.c_float(temperature), ctypes.c_float(g), _dev(draft_logits, "draft_logits"),
        _dev(tokens, "tokens", torch.int64, (B, k)), _opt(active, "active", torch.uint8, (B,)),
        _dev(o["c"], "c", torch.float32), _dev(o["cont"], "cont", torch.uint8),
        _opt(o.get("row_lse"), "row_lse", torch.float32), _opt(o.get("flags"), "flags", torch.uint8),
        w.data_ptr(), w.numel(), _stream(dev))
    _check(rc)
    return o


def gate_stage(draft_logits: torch.Tensor, cand: torch.Tensor, stage: int, k: int, temperature: float = 1.0,
               g: float = -0.5, active: Optional[torch.Tensor] = None, row_lse: Optional[torch.Tensor] = None,
               n_verify: Optional[torch.Tensor] = None, out: Optional[dict] = None,
               ws: Optional[torch.Tensor] = None):
    """One DLoop stage's gate on the looped layout (``dflash_gate_stage``):
    draft_logits [B, n_max, V], cand [B, n_max + 1]; stage s's rows are
    s*k .. s*k + k - 1. ``row_lse`` [B, n_max] and ``n_verify`` [B] are
    accumulated across stages. Returns c, cont, flags."""
    _dev(draft_logits, "draft_logits")
    B, n_max, V = draft_logits.shape
    dev = draft_logits.device
    dims = GateDims(B, k, V, _dtype_code(draft_logits))
    o = out if out is not None else {}
    o.setdefault("c", torch.empty(B, dtype=torch.float32, device=dev))
    o.setdefault("cont", torch.empty(B, dtype=torch.uint8, device=dev))
    o.setdefault("flags", torch.empty(B, dtype=torch.uint8, device=dev))
    need = lib().dflash_gate_workspace_size(ctypes.byref(dims))
    if need == 0:
        raise DflashError(ERR_INVALID_ARG, last_error())
    w = ws if ws is not None else workspace(dev, need)
    rc = lib().dflash_gate_stage(
        ctypes.byref(dims), int(stage), int(n_max), ctypes.c_float(temperature), ctypes.c_float(g),
        _dev(draft_logits, "draft_logits"), _dev(cand, "cand", torch.int64, (B, n_max + 1)),
        _opt(active, "active", torch.uint8, (B,)), _dev(o["c"], "c", torch.float32),
        _dev(o["cont"], "cont", torch.uint8), _opt(row_lse, "row_lse", torch.float32, (B, n_max)),
        _opt(o.get("flags"), "flags", torch.uint8), _opt(n_verify, "n_verify", torch.int32, (B,)),
        w.data_ptr(), w.numel(), _stream(dev))
    _check(rc)
    return o


def draft_select(draft_logits: torch.Tensor, anchor: torch.Tensor, temperature: float = 0.0,
                 u_draft: Optional[torch.Tensor] = None, n_draft: Optional[torch.Tensor] = None,
                 out: Optional[dict] = None, ws: Optional[torch.Tensor] = None):
    """Candidates from the draft's MASK-position logits (``dflash_draft_select``):
    argmax (temperature 0) or one inverse-CDF sample per row with ``u_draft``.
    Returns cand [B, n_max+1] int64, q_x and row_lse [B, n_max] float32, flags
    [B, n_max] uint8."""
    _dev(draft_logits, "draft_logits")
    B, n_max, V = draft_logits.shape
    dev = draft_logits.device
    dims = VerifyDims(B, n_max, V, _dtype_code(draft_logits))
    o = out if out is not None else {}
    if "cand" not in o:
        o["cand"] = torch.empty((B, n_max + 1), dtype=torch.int64, device=dev)
        o["q_x"] = torch.empty((B, n_max), dtype=torch.float32, device=dev)
        o["row_lse"] = torch.empty((B, n_max), dtype=torch.float32, device=dev)
        o["flags"] = torch.empty((B, n_max), dtype=torch.uint8, device=dev)
    need = lib().dflash_draft_select_workspace_size(ctypes.byref(dims))
    if need == 0:
        raise DflashError(ERR_INVALID_ARG, last_error())
    w = ws if ws is not None else workspace(dev, need)
    rc = lib().dflash_draft_select(
        ctypes.byref(dims), ctypes.c_float(temperature), _dev(draft_logits, "draft_logits"),
        _dev(anchor, "anchor", torch.int64, (B,)), _opt(n_draft, "n_draft", torch.int32, (B,)),
        _opt(u_draft if temperature > 0 else None, "u_draft", torch.float32, (B, n_max)),
        _dev(o["cand"], "cand", torch.int64, (B, n_max + 1)), _opt(o.get("q_x"), "q_x", torch.float32),
        _opt(o.get("row_lse"), "row_lse", torch.float32), _opt(o.get("flags"), "flags", torch.uint8),
        w.data_ptr(), w.numel(), _stream(dev))
    _check(rc)
    return o


# ---------------------------------------------------------------------------
# DDTree
# ---------------------------------------------------------------------------
def ddtree_topk(draft_logits: torch.Tensor, K: int, temperature: float = 1.0, out: Optional[dict] = None):
    """Top-K tokens and their log-probabilities of every drafted position
    (``dflash_ddtree_topk``): tok [B, n, K] int64, logp [B, n, K] float32."""
    _dev(draft_logits, "draft_logits")
    B, n, V = draft_logits.shape
    dev = draft_logits.device
    dims = TreeDims(B, n, V, _dtype_code(draft_logits), K, 1)
    o = out if out is not None else {}
    if "tok" not in o:
        o["tok"] = torch.empty((B, n, K), dtype=torch.int64, device=dev)
        o["logp"] = torch.empty((B, n, K), dtype=torch.float32, device=dev)
    _check(lib().dflash_ddtree_topk(ctypes.byref(dims), ctypes.c_float(temperature), _dev(draft_logits, "draft_logits"),
                                    _dev(o["tok"], "tok", torch.int64, (B, n, K)),
                                    _dev(o["logp"], "logp", torch.float32, (B, n, K)), _stream(dev)))
    return o


def ddtree_build(tok: torch.Tensor, logp: torch.Tensor, budget: int, V: int = 1, out: Optional[dict] = None):
    """Best-first draft tree within ``budget`` nodes (``dflash_ddtree_build``):
    node_token, node_parent, node_depth, node_logp [B, budget], n_nodes [B],
    flags [B]."""
    B, n, K = tok.shape
    dev = tok.device
    dims = TreeDims(B, n, max(V, K), BF16, K, budget)
    o = out if out is not None else {}
    if "node_token" not in o:
        o["node_token"] = torch.empty((B, budget), dtype=torch.int64, device=dev)
        o["node_parent"] = torch.empty((B, budget), dtype=torch.int32, device=dev)
        o["node_depth"] = torch.empty((B, budget), dtype=torch.int32, device=dev)
        o["node_logp"] = torch.empty((B, budget), dtype=torch.float32, device=dev)
        o["n_nodes"] = torch.empty(B, dtype=torch.int32, device=dev)
        o["flags"] = torch.empty(B, dtype=torch.uint8, device=dev)
    _check(lib().dflash_ddtree_build(
        ctypes.byref(dims), _dev(tok, "tok", torch.int64, (B, n, K)), _dev(logp, "logp", torch.float32, (B, n, K)),
        _dev(o["node_token"], "node_token", torch.int64), _dev(o["node_parent"], "node_parent", torch.int32),
        _dev(o["node_depth"], "node_depth", torch.int32), _dev(o["node_logp"], "node_logp", torch.float32),
        _dev(o["n_nodes"], "n_nodes", torch.int32), _opt(o.get("flags"), "flags", torch.uint8), _stream(dev)))
    return o


def ddtree_verify_greedy(target_logits: torch.Tensor, node_token: torch.Tensor, node_parent: torch.Tensor,
                         n_nodes: torch.Tensor, n: int, K: int, out: Optional[dict] = None,
                         ws: Optional[torch.Tensor] = None):
    """Greedy walk of the verified tree (``dflash_ddtree_verify_greedy``):
    accept_len, commit_len, bonus, path [B, budget], out_tokens [B, budget+1]."""
    _dev(target_logits, "target_logits")
    B, R, V = target_logits.shape
    budget = R - 1
    dev = target_logits.device
    dims = TreeDims(B, n, V, _dtype_code(target_logits), K, budget)
    o = out if out is not None else {}
    if "accept_len" not in o:
        o["accept_len"] = torch.empty(B, dtype=torch.int32, device=dev)
        o["bonus"] = torch.empty(B, dtype=torch.int64, device=dev)
        o["commit_len"] = torch.empty(B, dtype=torch.int32, device=dev)
        o["path"] = torch.empty((B, budget), dtype=torch.int32, device=dev)
        o["out_tokens"] = torch.empty((B, R), dtype=torch.int64, device=dev)
    need = lib().dflash_ddtree_verify_workspace_size(ctypes.byref(dims))
    if need == 0:
        raise DflashError(ERR_INVALID_ARG, last_error())
    w = ws if ws is not None else workspace(dev, need)
    _check(lib().dflash_ddtree_verify_greedy(
        ctypes.byref(dims), _dev(target_logits, "target_logits"),
        _dev(node_token, "node_token", torch.int64, (B, budget)), _dev(node_parent, "node_parent", torch.int32, (B, budget)),
        _dev(n_nodes, "n_nodes", torch.int32, (B,)), _dev(o["accept_len"], "accept_len", torch.int32),
        _dev(o["bonus"], "bonus", torch.int64), _dev(o["commit_len"], "commit_len", torch.int32),
        _opt(o.get("path"), "path", torch.int32), _opt(o.get("out_tokens"), "out_tokens", torch.int64),
        w.data_ptr(), w.numel(), _stream(dev)))
    return o


# ---------------------------------------------------------------------------
# rules on the verify rows' logits
# ---------------------------------------------------------------------------
def logits_rules(logits: torch.Tensor, cand: Optional[torch.Tensor] = None, n_draft: Optional[torch.Tensor] = None,
                 hist: Optional[torch.Tensor] = None, hist_len: Optional[torch.Tensor] = None,
                 prompt_len: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                 presence: Optional[torch.Tensor] = None, frequency: Optional[torch.Tensor] = None,
                 bias_tok: Optional[torch.Tensor] = None, bias_val: Optional[torch.Tensor] = None,
                 mask: Optional[torch.Tensor] = None, mask_on: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Penalties, biases and grammar masks on logits [B, R, V]
    (``dflash_logits_rules``); row r's history is hist[b, :hist_len[b]] and
    cand[b, 1 .. r]. hist [B, H], cand [B, R] int64; hist_len, prompt_len,
    n_draft [B] int32; repetition, presence, frequency [B] float32; bias_tok
    [B, n] int64 with bias_val [B, n] float32; mask [B, R, ceil(V / 32)] int32,
    bit 1 = allowed, for the sequences with mask_on[b] != 0 (uint8; None: all).
    Returns ``out``; ``out=logits`` works in place. If not given, ``out`` is a new
    tensor, which with ``n_draft`` is zeroed whole before the call, as its rows past
    n_draft[b] are not written: pass one to save that."""
    _dev(logits, "logits")
    B, R, V = logits.shape
    dev = logits.get_device()
    if (hist is None) != (hist_len is None):
        raise ValueError("hist and hist_len come together")
    if (bias_tok is None) != (bias_val is None):
        raise ValueError("bias_tok and bias_val come together")
    H = 0 if hist is None else hist.shape[1]
    nb = 0 if bias_tok is None else bias_tok.shape[1]
    if out is None:
        out = torch.empty_like(logits) if n_draft is None else torch.zeros_like(logits)
    seq = (B,)
    _launch(dev, lib().dflash_logits_rules, ctypes.byref(RulesDims(B, R, V, _dtype_code(logits), H, nb)),
            logits.data_ptr(), _arg(cand, "cand", dev, torch.int64, (B, R)),
            _arg(n_draft, "n_draft", dev, torch.int32, seq), _arg(hist, "hist", dev, torch.int64, (B, H)),
            _arg(hist_len, "hist_len", dev, torch.int32, seq), _arg(prompt_len, "prompt_len", dev, torch.int32, seq),
            _arg(repetition, "repetition", dev, torch.float32, seq),
            _arg(presence, "presence", dev, torch.float32, seq),
            _arg(frequency, "frequency", dev, torch.float32, seq),
            _arg(bias_tok, "bias_tok", dev, torch.int64, (B, nb)),
            _arg(bias_val, "bias_val", dev, torch.float32, (B, nb)),
            _arg(mask, "mask", dev, torch.int32, (B, R, (V + 31) // 32)),
            _arg(mask_on, "mask_on", dev, torch.uint8, seq), _arg(out, "out", dev, logits.dtype, (B, R, V)))
    return out


# ---------------------------------------------------------------------------
# block tables and slot maps
# ---------------------------------------------------------------------------
def pages_resize(length: torch.Tensor, page_table: torch.Tensor, n_pages: torch.Tensor, free_pages: torch.Tensor,
                 n_free: torch.Tensor, page_size: int, out: Optional[dict] = None) -> dict:
    """Grow or shrink every sequence's row of the block table to length[b]
    tokens (``dflash_pages_resize``). length, n_pages [B], page_table [B,
    max_pages], free_pages [num_pages], n_free [1], all int32; page_table and
    free_pages are changed in place. Returns n_pages [B] and n_free [1] int32
    (tensors that overlap no other one of the call), short [B] uint8."""
    _dev(page_table, "page_table", torch.int32)
    B, max_pages = page_table.shape
    dev = page_table.get_device()
    o = out if out is not None else {}
    num_pages = len(free_pages)
    i32, seq = torch.int32, (B,)
    _launch(dev, lib().dflash_pages_resize, ctypes.byref(PagesDims(B, page_size, max_pages, num_pages)),
            _arg(length, "length", dev, i32, seq), page_table.data_ptr(), _arg(n_pages, "n_pages", dev, i32, seq),
            _arg(free_pages, "free_pages", dev, i32, (num_pages,)), _arg(n_free, "n_free", dev, i32, (1,)),
            _out(o, "n_pages", page_table, dev, i32, seq), _out(o, "n_free", page_table, dev, i32, (1,)),
            _out(o, "short", page_table, dev, torch.uint8, seq))
    return o


def slot_map(start_pos: torch.Tensor, n_rows: torch.Tensor, page_table: torch.Tensor, page_size: int, num_pages: int,
             rows_max: int, out: Optional[dict] = None) -> dict:
    """Slot map of the ragged batch of rows start_pos[b] .. start_pos[b] +
    n_rows[b] - 1 (``dflash_slot_map``). Returns cu_rows [B + 1], row_seq and
    positions [rows_max] int32, slots [rows_max] int64 (-1 past the last row)."""
    _dev(page_table, "page_table", torch.int32)
    B, max_pages = page_table.shape
    dev = page_table.get_device()
    i32, rows = torch.int32, (max(rows_max, 0),)
    o = out if out is not None else {}
    _launch(dev, lib().dflash_slot_map, ctypes.byref(PagesDims(B, page_size, max_pages, num_pages)), rows_max,
            _arg(start_pos, "start_pos", dev, i32, (B,)), _arg(n_rows, "n_rows", dev, i32, (B,)),
            page_table.data_ptr(), _out(o, "cu_rows", page_table, dev, i32, (B + 1,)),
            _out(o, "row_seq", page_table, dev, i32, rows), _out(o, "positions", page_table, dev, i32, rows),
            _out(o, "slots", page_table, dev, torch.int64, rows))
    return o


# ---------------------------------------------------------------------------
# (b) block attention
# ---------------------------------------------------------------------------
def block_attn(q: torch.Tensor, k_blk: torch.Tensor, v_blk: torch.Tensor, k_pool: torch.Tensor,
               v_pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
               max_ctx: Optional[int] = None, scale: Optional[float] = None,
               out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
               causal: bool = False, active: Optional[torch.Tensor] = None) -> torch.Tensor:
    """GQA attention of the draft block over [paged context ; block]
    (``dflash_block_attn``): unmasked, or with ``causal`` the in-block causal
    variant (query i sees the context and block rows j <= i + n_kv - n_q).
    q [B, n_q, Hq, D]; k_blk, v_blk [B, n_kv, Hkv, D]; pools [num_pages, page,
    Hkv, D]; page_table [B, max_pages] int32; ctx_len [B] int32. ``max_ctx``
    bounds every ctx_len (defaults to the page table's capacity). With
    ``active`` [B] uint8 (``dflash_block_attn_active``) only the sequences with
    active[b] != 0 are computed; the other rows of ``out`` are left as they were."""
    _dev(q, "q")
    B, n_q, Hq, D = q.shape
    n_kv, Hkv = k_blk.shape[1], k_blk.shape[2]
    num_pages, page = k_pool.shape[0], k_pool.shape[1]
    max_pages = page_table.shape[1]
    if max_ctx is None:
        max_ctx = max_pages * page
    dt = _dtype_code(q)
    for name, t in (("k_blk", k_blk), ("v_blk", v_blk), ("k_pool", k_pool), ("v_pool", v_pool)):
        if t.dtype != q.dtype:
            raise TypeError(f"{name} must have the dtype of q")
    dims = AttnDims(B, n_q, n_kv, Hq, Hkv, D, page, max_pages, num_pages, int(max_ctx), dt, 1 if causal else 0)
    if out is None:
        out = torch.empty_like(q)
    need = lib().dflash_block_attn_workspace_size(ctypes.byref(dims))
    if need == 0:
        raise DflashError(ERR_INVALID_ARG, last_error())
    w = ws if ws is not None else workspace(q.device, need, slot=1)
    args = [ctypes.byref(dims), _dev(q, "q"), _dev(k_blk, "k_blk", None, (B, n_kv, Hkv, D)),
            _dev(v_blk, "v_blk", None, (B, n_kv, Hkv, D)), _dev(k_pool, "k_pool", None, (num_pages, page, Hkv, D)),
            _dev(v_pool, "v_pool", None, (num_pages, page, Hkv, D)),
            _dev(page_table, "page_table", torch.int32, (B, max_pages)),
            _dev(ctx_len, "ctx_len", torch.int32, (B,))]
    tail = [ctypes.c_float(scale if scale is not None else D ** -0.5), _dev(out, "out", q.dtype, q.shape),
            w.data_ptr(), w.numel(), _stream(q.device)]
    if active is None:
        rc = lib().dflash_block_attn(*args, *tail)
    else:
        rc = lib().dflash_block_attn_active(*args, _dev(active, "active", torch.uint8, (B,)), *tail)
    _check(rc)
    return out


def device_error_word(ws: torch.Tensor) -> int:
    """The sticky device-side error word of a workspace (0: no error; 1-99: a
    kernel gave up a bounded wait; DEVERR_BAD_PAGE: attention met a page-table
    entry outside the pools; DEVERR_BAD_N_DRAFT: a verify or draft-select call
    met an n_draft outside [0, n_max]; with the debug library also
    DEVERR_BAD_CTX_LEN, DEVERR_BAD_COMMIT_LEN, DEVERR_BAD_POSITION).
    Synchronises with the device to read it."""
    return int(ws[WS_ERROR_WORD_OFFSET:WS_COUNTER_BYTES].view(torch.int32).item())


def clear_counters(ws: torch.Tensor) -> None:
    """Zero a workspace's counter region (after a nonzero error word), on the
    current stream."""
    ws[:WS_COUNTER_BYTES].zero_()


def error_words() -> Dict[Tuple[int, int], int]:
    """Error word of the cached workspaces (see ``workspace``), keyed by (device,
    slot): the first nonzero one among a slot's outgrown workspaces, with which a
    captured graph may still replay, and its current one."""
    words: Dict[Tuple[int, int], int] = {}
    for key, ws in cached_workspaces():
        words[key] = words.get(key, 0) or device_error_word(ws)
    return words


# ---------------------------------------------------------------------------
# (a) context-KV materialisation
# ---------------------------------------------------------------------------
def materialize_ctx_kv(hidden: torch.Tensor, commit_len: torch.Tensor, start_pos: torch.Tensor,
                       W_f: torch.Tensor, b_f: Optional[torch.Tensor], W_kv: torch.Tensor,
                       k_norm_w: Optional[torch.Tensor], rms_eps: float, rope_theta: float,
                       k_pools: Sequence[torch.Tensor], v_pools: Sequence[torch.Tensor],
                       page_table: torch.Tensor, new_len: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None) -> None:
    """Write the committed rows' context K/V of every draft layer into the paged
    pools (``dflash_materialize_ctx_kv``). hidden [B, rows_max, m*d];
    W_f [d, m*d]; b_f [d] or None; W_kv [L, 2, Hkv*D, d]; k_norm_w [L, D] or
    None; pools: L tensors [num_pages, page, Hkv, D]; page_table [B, max_pages]."""
    _dev(hidden, "hidden")
    B, rows_max, md = hidden.shape
    d = W_f.shape[0]
    m = md // d
    L, two, HD, d2 = W_kv.shape
    if two != 2 or d2 != d or m * d != md:
        raise ValueError("inconsistent hidden / W_f / W_kv shapes")
    if len(k_pools) != L or len(v_pools) != L:
        raise ValueError("need one K and one V pool per draft layer")
    num_pages, page, Hkv, D = k_pools[0].shape
    if Hkv * D != HD:
        raise ValueError("pool head layout does not match W_kv")
    dt = _dtype_code(hidden)
    for name, t in (("W_f", W_f), ("W_kv", W_kv)):
        if t.dtype != hidden.dtype:
            raise TypeError(f"{name} must have the dtype of hidden")
    max_pages = page_table.shape[1]
    dims = CtxKvDims(B, rows_max, m, d, L, Hkv, D, page, max_pages, num_pages, dt)
    need = lib().dflash_materialize_workspace_size(ctypes.byref(dims))
    if need == 0:
        raise DflashError(ERR_INVALID_ARG, last_error())
    w = ws if ws is not None else workspace(hidden.device, need, slot=2)
    kp = (c_p * L)(*[_dev(t, f"k_pools[{i}]", hidden.dtype, (num_pages, page, Hkv, D)) for i, t in enumerate(k_pools)])
    vp = (c_p * L)(*[_dev(t, f"v_pools[{i}]", hidden.dtype, (num_pages, page, Hkv, D)) for i, t in enumerate(v_pools)])
    rc = lib().dflash_materialize_ctx_kv(
        ctypes.byref(dims), _dev(hidden, "hidden"), _dev(commit_len, "commit_len", torch.int32, (B,)),
        _dev(start_pos, "start_pos", torch.int32, (B,)), _dev(W_f, "W_f", None, (d, md)),
        _opt(b_f, "b_f", hidden.dtype, (d,)), _dev(W_kv, "W_kv"), _opt(k_norm_w, "k_norm_w", hidden.dtype, (L, D)),
        ctypes.c_float(rms_eps), ctypes.c_float(rope_theta), ctypes.cast(kp, c_p), ctypes.cast(vp, c_p),
        _dev(page_table, "page_table", torch.int32, (B, max_pages)), _opt(new_len, "new_len", torch.int32, (B,)),
        w.data_ptr(), w.numel(), _stream(hidden.device))
    _check(rc)


# ---------------------------------------------------------------------------
# 8-bit floating point with a scale per 128 values
# ---------------------------------------------------------------------------
_E4M3 = torch.float8_e4m3fn


def fp8_quant(x: torch.Tensor, block_rows: int = 1, q: Optional[torch.Tensor] = None,
              scale: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [T, K] in e4m3 with one float32 scale per ``block_rows`` x 128 values
    (``dflash_fp8_quant``): block_rows 1 for activations, 128 for weights.
    Returns q [T, K] float8_e4m3fn and scale [ceil(T / block_rows),
    ceil(K / 128)]; x is about q * scale. K is a multiple of 16."""
    _dev(x, "x")
    T, K = x.shape
    dev = x.get_device()
    o = {"q": q, "scale": scale}
    _launch(dev, lib().dflash_fp8_quant, ctypes.byref(Fp8QuantDims(T, K, _dtype_code(x), block_rows)), x.data_ptr(),
            _out(o, "q", x, dev, _E4M3, (T, K)),
            _out(o, "scale", x, dev, torch.float32, (-(-T // block_rows) if block_rows > 0 else T, -(-K // 128))))
    return o["q"], o["scale"]


def fp8_gemm(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
             bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
             out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x w^T + bias of e4m3 operands with block scales (``dflash_fp8_gemm``).
    x [T, K], w [N, K] float8_e4m3fn; x_scale [T, ceil(K / 128)], w_scale
    [ceil(N / 128), ceil(K / 128)] float32; bias [N] and the result [T, N] in
    ``out_dtype`` (bfloat16 or float32)."""
    _dev(x, "x", _E4M3)
    T, K = x.shape
    N = w.shape[0]
    dev = x.get_device()
    groups = -(-K // 128)
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in _DT:
        raise TypeError(f"unsupported dtype {out_dtype}; use float32 or bfloat16")
    o = {"out": out}
    w_ws = ws if ws is not None else workspace(x.device, WS_COUNTER_BYTES, slot=3)
    _launch(dev, lib().dflash_fp8_gemm, ctypes.byref(Fp8GemmDims(T, N, K, _DT[out_dtype])), x.data_ptr(),
            _arg(x_scale, "x_scale", dev, torch.float32, (T, groups)), _arg(w, "w", dev, _E4M3, (N, K)),
            _arg(w_scale, "w_scale", dev, torch.float32, (-(-N // 128), groups)),
            _arg(bias, "bias", dev, out_dtype, (N,)), _out(o, "out", x, dev, out_dtype, (T, N)),
            w_ws.data_ptr(), w_ws.numel())
    return o["out"]


def materialize_ctx_kv_fp8(hidden: torch.Tensor, commit_len: torch.Tensor, start_pos: torch.Tensor,
                           W_f: torch.Tensor, W_f_scale: torch.Tensor, b_f: Optional[torch.Tensor],
                           W_kv: torch.Tensor, W_kv_scale: torch.Tensor, k_norm_w: Optional[torch.Tensor],
                           rms_eps: float, rope_theta: float, k_pools: Sequence[torch.Tensor],
                           v_pools: Sequence[torch.Tensor], page_table: torch.Tensor,
                           new_len: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> None:
    """``materialize_ctx_kv`` with e4m3 weights (``dflash_materialize_ctx_kv_fp8``):
    W_f [d, m*d] and W_kv [L, 2, Hkv*D, d] float8_e4m3fn with the scales of
    ``fp8_quant(..., block_rows=128)`` over W_f and over W_kv.view(-1, d). Faster
    than the bf16 call where most of the B x rows_max rows are committed, slower
    where few of many are."""
    _dev(hidden, "hidden", torch.bfloat16)
    B, rows_max, md = hidden.shape
    dev = hidden.get_device()
    d = W_f.shape[0]
    m = md // d
    L, two, HD, d2 = W_kv.shape
    if two != 2 or d2 != d or m * d != md:
        raise ValueError("inconsistent hidden / W_f / W_kv shapes")
    if len(k_pools) != L or len(v_pools) != L:
        raise ValueError("need one K and one V pool per draft layer")
    num_pages, page, Hkv, D = k_pools[0].shape
    if Hkv * D != HD:
        raise ValueError("pool head layout does not match W_kv")
    max_pages = page_table.shape[1]
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    dims = CtxKvDims(B, rows_max, m, d, L, Hkv, D, page, max_pages, num_pages, BF16)
    need = lib().dflash_materialize_fp8_workspace_size(ctypes.byref(dims))
    if need == 0:
        raise DflashError(ERR_INVALID_ARG, last_error())
    w = ws if ws is not None else workspace(hidden.device, need, slot=4)
    pool = (num_pages, page, Hkv, D)
    kp = (c_p * L)(*[_arg(t, f"k_pools[{i}]", dev, bf, pool) for i, t in enumerate(k_pools)])
    vp = (c_p * L)(*[_arg(t, f"v_pools[{i}]", dev, bf, pool) for i, t in enumerate(v_pools)])
    groups = -(-d // 128)
    _launch(dev, lib().dflash_materialize_ctx_kv_fp8, ctypes.byref(dims), hidden.data_ptr(),
            _arg(commit_len, "commit_len", dev, i32, (B,)), _arg(start_pos, "start_pos", dev, i32, (B,)),
            _arg(W_f, "W_f", dev, _E4M3, (d, md)), _arg(W_f_scale, "W_f_scale", dev, f32, (groups, -(-md // 128))),
            _arg(b_f, "b_f", dev, bf, (d,)), _arg(W_kv, "W_kv", dev, _E4M3, (L, 2, HD, d)),
            _arg(W_kv_scale, "W_kv_scale", dev, f32, (-(-L * 2 * HD // 128), groups)),
            _arg(k_norm_w, "k_norm_w", dev, bf, (L, D)), rms_eps, rope_theta, ctypes.cast(kp, c_p),
            ctypes.cast(vp, c_p), _arg(page_table, "page_table", dev, i32, (B, max_pages)),
            _arg(new_len, "new_len", dev, i32, (B,)), w.data_ptr(), w.numel())
