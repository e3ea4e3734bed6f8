"""ctypes binding of libdg (include/dg.h): argument marshalling only.

Every function here has the name of the C entry point it calls and forwards torch tensors
as raw device pointers on the current (or given) CUDA stream.  All arithmetic runs in the
library's kernels; there is no fallback.  Loading fails loudly when the library has not been
built (run ``entropy_bounded_denoising_gb300.build.build()``).
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np
import torch

from . import build as _build

DG_OK, DG_ERR_INVALID_ARG, DG_ERR_ALIGNMENT, DG_ERR_WORKSPACE, DG_ERR_UNSUPPORTED, DG_ERR_CUDA = 0, -1, -2, -3, -4, -5
DG_BF16, DG_FP32 = 0, 1
DG_ACTIVE, DG_READ_ONLY, DG_SELF_COND, DG_SAMPLE_ALL = 1, 2, 4, 8
DG_DEV_NAN_INF_ROW, DG_DEV_EMPTY_ROW, DG_DEV_TIMEOUT, DG_DEV_BAD_PARAM = 1, 2, 4, 8

PARAM_FIELDS = ("temperature", "beta", "tau", "k", "max_steps", "min_accept", "step",
                "request_id", "flags")
_PARAM_FMT = "<fffiiiiII"
PARAM_BYTES = struct.calcsize(_PARAM_FMT)   # 36, sizeof(dg_canvas_params)

_lib = None


class _PagedKV(ctypes.Structure):   # dg_paged_kv
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class DGError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {status_string(code)} ({code})")
        self.code = code


def library_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Load libdg.so (built in-tree).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"libdg.so not found at {path}: build it with "
                           "entropy_bounded_denoising_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P, i32, i64, u32, u64, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                  ctypes.c_uint64, ctypes.c_size_t)
    st = ctypes.c_int
    PagedKV = ctypes.POINTER(_PagedKV)
    sig = {
        "dg_denoise_workspace_bytes": (sz, [i64, i32, i64, ctypes.c_int]),
        "dg_denoise_step": (st, [P, ctypes.c_int, i64, i64, i32, i64, P, u64] + [P] * 11 + [P, sz, P]),
        "dg_denoise_stats": (st, [P, ctypes.c_int, i64, i64, i32, i64, P, u64] + [P] * 11 + [P, sz, P]),
        "dg_denoise_samples": (st, [P, ctypes.c_int, i64, i64, i32, i64, P, u64, P, P, P, sz, P]),
        "dg_denoise_row_stats": (st, [P, ctypes.c_int, i64, i64, i32, i64, P, u64, P, P, P, P, P, sz, P]),
        "dg_denoise_accept": (st, [P, P, P, i64, i32, i64, P, u64] + [P] * 7 + [P, sz, P]),
        "dg_self_cond_zero_converged": (st, [P, P, i64, i32, i32, P, P]),
        "dg_denoise_step_choices": (st, [P, ctypes.c_int, i64, i64, i32, i64, P, u64] + [P] * 11
                                    + [P, i32, P] + [P, sz, P]),
        "dg_accept_from_entropy": (st, [P, P, P, i64, i32, i64, P, u64] + [P] * 7 + [P]),
        "dg_lm_head_workspace_bytes": (sz, [i64, i32, i64]),
        "dg_lm_head_logits": (st, [P, i64, P, i64, i64, i32, i64, i32, P, P, i64, P, sz, P]),
        "dg_lm_head_denoise_step": (st, [P, i64, P, i64, i64, i32, i64, i32, P, u64, P, i64]
                                    + [P] * 11 + [P, sz, P]),
        "dg_canvas_init": (st, [P, i64, i32, i64, P, u64, P]),
        "dg_advance_params": (st, [P, P, i64, P]),
        "dg_self_cond_workspace_bytes": (sz, [i64, i32, i32, i32]),
        "dg_self_cond_logits": (st, [P, ctypes.c_int, i64, P, P, P, i64, i32, i64, i32, i32,
                                     P, P, P, P, P, P, sz, P]),
        "dg_self_cond_prepare": (st, [P, P, i64, i32, i32, i32, P, P, sz, P]),
        "dg_self_cond_pe": (st, [P, ctypes.c_int, i64, P, P, i64, i32, i64, i32, i32, P, P, sz, P]),
        "dg_self_cond_mlp": (st, [i64, i32, i32, i32, P, P, P, P, P, sz, P]),
        "dg_self_cond_probs_workspace_bytes": (sz, [i64, i32, i32]),
        "dg_self_cond_probs": (st, [P, i64, i64, i64, i32, i32, P, P, P, P, P, P, sz, P]),
        "dg_gemm_workspace_bytes": (sz, [i64, i64]),
        "dg_gemm_bf16": (st, [P, i64, P, i64, ctypes.c_int, P, i64, i64, i64, i64, P, sz, P]),
        "dg_gemm_bf16_noalloc": (st, [P, i64, P, i64, ctypes.c_int, P, i64, i64, i64, i64, P]),
        "dg_choice_probs": (st, [P, ctypes.c_int, i64, P, P, i64, i32, i64, P, i32, P, P]),
        "dg_attention_workspace_bytes": (sz, [i32, i32]),
        "dg_attention": (st, [P, P, P, P, P, P, P, P, i32, i32, i64, i64, i32, i32, i32, i32, ctypes.c_float,
                              P, sz, P]),
        "dg_kv_append": (st, [P, i64, P, i64, P, i64, P, P, i32, i64, i32, i32, i32, P, i32, i32, PagedKV, P]),
        "dg_paged_attention_workspace_bytes": (sz, [i32, i32, i32, i32, i32]),
        "dg_paged_attention": (st, [P, PagedKV, P, P, P, P, i32, i32, i64, i32, i32, i32, i32, ctypes.c_float,
                                    P, sz, P]),
        "dg_adjust_logits": (st, [P, ctypes.c_int, i64, P, i64, i64, i32, i64, P, P, P, i64, P, P, P, P, i64,
                                  P, i64, i32, P, P]),
        "dg_embed_canvas": (st, [P, i64, i64, P, i32, P, ctypes.c_float, P, P]),
        "dg_commit": (st, [P, P, P, i64, i32, P, P, P, P, P]),
        "dg_philox_words": (st, [u64, u32, u32, u32, u32, u32, i64, P, P]),
        "dg_get_device_status": (st, [P, ctypes.POINTER(u32)]),
        "dg_clear_device_status": (st, [P]),
        "dg_probe_bounded_wait": (st, [u32, P, P]),
        "dg_status_string": (ctypes.c_char_p, [st]),
        "dg_version": (i32, []),
        "dg_launch_count": (u64, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def exported_symbols() -> list[str]:
    lib = load()
    return [n for n in ("dg_denoise_workspace_bytes", "dg_denoise_step", "dg_denoise_stats",
                        "dg_denoise_samples", "dg_denoise_step_choices", "dg_denoise_row_stats", "dg_denoise_accept",
                        "dg_self_cond_zero_converged", "dg_accept_from_entropy", "dg_lm_head_workspace_bytes",
                        "dg_lm_head_logits", "dg_lm_head_denoise_step",
                        "dg_canvas_init", "dg_advance_params", "dg_self_cond_workspace_bytes",
                        "dg_self_cond_logits", "dg_self_cond_prepare", "dg_self_cond_pe",
                        "dg_self_cond_mlp", "dg_self_cond_probs_workspace_bytes",
                        "dg_self_cond_probs", "dg_gemm_workspace_bytes", "dg_gemm_bf16",
                        "dg_gemm_bf16_noalloc", "dg_choice_probs", "dg_embed_canvas", "dg_commit", "dg_attention",
                        "dg_attention_workspace_bytes", "dg_kv_append", "dg_paged_attention",
                        "dg_paged_attention_workspace_bytes", "dg_adjust_logits",
                        "dg_philox_words", "dg_get_device_status", "dg_clear_device_status",
                        "dg_probe_bounded_wait",
                        "dg_status_string", "dg_version", "dg_launch_count") if hasattr(lib, n)]


# ------------------------------------------------------------------ marshalling helpers
def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    return t.data_ptr()


def _s(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn: str, code: int) -> None:
    if code != DG_OK:
        raise DGError(fn, code)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DG_BF16
    if t.dtype == torch.float32:
        return DG_FP32
    raise TypeError("logits must be bfloat16 or float32")


def status_string(code: int) -> str:
    return load().dg_status_string(int(code)).decode()


def version() -> int:
    return int(load().dg_version())


def dg_launch_count() -> int:
    return int(load().dg_launch_count())


def pack_params(p: dict) -> bytes:
    """Pack per-canvas parameter arrays into dg_canvas_params records (host bytes)."""
    n = len(p["flags"])
    return b"".join(struct.pack(_PARAM_FMT, *(np.asarray(p[f])[i].item() for f in PARAM_FIELDS))
                    for i in range(n))


def params_tensor(p: dict, device="cuda") -> torch.Tensor:
    """Per-canvas parameters as a device uint8 tensor [n * 36]."""
    raw = np.frombuffer(pack_params(p), dtype=np.uint8).copy()
    return torch.from_numpy(raw).to(device)


def unpack_params(t: torch.Tensor) -> dict:
    raw = t.detach().cpu().numpy().tobytes()
    n = len(raw) // PARAM_BYTES
    rows = [struct.unpack_from(_PARAM_FMT, raw, i * PARAM_BYTES) for i in range(n)]
    return {f: np.array([r[j] for r in rows]) for j, f in enumerate(PARAM_FIELDS)}


# ------------------------------------------------------------------ entry points
def dg_denoise_workspace_bytes(n_canvas: int, L: int, V: int, dtype: int = DG_BF16) -> int:
    return int(load().dg_denoise_workspace_bytes(n_canvas, L, V, dtype))


def _denoise_dims(logits, n_canvas, L, V, ld):
    n, Lx, ldx = logits.shape if logits.dim() == 3 else (n_canvas, L, ld)
    n_canvas = n if n_canvas is None else n_canvas
    L = Lx if L is None else L
    ld = ldx if ld is None else ld
    V = ld if V is None else V
    return n_canvas, L, V, ld


def _denoise_ws(workspace, logits, n_canvas, L, V):
    if workspace is None:  # the caller gave none: one sized by the library, on the logits' device
        workspace = torch.empty(dg_denoise_workspace_bytes(n_canvas, L, V, _dtype_code(logits)),
                                dtype=torch.uint8, device=logits.device)
    return workspace, workspace.numel() * workspace.element_size()


def _denoise_full(fn, logits, params, seed, canvas, prev_argmax, stable_count, accept_mask, argmax,
                  sample, entropy, lse, converged, mean_entropy, n_accept, workspace, n_canvas, L, V,
                  ld, stream, check):
    n_canvas, L, V, ld = _denoise_dims(logits, n_canvas, L, V, ld)
    workspace, ws_bytes = _denoise_ws(workspace, logits, n_canvas, L, V)
    rc = getattr(load(), fn)(_p(logits), _dtype_code(logits), ld, n_canvas, L, V, _p(params),
                             int(seed) & 0xFFFFFFFFFFFFFFFF, _p(canvas), _p(prev_argmax),
                             _p(stable_count), _p(accept_mask), _p(argmax), _p(sample), _p(entropy),
                             _p(lse), _p(converged), _p(mean_entropy), _p(n_accept),
                             _p(workspace), ws_bytes, _s(stream))
    if check:
        _check(fn, rc)
    return rc


def dg_denoise_step(logits, params, seed, canvas, prev_argmax, stable_count, accept_mask, argmax,
                    sample, entropy, lse, converged, mean_entropy=None, n_accept=None,
                    workspace=None, *, n_canvas=None, L=None, V=None, ld=None, stream=None,
                    check=True) -> int:
    return _denoise_full("dg_denoise_step", logits, params, seed, canvas, prev_argmax, stable_count,
                         accept_mask, argmax, sample, entropy, lse, converged, mean_entropy, n_accept,
                         workspace, n_canvas, L, V, ld, stream, check)


def dg_denoise_step_choices(logits, params, seed, canvas, prev_argmax, stable_count, accept_mask,
                            argmax, sample, entropy, lse, converged, choices, probs, mean_entropy=None,
                            n_accept=None, workspace=None, *, n_canvas=None, L=None, V=None, ld=None,
                            stream=None, check=True) -> int:
    """dg_denoise_step plus probs[c, i, k] = exp(logits[c, i, choices[c, i, k]] / T - lse[c, i])
    gathered in the statistics pass; choices [n, L, C] int32, probs [n, L, C] float32."""
    n_canvas, L, V, ld = _denoise_dims(logits, n_canvas, L, V, ld)
    workspace, ws_bytes = _denoise_ws(workspace, logits, n_canvas, L, V)
    C = choices.shape[-1]
    rc = load().dg_denoise_step_choices(_p(logits), _dtype_code(logits), ld, n_canvas, L, V, _p(params),
                                        int(seed) & 0xFFFFFFFFFFFFFFFF, _p(canvas), _p(prev_argmax),
                                        _p(stable_count), _p(accept_mask), _p(argmax), _p(sample),
                                        _p(entropy), _p(lse), _p(converged), _p(mean_entropy), _p(n_accept),
                                        _p(choices), C, _p(probs), _p(workspace), ws_bytes, _s(stream))
    if check:
        _check("dg_denoise_step_choices", rc)
    return rc


def dg_denoise_stats(logits, params, seed, canvas, prev_argmax, stable_count, accept_mask, argmax,
                     sample, entropy, lse, converged, mean_entropy=None, n_accept=None,
                     workspace=None, *, n_canvas=None, L=None, V=None, ld=None, stream=None,
                     check=True) -> int:
    """The statistics / acceptance half of dg_denoise_step (pass the same workspace to
    dg_denoise_samples afterwards)."""
    if workspace is None:
        raise ValueError("dg_denoise_stats needs the workspace that dg_denoise_samples will read")
    return _denoise_full("dg_denoise_stats", logits, params, seed, canvas, prev_argmax, stable_count,
                         accept_mask, argmax, sample, entropy, lse, converged, mean_entropy, n_accept,
                         workspace, n_canvas, L, V, ld, stream, check)


def dg_denoise_row_stats(logits, params, seed, argmax, sample, entropy, lse, workspace, *, n_canvas=None,
                         L=None, V=None, ld=None, stream=None, check=True) -> int:
    """K1 alone: per-position statistics (and DG_SAMPLE_ALL samples) into the given buffers;
    the workspace then goes to dg_denoise_accept and dg_denoise_samples."""
    n_canvas, L, V, ld = _denoise_dims(logits, n_canvas, L, V, ld)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().dg_denoise_row_stats(_p(logits), _dtype_code(logits), ld, n_canvas, L, V, _p(params),
                                     int(seed) & 0xFFFFFFFFFFFFFFFF, _p(argmax), _p(sample), _p(entropy),
                                     _p(lse), _p(workspace), ws_bytes, _s(stream))
    if check:
        _check("dg_denoise_row_stats", rc)
    return rc


def dg_denoise_accept(entropy, sample, argmax, params, seed, canvas, prev_argmax, stable_count, accept_mask,
                      converged, workspace, *, V, mean_entropy=None, n_accept=None, stream=None,
                      check=True) -> int:
    """Acceptance, renoise, convergence and the sampler's list after dg_denoise_row_stats."""
    n_canvas, L = entropy.shape
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().dg_denoise_accept(_p(entropy), _p(sample), _p(argmax), n_canvas, L, V, _p(params),
                                  int(seed) & 0xFFFFFFFFFFFFFFFF, _p(canvas), _p(prev_argmax), _p(stable_count),
                                  _p(accept_mask), _p(converged), _p(mean_entropy), _p(n_accept),
                                  _p(workspace), ws_bytes, _s(stream))
    if check:
        _check("dg_denoise_accept", rc)
    return rc


def dg_denoise_samples(logits, params, seed, canvas, sample, workspace, *, n_canvas=None, L=None,
                       V=None, ld=None, stream=None, check=True) -> int:
    n_canvas, L, V, ld = _denoise_dims(logits, n_canvas, L, V, ld)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().dg_denoise_samples(_p(logits), _dtype_code(logits), ld, n_canvas, L, V, _p(params),
                                   int(seed) & 0xFFFFFFFFFFFFFFFF, _p(canvas), _p(sample),
                                   _p(workspace), ws_bytes, _s(stream))
    if check:
        _check("dg_denoise_samples", rc)
    return rc


def dg_accept_from_entropy(entropy, sample, argmax, n_canvas, L, V, params, seed, canvas,
                           prev_argmax, stable_count, accept_mask, converged, mean_entropy=None,
                           n_accept=None, stream=None, check=True) -> int:
    rc = load().dg_accept_from_entropy(_p(entropy), _p(sample), _p(argmax), n_canvas, L, V,
                                       _p(params), int(seed) & 0xFFFFFFFFFFFFFFFF, _p(canvas),
                                       _p(prev_argmax), _p(stable_count), _p(accept_mask),
                                       _p(converged), _p(mean_entropy), _p(n_accept), _s(stream))
    if check:
        _check("dg_accept_from_entropy", rc)
    return rc


def dg_lm_head_workspace_bytes(n_canvas: int, L: int, V: int) -> int:
    return int(load().dg_lm_head_workspace_bytes(n_canvas, L, V))


def _lm_dims(hidden, W_lm, logits, V):
    n, L, ldh = hidden.shape
    d = W_lm.shape[1] if W_lm.dim() == 2 else None
    if hidden.stride(2) != 1 or W_lm.stride(1) != 1 or logits.stride(2) != 1:
        raise ValueError("rows must be contiguous")
    if hidden.stride(0) != L * hidden.stride(1) or logits.stride(0) != L * logits.stride(1):
        raise ValueError("canvases must follow each other at L row strides")
    V = W_lm.shape[0] if V is None else V
    return n, L, V, d, hidden.stride(1), W_lm.stride(0), logits.stride(1)


def dg_lm_head_logits(hidden, W_lm, params, logits, workspace=None, *, V=None, stream=None,
                      check=True) -> int:
    """logits[n, L, ld] = bf16(hidden[n, L, d] . W_lm[V, d]^T) for the active canvases."""
    n, L, V, d, ldh, ldw, ld = _lm_dims(hidden, W_lm, logits, V)
    if workspace is None:
        workspace = torch.empty(dg_lm_head_workspace_bytes(n, L, V), dtype=torch.uint8, device=hidden.device)
    rc = load().dg_lm_head_logits(_p(hidden), ldh, _p(W_lm), ldw, n, L, V, d, _p(params), _p(logits), ld,
                                  _p(workspace), workspace.numel(), _s(stream))
    if check:
        _check("dg_lm_head_logits", rc)
    return rc


def dg_lm_head_denoise_step(hidden, W_lm, params, seed, logits, canvas, prev_argmax, stable_count,
                            accept_mask, argmax, sample, entropy, lse, converged, mean_entropy=None,
                            n_accept=None, workspace=None, *, V=None, stream=None, check=True) -> int:
    """The LM head (logits stored into ``logits``) and one denoising step on its logits."""
    n, L, V, d, ldh, ldw, ld = _lm_dims(hidden, W_lm, logits, V)
    if workspace is None:
        workspace = torch.empty(dg_lm_head_workspace_bytes(n, L, V), dtype=torch.uint8, device=hidden.device)
    rc = load().dg_lm_head_denoise_step(_p(hidden), ldh, _p(W_lm), ldw, n, L, V, d, _p(params),
                                        int(seed) & 0xFFFFFFFFFFFFFFFF, _p(logits), ld, _p(canvas),
                                        _p(prev_argmax), _p(stable_count), _p(accept_mask), _p(argmax),
                                        _p(sample), _p(entropy), _p(lse), _p(converged), _p(mean_entropy),
                                        _p(n_accept), _p(workspace), workspace.numel(), _s(stream))
    if check:
        _check("dg_lm_head_denoise_step", rc)
    return rc


def dg_canvas_init(canvas, n_canvas, L, V, params, seed, stream=None, check=True) -> int:
    rc = load().dg_canvas_init(_p(canvas), n_canvas, L, V, _p(params),
                               int(seed) & 0xFFFFFFFFFFFFFFFF, _s(stream))
    if check:
        _check("dg_canvas_init", rc)
    return rc


def dg_advance_params(params, converged, n_canvas, stream=None, check=True) -> int:
    rc = load().dg_advance_params(_p(params), _p(converged), n_canvas, _s(stream))
    if check:
        _check("dg_advance_params", rc)
    return rc


def dg_choice_probs(logits, lse, params, choices, probs, *, V=None, stream=None, check=True) -> int:
    """probs[c, i, k] = exp(logits[c, i, choices[c, i, k]] / T - lse[c, i]); logits [n, L, ld]."""
    n, L, ld = logits.shape
    C = choices.shape[-1]
    rc = load().dg_choice_probs(_p(logits), _dtype_code(logits), ld, _p(lse), _p(params), n, L,
                                ld if V is None else V, _p(choices), C, _p(probs), _s(stream))
    if check:
        _check("dg_choice_probs", rc)
    return rc


def dg_attention_workspace_bytes(n_seq: int, max_q_len: int) -> int:
    return int(load().dg_attention_workspace_bytes(n_seq, max_q_len))


def dg_attention(q, k, v, o, cu_q, cu_kv, causal, max_q_len: int, *, lse=None, window: int = -1,
                 scale: float | None = None, workspace=None, stream=None, check=True) -> int:
    """o = attention over the allowed keys (per-sequence causality, optional symmetric window);
    q [total_q, Hq, D], k / v [total_kv, Hkv, D], o like q (bf16); cu_q / cu_kv [n + 1] int32 and
    causal [n] uint8 on the device."""
    total_q, Hq, D = q.shape
    total_kv, Hkv, _ = k.shape
    for t in (q, k, v, o):
        if not t.is_contiguous():
            raise ValueError("q, k, v and o must be contiguous")
    n = causal.numel()
    scale = 1.0 / float(D) ** 0.5 if scale is None else float(scale)
    if workspace is None:
        workspace = torch.empty(max(1, dg_attention_workspace_bytes(n, int(max_q_len))), dtype=torch.uint8,
                                device=q.device)
    rc = load().dg_attention(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(cu_q), _p(cu_kv), _p(causal), n,
                             int(max_q_len), total_q, total_kv, Hq, Hkv, D, int(window), scale, _p(workspace),
                             workspace.numel(), _s(stream))
    if check:
        _check("dg_attention", rc)
    return rc


# The serving calls below are made once a token: their checks are written out, with few calls, because a
# call of a few microseconds on the device waits for the host.
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _refuse(fn, name, t, dtype, shape, dev):
    """Why a tensor is not a contiguous one of dtype and shape (None = any extent) on device dev."""
    if t.dtype != dtype:
        raise TypeError(f"{fn}: {name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and s != w for s, w in zip(t.shape, shape)):
        raise ValueError(f"{fn}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be contiguous")
    raise ValueError(f"{fn}: {name} is on {t.device}, other tensors of the call on device {dev}")


def _whole(fn, name, t, dtype, shape, dev):
    """The address of a contiguous tensor of dtype and shape on device dev; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        _refuse(fn, name, t, dtype, shape, dev)
    return t.data_ptr()


# the current stream's handle without building a Stream object (3 us of a 15 us call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(fn, dev, stream):
    """The raw stream of a call whose tensors are on device dev, the current one."""
    if dev < 0:
        raise ValueError(f"{fn}: device tensors expected")
    if dev != _device():
        raise ValueError(f"{fn}: the tensors are on device {dev}, the current device is {_device()}")
    return _raw_stream(dev) if stream is None else _s(stream)


def _rows(fn, name, t, heads, d, dev):
    """Address and row stride of t [tokens, heads, d], whose rows hold [heads][d] without gaps."""
    if t.dtype is not _BF16:
        raise TypeError(f"{fn}: {name} must be bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d:
        raise ValueError(f"{fn}: {name} must have shape (tokens, {heads}, {d}), got {tuple(shape)}")
    row, head, one = t.stride()
    if one != 1 or (heads > 1 and head != d):
        raise ValueError(f"{fn}: {name}'s heads must follow each other")
    if t.get_device() != dev:
        _refuse(fn, name, t, t.dtype, shape, dev)
    return t.data_ptr(), row if shape[0] > 1 else heads * d


def _refuse_cache(fn, k_cache, v_cache):
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{fn}: {name} must be bfloat16, got {t.dtype}")
        if t.dim() != 4 or t.stride(3) != 1:
            raise ValueError(f"{fn}: {name} must be [n_pages, page_size, Hkv, D] with contiguous heads")
    raise ValueError(f"{fn}: k_cache and v_cache must have one layout")


def _paged_kv(fn, k_cache, v_cache, page_table, kv_len):
    """dg_paged_kv of k_cache, v_cache [n_pages, page_size, Hkv, D] (any strides of the first three) and
    page_table [n_seq, max_pages], kv_len [n_seq] int32; n_seq, Hkv, D and the device."""
    shape, strides = k_cache.shape, k_cache.stride()
    if (k_cache.dtype is not _BF16 or v_cache.dtype is not _BF16 or len(shape) != 4
            or strides[3] != 1 or v_cache.shape != shape or v_cache.stride() != strides):
        _refuse_cache(fn, k_cache, v_cache)
    n_pages, page_size, Hkv, D = shape
    dev = k_cache.get_device()
    if v_cache.get_device() != dev:
        _refuse(fn, "v_cache", v_cache, v_cache.dtype, (None,) * 4, dev)
    n = kv_len.numel()
    if kv_len.dtype is not _I32 or kv_len.dim() != 1 or not kv_len.is_contiguous() or kv_len.get_device() != dev:
        _refuse(fn, "kv_len", kv_len, _I32, (n,), dev)
    ts = page_table.shape
    if (page_table.dtype is not _I32 or len(ts) != 2 or ts[0] != n or not page_table.is_contiguous()
            or page_table.get_device() != dev):
        _refuse(fn, "page_table", page_table, _I32, (n, None), dev)
    # the stride of an extent of one says nothing: any valid one will do
    ps, ss, hs, _ = strides
    if n_pages == 1 or page_size == 1 or Hkv == 1:
        ps, ss, hs = (s if e > 1 else D for e, s in zip(shape, (ps, ss, hs)))
    return (_PagedKV(k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), kv_len.data_ptr(), n_pages, ps, ss,
                     hs, page_size, ts[1]), n, Hkv, D, dev)


def _scratch(fn, nbytes, workspace, dev, stream):
    """Address and size of the caller's workspace, or of one for this call; a fresh one lives until the
    call's stream passes it."""
    if workspace is None:
        workspace = torch.empty(max(1, nbytes), dtype=torch.uint8, device=dev)
        if stream is not None and _s(stream) != torch.cuda.current_stream().cuda_stream:
            # the allocator orders memory along the current stream: order the call's stream after it and
            # keep the memory until that stream is done with it
            st = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))
            st.wait_stream(torch.cuda.current_stream())
            workspace.record_stream(st)
        return workspace, nbytes
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(fn, "workspace", workspace, workspace.dtype, workspace.shape, dev)
    return workspace, workspace.nbytes


def dg_kv_append(k, v, k_cache, v_cache, page_table, cu_q, kv_len, *, inv_freq=None, interleaved=False, q=None,
                 q_out=None, stream=None, check=True) -> int:
    """Append k, v [total, Hkv, D] (rows of any stride) to the paged cache, keys rotated by position *
    inv_freq [rot_dim / 2] float64; q [total, Hq, D] is rotated into q_out (contiguous).  The cache:
    k_cache, v_cache [n_pages, page_size, Hkv, D] (any strides but the last), page_table [n_seq,
    max_pages], kv_len [n_seq] and cu_q [n_seq + 1] int32."""
    fn = "dg_kv_append"
    if (q is None) != (q_out is None):
        raise ValueError(f"{fn}: q and q_out come together")
    kv, n, Hkv, D, dev = _paged_kv(fn, k_cache, v_cache, page_table, kv_len)
    total = k.shape[0]
    kp, ldk = _rows(fn, "k", k, Hkv, D, dev)
    vp, ldv = _rows(fn, "v", v, Hkv, D, dev)
    Hq, qp, ldq, op = Hkv, None, 0, None
    if v.shape[0] != total or (q is not None and q.shape[0] != total):
        raise ValueError(f"{fn}: q, k and v must have as many rows")
    if q is not None:
        Hq = q.shape[1] if q.dim() == 3 else 0
        qp, ldq = _rows(fn, "q", q, Hq, D, dev)
        if (q_out.dtype is not _BF16 or q_out.shape != q.shape or not q_out.is_contiguous()
                or q_out.get_device() != dev):
            _refuse(fn, "q_out", q_out, _BF16, (total, Hq, D), dev)
        op = q_out.data_ptr()
    if cu_q.dtype is not _I32 or cu_q.shape != (n + 1,) or not cu_q.is_contiguous() or cu_q.get_device() != dev:
        _refuse(fn, "cu_q", cu_q, _I32, (n + 1,), dev)
    half, wp = 0, None
    if inv_freq is not None:
        half = inv_freq.numel()
        wp = _whole(fn, "inv_freq", inv_freq, torch.float64, (half,), dev)
    rc = load().dg_kv_append(kp, ldk, vp, ldv, qp, ldq, op, cu_q.data_ptr(), n, total, Hq, Hkv, D, wp, 2 * half,
                             1 if interleaved else 0, kv, _on(fn, dev, stream))
    if check and rc:
        _check(fn, rc)
    return rc


def dg_paged_attention_workspace_bytes(n_seq: int, max_q_len: int, Hq: int, Hkv: int, D: int) -> int:
    return int(load().dg_paged_attention_workspace_bytes(n_seq, max_q_len, Hq, Hkv, D))


def dg_paged_attention(q, k_cache, v_cache, o, page_table, cu_q, kv_len, causal, max_q_len: int, *, lse=None,
                       window: int = -1, scale: float | None = None, workspace=None, stream=None,
                       check=True) -> int:
    """dg_attention over the paged cache of dg_kv_append: q, o [total_q, Hq, D] bf16, cu_q [n + 1] and
    kv_len [n] int32, causal [n] uint8, lse [total_q, Hq] float32."""
    fn = "dg_paged_attention"
    kv, n, Hkv, D, dev = _paged_kv(fn, k_cache, v_cache, page_table, kv_len)
    rows = q.shape
    if q.dtype is not _BF16 or len(rows) != 3 or rows[2] != D or not q.is_contiguous() or q.get_device() != dev:
        _refuse(fn, "q", q, _BF16, (None, None, D), dev)
    total, Hq, _ = rows
    if o.dtype is not _BF16 or o.shape != rows or not o.is_contiguous() or o.get_device() != dev:
        _refuse(fn, "o", o, _BF16, rows, dev)
    if cu_q.dtype is not _I32 or cu_q.shape != (n + 1,) or not cu_q.is_contiguous() or cu_q.get_device() != dev:
        _refuse(fn, "cu_q", cu_q, _I32, (n + 1,), dev)
    cz = _whole(fn, "causal", causal, torch.uint8, (n,), dev)
    lp = None if lse is None else _whole(fn, "lse", lse, _F32, (total, Hq), dev)
    st = _on(fn, dev, stream)
    lib = load()
    max_q_len = int(max_q_len)
    scale = D ** -0.5 if scale is None else float(scale)
    need = 0 if workspace is not None else lib.dg_paged_attention_workspace_bytes(n, max_q_len, Hq, Hkv, D)
    workspace, ws_bytes = _scratch(fn, need, workspace, dev, stream)
    rc = lib.dg_paged_attention(q.data_ptr(), kv, o.data_ptr(), lp, cu_q.data_ptr(), cz, n, max_q_len, total, Hq, Hkv,
                                D, int(window), scale, workspace.data_ptr(), ws_bytes, st)
    if check and rc:
        _check(fn, rc)
    return rc


def dg_adjust_logits(logits, params, out=None, *, history=None, cu_history=None, penalties=None,
                     bias_tokens=None, bias_values=None, cu_bias=None, masks=None, mask_index=None, V=None,
                     stream=None, check=True) -> int:
    """Penalties for the tokens of history (penalties [n, 3]: repetition, frequency, presence), biases and
    masks (int32 words, bit set = allowed; mask_index [n, L], -1 = none) on logits [n, L, ld], into out
    (in place when None).  history / bias lists are packed, canvas c's at cu[c] .. cu[c + 1]."""
    fn = "dg_adjust_logits"
    out = logits if out is None else out
    if logits.dim() != 3 or out.dim() != 3:
        raise ValueError(f"{fn}: logits and out must be [n, L, ld]")
    dt, dtype = _dtype_code(logits), logits.dtype
    n, L, ld = logits.shape
    ldo = out.shape[2]
    V = ld if V is None else V
    if (history is None) != (cu_history is None) or (history is None) != (penalties is None):
        raise ValueError(f"{fn}: history, cu_history and penalties come together")
    if (bias_tokens is None) != (bias_values is None) or (bias_tokens is None) != (cu_bias is None):
        raise ValueError(f"{fn}: bias_tokens, bias_values and cu_bias come together")
    if (masks is None) != (mask_index is None):
        raise ValueError(f"{fn}: masks and mask_index come together")
    i32, f32, dev = torch.int32, torch.float32, logits.get_device()
    nh = 0 if history is None else history.numel()
    nb = 0 if bias_tokens is None else bias_tokens.numel()
    n_masks, words = (0, 0) if masks is None else masks.shape if masks.dim() == 2 else (-1, -1)
    xp = _whole(fn, "logits", logits, dtype, (n, L, ld), dev)
    op = _whole(fn, "out", out, dtype, (n, L, ldo), dev)
    pp = _whole(fn, "params", params, torch.uint8, (n * PARAM_BYTES,), dev)
    hp = _whole(fn, "history", history, i32, (nh,), dev)
    ch = _whole(fn, "cu_history", cu_history, i32, (n + 1,), dev)
    pen = _whole(fn, "penalties", penalties, f32, (n, 3), dev)
    bt = _whole(fn, "bias_tokens", bias_tokens, i32, (nb,), dev)
    bv = _whole(fn, "bias_values", bias_values, f32, (nb,), dev)
    cb = _whole(fn, "cu_bias", cu_bias, i32, (n + 1,), dev)
    mp = _whole(fn, "masks", masks, i32, (n_masks, words), dev)
    mi = _whole(fn, "mask_index", mask_index, i32, (n, L), dev)
    rc = load().dg_adjust_logits(xp, dt, ld, op, ldo, n, L, V, pp, hp, ch, nh, pen, bt, bv, cb, nb, mp, words,
                                 n_masks, mi, _on(fn, dev, stream))
    if check and rc:
        _check(fn, rc)
    return rc


def dg_embed_canvas(canvas, E, delta_emb, out, scale: float = 1.0, stream=None, check=True) -> int:
    """out = bf16(fma(scale, E[canvas], delta_emb)); canvas [..] int32, E [V, d], out [.., d]."""
    V, d = E.shape
    rc = load().dg_embed_canvas(_p(canvas), canvas.numel(), V, _p(E), d, _p(delta_emb), float(scale),
                                _p(out), _s(stream))
    if check:
        _check("dg_embed_canvas", rc)
    return rc


def dg_commit(params, converged, argmax, tokens, prev_argmax, stable_count, committed, stream=None,
              check=True) -> int:
    n, L = argmax.shape
    rc = load().dg_commit(_p(params), _p(converged), _p(argmax), n, L, _p(tokens), _p(prev_argmax),
                          _p(stable_count), _p(committed), _s(stream))
    if check:
        _check("dg_commit", rc)
    return rc


def dg_self_cond_workspace_bytes(n_canvas: int, L: int, d: int, h: int) -> int:
    return int(load().dg_self_cond_workspace_bytes(n_canvas, L, d, h))


def dg_self_cond_logits(logits, lse, params, converged, E, W_gate, W_up, W_down, delta_emb,
                        workspace, *, n_canvas=None, L=None, V=None, ld=None, stream=None,
                        check=True) -> int:
    n, Lx, ldx = logits.shape if logits.dim() == 3 else (n_canvas, L, ld)
    n_canvas = n if n_canvas is None else n_canvas
    L = Lx if L is None else L
    ld = ldx if ld is None else ld
    V = ld if V is None else V
    d = E.shape[1]
    h = W_gate.shape[0]
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().dg_self_cond_logits(_p(logits), _dtype_code(logits), ld, _p(lse), _p(params),
                                    _p(converged), n_canvas, L, V, d, h, _p(E), _p(W_gate),
                                    _p(W_up), _p(W_down), _p(delta_emb), _p(workspace), ws_bytes,
                                    _s(stream))
    if check:
        _check("dg_self_cond_logits", rc)
    return rc


def dg_self_cond_prepare(params, converged, n_canvas, L, d, h, delta_emb, workspace, stream=None,
                         check=True) -> int:
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().dg_self_cond_prepare(_p(params), _p(converged), n_canvas, L, d, h, _p(delta_emb),
                                     _p(workspace), ws_bytes, _s(stream))
    if check:
        _check("dg_self_cond_prepare", rc)
    return rc


def dg_self_cond_pe(logits, lse, params, E, h, workspace, *, n_canvas=None, L=None, V=None, ld=None,
                    stream=None, check=True) -> int:
    n, Lx, ldx = logits.shape if logits.dim() == 3 else (n_canvas, L, ld)
    n_canvas = n if n_canvas is None else n_canvas
    L = Lx if L is None else L
    ld = ldx if ld is None else ld
    V = ld if V is None else V
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().dg_self_cond_pe(_p(logits), _dtype_code(logits), ld, _p(lse), _p(params), n_canvas, L, V,
                                E.shape[1], h, _p(E), _p(workspace), ws_bytes, _s(stream))
    if check:
        _check("dg_self_cond_pe", rc)
    return rc


def dg_self_cond_mlp(n_canvas, L, W_gate, W_up, W_down, delta_emb, workspace, stream=None,
                     check=True) -> int:
    d = W_gate.shape[1]
    h = W_gate.shape[0]
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().dg_self_cond_mlp(n_canvas, L, d, h, _p(W_gate), _p(W_up), _p(W_down), _p(delta_emb),
                                 _p(workspace), ws_bytes, _s(stream))
    if check:
        _check("dg_self_cond_mlp", rc)
    return rc


def dg_self_cond_zero_converged(params, converged, delta_emb, stream=None, check=True) -> int:
    """Zero the feedback rows of canvases that got feedback and converged (delta_emb [n, L, d])."""
    n_canvas, L, d = delta_emb.shape
    rc = load().dg_self_cond_zero_converged(_p(params), _p(converged), n_canvas, L, d, _p(delta_emb), _s(stream))
    if check:
        _check("dg_self_cond_zero_converged", rc)
    return rc


def dg_self_cond_probs_workspace_bytes(n_rows: int, d: int, h: int) -> int:
    return int(load().dg_self_cond_probs_workspace_bytes(n_rows, d, h))


def dg_self_cond_probs(P, E, W_gate, W_up, W_down, delta_emb, workspace, *, V=None, stream=None,
                       check=True) -> int:
    n_rows, ld = P.shape
    V = ld if V is None else V
    d = E.shape[1]
    h = W_gate.shape[0]
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().dg_self_cond_probs(_p(P), ld, n_rows, V, d, h, _p(E), _p(W_gate), _p(W_up),
                                   _p(W_down), _p(delta_emb), _p(workspace), ws_bytes, _s(stream))
    if check:
        _check("dg_self_cond_probs", rc)
    return rc


def dg_gemm_workspace_bytes(M: int, N: int) -> int:
    return int(load().dg_gemm_workspace_bytes(M, N))


def dg_gemm_bf16(A, B, C, b_mn_major: bool, workspace, *, M=None, N=None, K=None, stream=None,
                 check=True) -> int:
    M = A.shape[0] if M is None else M
    K = A.shape[1] if K is None else K
    N = (B.shape[1] if b_mn_major else B.shape[0]) if N is None else N
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().dg_gemm_bf16(_p(A), A.stride(0), _p(B), B.stride(0), int(bool(b_mn_major)), _p(C),
                             C.stride(0), M, N, K, _p(workspace), ws_bytes, _s(stream))
    if check:
        _check("dg_gemm_bf16", rc)
    return rc


def dg_gemm_bf16_noalloc(A, B, C, b_mn_major: bool, *, M=None, N=None, K=None, stream=None,
                         check=True) -> int:
    M = A.shape[0] if M is None else M
    K = A.shape[1] if K is None else K
    N = (B.shape[1] if b_mn_major else B.shape[0]) if N is None else N
    rc = load().dg_gemm_bf16_noalloc(_p(A), A.stride(0), _p(B), B.stride(0), int(bool(b_mn_major)), _p(C),
                                     C.stride(0), M, N, K, _s(stream))
    if check:
        _check("dg_gemm_bf16_noalloc", rc)
    return rc


def dg_philox_words(seed, request_id, step, position, stream_id, block0, n_blocks, out,
                    stream=None, check=True) -> int:
    rc = load().dg_philox_words(int(seed) & 0xFFFFFFFFFFFFFFFF, request_id, step, position,
                                stream_id, block0, n_blocks, _p(out), _s(stream))
    if check:
        _check("dg_philox_words", rc)
    return rc


def dg_get_device_status(stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check("dg_get_device_status", load().dg_get_device_status(_s(stream), ctypes.byref(v)))
    return int(v.value)


def dg_clear_device_status(stream=None) -> None:
    _check("dg_clear_device_status", load().dg_clear_device_status(_s(stream)))


def dg_probe_bounded_wait(polls, result, stream=None, check=True) -> int:
    rc = load().dg_probe_bounded_wait(int(polls), _p(result), _s(stream))
    if check:
        _check("dg_probe_bounded_wait", rc)
    return rc
