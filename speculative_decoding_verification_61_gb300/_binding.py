"""ctypes marshalling for libspecverify.so (argument marshalling only)."""
from __future__ import annotations

import array
import ctypes
import functools
import math
import os

PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(PKG, "_build", "libspecverify.so")

F32, BF16 = 0, 1
MAX_K, MAX_B, MAX_V = 32, 4096, 1 << 24
MAX_TREE_NODES = 64
MAX_SHARDS = 64
MAX_BEAMS, MAX_CANDIDATES, MAX_STATES = 64, 128, 64
ROWS = {"target": 0, "draft": 1, "next": 2, "tree": 3}  # SPEC_ROWS_*
CACHE_ROWS = {"target": 0, "next": 2, "tree": 3, "prompt": 4}
NOALLOC_SCRATCH_BYTES = 48 << 20  # spec_verify_noalloc's fixed scratch array
ABI_VERSION = 1
SPEC_ERRORS = {0: "SPEC_OK", -1: "SPEC_ERR_INVALID_ARG", -2: "SPEC_ERR_ALIGNMENT",
               -3: "SPEC_ERR_CUDA", -4: "SPEC_ERR_TIMEOUT", -5: "SPEC_ERR_WORKSPACE"}

# every symbol include/spec_verify.h declares
EXPORTS = ("spec_verify", "spec_verify_ex", "spec_draft_sample", "spec_draft_sample_ex",
           "spec_round_host", "spec_workspace_bytes", "spec_workspace_status",
           "spec_status_string", "spec_abi_version", "spec_last_error", "spec_verify_noalloc",
           "spec_noalloc_bytes", "spec_adapt_state_bytes", "spec_adapt_init", "spec_adapt_update",
           "spec_draft_sample_lse", "spec_verify_lse", "spec_round", "spec_tree_verify",
           "spec_tree_draft_sample", "spec_shard_workspace_bytes", "spec_shard_stats",
           "spec_shard_decide", "spec_shard_draw", "spec_shutdown", "spec_selfcheck_wait_timeout",
           "spec_logits_process", "spec_logits_truncate", "spec_logits_process_truncate",
           "spec_penalty_reset", "spec_penalty_update", "spec_beam_workspace_bytes", "spec_beam_select",
           "spec_state_reorder", "spec_state_reorder_status", "spec_selfcheck_reorder_timeout", "spec_cache_write",
           "spec_cache_read")


class SpecError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {SPEC_ERRORS.get(code, code)}")
        self.code = code


class _Aux(ctypes.Structure):
    _fields_ = [("accept_prob", ctypes.c_void_p), ("residual_mass", ctypes.c_void_p),
                ("lse_target", ctypes.c_void_p), ("lse_draft", ctypes.c_void_p)]


class _Rows(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("B", ctypes.c_int), ("R", ctypes.c_int),
                ("offsets", ctypes.c_void_p), ("parent", ctypes.c_void_p),
                ("draft_tokens", ctypes.c_void_p), ("n_tokens", ctypes.c_int)]


class _Logits(ctypes.Structure):
    _fields_ = [("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("counts", ctypes.c_void_p), ("seen", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("S", ctypes.c_int), ("bias_offsets", ctypes.c_void_p), ("bias_tokens", ctypes.c_void_p),
                ("bias_values", ctypes.c_void_p), ("n_bias", ctypes.c_int), ("mask", ctypes.c_void_p),
                ("mask_rows", ctypes.c_void_p), ("M", ctypes.c_int)]


class _Truncate(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
                ("min_p", ctypes.c_void_p)]


class _State(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("planes", ctypes.c_int64), ("runs", ctypes.c_int64),
                ("T", ctypes.c_int64), ("unit", ctypes.c_int64)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("L", ctypes.c_int), ("P", ctypes.c_int), ("T", ctypes.c_int),
                ("H", ctypes.c_int), ("D", ctypes.c_int), ("pages", ctypes.c_void_p), ("S", ctypes.c_int),
                ("M", ctypes.c_int), ("lengths", ctypes.c_void_p)]


_lib = None


def lib_path() -> str:
    return _LIB_PATH


def lib():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"CUDA library not built: {_LIB_PATH} is missing "
                           "(run __graft_entry__.build() or python -m "
                           "speculative_decoding_verification_61_gb300.build)")
    L = ctypes.CDLL(_LIB_PATH)
    vp, ip, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.spec_verify.argtypes = [vp, vp, vp, vp, vp, vp, ip, vp, ip, ip, vp, vp, vp]
    L.spec_verify_ex.argtypes = [vp, vp, vp, vp, vp, vp, ip, vp, ip, ip, vp, vp,
                                 ctypes.POINTER(_Aux), vp, sz, vp]
    L.spec_draft_sample.argtypes = [vp, vp, vp, ip, vp, ip, ip, vp, vp]
    L.spec_draft_sample_ex.argtypes = [vp, vp, vp, ip, vp, ip, ip, vp, vp, sz, vp]
    L.spec_round_host.argtypes = [vp, vp, vp, vp, vp, vp, ip, vp, ip, ip, vp, vp, vp, vp]
    L.spec_draft_sample_lse.argtypes = [vp, vp, vp, ip, vp, ip, ip, vp, vp, vp, sz, vp]
    L.spec_verify_lse.argtypes = [vp, vp, vp, vp, vp, vp, vp, ip, vp, ip, ip, vp, vp,
                                  ctypes.POINTER(_Aux), vp, sz, vp]
    L.spec_round.argtypes = [vp, vp, vp, vp, vp, vp, ip, vp, ip, ip, vp, vp, vp, vp]
    L.spec_tree_verify.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ip, ip, ip, ip, vp, vp, vp, vp]
    L.spec_tree_draft_sample.argtypes = [vp, vp, vp, vp, vp, ip, ip, ip, ip, vp, vp]
    L.spec_shard_workspace_bytes.argtypes = [ip, ip, ip]
    L.spec_shard_workspace_bytes.restype = sz
    L.spec_shard_stats.argtypes = [vp, vp, vp, vp, ip, vp, vp, ip, ip, ip, vp, vp, sz, vp]
    L.spec_shard_decide.argtypes = [vp, vp, vp, vp, vp, vp, ip, vp, vp, ip, ip, ip, vp, vp, vp, vp, sz, vp]
    L.spec_shard_draw.argtypes = [vp, vp, vp, vp, ip, vp, vp, ip, ip, ip, vp, vp, sz, vp]
    L.spec_workspace_bytes.argtypes = [ip, ip, ip]
    L.spec_workspace_bytes.restype = sz
    L.spec_noalloc_bytes.argtypes = [ip, ip, ip]
    L.spec_noalloc_bytes.restype = sz
    L.spec_workspace_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int), ip]
    L.spec_status_string.argtypes = [ip]
    L.spec_status_string.restype = ctypes.c_char_p
    L.spec_abi_version.argtypes = []
    L.spec_shutdown.argtypes = []
    L.spec_shutdown.restype = ip
    L.spec_selfcheck_wait_timeout.argtypes = [vp, sz, vp]
    L.spec_selfcheck_wait_timeout.restype = ip
    L.spec_verify_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, ip, vp, ip, ip, vp, vp, vp]
    L.spec_verify_noalloc.restype = ip
    L.spec_last_error.argtypes = []
    L.spec_last_error.restype = ctypes.c_char_p
    L.spec_adapt_state_bytes.argtypes = [ip]
    L.spec_adapt_state_bytes.restype = sz
    L.spec_adapt_init.argtypes = [vp, ip, ip, ip, vp, vp]
    L.spec_adapt_init.restype = ip
    L.spec_adapt_update.argtypes = [vp, vp, ip, ip, ip, vp, vp]
    L.spec_adapt_update.restype = ip
    rp, gp, tp = ctypes.POINTER(_Rows), ctypes.POINTER(_Logits), ctypes.POINTER(_Truncate)
    L.spec_logits_process.argtypes = [vp, rp, gp, ip, ip, vp, vp]
    L.spec_logits_truncate.argtypes = [vp, rp, tp, ip, ip, vp, vp]
    L.spec_logits_process_truncate.argtypes = [vp, rp, gp, tp, ip, ip, vp, vp]
    L.spec_penalty_reset.argtypes = [vp, vp, ip, ip, vp, ip, vp, vp, ip, vp, vp, ip, vp]
    L.spec_penalty_update.argtypes = [vp, vp, ip, ip, vp, rp, vp, vp, vp]
    for name in ("spec_logits_process", "spec_logits_truncate", "spec_logits_process_truncate",
                 "spec_penalty_reset", "spec_penalty_update"):
        getattr(L, name).restype = ip
    i64, cp = ctypes.c_int64, ctypes.POINTER(_Cache)
    L.spec_beam_workspace_bytes.argtypes = [ip, ip, ip]
    L.spec_beam_workspace_bytes.restype = sz
    L.spec_beam_select.argtypes = [vp, vp, vp, ip, vp, ip, ip, ip, ip, ip, vp, vp, vp, vp, vp, sz, vp]
    L.spec_state_reorder.argtypes = [vp, ip, ip, vp, vp, ip, ip, vp, vp, vp]
    L.spec_selfcheck_reorder_timeout.argtypes = L.spec_state_reorder.argtypes
    L.spec_state_reorder_status.argtypes = [ctypes.POINTER(ctypes.c_int), ip]
    L.spec_cache_write.argtypes = [cp, vp, vp, i64, i64, ip, rp, vp, vp, vp, vp, vp]
    L.spec_cache_read.argtypes = [cp, vp, ip, ip, vp, vp, ip, vp, vp, vp]
    for name in ("spec_beam_select", "spec_state_reorder", "spec_state_reorder_status", "spec_selfcheck_reorder_timeout",
                 "spec_cache_write", "spec_cache_read"):
        getattr(L, name).restype = ip
    for name in ("spec_verify", "spec_verify_ex", "spec_draft_sample", "spec_draft_sample_ex",
                 "spec_round_host", "spec_workspace_status", "spec_abi_version",
                 "spec_draft_sample_lse", "spec_verify_lse", "spec_round", "spec_tree_verify",
                 "spec_tree_draft_sample", "spec_shard_stats", "spec_shard_decide", "spec_shard_draw"):
        getattr(L, name).restype = ip
    _lib = L
    return L


def exported_symbols():
    L = lib()
    return {name: hasattr(L, name) for name in EXPORTS}


# ----------------------------------------------------------------- helpers
def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_dev(name, t, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _new(shape, dtype, dev, stream, fill=None):
    """A call's output: memory of the stream that the call runs on (what the current stream has freed may still
    be in use there), not given to others before the current stream, too, is done with it."""
    import torch
    if stream is None and fill is None:
        return torch.empty(shape, dtype=dtype, device=dev)

    def make():
        return torch.empty(shape, dtype=dtype, device=dev) if fill is None else torch.full(shape, fill, dtype=dtype, device=dev)

    here = None if stream is None else torch.cuda.current_stream(dev)
    if here is None or here.cuda_stream == stream.cuda_stream:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(here)
    return t


def _raise(rc, what):
    if rc != 0:
        detail = lib().spec_last_error().decode() if rc == -3 else ""
        raise SpecError(rc, f"{what} [{detail}]" if detail else what)


# ----------------------------------------------------------------- API
def spec_verify(target_logits, draft_logits, draft_tokens, u_accept, u_resample,
                temperature, k_offsets, out_tokens=None, out_num_accepted=None,
                aux: bool = False, workspace=None, stream=None):
    """Verify-and-resample (device tensors).  Returns (out_tokens [R_t] int32,
    out_num_accepted [B] int32) and, with aux=True, a dict of accept_prob,
    residual_mass, lse_target, lse_draft (float32)."""
    import torch
    B = temperature.numel()
    V = target_logits.shape[-1]
    dt = _dtype_code(target_logits)
    for name, t in (("target_logits", target_logits), ("draft_logits", draft_logits)):
        _check_dev(name, t, target_logits.dtype)
    _check_dev("draft_tokens", draft_tokens, torch.int32)
    _check_dev("u_accept", u_accept, torch.float32)
    _check_dev("u_resample", u_resample, torch.float32)
    _check_dev("temperature", temperature, torch.float32)
    _check_dev("k_offsets", k_offsets, torch.int32)
    if k_offsets.numel() != B + 1:
        raise ValueError("k_offsets must have B + 1 entries")
    R_t = u_resample.numel()
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = _new(R_t, torch.int32, dev, stream)
    if out_num_accepted is None:
        out_num_accepted = _new(B, torch.int32, dev, stream)
    L = lib()
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (_p(workspace), workspace.numel() * workspace.element_size())
    aux_out, ax = _aux_buffers(B, R_t, draft_tokens.numel(), dev, stream) if aux else (None, None)
    if ax is None and workspace is None:
        rc = L.spec_verify(_p(target_logits), _p(draft_logits), _p(draft_tokens), _p(u_accept),
                           _p(u_resample), _p(temperature), B, _p(k_offsets), V, dt,
                           _p(out_tokens), _p(out_num_accepted), _stream(stream))
    else:
        rc = L.spec_verify_ex(_p(target_logits), _p(draft_logits), _p(draft_tokens), _p(u_accept),
                              _p(u_resample), _p(temperature), B, _p(k_offsets), V, dt,
                              _p(out_tokens), _p(out_num_accepted),
                              ctypes.byref(ax) if ax is not None else None, ws_ptr, ws_bytes,
                              _stream(stream))
    _raise(rc, "spec_verify")
    if aux:
        return out_tokens, out_num_accepted, aux_out
    return out_tokens, out_num_accepted


def spec_draft_sample(draft_logits, temperature, u_draft, k_offsets, out_draft_tokens=None,
                      workspace=None, stream=None):
    """Draft-side softmax + multinomial (argmax for T = 0).  Returns int32 [R_d]."""
    import torch
    B = temperature.numel()
    V = draft_logits.shape[-1]
    dt = _dtype_code(draft_logits)
    _check_dev("draft_logits", draft_logits)
    _check_dev("temperature", temperature, torch.float32)
    _check_dev("u_draft", u_draft, torch.float32)
    _check_dev("k_offsets", k_offsets, torch.int32)
    if out_draft_tokens is None:
        out_draft_tokens = _new(u_draft.numel(), torch.int32, draft_logits.device, stream)
    L = lib()
    if workspace is None:
        rc = L.spec_draft_sample(_p(draft_logits), _p(temperature), _p(u_draft), B, _p(k_offsets), V,
                                 dt, _p(out_draft_tokens), _stream(stream))
    else:
        rc = L.spec_draft_sample_ex(_p(draft_logits), _p(temperature), _p(u_draft), B, _p(k_offsets),
                                    V, dt, _p(out_draft_tokens), _p(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    _raise(rc, "spec_draft_sample")
    return out_draft_tokens


def _aux_buffers(B, R_t, R_d, dev, stream):
    import torch
    out = dict(accept_prob=_new((R_d,), torch.float32, dev, stream, float("nan")),
               residual_mass=_new((B,), torch.float32, dev, stream, float("nan")),
               lse_target=_new((R_t,), torch.float32, dev, stream, float("nan")),
               lse_draft=_new((R_d,), torch.float32, dev, stream, float("nan")))
    ax = _Aux(*(ctypes.c_void_p(out[k].data_ptr()) for k in
                ("accept_prob", "residual_mass", "lse_target", "lse_draft")))
    return out, ax


def spec_draft_sample_lse(draft_logits, temperature, u_draft, k_offsets, out_draft_tokens=None,
                          out_draft_lse2=None, workspace=None, stream=None):
    """Draft sampling that also returns each draft row's log2-domain
    log-sum-exp (float64 [R_d], NaN for greedy/invalid rows), for
    spec_verify_lse.  Returns (draft_tokens int32 [R_d], draft_lse2)."""
    import torch
    B = temperature.numel()
    V = draft_logits.shape[-1]
    dt = _dtype_code(draft_logits)
    _check_dev("draft_logits", draft_logits)
    _check_dev("temperature", temperature, torch.float32)
    _check_dev("u_draft", u_draft, torch.float32)
    _check_dev("k_offsets", k_offsets, torch.int32)
    R_d = u_draft.numel()
    dev = draft_logits.device
    if out_draft_tokens is None:
        out_draft_tokens = _new(R_d, torch.int32, dev, stream)
    if out_draft_lse2 is None:
        out_draft_lse2 = _new(max(R_d, 1), torch.float64, dev, stream)
    _check_dev("out_draft_lse2", out_draft_lse2, torch.float64)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (_p(workspace), workspace.numel() * workspace.element_size())
    rc = lib().spec_draft_sample_lse(_p(draft_logits), _p(temperature), _p(u_draft), B, _p(k_offsets), V, dt,
                                     _p(out_draft_tokens), _p(out_draft_lse2), ws_ptr, ws_bytes, _stream(stream))
    _raise(rc, "spec_draft_sample_lse")
    return out_draft_tokens, out_draft_lse2[:R_d]


def spec_verify_lse(target_logits, draft_logits, draft_lse2, draft_tokens, u_accept, u_resample,
                    temperature, k_offsets, out_tokens=None, out_num_accepted=None, aux: bool = False,
                    workspace=None, stream=None):
    """spec_verify with the draft rows' normalisers given (from
    spec_draft_sample_lse): only the target rows are streamed.  Same
    returns as spec_verify."""
    import torch
    B = temperature.numel()
    V = target_logits.shape[-1]
    dt = _dtype_code(target_logits)
    for name, t in (("target_logits", target_logits), ("draft_logits", draft_logits)):
        _check_dev(name, t, target_logits.dtype)
    _check_dev("draft_lse2", draft_lse2, torch.float64)
    _check_dev("draft_tokens", draft_tokens, torch.int32)
    _check_dev("u_accept", u_accept, torch.float32)
    _check_dev("u_resample", u_resample, torch.float32)
    _check_dev("temperature", temperature, torch.float32)
    _check_dev("k_offsets", k_offsets, torch.int32)
    if k_offsets.numel() != B + 1:
        raise ValueError("k_offsets must have B + 1 entries")
    R_t, R_d = u_resample.numel(), draft_tokens.numel()
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = _new(R_t, torch.int32, dev, stream)
    if out_num_accepted is None:
        out_num_accepted = _new(B, torch.int32, dev, stream)
    aux_out, ax = _aux_buffers(B, R_t, R_d, dev, stream) if aux else (None, None)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (_p(workspace), workspace.numel() * workspace.element_size())
    rc = lib().spec_verify_lse(_p(target_logits), _p(draft_logits), _p(draft_lse2), _p(draft_tokens),
                               _p(u_accept), _p(u_resample), _p(temperature), B, _p(k_offsets), V, dt,
                               _p(out_tokens), _p(out_num_accepted),
                               ctypes.byref(ax) if ax is not None else None, ws_ptr, ws_bytes, _stream(stream))
    _raise(rc, "spec_verify_lse")
    if aux:
        return out_tokens, out_num_accepted, aux_out
    return out_tokens, out_num_accepted


def spec_round(target_logits, draft_logits, u_draft, u_accept, u_resample, temperature, k_offsets,
               out_draft_tokens=None, out_tokens=None, out_num_accepted=None, stream=None):
    """One sampling round on device tensors: draft sampling, then verify
    with the draft rows' normalisers kept between the passes (every row
    read once).  Returns (draft_tokens [R_d], out_tokens [R_t],
    out_num_accepted [B])."""
    import torch
    B = temperature.numel()
    V = target_logits.shape[-1]
    dt = _dtype_code(target_logits)
    for name, t in (("target_logits", target_logits), ("draft_logits", draft_logits)):
        _check_dev(name, t, target_logits.dtype)
    for name, t in (("u_draft", u_draft), ("u_accept", u_accept), ("u_resample", u_resample),
                    ("temperature", temperature)):
        _check_dev(name, t, torch.float32)
    _check_dev("k_offsets", k_offsets, torch.int32)
    if k_offsets.numel() != B + 1:
        raise ValueError("k_offsets must have B + 1 entries")
    R_t, R_d = u_resample.numel(), u_accept.numel()
    dev = target_logits.device
    if out_draft_tokens is None:
        out_draft_tokens = _new(R_d, torch.int32, dev, stream)
    if out_tokens is None:
        out_tokens = _new(R_t, torch.int32, dev, stream)
    if out_num_accepted is None:
        out_num_accepted = _new(B, torch.int32, dev, stream)
    rc = lib().spec_round(_p(target_logits), _p(draft_logits), _p(u_draft), _p(u_accept), _p(u_resample),
                          _p(temperature), B, _p(k_offsets), V, dt, _p(out_draft_tokens), _p(out_tokens),
                          _p(out_num_accepted), _stream(stream))
    _raise(rc, "spec_round")
    return out_draft_tokens, out_tokens, out_num_accepted


def spec_tree_verify(target_logits, draft_logits, node_offsets, parent, tokens, u_accept, u_resample,
                     temperature, out_tokens=None, out_num_accepted=None, out_last_node=None,
                     stream=None):
    """Tree (multi-candidate) verify (device tensors, one target and one
    draft row per node).  Returns (out_tokens [N] int32, out_num_accepted [B]
    int32, out_last_node [B] int32)."""
    import torch
    B = temperature.numel()
    N = parent.numel()
    V = target_logits.shape[-1]
    dt = _dtype_code(target_logits)
    for name, t in (("target_logits", target_logits), ("draft_logits", draft_logits)):
        _check_dev(name, t, target_logits.dtype)
    for name, t in (("node_offsets", node_offsets), ("parent", parent), ("tokens", tokens)):
        _check_dev(name, t, torch.int32)
    for name, t in (("u_accept", u_accept), ("u_resample", u_resample), ("temperature", temperature)):
        _check_dev(name, t, torch.float32)
    if node_offsets.numel() != B + 1:
        raise ValueError("node_offsets must have B + 1 entries")
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = _new(N, torch.int32, dev, stream)
    if out_num_accepted is None:
        out_num_accepted = _new(B, torch.int32, dev, stream)
    if out_last_node is None:
        out_last_node = _new(B, torch.int32, dev, stream)
    rc = lib().spec_tree_verify(_p(target_logits), _p(draft_logits), _p(node_offsets), _p(parent), _p(tokens),
                                _p(u_accept), _p(u_resample), _p(temperature), B, N, V, dt, _p(out_tokens),
                                _p(out_num_accepted), _p(out_last_node), _stream(stream))
    _raise(rc, "spec_tree_verify")
    return out_tokens, out_num_accepted, out_last_node


def spec_tree_draft_sample(draft_logits, node_offsets, parent, temperature, u_draft, out_tokens=None,
                           stream=None):
    """Tree drafting: each non-root node's token from its parent's draft
    row.  Returns int32 [N] (-1 for roots)."""
    import torch
    B = temperature.numel()
    N = parent.numel()
    V = draft_logits.shape[-1]
    dt = _dtype_code(draft_logits)
    _check_dev("draft_logits", draft_logits)
    for name, t in (("node_offsets", node_offsets), ("parent", parent)):
        _check_dev(name, t, torch.int32)
    _check_dev("temperature", temperature, torch.float32)
    _check_dev("u_draft", u_draft, torch.float32)
    if out_tokens is None:
        out_tokens = _new(N, torch.int32, draft_logits.device, stream)
    rc = lib().spec_tree_draft_sample(_p(draft_logits), _p(node_offsets), _p(parent), _p(temperature), _p(u_draft),
                                      B, N, V, dt, _p(out_tokens), _stream(stream))
    _raise(rc, "spec_tree_draft_sample")
    return out_tokens


def spec_round_host(target_logits, draft_logits, u_draft, u_accept, u_resample, temperature,
                    k_offsets, out_draft_tokens=None, out_tokens=None, out_num_accepted=None,
                    stream=None):
    """One sampling round from host (CPU, ideally pinned) tensors: draft
    sampling then verify on the GPU, results copied back to host tensors."""
    import torch
    B = temperature.numel()
    V = target_logits.shape[-1]
    dt = _dtype_code(target_logits)
    for name, t in (("target_logits", target_logits), ("draft_logits", draft_logits),
                    ("u_draft", u_draft), ("u_accept", u_accept), ("u_resample", u_resample),
                    ("temperature", temperature), ("k_offsets", k_offsets)):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor")
    R_d, R_t = u_accept.numel(), u_resample.numel()
    if out_draft_tokens is None:
        out_draft_tokens = torch.empty(R_d, dtype=torch.int32)
    if out_tokens is None:
        out_tokens = torch.empty(R_t, dtype=torch.int32)
    if out_num_accepted is None:
        out_num_accepted = torch.empty(B, dtype=torch.int32)
    rc = lib().spec_round_host(_p(target_logits), _p(draft_logits), _p(u_draft), _p(u_accept),
                               _p(u_resample), _p(temperature), B, _p(k_offsets), V, dt,
                               _p(out_draft_tokens), _p(out_tokens), _p(out_num_accepted),
                               _stream(stream))
    _raise(rc, "spec_round_host")
    return out_draft_tokens, out_tokens, out_num_accepted


# ------------------------------------------------------- vocab-sharded verify
def _bounds(shard_bounds):
    b = [int(x) for x in shard_bounds]
    return (ctypes.c_int32 * len(b))(*b), len(b) - 1


def _ws_args(workspace):
    _check_dev("workspace", workspace)
    return _p(workspace), workspace.numel() * workspace.element_size()


def shard_workspace_bytes(B: int, Vs: int, dtype: int) -> int:
    """Workspace bytes of one rank's vocab-sharded verify (Vs columns)."""
    return int(lib().spec_shard_workspace_bytes(B, Vs, dtype))


def shard_workspace(B: int, Vs: int, dtype: int, device="cuda"):
    """A zero-filled workspace tensor for spec_shard_* (the caching
    allocator's blocks are 512-byte aligned; the zeros clear the status
    word that workspace_status reads)."""
    import torch
    n = shard_workspace_bytes(B, Vs, dtype)
    if n == 0:
        raise ValueError(f"invalid shard workspace arguments B={B}, Vs={Vs}, dtype={dtype}")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def spec_shard_stats(target_shard, draft_shard, draft_tokens, temperature, k_offsets, shard_bounds, rank,
                     workspace, out_stats=None, stream=None):
    """Step 1 of the vocab-sharded verify on this rank's columns.  Returns
    the row records as int32 [R_t + R_d, 4] (fields m, s, zx as float bits,
    then arg)."""
    import torch
    B = temperature.numel()
    dt = _dtype_code(target_shard)
    for name, t in (("target_shard", target_shard), ("draft_shard", draft_shard)):
        _check_dev(name, t, target_shard.dtype)
    _check_dev("draft_tokens", draft_tokens, torch.int32)
    _check_dev("temperature", temperature, torch.float32)
    _check_dev("k_offsets", k_offsets, torch.int32)
    rows = target_shard.shape[0] + draft_shard.shape[0]
    if out_stats is None:
        out_stats = _new((rows, 4), torch.int32, target_shard.device, stream)
    bounds, G = _bounds(shard_bounds)
    wp, wb = _ws_args(workspace)
    rc = lib().spec_shard_stats(_p(target_shard), _p(draft_shard), _p(draft_tokens), _p(temperature), B,
                                _p(k_offsets), bounds, G, rank, dt, _p(out_stats), wp, wb, _stream(stream))
    _raise(rc, "spec_shard_stats")
    return out_stats


def spec_shard_decide(target_shard, draft_shard, all_stats, draft_tokens, u_accept, temperature, k_offsets,
                      shard_bounds, rank, workspace, out_tokens=None, out_num_accepted=None, out_mass=None,
                      stream=None):
    """Step 2: the decision from the gathered records (all_stats: the G
    ranks' records, rank-major).  Returns (out_tokens [R_t] int32,
    out_num_accepted [B] int32, out_mass [B, 2] float64)."""
    import torch
    B = temperature.numel()
    dt = _dtype_code(target_shard)
    bounds, G = _bounds(shard_bounds)
    R_t, R_d = target_shard.shape[0], draft_shard.shape[0]
    _check_dev("all_stats", all_stats, torch.int32)
    if all_stats.numel() != G * (R_t + R_d) * 4:
        raise ValueError("all_stats must hold G * (R_t + R_d) records")
    for name, t in (("draft_tokens", draft_tokens), ("k_offsets", k_offsets)):
        _check_dev(name, t, torch.int32)
    for name, t in (("u_accept", u_accept), ("temperature", temperature)):
        _check_dev(name, t, torch.float32)
    dev = target_shard.device
    if out_tokens is None:
        out_tokens = _new(R_t, torch.int32, dev, stream)
    if out_num_accepted is None:
        out_num_accepted = _new(B, torch.int32, dev, stream)
    if out_mass is None:
        out_mass = _new((B, 2), torch.float64, dev, stream)
    wp, wb = _ws_args(workspace)
    rc = lib().spec_shard_decide(_p(target_shard), _p(draft_shard), _p(all_stats), _p(draft_tokens), _p(u_accept),
                                 _p(temperature), B, _p(k_offsets), bounds, G, rank, dt, _p(out_tokens),
                                 _p(out_num_accepted), _p(out_mass), wp, wb, _stream(stream))
    _raise(rc, "spec_shard_decide")
    return out_tokens, out_num_accepted, out_mass


def spec_shard_draw(target_shard, draft_shard, all_mass, u_resample, k_offsets, shard_bounds, rank, workspace,
                    out_tokens, stream=None):
    """Step 3: the draw by the rank owning the crossing (all_mass: the G
    ranks' out_mass, rank-major).  Writes the drawn token into out_tokens
    on that rank; returns out_tokens."""
    import torch
    B = k_offsets.numel() - 1
    dt = _dtype_code(target_shard)
    bounds, G = _bounds(shard_bounds)
    _check_dev("all_mass", all_mass, torch.float64)
    if all_mass.numel() != G * B * 2:
        raise ValueError("all_mass must hold G * B * 2 values")
    _check_dev("u_resample", u_resample, torch.float32)
    _check_dev("k_offsets", k_offsets, torch.int32)
    _check_dev("out_tokens", out_tokens, torch.int32)
    wp, wb = _ws_args(workspace)
    rc = lib().spec_shard_draw(_p(target_shard), _p(draft_shard), _p(all_mass), _p(u_resample), B, _p(k_offsets),
                               bounds, G, rank, dt, _p(out_tokens), wp, wb, _stream(stream))
    _raise(rc, "spec_shard_draw")
    return out_tokens


def selfcheck_wait_timeout(workspace, stream=None):
    """Run the device-side bounded waits until they give up (about 4 s);
    afterwards workspace_status(workspace) is SPEC_ERR_TIMEOUT."""
    wp, wb = _ws_args(workspace)
    _raise(lib().spec_selfcheck_wait_timeout(wp, wb, _stream(stream)), "spec_selfcheck_wait_timeout")


def shutdown():
    """Free the library-owned device buffers (they are allocated again on
    the next call that needs them)."""
    _raise(lib().spec_shutdown(), "spec_shutdown")


def workspace_bytes(B: int, V: int, dtype: int) -> int:
    return int(lib().spec_workspace_bytes(B, V, dtype))


def noalloc_bytes(B: int, V: int, dtype: int) -> int:
    """Scratch a spec_verify_noalloc call uses (refused above NOALLOC_SCRATCH_BYTES)."""
    return int(lib().spec_noalloc_bytes(B, V, dtype))


def workspace_status(workspace=None, clear: bool = False) -> int:
    """Device status word of a workspace tensor (None: the library-owned one)."""
    v = ctypes.c_int(0)
    rc = lib().spec_workspace_status(None if workspace is None else _p(workspace), ctypes.byref(v),
                                     1 if clear else 0)
    _raise(rc, "spec_workspace_status")
    return v.value


def spec_verify_noalloc(target_logits, draft_logits, draft_tokens, u_accept, u_resample,
                        temperature, k_offsets, out_tokens=None, out_num_accepted=None,
                        stream=None):
    """spec_verify without any device allocation inside the call, for callers
    that cannot allocate while they verify (a serving loop that keeps
    allocation off its hot path, a runtime whose memory pool owns the
    device).  Scratch comes from a fixed array in the library (48 MiB);
    larger batches raise SpecError (SPEC_ERR_WORKSPACE).  Calls share that
    array, so keep them ordered on one stream.  Pass out_tokens and
    out_num_accepted to keep this wrapper from allocating them; the inputs
    are checked as spec_verify checks them."""
    import torch
    B = temperature.numel()
    V = target_logits.shape[-1]
    dt = _dtype_code(target_logits)
    for name, t in (("target_logits", target_logits), ("draft_logits", draft_logits)):
        _check_dev(name, t, target_logits.dtype)
    _check_dev("draft_tokens", draft_tokens, torch.int32)
    _check_dev("u_accept", u_accept, torch.float32)
    _check_dev("u_resample", u_resample, torch.float32)
    _check_dev("temperature", temperature, torch.float32)
    _check_dev("k_offsets", k_offsets, torch.int32)
    if k_offsets.numel() != B + 1:
        raise ValueError("k_offsets must have B + 1 entries")
    R_t = u_resample.numel()
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = _new(R_t, torch.int32, dev, stream)
    if out_num_accepted is None:
        out_num_accepted = _new(B, torch.int32, dev, stream)
    _check_dev("out_tokens", out_tokens, torch.int32)
    _check_dev("out_num_accepted", out_num_accepted, torch.int32)
    if out_tokens.numel() < R_t or out_num_accepted.numel() < B:
        raise ValueError("out_tokens needs R_t = u_resample.numel() entries and out_num_accepted B")
    rc = lib().spec_verify_noalloc(_p(target_logits), _p(draft_logits), _p(draft_tokens), _p(u_accept),
                                   _p(u_resample), _p(temperature), B, _p(k_offsets), V, dt,
                                   _p(out_tokens), _p(out_num_accepted), _stream(stream))
    _raise(rc, "spec_verify_noalloc")
    return out_tokens, out_num_accepted


class AdaptiveK:
    """Device-side adaptive draft length for a batch of B sequences (the
    spec_adapt_* entry points): holds the state buffer and the next round's
    k_offsets on the device."""

    def __init__(self, B: int, min_k: int = 1, max_k: int = 10, device="cuda", stream=None):
        import torch
        nbytes = int(lib().spec_adapt_state_bytes(B))
        if nbytes == 0:
            raise SpecError(-1, "spec_adapt_state_bytes")
        self.B, self.min_k, self.max_k = B, min_k, max_k
        self.state = _new(nbytes, torch.uint8, device, stream)
        self.k_offsets = _new(B + 1, torch.int32, device, stream)
        _raise(lib().spec_adapt_init(_p(self.state), B, min_k, max_k, _p(self.k_offsets), _stream(stream)),
               "spec_adapt_init")

    def update(self, num_accepted, stream=None):
        """Feed one round's out_num_accepted ([B] int32, device); returns the
        next round's k_offsets ([B+1] int32, device, updated in place)."""
        import torch
        _check_dev("num_accepted", num_accepted, torch.int32)
        _raise(lib().spec_adapt_update(_p(self.state), _p(num_accepted), self.B, self.min_k, self.max_k,
                                       _p(self.k_offsets), _stream(stream)), "spec_adapt_update")
        return self.k_offsets


# ------------------------------------------------------------- logit operators
# A decoding step's calls are microseconds on the device, so their checks are
# written to cost little: one test per tensor, its reasons found when it fails.
def _ptr(t, name, dtype, dev, n=-1):
    """data_ptr of a contiguous tensor of its type on the call's device, with n entries if n >= 0; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or (n >= 0 and t.numel() != n):
        _check_dev(name, t, dtype)
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{dev}")
        raise ValueError(f"{name} must have {n} entries, got {t.numel()}")
    return t.data_ptr()


def _size(n, name):
    """A number of entries, which the C ABI takes as an int."""
    if n > 0x7fffffff:
        raise ValueError(f"{name} has {n} entries, more than 2147483647")
    return n


def _launch(dev, stream, fn, what, *args):
    """Calls fn(*args, stream) with device `dev` current, on its current stream if none is given."""
    import torch
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc != 0:
        _raise(rc, what)


def _rows_arg(logits, offsets, rows, draft_tokens, parent, i32):
    mode = ROWS.get(rows)
    if mode is None:
        raise ValueError(f"rows must be one of {sorted(ROWS)}, got {rows!r}")
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, V]")
    if not logits.is_cuda or not logits.is_contiguous():
        _check_dev("logits", logits)
    dev = logits.get_device()
    R, B = _size(logits.shape[0], "logits"), _size(offsets.numel() - 1, "offsets")
    _size(logits.shape[1], "a row")
    if B < 0:
        raise ValueError("offsets must have B + 1 entries")
    n_tokens = 0 if draft_tokens is None else _size(draft_tokens.numel(), "draft_tokens")
    if mode == 3 and parent is not None:
        if parent.numel() > R:
            raise ValueError("parent has more nodes than logits has rows")
        n_tokens = min(n_tokens, parent.numel())
    return _Rows(mode, B, R, _ptr(offsets, "offsets", i32, dev), _ptr(parent, "parent", i32, dev),
                 _ptr(draft_tokens, "draft_tokens", i32, dev), n_tokens)


def _out_arg(logits, out, stream):
    if out is None:
        out = _new(logits.shape, logits.dtype, logits.device, stream)
        return out, out.data_ptr()
    return out, _ptr(out, "out", logits.dtype, logits.get_device(), logits.numel())


def _logits_arg(logits, rw, rows, draft_tokens, parent, repetition, frequency, presence, counts, seen, slots,
                bias_offsets, bias_tokens, bias_values, mask, mask_rows, i32, f32):
    dev, V, B, R = logits.get_device(), logits.shape[1], rw.B, rw.R
    W = (V + 31) // 32
    pen, bias, masks = (None, None, None, None, None, None, 0), (None, None, None, 0), (None, None, 0)
    if counts is not None:
        if seen is None or draft_tokens is None:
            raise ValueError("penalties need counts, seen and draft_tokens")
        if rows == "tree" and parent is None:
            raise ValueError("penalties on a tree need parent")
        S = _size(counts.shape[0], "counts")
        pen = (_ptr(repetition, "repetition", f32, dev, B), _ptr(frequency, "frequency", f32, dev, B),
               _ptr(presence, "presence", f32, dev, B), _ptr(counts, "counts", i32, dev, S * V),
               _ptr(seen, "seen", i32, dev, S * 2 * W), _ptr(slots, "slots", i32, dev, B), S)
    elif not (repetition is None and frequency is None and presence is None and seen is None and slots is None):
        raise ValueError("penalties need counts, seen and draft_tokens")
    if bias_offsets is not None:
        if bias_tokens is None or bias_values is None:
            raise ValueError("biases need bias_offsets, bias_tokens and bias_values")
        n = _size(bias_tokens.numel(), "bias_tokens")
        bias = (_ptr(bias_offsets, "bias_offsets", i32, dev, B + 1), _ptr(bias_tokens, "bias_tokens", i32, dev),
                _ptr(bias_values, "bias_values", f32, dev, n), n)
    elif not (bias_tokens is None and bias_values is None):
        raise ValueError("biases need bias_offsets, bias_tokens and bias_values")
    if mask is not None:
        M = _size(mask.shape[0], "mask")
        if mask_rows is None and M < R:
            raise ValueError("mask needs a row for each row of logits, or mask_rows")
        pm, pr = _ptr(mask, "mask", i32, dev, M * W), _ptr(mask_rows, "mask_rows", i32, dev, R)
        masks = pm or pr, pr, M  # (no mask to name: an address that is not read)
    elif mask_rows is not None:
        raise ValueError("mask_rows without mask")
    return _Logits(*pen, *bias, *masks)


def _truncate_arg(dev, B, temperature, top_k, top_p, min_p, i32, f32):
    return _Truncate(_ptr(temperature, "temperature", f32, dev, B), _ptr(top_k, "top_k", i32, dev, B),
                     _ptr(top_p, "top_p", f32, dev, B), _ptr(min_p, "min_p", f32, dev, B))


def spec_logits_process(logits, offsets, draft_tokens=None, *, rows="target", parent=None, repetition=None,
                        frequency=None, presence=None, counts=None, seen=None, slots=None, bias_offsets=None,
                        bias_tokens=None, bias_values=None, mask=None, mask_rows=None, out=None, stream=None):
    """Penalties for repeated tokens, biases and grammar masks on packed logit
    rows [R, V] (device tensors).  rows: "target" or "draft" (offsets =
    k_offsets), "next" (one row per sequence, after all its drafted tokens)
    or "tree" (offsets = node_offsets).  counts [S, V] and seen [S, 2, W] are
    a PenaltyState's; biases are a ragged list per sequence; mask [M, W] holds
    a bit per token (set: allowed) and mask_rows [R] the mask of each row (-1:
    none).  out: the result's buffer, logits itself for in place; else a new
    one, whose rows behind the last sequence's are not written.  Returns out."""
    import torch
    i32, f32 = torch.int32, torch.float32
    rw = _rows_arg(logits, offsets, rows, draft_tokens, parent, i32)
    dt = _dtype_code(logits)
    ps = _logits_arg(logits, rw, rows, draft_tokens, parent, repetition, frequency, presence, counts, seen, slots,
                     bias_offsets, bias_tokens, bias_values, mask, mask_rows, i32, f32)
    out, po = _out_arg(logits, out, stream)
    _launch(logits.get_device(), stream, lib().spec_logits_process, "spec_logits_process", logits.data_ptr(),
            ctypes.byref(rw), ctypes.byref(ps), logits.shape[1], dt, po)
    return out


def spec_logits_truncate(logits, temperature, offsets, *, rows="target", top_k=None, top_p=None, min_p=None,
                         out=None, stream=None):
    """Top-k, top-p and min-p on packed logit rows [R, V] (device tensors, a
    setting per sequence): tokens outside the kept set become -inf, ties go
    to the lowest index.  rows, out: as in spec_logits_process.  Greedy
    sequences' rows (temperature 0) stay as they are.  Returns out."""
    import torch
    rw = _rows_arg(logits, offsets, rows, None, None, torch.int32)
    dt = _dtype_code(logits)
    tr = _truncate_arg(logits.get_device(), rw.B, temperature, top_k, top_p, min_p, torch.int32, torch.float32)
    out, po = _out_arg(logits, out, stream)
    _launch(logits.get_device(), stream, lib().spec_logits_truncate, "spec_logits_truncate", logits.data_ptr(),
            ctypes.byref(rw), ctypes.byref(tr), logits.shape[1], dt, po)
    return out


def spec_logits_process_truncate(logits, temperature, offsets, draft_tokens=None, *, rows="target", parent=None,
                                 repetition=None, frequency=None, presence=None, counts=None, seen=None, slots=None,
                                 bias_offsets=None, bias_tokens=None, bias_values=None, mask=None, mask_rows=None,
                                 top_k=None, top_p=None, min_p=None, out=None, stream=None):
    """spec_logits_process, then spec_logits_truncate on its result, in one
    call (the same outputs, bit for bit).  Returns out."""
    import torch
    i32, f32 = torch.int32, torch.float32
    rw = _rows_arg(logits, offsets, rows, draft_tokens, parent, i32)
    dt = _dtype_code(logits)
    ps = _logits_arg(logits, rw, rows, draft_tokens, parent, repetition, frequency, presence, counts, seen, slots,
                     bias_offsets, bias_tokens, bias_values, mask, mask_rows, i32, f32)
    tr = _truncate_arg(logits.get_device(), rw.B, temperature, top_k, top_p, min_p, i32, f32)
    out, po = _out_arg(logits, out, stream)
    _launch(logits.get_device(), stream, lib().spec_logits_process_truncate, "spec_logits_process_truncate",
            logits.data_ptr(), ctypes.byref(rw), ctypes.byref(ps), ctypes.byref(tr), logits.shape[1], dt, po)
    return out


def _state_arg(counts, seen, i32):
    if counts.dim() != 2:
        raise ValueError("counts must be [S, V]")
    S, V = _size(counts.shape[0], "counts"), _size(counts.shape[1], "a row")
    if not counts.is_cuda:
        _check_dev("counts", counts)
    dev = counts.get_device()
    return S, V, dev, _ptr(counts, "counts", i32, dev), _ptr(seen, "seen", i32, dev, S * 2 * ((V + 31) // 32))


def spec_penalty_reset(counts, seen, slots, prompt_offsets=None, prompt_tokens=None, output_offsets=None,
                       output_tokens=None, stream=None):
    """New sequences in the given slots of a penalty state: their counts are
    cleared, their prompts' tokens (a ragged list) marked, and tokens they
    have emitted already counted.  Returns (counts, seen)."""
    import torch
    i32 = torch.int32
    S, V, dev, pc, ps = _state_arg(counts, seen, i32)
    n = _size(slots.numel(), "slots")
    if (prompt_offsets is None) != (prompt_tokens is None) or (output_offsets is None) != (output_tokens is None):
        raise ValueError("offsets and tokens go together")
    _launch(dev, stream, lib().spec_penalty_reset, "spec_penalty_reset", pc, ps, S, V, _ptr(slots, "slots", i32, dev), n,
            _ptr(prompt_offsets, "prompt_offsets", i32, dev, n + 1), _ptr(prompt_tokens, "prompt_tokens", i32, dev),
            0 if prompt_tokens is None else _size(prompt_tokens.numel(), "prompt_tokens"),
            _ptr(output_offsets, "output_offsets", i32, dev, n + 1), _ptr(output_tokens, "output_tokens", i32, dev),
            0 if output_tokens is None else _size(output_tokens.numel(), "output_tokens"))
    return counts, seen


def spec_penalty_update(counts, seen, out_tokens, out_num_accepted, offsets, *, rows="target", slots=None,
                        stream=None):
    """Counts the tokens that a verify emitted (its out_tokens and
    out_num_accepted, with its k_offsets, or node_offsets for rows="tree") in
    the sequences' slots.  Returns (counts, seen)."""
    import torch
    i32 = torch.int32
    S, V, dev, pc, ps = _state_arg(counts, seen, i32)
    if rows not in ("target", "tree"):
        raise ValueError(f"rows must be 'target' or 'tree', got {rows!r}")
    B = _size(offsets.numel() - 1, "offsets")
    if B < 0:
        raise ValueError("offsets must have B + 1 entries")
    rw = _Rows(ROWS[rows], B, _size(out_tokens.numel(), "out_tokens"), _ptr(offsets, "offsets", i32, dev), None, None, 0)
    _launch(dev, stream, lib().spec_penalty_update, "spec_penalty_update", pc, ps, S, V,
            _ptr(slots, "slots", i32, dev, B), ctypes.byref(rw), _ptr(out_tokens, "out_tokens", i32, dev),
            _ptr(out_num_accepted, "out_num_accepted", i32, dev, B))
    return counts, seen


class PenaltyState:
    """What S slots of a running batch have emitted and been prompted with:
    counts [S, V] and the bit arrays seen [S, 2, W] that spec_logits_process
    reads.  Starts empty."""

    def __init__(self, S: int, V: int, device="cuda"):
        import torch
        if S <= 0 or not 0 < V <= MAX_V:
            raise ValueError(f"invalid penalty state S={S}, V={V}")
        self.counts = torch.zeros((S, V), dtype=torch.int32, device=device)
        self.seen = torch.zeros((S, 2, (V + 31) // 32), dtype=torch.int32, device=device)

    def reset(self, slots, prompt_offsets=None, prompt_tokens=None, output_offsets=None, output_tokens=None,
              stream=None):
        """spec_penalty_reset on this state."""
        spec_penalty_reset(self.counts, self.seen, slots, prompt_offsets, prompt_tokens, output_offsets,
                           output_tokens, stream)

    def update(self, out_tokens, out_num_accepted, offsets, *, rows="target", slots=None, stream=None):
        """spec_penalty_update on this state."""
        spec_penalty_update(self.counts, self.seen, out_tokens, out_num_accepted, offsets, rows=rows, slots=slots,
                            stream=stream)

    def reorder(self, rows, offsets, *, slots=None, stream=None):
        """spec_state_reorder on this state: the counts and prompts follow the
        hypotheses that a beam kept."""
        spec_state_reorder([self.counts, self.seen], rows, offsets, slots=slots, stream=stream)


# --------------------------------------------------- beams, states, the cache
@functools.lru_cache(maxsize=256)
def beam_workspace_bytes(R: int, V: int, dtype: int) -> int:
    return int(lib().spec_beam_workspace_bytes(R, V, dtype))


def spec_beam_select(logits, scores, offsets, n, *, ended=None, end_token=0, lse=False, workspace=None, stream=None):
    """The n best continuations of each group of hypotheses: logits [R, V] and
    scores [R] (float32) hold a row per hypothesis, offsets [B+1] says which
    rows a group has; ended [R] (bool): hypotheses that have ended go on with
    end_token and their score.  Returns (scores [B, n] float32, tokens [B, n]
    int32, rows [B, n] int32: the row each comes from), best first, -inf and
    -1 where there are fewer, and with lse=True each row's log-sum-exp [R] (of
    rows behind the last group's nothing is written: fresh memory, of any contents).
    Invalid offsets make everything NaN and -1."""
    import torch
    i32, f32 = torch.int32, torch.float32
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, V]")
    if not logits.is_cuda or not logits.is_contiguous():
        _check_dev("logits", logits)
    dt, dev, device = _dtype_code(logits), logits.get_device(), logits.device
    R, V = logits.shape
    B = _size(offsets.numel() - 1, "offsets")
    _size(R, "logits"), _size(V, "a row")
    if B < 0:
        raise ValueError("offsets must have B + 1 entries")
    if not 1 <= n <= MAX_CANDIDATES:
        raise ValueError(f"n must be 1 to {MAX_CANDIDATES}, got {n}")
    truth = torch.bool if ended is not None and ended.dtype is torch.bool else torch.uint8
    ps, pe, po = _ptr(scores, "scores", f32, dev, R), _ptr(ended, "ended", truth, dev, R), _ptr(offsets, "offsets", i32, dev)
    if workspace is None:
        workspace = _new(max(256, beam_workspace_bytes(R, V, dt)), torch.uint8, device, stream)
        pw = workspace.data_ptr()
    else:
        pw = _ptr(workspace, "workspace", torch.uint8, dev)
    if stream is None:
        out_scores, out_tokens = torch.empty((B, n), dtype=f32, device=device), torch.empty((B, n), dtype=i32, device=device)
        out_rows, out_lse = torch.empty_like(out_tokens), torch.empty(R, dtype=f32, device=device) if lse else None
    else:
        out_scores, out_tokens, out_rows = (_new((B, n), d, device, stream) for d in (f32, i32, i32))
        out_lse = _new(R, f32, device, stream) if lse else None
    _launch(dev, stream, lib().spec_beam_select, "spec_beam_select", logits.data_ptr(), ps, pe, end_token, po, B, R, V, dt,
            n, out_scores.data_ptr(), out_tokens.data_ptr(), out_rows.data_ptr(), out_lse.data_ptr() if lse else None, pw,
            workspace.numel())
    return (out_scores, out_tokens, out_rows, out_lse) if lse else (out_scores, out_tokens, out_rows)


def _state_of(x, S, dev):
    """A tensor with the slots first, or (tensor, slot dimension, position dimension or None), as a _State's fields."""
    t, at, pos = x if isinstance(x, (tuple, list)) else (x, 0, None)
    if not t.is_cuda or not t.is_contiguous():
        _check_dev("a state", t)
    if t.get_device() != dev:
        raise ValueError(f"a state is on {t.device}, the call's other tensors on cuda:{dev}")
    shape = tuple(t.shape)
    if not 0 <= at < len(shape) or (pos is not None and not at < pos < len(shape)):
        raise ValueError("a state is (tensor, slot dimension, position dimension behind it or None)")
    if shape[at] != S:
        raise ValueError(f"a state has {shape[at]} slots, another {S}")
    planes = math.prod(shape[:at])
    if pos is None:  # one position: everything a slot holds
        return t.data_ptr(), planes, 1, 1, math.prod(shape[at + 1:]) * t.element_size()
    return (t.data_ptr(), planes, math.prod(shape[at + 1:pos]), shape[pos],
            math.prod(shape[pos + 1:]) * t.element_size())


def spec_state_reorder(states, rows, offsets, *, slots=None, lengths=None, stream=None):
    """The states of the hypotheses put in the order of what a beam kept, in
    place: slot slots[i] (None: i) of every state gets what slot
    slots[rows[i]] held, for the entries i of each group (offsets [B+1]);
    rows[i] is -1 or an entry of the same group.  A state is a tensor with the
    slots first, or (tensor, slot dimension, position dimension or None); of a state
    with positions the first lengths[slot] (int32 [S], by source) are moved,
    without lengths all.  Lengths go with the slots of all states; a state without
    positions moves as one whole where its source's length is not 0.  Returns states.
    (state_reorder_status: whether a device-side wait has run out.)"""
    import torch
    i32 = torch.int32
    R, B = _size(rows.numel(), "rows"), _size(offsets.numel() - 1, "offsets")
    if B < 0:
        raise ValueError("offsets must have B + 1 entries")
    if not rows.is_cuda:
        _check_dev("rows", rows)
    dev = rows.get_device()
    args = (_ptr(rows, "rows", i32, dev), _ptr(offsets, "offsets", i32, dev), B, R, _ptr(slots, "slots", i32, dev, R))
    if not states:
        return states
    first = states[0]
    S = _size(first.shape[0] if not isinstance(first, (tuple, list)) else first[0].shape[first[1]], "a state")
    pl = _ptr(lengths, "lengths", i32, dev, S)
    made = array.array("q")  # five fields of 64 bits each, as in _State
    for x in states:
        made.extend(_state_of(x, S, dev))
    if len(states) > MAX_STATES:  # each launch looks at its own states only
        parts = sorted((made[i], made[i] + S * math.prod(made[i + 1:i + 5])) for i in range(0, len(made), 5) if math.prod(made[i + 1:i + 5]))
        if any(b[0] < a[1] for a, b in zip(parts, parts[1:])):
            raise ValueError("no two states may overlap")
    start, size = made.buffer_info()[0], ctypes.sizeof(_State)
    for at in range(0, len(states), MAX_STATES):
        _launch(dev, stream, lib().spec_state_reorder, "spec_state_reorder", start + at * size,
                min(len(states) - at, MAX_STATES), S, *args, pl)
    return states


def state_reorder_status(clear: bool = False) -> int:
    """SPEC_OK, or SPEC_ERR_TIMEOUT if a spec_state_reorder call's wait has run out on the current device (its
    states are then no longer to be used).  Waits for the device."""
    v = ctypes.c_int(0)
    _raise(lib().spec_state_reorder_status(ctypes.byref(v), 1 if clear else 0), "spec_state_reorder_status")
    return v.value


def selfcheck_reorder_timeout(state, rows, offsets, stream=None):
    """spec_state_reorder of one tensor with waits that give up (2 to 6 s);
    afterwards state_reorder_status() is SPEC_ERR_TIMEOUT."""
    import torch
    dev, i32 = state.get_device(), torch.int32
    S = state.shape[0]
    made = _State(*_state_of(state, S, dev))
    _launch(dev, stream, lib().spec_selfcheck_reorder_timeout, "spec_selfcheck_reorder_timeout", ctypes.byref(made), 1, S,
            _ptr(rows, "rows", i32, dev), _ptr(offsets, "offsets", i32, dev), offsets.numel() - 1, rows.numel(), None, None)


def _cache_arg(k, k_scale, v, v_scale, lengths, pages):
    import torch
    if k.dim() != 5:
        raise ValueError("k must be [L, P, T, H, D]")
    if not k.is_cuda:
        _check_dev("k", k)
    dev, i32 = k.get_device(), torch.int32
    L, P, T, H, D = shape = tuple(k.shape)
    if (v is None) != (v_scale is None):
        raise ValueError("v and v_scale go together")
    scales = L * P * T * H * ((D + 31) // 32)
    if pages is None:
        S, M = P, 1
    else:
        if pages.dim() != 2:
            raise ValueError("pages must be [S, M]")
        S, M = pages.shape
    if max(*shape, S, M) > 0x7fffffff:
        raise ValueError(f"k {shape} and pages [{S}, {M}] must have dimensions below 2147483648")
    f8, u8 = torch.float8_e4m3fn, torch.uint8
    return dev, _Cache(_ptr(k, "k", f8, dev), _ptr(k_scale, "k_scale", u8, dev, scales), _ptr(v, "v", f8, dev, k.numel()),
                       _ptr(v_scale, "v_scale", u8, dev, scales), L, P, T, H, D, _ptr(pages, "pages", i32, dev), S, M,
                       _ptr(lengths, "lengths", i32, dev, S))


def _lines_of(t, name, dev, L, H, D):
    """(rows, elements from one layer to the next, from one row to the next) of keys or values [L, R, H, D] or [R, H, D]."""
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be on the cache's device")
    shape, strides = tuple(t.shape), t.stride()
    if len(shape) == 3 and L == 1:
        shape, strides = (1, *shape), (0, *strides)
    if len(shape) != 4 or shape[0] != L or shape[2] != H or shape[3] != D:
        raise ValueError(f"{name} must be [{L}, R, {H}, {D}], got {tuple(t.shape)}")
    R = shape[1]
    if R and L and (strides[3] != 1 or (H > 1 and strides[2] != D)):
        raise ValueError(f"{name} must be contiguous in heads and elements")
    return R, strides[0] if L > 1 else 0, strides[1] if R > 1 else H * D


def spec_cache_write(k, k_scale, v, v_scale, lengths, keys, values, offsets=None, *, rows="target", num_accepted=None,
                     parent=None, last_node=None, slots=None, pages=None, out_lengths=None, stream=None):
    """Writes the rows that a round kept into an 8-bit cache: k, v e4m3
    [L, P, T, H, D] with a scale's byte per 32 elements of a head (k_scale,
    v_scale uint8), lengths [S] the positions held, pages [S, M] or None (slot s
    is page s).  keys, values [L, R, H, D], or [R, H, D] for L = 1; strided in
    layers and rows.  rows: "target" (a verify's rows with its k_offsets and
    num_accepted: the first num_accepted + 1 of each sequence), "tree"
    (node_offsets, parent, num_accepted, last_node: the accepted path), "next"
    (a row per sequence) or "prompt" (offsets of any lengths: all).  out_lengths: the lengths after it
    (lengths for in place), None: not written.  v, v_scale, values None: a
    cache of one tensor.  Returns out_lengths."""
    import torch
    i32 = torch.int32
    dev, cache = _cache_arg(k, k_scale, v, v_scale, lengths, pages)
    mode = CACHE_ROWS.get(rows)
    if mode is None:
        raise ValueError(f"rows must be one of {sorted(CACHE_ROWS)}, got {rows!r}")
    if (values is None) != (v is None):
        raise ValueError("values and v go together")
    L, H, D = cache.L, cache.H, cache.D
    R, layer, row = layout = _lines_of(keys, "keys", dev, L, H, D)
    if values is not None and (_lines_of(values, "values", dev, L, H, D) != layout or values.dtype is not keys.dtype):
        raise ValueError("keys and values must have one type and one layout")
    dt = _dtype_code(keys)
    if mode == 2:
        if slots is None:
            raise ValueError("rows 'next' need slots: one per sequence")
        B = _size(slots.numel(), "slots")
        if B > R:
            raise ValueError("keys have fewer rows than there are sequences")
    else:
        if offsets is None:
            raise ValueError("offsets must have B + 1 entries")
        B = _size(offsets.numel() - 1, "offsets")
    if B < 0:
        raise ValueError("offsets must have B + 1 entries")
    if (mode in (0, 3)) != (num_accepted is not None) or (mode == 3) != (last_node is not None and parent is not None):
        raise ValueError("num_accepted goes with rows 'target' and 'tree', parent and last_node with 'tree'")
    if parent is not None and parent.numel() < R:
        raise ValueError("parent must have an entry for each row")
    rw = _Rows(mode, B, _size(R, "keys"), _ptr(offsets, "offsets", i32, dev), _ptr(parent, "parent", i32, dev), None, 0)
    _launch(dev, stream, lib().spec_cache_write, "spec_cache_write", ctypes.byref(cache), keys.data_ptr(),
            None if values is None else values.data_ptr(), layer, row, dt,
            ctypes.byref(rw), _ptr(num_accepted, "num_accepted", i32, dev, B), _ptr(last_node, "last_node", i32, dev, B),
            _ptr(slots, "slots", i32, dev, B), _ptr(out_lengths, "out_lengths", i32, dev, cache.S))
    return out_lengths


def spec_cache_read(k, k_scale, v, v_scale, lengths, offsets, R, *, first=None, slots=None, pages=None, dtype=None,
                    out=None, stream=None):
    """Positions of an 8-bit cache (as in spec_cache_write) read back: row
    offsets[b] + i of the outputs gets position first[b] + i (first None: 0) of
    sequence b's slot, NaN where it holds none.  R: rows of the outputs, at least
    offsets[B].  dtype: bfloat16 (None) or float32.  Returns (keys, values)
    [L, R, H, D], values None for a cache of one tensor; out: the two to write to.
    Rows behind offsets[B] are not written, and no row is if the offsets are
    invalid: they are as `out` had them, without `out` fresh memory of any contents."""
    import torch
    i32 = torch.int32
    dev, cache = _cache_arg(k, k_scale, v, v_scale, lengths, pages)
    B = _size(offsets.numel() - 1, "offsets")
    if B < 0:
        raise ValueError("offsets must have B + 1 entries")
    R = _size(R, "the output")
    shape = (cache.L, R, cache.H, cache.D)
    if out is None:
        kind = torch.bfloat16 if dtype is None else dtype
        out_k = _new(shape, kind, k.device, stream)
        out = out_k, None if v is None else torch.empty_like(out_k) if stream is None else _new(shape, kind, k.device, stream)
    dt = _dtype_code(out[0])
    if (out[1] is None) != (v is None) or (dtype is not None and out[0].dtype != dtype):
        raise ValueError("out must be (keys, values) of the type asked for, values None if there is no v")
    size = cache.L * R * cache.H * cache.D
    _launch(dev, stream, lib().spec_cache_read, "spec_cache_read", ctypes.byref(cache),
            _ptr(offsets, "offsets", i32, dev), B, R, _ptr(first, "first", i32, dev, B), _ptr(slots, "slots", i32, dev, B), dt,
            _ptr(out[0], "out", out[0].dtype, dev, size), _ptr(out[1], "out", out[0].dtype, dev, size))
    return out


class CacheState:
    """An 8-bit cache of keys and values for S slots (spec_cache_write's
    layout): T positions per slot, or, with pages, `pages` pages of T
    positions that the caller gives out through page_table [S, M] (-1:
    none).  Starts empty."""

    def __init__(self, L: int, S: int, T: int, H: int, D: int, *, pages=None, max_pages=None, values: bool = True,
                 device="cuda"):
        import torch
        if min(L, S, T, H) <= 0 or D <= 0 or D % 16 or D > 1024 or H * D > 65536 or L * (1 + values) * H * ((D + 31) // 32) >= 1 << 23:
            raise ValueError(f"invalid cache L={L}, S={S}, T={T}, H={H}, D={D}")
        if (pages is None) != (max_pages is None):
            raise ValueError("pages and max_pages go together")
        P = S if pages is None else pages
        shape, scales = (L, P, T, H, D), (L, P, T, H, (D + 31) // 32)
        self.k = torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        self.k_scale = torch.zeros(scales, dtype=torch.uint8, device=device)
        self.v = torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) if values else None
        self.v_scale = torch.zeros(scales, dtype=torch.uint8, device=device) if values else None
        self.lengths = torch.zeros(S, dtype=torch.int32, device=device)
        self.page_table = None if pages is None else torch.full((S, max_pages), -1, dtype=torch.int32, device=device)

    def write(self, keys, values, offsets=None, *, rows="target", num_accepted=None, parent=None, last_node=None,
              slots=None, stream=None):
        """spec_cache_write of all layers; the lengths grow in place."""
        spec_cache_write(self.k, self.k_scale, self.v, self.v_scale, self.lengths, keys, values, offsets, rows=rows,
                         num_accepted=num_accepted, parent=parent, last_node=last_node, slots=slots,
                         pages=self.page_table, out_lengths=self.lengths, stream=stream)

    def read(self, offsets, R, *, first=None, slots=None, dtype=None, out=None, stream=None):
        """spec_cache_read (rows behind offsets[B], all if the offsets are invalid, are not written)."""
        return spec_cache_read(self.k, self.k_scale, self.v, self.v_scale, self.lengths, offsets, R, first=first,
                               slots=slots, pages=self.page_table, dtype=dtype, out=out, stream=stream)

    def reorder(self, rows, offsets, *, slots=None, stream=None):
        """spec_state_reorder of the held positions and of the lengths (a cache
        without pages; with pages it is the caller that gives them out)."""
        if self.page_table is not None:
            raise ValueError("a cache with pages is reordered through its page table")
        states = [(t, 1, 2) for t in (self.k, self.k_scale, self.v, self.v_scale) if t is not None]
        spec_state_reorder(states, rows, offsets, slots=slots, lengths=self.lengths, stream=stream)
        spec_state_reorder([self.lengths], rows, offsets, slots=slots, stream=stream)
