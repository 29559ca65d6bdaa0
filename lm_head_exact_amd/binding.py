"""ctypes binding of libflashsample (C ABI in include/flashsample.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, outputs and workspaces are allocated with torch, and the call
goes to the library on torch's current HIP stream.  Every step of the
sampler runs in the library's kernels.  If the library is missing or fails
to load, every function raises; there is no fallback path.
"""
import bisect
import ctypes
import math
import os
import re
from typing import Optional, Tuple

import torch  # loaded first, so the library binds to the same HIP runtime

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libflashsample.so")
_HEADER = os.path.join(os.path.dirname(_HERE), "include", "flashsample.h")

FS_OK, FS_ERR_INVALID_ARG, FS_ERR_UNSUPPORTED, FS_ERR_WORKSPACE, FS_ERR_HIP = range(5)


class FlashSampleError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_status_name(status)}: {message}")
        self.status = status


_lib = None


def library_path() -> str:
    return _LIB_PATH


def exported_names_from_header():
    """Names of every function the public header declares."""
    text = open(_HEADER).read()
    return sorted(set(re.findall(r"FS_API\s+[\w\s\*]+?\b(fs_\w+)\s*\(", text)))


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise FlashSampleError(FS_ERR_UNSUPPORTED,
                               f"{_LIB_PATH} is missing: run lm_head_exact_amd/build.py")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i32, u32, i64, u64, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32,
                                  ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t)
    f64 = ctypes.c_double
    sample_args = [vp, vp, i32, i32, i32, i32, vp, u64, u64, vp, vp, vp, sz, vp]
    for name, args, res in [
        ("fs_workspace_bytes", [i32, i32, i32], sz),
        ("fs_unfused_workspace_bytes", [i32, i32, i32], sz),
        ("fs_sample", sample_args, ctypes.c_int),
        ("fs_sample_partial", sample_args, ctypes.c_int),
        ("fs_sample_unfused", sample_args, ctypes.c_int),
        ("fs_merge", [vp, vp, i32, i32, vp, vp, vp], ctypes.c_int),
        ("fs_sample_partial_lse", [vp, vp, i32, i32, i32, i32, vp, u64, u64, vp, vp, vp, vp,
                                   sz, vp], ctypes.c_int),
        ("fs_sample_partial_lse_packed", [vp, vp, i32, i32, i32, i32, vp, u64, u64, vp, vp, vp,
                                          vp, sz, vp], ctypes.c_int),
        ("fs_merge_lse", [vp, vp, vp, i32, i32, vp, u64, u64, vp, vp, vp, vp], ctypes.c_int),
        ("fs_groups_workspace_bytes", [i32, i32, i32, i32], sz),
        ("fs_sample_groups_lse", [vp, vp, i32, i32, i32, i32, vp, u64, u64, vp, i32, vp, vp, vp,
                                  vp, sz, vp], ctypes.c_int),
        ("fs_sample_groups_lse_packed", [vp, vp, i32, i32, i32, i32, vp, u64, u64, vp, i32, vp,
                                         vp, vp, vp, sz, vp], ctypes.c_int),
        ("fs_packed_weights_bytes", [i32, i32, i32], sz),
        ("fs_pack_weights", [vp, i32, i32, i32, vp, sz, vp], ctypes.c_int),
        ("fs_sample_packed", sample_args, ctypes.c_int),
        ("fs_sample_packed_noalloc", [vp, vp, i32, i32, i32, i32, vp, u64, u64, vp, vp, vp],
         ctypes.c_int),
        ("fs_online_bounds_workspace_bytes", [i32, i32], sz),
        ("fs_online_workspace_bytes", [i32, i32, i32, i32], sz),
        ("fs_online_bounds", [vp, i32, i32, vp, i32, vp, vp, sz, vp], ctypes.c_int),
        ("fs_online_bounds_packed", [vp, i32, i32, i32, vp, i32, vp, vp, sz, vp], ctypes.c_int),
        ("fs_sample_online", [vp, vp, i32, i32, i32, i32, vp, u64, u64, vp, i32, vp, vp, vp,
                              vp, vp, sz, vp], ctypes.c_int),
        ("fs_sample_online_packed", [vp, vp, i32, i32, i32, i32, vp, u64, u64, vp, i32, vp, vp,
                                     vp, vp, vp, sz, vp], ctypes.c_int),
        ("fs_token_logprobs_workspace_bytes", [i32, i32, i32], sz),
        ("fs_token_logprobs", [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp],
         ctypes.c_int),
        ("fs_token_logprobs_packed", [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp],
         ctypes.c_int),
        ("fs_token_logprobs_backward_workspace_bytes", [i32, i32, i32], sz),
        ("fs_token_logprobs_backward", [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                        sz, vp], ctypes.c_int),
        ("fs_fp8_weights_bytes", [i32, i32, i32], sz),
        ("fs_quantize_weights_fp8", [vp, i32, i32, i32, vp, sz, vp, vp], ctypes.c_int),
        ("fs_pack_weights_fp8", [vp, i32, i32, vp, sz, vp], ctypes.c_int),
        ("fs_fp8_workspace_bytes", [i32, i32, i32], sz),
        ("fs_logits_fp8", [vp, vp, vp, i32, i32, i32, i32, vp, i64, vp, sz, vp], ctypes.c_int),
        ("fs_token_logprobs_fp8", [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp],
         ctypes.c_int),
        ("fs_sample_fp8", [vp, vp, vp, i32, i32, i32, i32, vp, u64, u64, vp, vp, vp, sz, vp],
         ctypes.c_int),
        ("fs_cross_entropy_workspace_bytes", [i32, i32, i32, i32], sz),
        ("fs_cross_entropy", [vp, vp, i32, i32, i32, vp, f64, f64, i32, f64, vp, vp, vp, vp, vp, sz,
                              vp], ctypes.c_int),
        ("fs_loss_workspace_bytes", [i32, i32], sz),
        ("fs_policy_loss", [vp, vp, vp, vp, vp, vp, i32, i32, i32, f64, f64, f64, f64, ctypes.c_int,
                            ctypes.c_int, f64, i32, vp, vp, vp, sz, vp], ctypes.c_int),
        ("fs_preference_loss", [vp, vp, vp, vp, i32, i32, ctypes.c_int, f64, f64, f64, i32, f64, i32,
                                vp, vp, vp, vp, sz, vp], ctypes.c_int),
        ("fs_clip_grad_norm_workspace_bytes", [vp, i32], sz),
        ("fs_clip_grad_norm", [vp, vp, vp, vp, i32, ctypes.c_float, vp, vp, sz, vp], ctypes.c_int),
        ("fs_debug_noise", [u64, u64, u32, u32, i64, vp, vp, vp], ctypes.c_int),
        ("fs_debug_gumbel", [vp, i64, vp, vp], ctypes.c_int),
        ("fs_device_info", [i32, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)],
         ctypes.c_int),
        ("fs_num_configs", [], i32),
        ("fs_config_name", [i32], ctypes.c_char_p),
        ("fs_force_config", [i32], ctypes.c_int),
        ("fs_selected_config", [i32, i32, i32], i32),
        ("fs_selected_config_packed", [i32, i32, i32], i32),
        ("fs_selected_config_groups", [i32, i32, i32, i32], i32),
        ("fs_profile_enable", [i32], ctypes.c_int),
        ("fs_profile_read", [ctypes.POINTER(ctypes.c_int32)] + [ctypes.POINTER(ctypes.c_double)] * 3,
         ctypes.c_int),
        ("fs_status_string", [ctypes.c_int], ctypes.c_char_p),
        ("fs_last_error", [], ctypes.c_char_p),
    ]:
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _status_name(s: int) -> str:
    try:
        return lib().fs_status_string(s).decode()
    except Exception:
        return f"status {s}"


def _check(status: int):
    if status != FS_OK:
        raise FlashSampleError(status, lib().fs_last_error().decode())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _req(t: torch.Tensor, name: str, dtype, ndim: int):
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.dim() == ndim
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def workspace_bytes(B: int, D: int, V: int) -> int:
    return int(lib().fs_workspace_bytes(B, D, V))


def unfused_workspace_bytes(B: int, D: int, V: int) -> int:
    return int(lib().fs_unfused_workspace_bytes(B, D, V))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    # torch's caching allocator returns 256-byte (or better) aligned blocks
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _sample_common(fn_name, h, W, temperature, seed, step, vocab_offset, out_a, out_b,
                   workspace, ws_fn):
    _req(h, "h", torch.bfloat16, 2)
    _req(W, "W", torch.bfloat16, 2)
    _req(temperature, "temperature", torch.float32, 1)
    B, D = h.shape
    V, D2 = W.shape
    if D2 != D:
        raise ValueError(f"h is B x {D} but W is V x {D2}")
    if temperature.shape[0] != B:
        raise ValueError("temperature must have B entries")
    if not (h.device == W.device == temperature.device == out_a.device == out_b.device):
        raise ValueError("all tensors must be on one device")
    if workspace is None:
        workspace = alloc_workspace(ws_fn(B, D, V), h.device)
    fn = getattr(lib(), fn_name)
    _check(fn(_ptr(h), _ptr(W), B, D, V, int(vocab_offset), _ptr(temperature),
              int(seed) & (2**64 - 1), int(step) & (2**64 - 1), _ptr(out_a), _ptr(out_b),
              _ptr(workspace), workspace.numel() * workspace.element_size(),
              _stream(h.device)))


def sample(h: torch.Tensor, W: torch.Tensor, temperature: torch.Tensor, seed: int, step: int,
           vocab_offset: int = 0, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
           workspace: Optional[torch.Tensor] = None):
    """Fused LM-head + Gumbel-Max sampling: returns (ids int32[B], maxval fp32[B])."""
    B = h.shape[0]
    if out is None:
        out = (torch.empty(B, dtype=torch.int32, device=h.device),
               torch.empty(B, dtype=torch.float32, device=h.device))
    ids, val = out
    _sample_common("fs_sample", h, W, temperature, seed, step, vocab_offset, ids, val,
                   workspace, workspace_bytes)
    return ids, val


def sample_partial(h, W, temperature, seed, step, vocab_offset, partial_val, partial_idx,
                   workspace=None):
    """One shard's per-row (max, global argmax) into partial_val / partial_idx (B each)."""
    _req(partial_val, "partial_val", torch.float32, 1)
    _req(partial_idx, "partial_idx", torch.int32, 1)
    _sample_common("fs_sample_partial", h, W, temperature, seed, step, vocab_offset,
                   partial_val, partial_idx, workspace, workspace_bytes)
    return partial_val, partial_idx


def sample_partial_lse(h, W, temperature, seed, step, vocab_offset, partial_val, partial_idx,
                       partial_lse, workspace=None, V=None):
    """One vocabulary group's per-row (max, global argmax) and log-sum-exp of the
    scaled logits into partial_val / partial_idx / partial_lse (B each).  W is the
    group's row-major V x D rows, or (1-D, with V given) their fragment-order
    copy from pack_weights at the same vocab_offset."""
    _req(partial_val, "partial_val", torch.float32, 1)
    _req(partial_idx, "partial_idx", torch.int32, 1)
    _req(partial_lse, "partial_lse", torch.float32, 1)
    _req(h, "h", torch.bfloat16, 2)
    packed = W.dim() == 1
    _req(W, "W", torch.bfloat16, 1 if packed else 2)
    _req(temperature, "temperature", torch.float32, 1)
    B, D = h.shape
    if packed:
        if V is None:
            raise ValueError("V is required with fragment-order W")
        need = packed_weights_bytes(V, D, vocab_offset)
        if need == 0 or W.numel() * 2 < need:
            raise ValueError(f"W_packed holds {W.numel() * 2} bytes; {need} needed")
    else:
        V, D2 = W.shape
        if D2 != D:
            raise ValueError(f"h is B x {D} but W is V x {D2}")
    if not (temperature.shape[0] == partial_val.shape[0] == partial_idx.shape[0] ==
            partial_lse.shape[0] == B):
        raise ValueError("temperature and the partials must have B entries")
    devs = {t.device for t in (h, W, temperature, partial_val, partial_idx, partial_lse)}
    if len(devs) != 1:
        raise ValueError("all tensors must be on one device")
    if workspace is None:
        workspace = alloc_workspace(workspace_bytes(B, D, V), h.device)
    fn = lib().fs_sample_partial_lse_packed if packed else lib().fs_sample_partial_lse
    _check(fn(
        _ptr(h), _ptr(W), B, D, V, int(vocab_offset), _ptr(temperature),
        int(seed) & (2**64 - 1), int(step) & (2**64 - 1), _ptr(partial_val), _ptr(partial_idx),
        _ptr(partial_lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(h.device)))
    return partial_val, partial_idx, partial_lse


def groups_workspace_bytes(B: int, D: int, V: int, n_groups: int) -> int:
    return int(lib().fs_groups_workspace_bytes(B, D, V, n_groups))


def sample_groups_lse(h: torch.Tensor, W: torch.Tensor, temperature: torch.Tensor, seed: int,
                      step: int, cuts, vocab_offset: int = 0, out=None, workspace=None,
                      V: Optional[int] = None):
    """fs_sample_groups_lse: the grouped sampler's per-group partials for the
    groups W[cuts[g]:cuts[g+1]] in one launch.  Returns (val fp32 [G][B],
    idx int32 [G][B], lse fp32 [G][B]), slot g as fs_sample_partial_lse over
    group g.  W is the row-major V x D matrix, or (1-D, V given) its
    fragment-order copy (group starts multiples of 16)."""
    packed = W.dim() == 1
    _req(h, "h", torch.bfloat16, 2)
    _req(W, "W", torch.bfloat16, 1 if packed else 2)
    _req(temperature, "temperature", torch.float32, 1)
    B, D = h.shape
    if packed:
        if V is None:
            raise ValueError("V is required with fragment-order W")
    else:
        V = W.shape[0]
        if W.shape[1] != D:
            raise ValueError("h and W must have the same D")
    c, G = _host_cuts(cuts)
    dev = h.device
    if out is None:
        out = (torch.empty(G, B, dtype=torch.float32, device=dev),
               torch.empty(G, B, dtype=torch.int32, device=dev),
               torch.empty(G, B, dtype=torch.float32, device=dev))
    pv, pi, pl = out
    if workspace is None:
        workspace = alloc_workspace(groups_workspace_bytes(B, D, V, G), dev)
    fn = lib().fs_sample_groups_lse_packed if packed else lib().fs_sample_groups_lse
    _check(fn(_ptr(h), _ptr(W), B, D, V, int(vocab_offset), _ptr(temperature),
              int(seed) & (2**64 - 1), int(step) & (2**64 - 1), c, G, _ptr(pv), _ptr(pi),
              _ptr(pl), _ptr(workspace), workspace.numel() * workspace.element_size(),
              _stream(dev)))
    return pv, pi, pl


def merge_lse(partial_val, partial_idx, partial_lse, temperature, seed, step, out=None):
    """Grouped merge of P x B group partials: returns (ids int32[B], maxval fp32[B],
    total log-sum-exp fp32[B])."""
    _req(partial_val, "partial_val", torch.float32, 2)
    _req(partial_idx, "partial_idx", torch.int32, 2)
    _req(partial_lse, "partial_lse", torch.float32, 2)
    _req(temperature, "temperature", torch.float32, 1)
    if not (partial_val.shape == partial_idx.shape == partial_lse.shape):
        raise ValueError("the partials must have the same shape")
    P, B = partial_val.shape
    if temperature.shape[0] != B:
        raise ValueError("temperature must have B entries")
    dev = partial_val.device
    if out is None:
        out = (torch.empty(B, dtype=torch.int32, device=dev),
               torch.empty(B, dtype=torch.float32, device=dev),
               torch.empty(B, dtype=torch.float32, device=dev))
    ids, val, lse = out
    _check(lib().fs_merge_lse(_ptr(partial_val), _ptr(partial_idx), _ptr(partial_lse), P, B,
                              _ptr(temperature), int(seed) & (2**64 - 1),
                              int(step) & (2**64 - 1), _ptr(ids), _ptr(val), _ptr(lse),
                              _stream(dev)))
    return ids, val, lse


def sample_unfused(h, W, temperature, seed, step, vocab_offset=0, out=None, workspace=None):
    """Unfused baseline (logits and probabilities in device memory)."""
    B = h.shape[0]
    if out is None:
        out = (torch.empty(B, dtype=torch.int32, device=h.device),
               torch.empty(B, dtype=torch.float32, device=h.device))
    ids, val = out
    _sample_common("fs_sample_unfused", h, W, temperature, seed, step, vocab_offset, ids, val,
                   workspace, unfused_workspace_bytes)
    return ids, val


def merge(partial_val: torch.Tensor, partial_idx: torch.Tensor, out=None):
    """Per-row argmax over P x B partials (largest value, then smallest id)."""
    _req(partial_val, "partial_val", torch.float32, 2)
    _req(partial_idx, "partial_idx", torch.int32, 2)
    if partial_val.shape != partial_idx.shape:
        raise ValueError("partial_val and partial_idx must have the same shape")
    P, B = partial_val.shape
    dev = partial_val.device
    if out is None:
        out = (torch.empty(B, dtype=torch.int32, device=dev),
               torch.empty(B, dtype=torch.float32, device=dev))
    ids, val = out
    _check(lib().fs_merge(_ptr(partial_val), _ptr(partial_idx), P, B, _ptr(ids), _ptr(val),
                          _stream(dev)))
    return ids, val


def packed_weights_bytes(V: int, D: int, vocab_offset: int = 0) -> int:
    return int(lib().fs_packed_weights_bytes(V, D, vocab_offset))


def pack_weights(W: torch.Tensor, vocab_offset: int = 0) -> torch.Tensor:
    """W (V x D bf16) in the kernels' fragment order, as a flat bf16 tensor;
    sample it with sample_packed at the same vocab_offset (mod 4)."""
    _req(W, "W", torch.bfloat16, 2)
    V, D = W.shape
    n = packed_weights_bytes(V, D, vocab_offset)
    if n == 0:
        raise FlashSampleError(FS_ERR_INVALID_ARG, f"cannot pack a {V} x {D} W (D % 32 != 0?)")
    Wp = torch.empty(n // 2, dtype=torch.bfloat16, device=W.device)
    _check(lib().fs_pack_weights(_ptr(W), V, D, int(vocab_offset), _ptr(Wp), n,
                                 _stream(W.device)))
    return Wp


def sample_packed(h: torch.Tensor, W_packed: torch.Tensor, V: int, temperature: torch.Tensor,
                  seed: int, step: int, vocab_offset: int = 0, out=None, workspace=None):
    """fs_sample on fragment-order weights (pack_weights): returns (ids, maxval),
    identical to sample() on the row-major W."""
    _req(h, "h", torch.bfloat16, 2)
    _req(W_packed, "W_packed", torch.bfloat16, 1)
    _req(temperature, "temperature", torch.float32, 1)
    B, D = h.shape
    need = packed_weights_bytes(V, D, vocab_offset)
    if need == 0 or W_packed.numel() * 2 < need:
        raise ValueError(f"W_packed holds {W_packed.numel() * 2} bytes; {need} needed")
    if temperature.shape[0] != B:
        raise ValueError("temperature must have B entries")
    dev = h.device
    if out is None:
        out = (torch.empty(B, dtype=torch.int32, device=dev),
               torch.empty(B, dtype=torch.float32, device=dev))
    ids, val = out
    if len({t.device for t in (h, W_packed, temperature, ids, val)}) != 1:
        raise ValueError("all tensors must be on one device")
    if workspace is None:
        workspace = alloc_workspace(workspace_bytes(B, D, V), dev)
    _check(lib().fs_sample_packed(_ptr(h), _ptr(W_packed), B, D, V, int(vocab_offset),
                                  _ptr(temperature), int(seed) & (2**64 - 1),
                                  int(step) & (2**64 - 1), _ptr(ids), _ptr(val), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(dev)))
    return ids, val


def sample_packed_noalloc(h: torch.Tensor, W_packed: torch.Tensor, V: int,
                          temperature: torch.Tensor, seed: int, step: int, vocab_offset: int = 0,
                          out=None):
    """fs_sample_packed_noalloc: sample_packed with the tile partials in the
    library's own per-device scratch array instead of a workspace (calls that
    overlap on one device race).  Allocates nothing when `out` is given."""
    _req(h, "h", torch.bfloat16, 2)
    _req(W_packed, "W_packed", torch.bfloat16, 1)
    _req(temperature, "temperature", torch.float32, 1)
    B, D = h.shape
    need = packed_weights_bytes(V, D, vocab_offset)
    if need == 0 or W_packed.numel() * 2 < need:
        raise ValueError(f"W_packed holds {W_packed.numel() * 2} bytes; {need} needed")
    if temperature.shape[0] != B:
        raise ValueError("temperature must have B entries")
    dev = h.device
    if out is None:
        out = (torch.empty(B, dtype=torch.int32, device=dev),
               torch.empty(B, dtype=torch.float32, device=dev))
    ids, val = out
    if len({t.device for t in (h, W_packed, temperature, ids, val)}) != 1:
        raise ValueError("all tensors must be on one device")
    _check(lib().fs_sample_packed_noalloc(_ptr(h), _ptr(W_packed), B, D, V, int(vocab_offset),
                                          _ptr(temperature), int(seed) & (2**64 - 1),
                                          int(step) & (2**64 - 1), _ptr(ids), _ptr(val),
                                          _stream(dev)))
    return ids, val


def _host_cuts(cuts):
    """cuts as a host int32 ctypes array (kept alive by the caller) and the chunk count."""
    c = [int(x) for x in (cuts.tolist() if hasattr(cuts, "tolist") else cuts)]
    if len(c) < 2:
        raise ValueError("cuts needs at least two entries (0 and V)")
    return (ctypes.c_int32 * len(c))(*c), len(c) - 1


def online_bounds(W: torch.Tensor, cuts, workspace: Optional[torch.Tensor] = None,
                  V: Optional[int] = None, D: Optional[int] = None, vocab_offset: int = 0):
    """later_norm (fp64 [n_chunks], device) for the online sampler over the
    chunks W[cuts[c]:cuts[c+1]]: the largest row norm after each chunk.  W is
    the row-major V x D matrix, or (1-D, with V and D given) its fragment-order
    copy from pack_weights at vocab_offset."""
    packed = W.dim() == 1
    _req(W, "W", torch.bfloat16, 1 if packed else 2)
    if packed:
        if V is None or D is None:
            raise ValueError("V and D are required with fragment-order W")
        need = packed_weights_bytes(V, D, vocab_offset)
        if need == 0 or W.numel() * 2 < need:
            raise ValueError(f"W_packed holds {W.numel() * 2} bytes; {need} needed")
    else:
        V, D = W.shape
    arr, n = _host_cuts(cuts)
    later = torch.empty(n, dtype=torch.float64, device=W.device)
    if workspace is None:
        workspace = alloc_workspace(int(lib().fs_online_bounds_workspace_bytes(V, n)), W.device)
    nbytes = workspace.numel() * workspace.element_size()
    if packed:
        _check(lib().fs_online_bounds_packed(_ptr(W), V, D, int(vocab_offset), arr, n,
                                             _ptr(later), _ptr(workspace), nbytes,
                                             _stream(W.device)))
    else:
        _check(lib().fs_online_bounds(_ptr(W), V, D, arr, n, _ptr(later), _ptr(workspace), nbytes,
                                      _stream(W.device)))
    return later


def online_workspace_bytes(B: int, D: int, V: int, n_chunks: int) -> int:
    return int(lib().fs_online_workspace_bytes(B, D, V, n_chunks))


def sample_online(h, W, temperature, seed, step, cuts, later_norm, vocab_offset=0, out=None,
                  workspace=None, V=None):
    """Online sampler with early finalisation over the chunks W[cuts[c]:cuts[c+1]]:
    returns (ids int32[B], maxval fp32[B], chunks int32[B]).  W is the row-major
    V x D matrix, or (1-D, with V given) its fragment-order copy from
    pack_weights, whose chunk starts must be multiples of 16."""
    _req(h, "h", torch.bfloat16, 2)
    packed = W.dim() == 1
    _req(W, "W", torch.bfloat16, 1 if packed else 2)
    _req(temperature, "temperature", torch.float32, 1)
    _req(later_norm, "later_norm", torch.float64, 1)
    B, D = h.shape
    if packed:
        if V is None:
            raise ValueError("V is required with fragment-order W")
        need = packed_weights_bytes(V, D, vocab_offset)
        if need == 0 or W.numel() * 2 < need:
            raise ValueError(f"W_packed holds {W.numel() * 2} bytes; {need} needed")
    else:
        V, D2 = W.shape
        if D2 != D:
            raise ValueError(f"h is B x {D} but W is V x {D2}")
    if temperature.shape[0] != B:
        raise ValueError("temperature must have B entries")
    arr, n = _host_cuts(cuts)
    if later_norm.shape[0] != n:
        raise ValueError("later_norm must have one entry per chunk")
    dev = h.device
    if out is None:
        out = (torch.empty(B, dtype=torch.int32, device=dev),
               torch.empty(B, dtype=torch.float32, device=dev),
               torch.empty(B, dtype=torch.int32, device=dev))
    ids, val, chunks = out
    if len({t.device for t in (h, W, temperature, later_norm, ids, val, chunks)}) != 1:
        raise ValueError("all tensors must be on one device")
    if workspace is None:
        workspace = alloc_workspace(online_workspace_bytes(B, D, V, n), dev)
    fn = lib().fs_sample_online_packed if packed else lib().fs_sample_online
    _check(fn(
        _ptr(h), _ptr(W), B, D, V, int(vocab_offset), _ptr(temperature),
        int(seed) & (2**64 - 1), int(step) & (2**64 - 1), arr, n, _ptr(later_norm), _ptr(ids),
        _ptr(val), _ptr(chunks), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(dev)))
    return ids, val, chunks


def debug_noise(seed: int, step: int, row: int, gv0: int, n: int, device="cuda"):
    """Device noise words (as int32 bit patterns) and Gumbel values for ids gv0..gv0+n-1."""
    bits = torch.empty(n, dtype=torch.int32, device=device)
    g = torch.empty(n, dtype=torch.float32, device=device)
    _check(lib().fs_debug_noise(int(seed), int(step), int(row), int(gv0), int(n), _ptr(bits),
                                _ptr(g), _stream(bits.device)))
    return bits, g


def debug_gumbel(bits: torch.Tensor):
    _req(bits, "bits", torch.int32, 1)
    g = torch.empty(bits.shape[0], dtype=torch.float32, device=bits.device)
    _check(lib().fs_debug_gumbel(_ptr(bits), bits.shape[0], _ptr(g), _stream(bits.device)))
    return g


def device_info(device: int = 0):
    """(compute units, peak shader clock in kHz) the HIP runtime reports."""
    cus, clk = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib().fs_device_info(int(device), ctypes.byref(cus), ctypes.byref(clk)))
    return cus.value, clk.value


def profile_enable(capacity: int):
    """Time the next `capacity` fused-kernel launches with HIP events."""
    _check(lib().fs_profile_enable(int(capacity)))


def profile_read():
    """(launches, total_ms, min_ms, max_ms) of the launches timed so far."""
    n = ctypes.c_int32()
    tot, lo, hi = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
    _check(lib().fs_profile_read(ctypes.byref(n), ctypes.byref(tot), ctypes.byref(lo),
                                 ctypes.byref(hi)))
    return n.value, tot.value, lo.value, hi.value


def num_configs() -> int:
    return int(lib().fs_num_configs())


def config_name(i: int) -> str:
    r = lib().fs_config_name(i)
    return r.decode() if r else ""


def force_config(i: int):
    _check(lib().fs_force_config(int(i)))


def selected_config(B: int, D: int, V: int, packed: bool = False, grouped: bool = False) -> int:
    """Configuration fs_sample (packed: fs_sample_packed) would use; grouped:
    the one fs_sample_groups_lse (or its packed form) would use."""
    if grouped:
        return int(lib().fs_selected_config_groups(B, D, V, int(packed)))
    fn = lib().fs_selected_config_packed if packed else lib().fs_selected_config
    return int(fn(B, D, V))


# ---- training on sampled tokens ----
# These calls run on the device of their tensors, whatever the current device
# is, and on torch's current stream of that device.  The loss and clipping
# kernels take a few microseconds, so what the calls do on the host is kept
# short: addresses go to ctypes as plain integers, and the device is switched
# only where it differs.

def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _call(fn, dev, *args):
    """fn(*args, stream) on device `dev` and its current stream."""
    index = dev.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch.cuda.current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status != FS_OK:
        _check(status)


def _out(t: Optional[torch.Tensor], name: str, shape, dtype, device) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _req(t, name, dtype, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.device != device:
        raise ValueError("all tensors must be on one device")
    return t


def _workspace(t: Optional[torch.Tensor], nbytes: int, device) -> torch.Tensor:
    if t is None:
        return alloc_workspace(nbytes, device) if nbytes else None
    if not isinstance(t, torch.Tensor) or t.device != device or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return t


def _int32(*values: int):
    """The call's sizes and offsets fit the library's 32-bit arguments (ctypes would
    drop their upper bits)."""
    for v in values:
        if not -2 ** 31 <= v < 2 ** 31:
            raise ValueError(f"sizes and offsets must be below 2^31 (got {v})")


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _apart(written, read):
    """The given tensors that a call writes overlap neither one another nor one
    that it reads."""
    spans = [(t.data_ptr(), t.data_ptr() + _nbytes(t), i < len(written))
             for i, t in enumerate((*written, *read)) if t is not None and t.numel()]
    for i, (a, b, w) in enumerate(spans):
        if w and any(a < d and c < b for c, d, _ in spans[i + 1:]):
            raise ValueError("outputs and workspace must overlap neither each other nor an input")


def _changed(*tensors: Optional[torch.Tensor]):
    """Tells autograd that these tensors of the caller's were written: a graph that
    saved one refuses its backward pass."""
    torch.autograd.graph.increment_version([t for t in tensors if t is not None])


def _row(t: Optional[torch.Tensor], name: str, dtype, n: int, device):
    if t is None:
        return
    _req(t, name, dtype, 1)
    if t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries (got {t.shape[0]})")
    if t.device != device:
        raise ValueError("all tensors must be on one device")


def token_logprobs_workspace_bytes(B: int, D: int, V: int) -> int:
    _int32(B, D, V)
    return int(lib().fs_token_logprobs_workspace_bytes(B, D, V))


def token_logprobs(h: torch.Tensor, W: torch.Tensor, temperature: Optional[torch.Tensor],
                   token_ids: torch.Tensor, vocab_offset: int = 0, out=None,
                   workspace: Optional[torch.Tensor] = None, V: Optional[int] = None):
    """fs_token_logprobs: (log-probability fp32 [B] of each row's token under
    softmax(W h / T), log-sum-exp fp32 [B]), with no logits in memory.
    token_ids are global ids (int32); rows with a negative id have none and get
    log-probability 0, ids outside this W's rows get -inf.  temperature None
    means 1.  W is row-major V x D, or (1-D, with V given) its fragment-order
    copy from pack_weights at the same vocab_offset.

    Where torch records gradients and h or W requires one, the log-probabilities
    carry a graph whose backward pass is token_logprobs_backward (not within a
    graph capture: capture that call).  None leads through the log-sum-exps, the
    temperatures or a fragment-order W: its backward pass raises.  Results
    written to `out` carry no graph."""
    if out is None and torch.is_grad_enabled() and any(
            isinstance(t, torch.Tensor) and t.requires_grad for t in (h, W, temperature)):
        return _TokenLogprobs.apply(h, W, temperature, token_ids, vocab_offset, workspace, V)
    _req(h, "h", torch.bfloat16, 2)
    packed = isinstance(W, torch.Tensor) and W.dim() == 1
    _req(W, "W", torch.bfloat16, 1 if packed else 2)
    B, D = h.shape
    _int32(vocab_offset)
    if packed:
        if V is None:
            raise ValueError("V is required with fragment-order W")
        _int32(D, V)
        need = packed_weights_bytes(V, D, vocab_offset)
        if need == 0 or W.numel() * 2 < need:
            raise ValueError(f"W_packed holds {W.numel() * 2} bytes; {need} needed")
    else:
        if V is not None and V != W.shape[0]:
            raise ValueError(f"V is {V} but W has {W.shape[0]} rows")
        V = W.shape[0]
        if W.shape[1] != D:
            raise ValueError(f"h is B x {D} but W is V x {W.shape[1]}")
    dev = h.device
    if W.device != dev:
        raise ValueError("all tensors must be on one device")
    _row(temperature, "temperature", torch.float32, B, dev)
    _row(token_ids, "token_ids", torch.int32, B, dev)
    lp, lse = (None, None) if out is None else out
    lp = _out(lp, "logprob", (B,), torch.float32, dev)
    lse = _out(lse, "lse", (B,), torch.float32, dev)
    ws = _workspace(workspace, token_logprobs_workspace_bytes(B, D, V), dev)
    if out is not None or workspace is not None:
        _apart((lp, lse, ws), (h, W, temperature, token_ids))
    fn = lib().fs_token_logprobs_packed if packed else lib().fs_token_logprobs
    _call(fn, dev, _addr(h), _addr(W), B, D, V, int(vocab_offset), _addr(temperature),
          _addr(token_ids), _addr(lp), _addr(lse), _addr(ws), _nbytes(ws))
    if out is not None:
        _changed(*out)
    return lp, lse


def token_logprobs_backward_workspace_bytes(B: int, D: int, V: int) -> int:
    _int32(B, D, V)
    return int(lib().fs_token_logprobs_backward_workspace_bytes(B, D, V))


class _TokenLogprobs(torch.autograd.Function):
    """token_logprobs with its backward pass."""

    @staticmethod
    def forward(ctx, h, W, temperature, token_ids, vocab_offset, workspace, V):
        lp, lse = token_logprobs(h, W, temperature, token_ids, vocab_offset, None, workspace, V)
        ctx.save_for_backward(h, W, temperature, token_ids, lp, lse)
        ctx.vocab_offset = vocab_offset
        ctx.set_materialize_grads(False)  # (a gradient of lse is one that somebody asked for)
        return lp, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_logprob, grad_lse):
        h, W, temperature, token_ids, lp, lse = ctx.saved_tensors
        if grad_lse is not None:
            raise RuntimeError("token_logprobs: no gradient leads through the log-sum-exps")
        if ctx.needs_input_grad[2]:
            raise RuntimeError("token_logprobs: no gradient leads to the temperatures")
        if W.dim() == 1:
            raise RuntimeError("token_logprobs: no gradient leads through a fragment-order W; "
                               "score with the row-major one")
        if torch.cuda.is_current_stream_capturing():
            # (accumulating into leaves that an eager graph holds too would leave the capture)
            raise RuntimeError("token_logprobs: its backward pass cannot be captured; capture "
                               "token_logprobs_backward")
        if grad_logprob is None:
            return (None,) * 7
        gh, gw = token_logprobs_backward(h, W, temperature, token_ids, lp, lse,
                                         grad_logprob.contiguous(), ctx.vocab_offset,
                                         ctx.needs_input_grad[0], ctx.needs_input_grad[1])
        return gh, gw, None, None, None, None, None


def token_logprobs_backward(h: torch.Tensor, W: torch.Tensor, temperature: Optional[torch.Tensor],
                            token_ids: torch.Tensor, logprob: torch.Tensor, lse: torch.Tensor,
                            grad_logprob: torch.Tensor, vocab_offset: int = 0, need_h: bool = True,
                            need_W: bool = True, out=None,
                            workspace: Optional[torch.Tensor] = None):
    """fs_token_logprobs_backward: (grad_h bf16 [B][D], grad_W bf16 [V][D]) from
    the gradient of the log-probabilities; logprob and lse are the forward
    call's.  need_h / need_W false: that product is skipped and None returned.
    out: (grad_h, grad_W) to write into, either None."""
    _req(h, "h", torch.bfloat16, 2)
    _req(W, "W", torch.bfloat16, 2)
    B, D = h.shape
    V = W.shape[0]
    _int32(vocab_offset)
    if W.shape[1] != D:
        raise ValueError(f"h is B x {D} but W is V x {W.shape[1]}")
    dev = h.device
    if W.device != dev:
        raise ValueError("all tensors must be on one device")
    _row(temperature, "temperature", torch.float32, B, dev)
    _row(token_ids, "token_ids", torch.int32, B, dev)
    for t, name in ((logprob, "logprob"), (lse, "lse"), (grad_logprob, "grad_logprob")):
        _row(t, name, torch.float32, B, dev)
    gh, gw = (None, None) if out is None else out
    gh = _out(gh, "grad_h", (B, D), torch.bfloat16, dev) if need_h else None
    gw = _out(gw, "grad_W", (V, D), torch.bfloat16, dev) if need_W else None
    ws = _workspace(workspace, token_logprobs_backward_workspace_bytes(B, D, V), dev)
    if out is not None or workspace is not None:
        _apart((gh, gw, ws), (h, W, temperature, token_ids, logprob, lse, grad_logprob))
    _call(lib().fs_token_logprobs_backward, dev, _addr(h), _addr(W), B, D, V, int(vocab_offset),
          _addr(temperature), _addr(token_ids), _addr(logprob), _addr(lse), _addr(grad_logprob),
          _addr(gh), _addr(gw), _addr(ws), _nbytes(ws))
    if out is not None:
        _changed(gh, gw)
    return gh, gw


def cross_entropy_workspace_bytes(B: int, D: int, V: int, grads: bool = True) -> int:
    _int32(B, D, V)
    return int(lib().fs_cross_entropy_workspace_bytes(B, D, V, int(grads)))


def cross_entropy(h: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                  label_smoothing: float = 0.0, z_loss: float = 0.0, reduction: str = "mean",
                  grad_scale: float = 1.0, need_h: bool = True, need_W: bool = True, out=None,
                  workspace: Optional[torch.Tensor] = None):
    """fs_cross_entropy of the head W (bf16 [V][D]) on hidden states h (bf16
    [B][D]) and targets (int32 [B]; negative: the row has none): returns (stats
    fp32 [3], losses fp32 [B], grad_h bf16 [B][D], grad_W bf16 [V][D]).  stats are
    the loss (reduction "mean" or "sum" over the rows that have a target), their
    mean negative log-probability and their mean squared log-sum-exp; the
    gradients are those of grad_scale * loss.  need_h / need_W false: None in that
    gradient's place, and without both the loss alone is computed.  Nothing
    returned carries a graph (an h with one goes on by h.backward(grad_h), W by
    W.grad = grad_W).  out: (stats, losses, grad_h, grad_W) to write into, each may
    be None."""
    _req(h, "h", torch.bfloat16, 2)
    _req(W, "W", torch.bfloat16, 2)
    B, D = h.shape
    V = W.shape[0]
    if W.shape[1] != D:
        raise ValueError(f"h is B x {D} but W is V x {W.shape[1]}")
    dev = h.device
    if W.device != dev:
        raise ValueError("all tensors must be on one device")
    _row(targets, "targets", torch.int32, B, dev)
    if targets is None:
        raise TypeError("targets must be a tensor")
    mean = _choice(_LOSS_REDUCTIONS, reduction, "reduction")
    stats, losses, gh, gw = (None,) * 4 if out is None else out
    stats = _out(stats, "stats", (3,), torch.float32, dev)
    losses = _out(losses, "losses", (B,), torch.float32, dev)
    gh = _out(gh, "grad_h", (B, D), torch.bfloat16, dev) if need_h else None
    gw = _out(gw, "grad_W", (V, D), torch.bfloat16, dev) if need_W else None
    ws = _workspace(workspace, cross_entropy_workspace_bytes(B, D, V, need_h or need_W), dev)
    if out is not None or workspace is not None:
        _apart((stats, losses, gh, gw, ws), (h, W, targets))
    _call(lib().fs_cross_entropy, dev, _addr(h), _addr(W), B, D, V, _addr(targets), label_smoothing,
          z_loss, mean, grad_scale, _addr(stats), _addr(losses), _addr(gh), _addr(gw), _addr(ws),
          _nbytes(ws))
    if out is not None:
        _changed(stats, losses, gh, gw)
    return stats, losses, gh, gw


def loss_workspace_bytes(n_sequences: int, n_tokens: int) -> int:
    _int32(n_sequences, n_tokens)
    return int(lib().fs_loss_workspace_bytes(n_sequences, n_tokens))


def _sequences(logprob, cu_seqlens, mask, **rows):
    """Common checks of the losses; returns (device, tokens, mask as uint8)."""
    _req(logprob, "logprob", torch.float32, 1)
    dev, N = logprob.device, logprob.shape[0]
    _req(cu_seqlens, "cu_seqlens", torch.int32, 1)
    if cu_seqlens.device != dev:
        raise ValueError("all tensors must be on one device")
    if cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must have at least one entry")
    for name, t in rows.items():
        _row(t, name, torch.float32, N, dev)
    if mask is not None:
        if mask.dtype == torch.bool:
            mask = mask.view(torch.uint8)
        _row(mask, "mask", torch.uint8, N, dev)
    return dev, N, mask


_KL = {"k1": 1, "k2": 2, "k3": 3}
_LOSS_REDUCTIONS = {"sum": 0, "mean": 1}
_REDUCTIONS = {"token": 0, "sequence": 1}
_PREFERENCES = {"sigmoid": 0, "hinge": 1, "ipo": 2}


def _choice(table, value, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)} (got {value!r})")
    return table[value]


def policy_loss(logprob: torch.Tensor, old_logprob: torch.Tensor, advantages: torch.Tensor,
                cu_seqlens: torch.Tensor, ref_logprob: Optional[torch.Tensor] = None,
                mask: Optional[torch.Tensor] = None, per_token: bool = False,
                clip_low: float = 0.2, clip_high: float = 0.2, dual_clip: float = 0.0,
                kl_coef: float = 0.0, kl: str = "k3", reduction: str = "token",
                grad_scale: float = 1.0, out=None, workspace: Optional[torch.Tensor] = None):
    """fs_policy_loss over packed sequences (tokens cu_seqlens[s] to
    cu_seqlens[s + 1] of the flat fp32 arrays): returns (stats fp32 [4], grad
    fp32 [tokens]); stats are the loss, the mean surrogate, the mean KL and
    the clipped share, grad is grad_scale * d loss / d logprob; neither carries
    a graph (a logprob with one goes on by logprob.backward(grad)).  advantages
    holds one value per sequence, or with per_token one per token.  mask (bool
    or uint8): the tokens that count.  Entries of grad before the first and
    behind the last sequence are 0; in a grad given by `out` = (stats, grad)
    they are left as they were."""
    dev, N, m = _sequences(logprob, cu_seqlens, mask, old_logprob=old_logprob,
                           ref_logprob=ref_logprob)
    S = cu_seqlens.shape[0] - 1
    _row(advantages, "advantages", torch.float32, N if per_token else S, dev)
    stats, given = (None, None) if out is None else out
    stats = _out(stats, "stats", (4,), torch.float32, dev)
    grad = _out(given, "grad", (N,), torch.float32, dev)
    ws = _workspace(workspace, loss_workspace_bytes(S, N), dev)
    if out is not None or workspace is not None:
        _apart((stats, grad, ws), (logprob, old_logprob, ref_logprob, advantages, m, cu_seqlens))
    _call(lib().fs_policy_loss, dev, _addr(logprob), _addr(old_logprob), _addr(ref_logprob),
          _addr(advantages), _addr(m), _addr(cu_seqlens), S, N, int(per_token), clip_low, clip_high,
          dual_clip, kl_coef, _choice(_KL, kl, "kl"), _choice(_REDUCTIONS, reduction, "reduction"),
          grad_scale, int(given is None), _addr(stats), _addr(grad), _addr(ws), _nbytes(ws))
    if out is not None:
        _changed(*out)
    return stats, grad


def preference_loss(logprob: torch.Tensor, cu_seqlens: torch.Tensor,
                    ref_logprob: Optional[torch.Tensor] = None,
                    mask: Optional[torch.Tensor] = None, kind: str = "sigmoid", beta: float = 0.1,
                    margin: float = 0.0, label_smoothing: float = 0.0,
                    length_normalised: bool = False, grad_scale: float = 1.0, out=None,
                    workspace: Optional[torch.Tensor] = None):
    """fs_preference_loss over packed sequences, the chosen answers first and
    then the rejected ones in the same order (cu_seqlens has 2 P + 1 entries):
    returns (stats fp32 [3], rewards fp32 [2 P], grad fp32 [tokens]); stats are
    the loss, the share of pairs that prefer the chosen answer and the mean
    margin of rewards; none carries a graph (logprob.backward(grad)).  Entries of grad before the first and behind the last
    sequence are 0; in a grad given by `out` = (stats, rewards, grad) they are
    left as they were."""
    dev, N, m = _sequences(logprob, cu_seqlens, mask, ref_logprob=ref_logprob)
    S = cu_seqlens.shape[0] - 1
    if S % 2:
        raise ValueError("cu_seqlens must describe chosen and rejected answers: 2 P + 1 entries")
    stats, rewards, given = (None, None, None) if out is None else out
    stats = _out(stats, "stats", (3,), torch.float32, dev)
    rewards = _out(rewards, "rewards", (S,), torch.float32, dev)
    grad = _out(given, "grad", (N,), torch.float32, dev)
    ws = _workspace(workspace, loss_workspace_bytes(S, N), dev)
    if out is not None or workspace is not None:
        _apart((stats, rewards, grad, ws), (logprob, ref_logprob, m, cu_seqlens))
    _call(lib().fs_preference_loss, dev, _addr(logprob), _addr(ref_logprob), _addr(m),
          _addr(cu_seqlens), S // 2, N, _choice(_PREFERENCES, kind, "kind"), beta, margin,
          label_smoothing, int(length_normalised), grad_scale, int(given is None), _addr(stats),
          _addr(rewards), _addr(grad), _addr(ws), _nbytes(ws))
    if out is not None:
        _changed(*out)
    return stats, rewards, grad


_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def clip_grad_norm(grads, max_norm: float, out=None, norm: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """fs_clip_grad_norm: scales the gradients (a list of contiguous bf16, fp16
    or fp32 device tensors) in place, or into the tensors of `out`, by min(1,
    max_norm / (norm + 1e-6)) and returns their global norm before that (fp32
    [1], on the device).  A norm that is not finite scales nothing."""
    grads = list(grads)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    dev = grads[0].device
    n = len(grads)
    outs = grads if out is None else list(out)
    if len(outs) != n:
        raise ValueError(f"out must hold {n} tensors (got {len(outs)})")
    try:
        types = [_DTYPES[g.dtype] for g in grads]
    except (KeyError, AttributeError):
        raise TypeError("grads must be bf16, fp16 or fp32 tensors") from None
    on = dev.type == "cuda"
    for i, g in enumerate(grads):
        if not (on and g.is_contiguous() and g.device == dev):
            raise ValueError(f"grads[{i}] must be contiguous and on the first gradient's device")
    if out is not None:
        for i, (g, o) in enumerate(zip(grads, outs)):
            if not (o.dtype is g.dtype and o.shape == g.shape and o.is_contiguous()
                    and o.device == dev):
                raise ValueError(f"out[{i}] must be contiguous, of the type and shape of grads[{i}] "
                                 "and on its device")
    count = [g.numel() for g in grads]
    src = [g.data_ptr() for g in grads]
    dst = src if out is None else [o.data_ptr() for o in outs]
    # a written tensor's bytes end before the next one's begin ...
    ends = 0
    written = sorted([p for p in zip(dst, types, count) if p[2]])
    for p, t, k in written:
        if p < ends:
            raise ValueError("the tensors written must not overlap")
        ends = p + (k << (1 + (t == 2)))
    if out is not None:  # ... and touch no tensor read but their own
        starts = [p for p, _, _ in written]
        for p, q, t, k in zip(src, dst, types, count):
            if k and p != q:
                i = bisect.bisect_left(starts, p + (k << (1 + (t == 2)))) - 1
                if i >= 0 and starts[i] + (written[i][2] << (1 + (written[i][1] == 2))) > p:
                    raise ValueError("a tensor of out overlaps one of grads that is not its own")
    array = ctypes.c_void_p * n
    sizes = (ctypes.c_int64 * n)(*count)
    given = norm is not None or workspace is not None
    norm = _out(norm, "norm", (1,), torch.float32, dev)
    ws = _workspace(workspace, int(lib().fs_clip_grad_norm_workspace_bytes(sizes, n)), dev)
    if given:
        _apart((norm, ws), grads if out is None else (*grads, *outs))
        _changed(norm)
    types = (ctypes.c_int * n)(*types)
    _call(lib().fs_clip_grad_norm, dev, array(*src), None if out is None else array(*dst), sizes,
          types, n, max_norm, _addr(norm), _addr(ws), _nbytes(ws))
    if out is not None or max_norm != math.inf:  # (an infinite limit in place: the norm alone)
        torch.autograd.graph.increment_version(outs)
    return norm


# ---- the LM head in 8-bit floating point ----
def _fp8_types():
    """(e4m3, e8m0): torch has the scales' type from 2.7 on, and the bf16 calls do not need it."""
    try:
        return torch.float8_e4m3fn, torch.float8_e8m0fnu
    except AttributeError as e:
        raise RuntimeError("the 8-bit head needs torch.float8_e4m3fn and torch.float8_e8m0fnu, which "
                           f"torch {torch.__version__} does not have") from e


def _blocks(n: int) -> int:
    return -(-n // 128)


def quantize_weights_fp8(W: torch.Tensor, packed: bool = True, out=None):
    """fs_quantize_weights_fp8 of W (bf16 [V][D]): returns (values, scales).  The
    scales are powers of two, one per block of 128 x 128 (float8_e8m0fnu [ceil(V /
    128)][ceil(D / 128)]); the values float8_e4m3fn, in the fragment order that
    logits_fp8, sample_fp8 and token_logprobs_fp8 read (1-D; D % 64 == 0), or with
    packed false row-major [V][D].  out: (values, scales) to write into."""
    e4m3, e8m0 = _fp8_types()
    _req(W, "W", torch.bfloat16, 2)
    V, D = W.shape
    _int32(V, D)
    dev = W.device
    need = int(lib().fs_fp8_weights_bytes(V, D, int(packed)))
    if need == 0 and V > 0:
        _check(lib().fs_quantize_weights_fp8(None, V, D, int(packed), None, 0, None, None))
    q, scale = (None, None) if out is None else out
    q = _out(q, "values", (need,) if packed else (V, D), e4m3, dev)
    scale = _out(scale, "scales", (_blocks(V), _blocks(D)), e8m0, dev)
    if out is not None:
        _apart((q, scale), (W,))
    _call(lib().fs_quantize_weights_fp8, dev, _addr(W), V, D, int(packed), _addr(q), _nbytes(q),
          _addr(scale))
    if out is not None:
        _changed(q, scale)
    return q, scale


def pack_weights_fp8(q: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """fs_pack_weights_fp8: row-major e4m3 weights [V][D] in the fragment order of
    the 8-bit products (once, as at model load)."""
    e4m3, _ = _fp8_types()
    _req(q, "q", e4m3, 2)
    V, D = q.shape
    _int32(V, D)
    given, need = out, int(lib().fs_fp8_weights_bytes(V, D, 1))
    if need == 0:
        _check(lib().fs_pack_weights_fp8(None, V, D, None, 0, None))
    out = _out(out, "out", (need,), e4m3, q.device)
    if given is not None:
        _apart((out,), (q,))
    _call(lib().fs_pack_weights_fp8, q.device, _addr(q), V, D, _addr(out), _nbytes(out))
    if given is not None:
        _changed(out)
    return out


def fp8_workspace_bytes(B: int, D: int, V: int) -> int:
    _int32(B, D, V)
    return int(lib().fs_fp8_workspace_bytes(B, D, V))


def _fp8_head(h, W_packed, W_scale, V, vocab_offset, workspace):
    """Checks of the 8-bit products: (device, B, D, workspace)."""
    e4m3, e8m0 = _fp8_types()
    _req(h, "h", torch.bfloat16, 2)
    if isinstance(W_packed, torch.Tensor) and W_packed.dim() == 2:
        raise ValueError("W_packed must be in fragment order (quantize_weights_fp8, pack_weights_fp8)")
    _req(W_packed, "W_packed", e4m3, 1)
    _req(W_scale, "W_scale", e8m0, 2)
    B, D = h.shape
    _int32(B, D, V, vocab_offset)
    need = int(lib().fs_fp8_weights_bytes(V, D, 1))
    if need and W_packed.numel() != need:
        raise ValueError(f"W_packed holds {W_packed.numel()} bytes; {need} are those of {V} x {D}")
    if V > 0 and D > 0 and tuple(W_scale.shape) != (_blocks(V), _blocks(D)):
        raise ValueError(f"W_scale must have shape {(_blocks(V), _blocks(D))} (got {tuple(W_scale.shape)})")
    dev = h.device
    if W_packed.device != dev or W_scale.device != dev:
        raise ValueError("all tensors must be on one device")
    return dev, B, D, _workspace(workspace, fp8_workspace_bytes(B, D, V), dev)


class _NoGradient(torch.autograd.Function):
    """Results of the 8-bit products of an h that requires a gradient."""

    @staticmethod
    def forward(ctx, h, name, call):
        ctx.name = name
        return call()

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name}: no gradient leads through the 8-bit head")


def _records(h, out) -> bool:
    return (out is None and isinstance(h, torch.Tensor) and h.requires_grad
            and torch.is_grad_enabled())


def logits_fp8(h: torch.Tensor, W_packed: torch.Tensor, W_scale: torch.Tensor, V: int,
               dtype=torch.float32, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """fs_logits_fp8: logits [B][V] (fp32 or bf16) of hidden states h (bf16 [B][D],
    quantised by the call) and the 8-bit head of quantize_weights_fp8.  out: a
    tensor [B][V] of either type to write into, whose rows may lie further apart
    than V.  No gradient leads through the 8-bit head: where torch records them and h
    requires one, the backward pass of the result raises."""
    if _records(h, out):
        return _NoGradient.apply(h, "logits_fp8", lambda: logits_fp8(h, W_packed, W_scale, V, dtype,
                                                                     None, workspace))
    dev, B, D, ws = _fp8_head(h, W_packed, W_scale, V, 0, workspace)
    given = out
    if out is None:
        if dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"dtype must be torch.float32 or torch.bfloat16 (got {dtype})")
        out = torch.empty(B, V, dtype=dtype, device=dev)
    else:
        if not isinstance(out, torch.Tensor) or out.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("out must be an fp32 or bf16 tensor")
        if tuple(out.shape) != (B, V) or out.device != dev:
            raise ValueError(f"out must have shape {(B, V)} and be on h's device")
        if (V > 1 and out.stride(1) != 1) or (B > 1 and out.stride(0) < V):
            raise ValueError("out must have contiguous rows that do not overlap")
    pitch = out.stride(0) if B > 1 else V
    if given is not None or workspace is not None:
        _apart_rows(out, ws, (h, W_packed, W_scale))
    _call(lib().fs_logits_fp8, dev, _addr(h), _addr(W_packed), _addr(W_scale), B, D, V,
          int(out.dtype == torch.float32), _addr(out), pitch, _addr(ws), _nbytes(ws))
    if given is not None:
        _changed(out)
    return out


def _apart_rows(out, ws, read):
    """_apart for an output whose rows may lie apart: its whole span counts."""
    n = out.numel() and (out.shape[0] - 1) * out.stride(0) + out.shape[1]
    _apart((torch.as_strided(out, (n,), (1,)), ws), read)


def token_logprobs_fp8(h: torch.Tensor, W_packed: torch.Tensor, W_scale: torch.Tensor, V: int,
                       temperature: Optional[torch.Tensor], token_ids: torch.Tensor,
                       vocab_offset: int = 0, out=None, workspace: Optional[torch.Tensor] = None):
    """fs_token_logprobs_fp8: token_logprobs on the 8-bit head of
    quantize_weights_fp8 (what a rollout stores when it samples with sample_fp8):
    (logprob, lse).  No gradient leads through the 8-bit head: where torch records
    them and h requires one, the backward pass of the results raises."""
    if _records(h, out):
        return _NoGradient.apply(h, "token_logprobs_fp8", lambda: token_logprobs_fp8(
            h, W_packed, W_scale, V, temperature, token_ids, vocab_offset, None, workspace))
    dev, B, D, ws = _fp8_head(h, W_packed, W_scale, V, vocab_offset, workspace)
    _row(temperature, "temperature", torch.float32, B, dev)
    if token_ids is None:
        raise TypeError("token_ids must be a tensor")
    _row(token_ids, "token_ids", torch.int32, B, dev)
    lp, lse = (None, None) if out is None else out
    lp = _out(lp, "logprob", (B,), torch.float32, dev)
    lse = _out(lse, "lse", (B,), torch.float32, dev)
    if out is not None or workspace is not None:
        _apart((lp, lse, ws), (h, W_packed, W_scale, temperature, token_ids))
    _call(lib().fs_token_logprobs_fp8, dev, _addr(h), _addr(W_packed), _addr(W_scale), B, D, V,
          int(vocab_offset), _addr(temperature), _addr(token_ids), _addr(lp), _addr(lse), _addr(ws),
          _nbytes(ws))
    if out is not None:
        _changed(*out)
    return lp, lse


def sample_fp8(h: torch.Tensor, W_packed: torch.Tensor, W_scale: torch.Tensor, V: int,
               temperature: torch.Tensor, seed: int, step: int, vocab_offset: int = 0, out=None,
               workspace: Optional[torch.Tensor] = None):
    """fs_sample_fp8: sample on the 8-bit head of quantize_weights_fp8, with the same
    noise field: (ids int32 [B], winning scores fp32 [B])."""
    dev, B, D, ws = _fp8_head(h, W_packed, W_scale, V, vocab_offset, workspace)
    if temperature is None:
        raise TypeError("temperature must be a tensor")
    _row(temperature, "temperature", torch.float32, B, dev)
    ids, val = (None, None) if out is None else out
    ids = _out(ids, "ids", (B,), torch.int32, dev)
    val = _out(val, "maxval", (B,), torch.float32, dev)
    if out is not None or workspace is not None:
        _apart((ids, val, ws), (h, W_packed, W_scale, temperature))
    _call(lib().fs_sample_fp8, dev, _addr(h), _addr(W_packed), _addr(W_scale), B, D, V,
          int(vocab_offset), _addr(temperature), seed, step, _addr(ids), _addr(val), _addr(ws),
          _nbytes(ws))
    if out is not None:
        _changed(*out)
    return ids, val
