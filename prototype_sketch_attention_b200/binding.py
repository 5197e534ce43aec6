"""ctypes binding of libsa_sketch.so (argument marshalling only).

The functions named ``sa_*`` mirror the C ABI in include/sa_sketch.h one to one.
They take raw device pointers (ints), sizes and a stream handle, and return the
library's status code. ``forward`` and ``backward`` are conveniences for torch
users: they allocate outputs and workspace with torch (the library itself
allocates nothing), call the C ABI on the current stream and raise on errors.
Every step of the computation runs in the library's CUDA kernels. There is no
fallback: if the library is missing, importing this module raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os
import warnings

import torch

from .build import calls_path

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsa_sketch.so")

SA_F32 = 0
SA_BF16 = 1
SA_OK = 0
SA_ERR_INVALID_ARG = 1
SA_ERR_UNSUPPORTED = 2
SA_ERR_WORKSPACE = 3
SA_ERR_CUDA = 4
SA_ERR_TIMEOUT = 5
SA_ERR_BAD_OFFSETS = 6
SA_ERR_NO_DEVICE = 7
SA_ERR_BAD_PAGES = 8

EXPORTED = ("sa_sketch_workspace_size", "sa_sketch_forward", "sa_sketch_backward",
            "sa_sketch_get_device_status", "sa_status_string", "sa_sketch_debug_wait_timeout",
            "sa_sketch_profile_events", "sa_sketch_forward_noalloc", "sa_sketch_combine",
            "sa_sketch_debug_gemm", "sa_stca_workspace_size", "sa_stca_forward",
            "sa_stca_backward", "sa_sketch_pack", "sa_sketch_unpack",
            "sa_sketch_forward_host_buffer_size", "sa_sketch_forward_host",
            "sa_sketch_forward_host_status", "sa_sketch_host_parts", "sa_sketch_forward_grid",
            "sa_stca_keys_workspace_size", "sa_stca_keys_forward", "sa_stca_keys_backward",
            "sa_stca_recent_ranges", "sa_cross_attn_workspace_size", "sa_cross_attn_forward",
            "sa_cross_attn_backward", "sa_page_tables", "sa_paged_append",
            "sa_paged_attn_workspace_size", "sa_paged_attn")
SA_CODEC_BF16 = 0
SA_CODEC_FP8 = 1


class SketchAttentionError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {sa_status_string(status)} ({status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is not built; run `python -m prototype_sketch_attention_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.sa_sketch_workspace_size.restype = sz
    lib.sa_sketch_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32]
    lib.sa_sketch_forward.restype = i32
    lib.sa_sketch_forward.argtypes = [vp, vp, i32, i64, i32, vp, i32, vp, vp, i32,
                                      vp, vp, vp, vp, vp, sz, vp]
    lib.sa_sketch_backward.restype = i32
    lib.sa_sketch_backward.argtypes = [vp, vp, i32, i64, i32, vp, i32, vp, vp, i32,
                                       vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.sa_sketch_debug_gemm.restype = i32
    lib.sa_sketch_debug_gemm.argtypes = [vp, i32, vp, i32, i32, i32, i32, i32, vp, vp, vp]
    lib.sa_sketch_combine.restype = i32
    lib.sa_sketch_combine.argtypes = [vp, vp, i32, i32, i32, vp, i32, vp, vp]
    lib.sa_sketch_get_device_status.restype = i32
    lib.sa_sketch_get_device_status.argtypes = [vp, vp]
    lib.sa_status_string.restype = ctypes.c_char_p
    lib.sa_status_string.argtypes = [i32]
    lib.sa_sketch_debug_wait_timeout.restype = i32
    lib.sa_sketch_debug_wait_timeout.argtypes = [vp, ctypes.c_longlong, vp]
    lib.sa_sketch_profile_events.restype = i32
    lib.sa_sketch_profile_events.argtypes = [vp, vp]
    lib.sa_sketch_forward_noalloc.restype = i32
    lib.sa_sketch_forward_noalloc.argtypes = [vp, vp, i32, i64, i32, vp, i32, vp, vp, i32,
                                              vp, vp, vp, vp, vp, vp]
    lib.sa_stca_workspace_size.restype = sz
    lib.sa_stca_workspace_size.argtypes = [i32, i64, i32, i32, i32]
    lib.sa_sketch_pack.restype = i32
    lib.sa_sketch_pack.argtypes = [vp, i64, i32, i32, vp, vp, vp]
    lib.sa_sketch_unpack.restype = i32
    lib.sa_sketch_unpack.argtypes = [vp, vp, i64, i32, i32, vp, vp]
    lib.sa_stca_backward.restype = i32
    lib.sa_stca_backward.argtypes = [vp, vp, vp, i32, i64, i32, vp, i32, vp, vp, vp, vp, vp, vp,
                                     vp, vp, vp, vp, sz, vp]
    lib.sa_stca_forward.restype = i32
    lib.sa_stca_forward.argtypes = [vp, vp, i32, i64, i32, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.sa_sketch_forward_host_buffer_size.restype = sz
    lib.sa_sketch_forward_host_buffer_size.argtypes = [i32, i64, i32, i32, i32, i32]
    lib.sa_sketch_forward_host.restype = i32
    lib.sa_sketch_forward_host.argtypes = [vp, vp, i32, i64, i32, vp, i32, vp, vp, i32, vp, vp,
                                           vp, sz, i32, vp, vp, vp]
    lib.sa_sketch_forward_host_status.restype = i32
    lib.sa_sketch_forward_host_status.argtypes = [vp, i32, i64, i32, i32, i32, i32, vp]
    lib.sa_sketch_forward_grid.restype = i32
    lib.sa_sketch_forward_grid.argtypes = [i32, i32, i32, vp, vp, vp, vp]
    lib.sa_sketch_host_parts.restype = i32
    lib.sa_sketch_host_parts.argtypes = [vp, i32, i32, vp]
    lib.sa_stca_keys_workspace_size.restype = sz
    lib.sa_stca_keys_workspace_size.argtypes = [i32, i64, i32, i32]
    lib.sa_stca_keys_forward.restype = i32
    lib.sa_stca_keys_forward.argtypes = [vp, vp, i32, i64, i32, vp, i64, vp, vp, vp, vp, vp, vp,
                                         vp, vp, sz, vp]
    lib.sa_stca_keys_backward.restype = i32
    lib.sa_stca_keys_backward.argtypes = [vp, vp, i32, i64, i32, vp, i64, vp, vp, vp, vp, vp, vp,
                                          vp, vp, i32, vp, vp, vp, vp, sz, vp]
    lib.sa_stca_recent_ranges.restype = i32
    lib.sa_stca_recent_ranges.argtypes = [vp, i32, i64, vp, vp, vp]
    f32 = ctypes.c_float
    lib.sa_cross_attn_workspace_size.restype = sz
    lib.sa_cross_attn_workspace_size.argtypes = [i32, i64, i64, i32, i32, i32, i32]
    cross = [vp, i64, vp, i32, i64, i32, i32, vp, i64, vp, i64, vp, i64, i32, vp, f32]
    lib.sa_cross_attn_forward.restype = i32
    lib.sa_cross_attn_forward.argtypes = cross + [vp, vp, vp, vp, sz, vp]
    lib.sa_cross_attn_backward.restype = i32
    lib.sa_cross_attn_backward.argtypes = cross + [vp] * 8 + [sz, vp]
    lib.sa_page_tables.restype = i32
    lib.sa_page_tables.argtypes = [vp, vp, i32, i32, vp, i64, vp, vp, i32, i64, vp, vp, vp, vp, vp,
                                   sz, vp]
    lib.sa_paged_append.restype = i32
    lib.sa_paged_append.argtypes = [vp, i64, vp, i64, vp, i64, i32, i32, i32, vp, vp, vp, vp, i64,
                                    i32, vp]
    lib.sa_paged_attn_workspace_size.restype = sz
    lib.sa_paged_attn_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.sa_paged_attn.restype = i32
    lib.sa_paged_attn.argtypes = [vp, i64, i32, i32, i32, vp, vp, vp, vp, i32, i64, i32, i32, vp,
                                  i32, vp, i64, f32, vp, vp, vp, sz, vp]
    return lib


_lib = _load()


def _load_calls():
    """The usual calls of the attention with heads, in C++ (csrc/sa_calls.cpp): checks, allocations
    and the C ABI call in a third of the host time. They return None for any other call, which
    the functions below then check step by step and make themselves, as they make all of them
    where the extension is missing (None)."""
    path, name = calls_path(), f"{__package__}._calls"
    try:
        spec = importlib.util.spec_from_file_location(
            name, path, loader=importlib.machinery.ExtensionFileLoader(name, path))
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        return module
    except ImportError as e:
        if torch.version.cuda is not None:
            warnings.warn(f"no extension for the short calls ({e}): they take longer on the host; "
                          "run python -m prototype_sketch_attention_b200.build", RuntimeWarning)
        return None


_calls = _load_calls()


# ---------------------------------------------------------------- raw C ABI
def sa_sketch_workspace_size(R: int, n_total: int, k: int, d: int, dt: int, backward: int) -> int:
    return int(_lib.sa_sketch_workspace_size(R, n_total, k, d, dt, backward))


def sa_sketch_forward(X, offsets, R, n_total, d, P, k, Wk, Wv, dt, sketch, mass, lse, xsketch,
                      workspace, ws_bytes, stream) -> int:
    return int(_lib.sa_sketch_forward(X, offsets, R, n_total, d, P, k, Wk, Wv, dt, sketch, mass,
                                      lse, xsketch, workspace, ws_bytes, stream))


def sa_sketch_backward(X, offsets, R, n_total, d, P, k, Wk, Wv, dt, sketch, mass, lse, xsketch,
                       dsketch, dmass, dX, dP, dWk, dWv, workspace, ws_bytes, stream) -> int:
    return int(_lib.sa_sketch_backward(X, offsets, R, n_total, d, P, k, Wk, Wv, dt, sketch, mass,
                                       lse, xsketch, dsketch, dmass, dX, dP, dWk, dWv, workspace,
                                       ws_bytes, stream))


def sa_sketch_debug_gemm(A, a_mn, B, b_mn, M, N, K, splits, out, workspace, stream) -> int:
    return int(_lib.sa_sketch_debug_gemm(A, a_mn, B, b_mn, M, N, K, splits, out, workspace, stream))


def sa_sketch_combine(xsketch, mass, R, k, d, Wv, dt, sketch, stream) -> int:
    return int(_lib.sa_sketch_combine(xsketch, mass, R, k, d, Wv, dt, sketch, stream))


def sa_stca_workspace_size(R: int, n_cand: int, k: int, d: int, backward: int = 0) -> int:
    return int(_lib.sa_stca_workspace_size(R, n_cand, k, d, backward))


def sa_stca_backward(Q, cand_offsets, cand_offsets_host, R, n_cand, d, S, k, Wq, WK, WV, dout, dQ,
                     dS, dWq, dWK, dWV, workspace, ws_bytes, stream) -> int:
    return int(_lib.sa_stca_backward(Q, cand_offsets, cand_offsets_host, R, n_cand, d, S, k, Wq, WK,
                                     WV, dout, dQ, dS, dWq, dWK, dWV, workspace, ws_bytes, stream))


def sa_stca_forward(Q, cand_offsets, R, n_cand, d, S, k, Wq, WK, WV, out, lse, workspace,
                    ws_bytes, stream) -> int:
    return int(_lib.sa_stca_forward(Q, cand_offsets, R, n_cand, d, S, k, Wq, WK, WV, out, lse,
                                    workspace, ws_bytes, stream))


def sa_stca_keys_workspace_size(R: int, n_cand: int, d: int, backward: int = 0) -> int:
    return int(_lib.sa_stca_keys_workspace_size(R, n_cand, d, backward))


def sa_stca_keys_forward(Q, cand_offsets, R, n_cand, d, Kx, n_keys, key_begin, key_end, Wq, WK,
                         WV, out, lse, workspace, ws_bytes, stream) -> int:
    return int(_lib.sa_stca_keys_forward(Q, cand_offsets, R, n_cand, d, Kx, n_keys, key_begin,
                                         key_end, Wq, WK, WV, out, lse, workspace, ws_bytes,
                                         stream))


def sa_stca_keys_backward(Q, cand_offsets, R, n_cand, d, Kx, n_keys, key_begin, key_end, Wq, WK,
                          WV, dout, dQ, dKx, accumulate, dWq, dWK, dWV, workspace, ws_bytes,
                          stream) -> int:
    return int(_lib.sa_stca_keys_backward(Q, cand_offsets, R, n_cand, d, Kx, n_keys, key_begin,
                                          key_end, Wq, WK, WV, dout, dQ, dKx, int(accumulate),
                                          dWq, dWK, dWV, workspace, ws_bytes, stream))


def sa_stca_recent_ranges(offsets, R, L, key_begin, key_end, stream) -> int:
    return int(_lib.sa_stca_recent_ranges(offsets, R, L, key_begin, key_end, stream))


def sa_sketch_forward_host_buffer_size(R, n_total, k, d, dt, parts) -> int:
    return int(_lib.sa_sketch_forward_host_buffer_size(R, n_total, k, d, dt, parts))


def sa_sketch_forward_host(X_host, offsets_host, R, n_total, d, P, k, Wk, Wv, dt, sketch_host,
                           mass_host, device_buffer, device_bytes, parts, stream, h2d_stream,
                           d2h_stream) -> int:
    return int(_lib.sa_sketch_forward_host(X_host, offsets_host, R, n_total, d, P, k, Wk, Wv, dt,
                                           sketch_host, mass_host, device_buffer, device_bytes,
                                           parts, stream, h2d_stream, d2h_stream))


def sa_sketch_forward_host_status(device_buffer, R, n_total, k, d, dt, parts, stream) -> int:
    return int(_lib.sa_sketch_forward_host_status(device_buffer, R, n_total, k, d, dt, parts,
                                                  stream))


def sa_sketch_forward_grid(k, d, dt, clusters, cluster_size, helpers=None, helper_share=None) -> int:
    return int(_lib.sa_sketch_forward_grid(k, d, dt, clusters, cluster_size, helpers, helper_share))


def forward_grid(k: int, d: int, dtype=torch.bfloat16) -> tuple[int, int, int, int]:
    """(clusters, cluster_size, helpers, helper_share) of the bf16 forward on the current
    device: tile ranges as sa_sketch_forward_grid describes."""
    c, s, h, f = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    st = sa_sketch_forward_grid(k, d, SA_BF16 if dtype == torch.bfloat16 else SA_F32,
                                ctypes.addressof(c), ctypes.addressof(s), ctypes.addressof(h),
                                ctypes.addressof(f))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_sketch_forward_grid")
    return c.value, s.value, h.value, f.value


def sa_sketch_host_parts(offsets_host, R, parts, bounds) -> int:
    return int(_lib.sa_sketch_host_parts(offsets_host, R, parts, bounds))


def sa_sketch_pack(sketch, rows, d, fmt, codes, scales, stream) -> int:
    return int(_lib.sa_sketch_pack(sketch, rows, d, fmt, codes, scales, stream))


def sa_sketch_unpack(codes, scales, rows, d, fmt, sketch, stream) -> int:
    return int(_lib.sa_sketch_unpack(codes, scales, rows, d, fmt, sketch, stream))


def sketch_pack(S: torch.Tensor, fmt: int = SA_CODEC_FP8, stream=None) -> dict:
    """Packs fp32 sketches [..., d] (contiguous, CUDA) for the cache: codes (uint8 for
    fp8, bfloat16 for bf16) and, for fp8, one fp32 scale per row."""
    where = "sketch_pack"
    _require(isinstance(S, torch.Tensor) and S.dim() >= 2, where, "S must be [..., d]")
    d = S.shape[-1]
    rows = S.numel() // d if d else 0
    _check_tensor(where, "S", S, tuple(S.shape), torch.float32, S.device)
    _check_cuda(where, S)
    dt = torch.uint8 if fmt == SA_CODEC_FP8 else torch.bfloat16
    with _on(where, S.device, stream):
        out = {"codes": torch.empty(S.shape, dtype=dt, device=S.device),
               "scales": (torch.empty(S.shape[:-1], dtype=torch.float32, device=S.device)
                          if fmt == SA_CODEC_FP8 else None), "format": fmt}
        st = sa_sketch_pack(_ptr(S), rows, d, fmt, _ptr(out["codes"]), _ptr(out["scales"]),
                            _stream(stream, S.device))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_sketch_pack")
    _used_on(stream, S.device, S, out)
    return out


def sketch_unpack(packed: dict, stream=None) -> torch.Tensor:
    """The fp32 sketches back from sketch_pack's output."""
    where = "sketch_unpack"
    codes, fmt = packed["codes"], packed["format"]
    _require(fmt in (SA_CODEC_BF16, SA_CODEC_FP8), where, f"unknown format {fmt}")
    _require(isinstance(codes, torch.Tensor) and codes.dim() >= 2 and codes.shape[-1] > 0, where,
             "codes must be [..., d]")
    d, size = codes.shape[-1], 1 if fmt == SA_CODEC_FP8 else 2
    _require(codes.element_size() == size, where, f"{codes.dtype} codes; format {fmt} has {size} bytes a code")
    _check_tensor(where, "codes", codes, tuple(codes.shape), codes.dtype)
    scales = packed.get("scales") if fmt == SA_CODEC_FP8 else None
    if fmt == SA_CODEC_FP8:
        _check_tensor(where, "scales", scales, tuple(codes.shape[:-1]), torch.float32, codes.device)
    _check_cuda(where, codes)
    with _on(where, codes.device, stream):
        S = torch.empty(codes.shape, dtype=torch.float32, device=codes.device)
        st = sa_sketch_unpack(_ptr(codes), _ptr(scales), codes.numel() // d, d, fmt, _ptr(S),
                              _stream(stream, codes.device))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_sketch_unpack")
    _used_on(stream, codes.device, codes, scales, S)
    return S


def sa_cross_attn_workspace_size(R, n_q, n_kv, H, Hkv, d, backward) -> int:
    return int(_lib.sa_cross_attn_workspace_size(R, n_q, n_kv, H, Hkv, d, int(backward)))


def sa_cross_attn_forward(Q, q_stride, q_offsets, R, n_q, H, d, K, k_stride, V, v_stride,
                          kv_offsets, n_kv, Hkv, key_mask, scale, out, out_rest, lse, workspace,
                          ws_bytes, stream) -> int:
    return int(_lib.sa_cross_attn_forward(Q, q_stride, q_offsets, R, n_q, H, d, K, k_stride, V,
                                          v_stride, kv_offsets, n_kv, Hkv, key_mask, scale, out,
                                          out_rest, lse, workspace, ws_bytes, stream))


def sa_cross_attn_backward(Q, q_stride, q_offsets, R, n_q, H, d, K, k_stride, V, v_stride,
                           kv_offsets, n_kv, Hkv, key_mask, scale, out, out_rest, lse, dout, dQ,
                           dK, dV, workspace, ws_bytes, stream) -> int:
    return int(_lib.sa_cross_attn_backward(Q, q_stride, q_offsets, R, n_q, H, d, K, k_stride, V,
                                           v_stride, kv_offsets, n_kv, Hkv, key_mask, scale, out,
                                           out_rest, lse, dout, dQ, dK, dV, workspace, ws_bytes,
                                           stream))


def sa_page_tables(cached_lens, new_lens, R, page_size, free_pages, n_free, free_used, block_table,
                   max_pages, n_slots, slots, new_offsets, seq_lens, free_used_out, workspace,
                   ws_bytes, stream) -> int:
    return int(_lib.sa_page_tables(cached_lens, new_lens, R, page_size, free_pages, n_free,
                                   free_used, block_table, max_pages, n_slots, slots, new_offsets,
                                   seq_lens, free_used_out, workspace, ws_bytes, stream))


def sa_paged_append(K, k_stride, V, v_stride, slots, n, Hkv, d, fmt, k_cache, v_cache, k_scales,
                    v_scales, n_pages, page_size, stream) -> int:
    return int(_lib.sa_paged_append(K, k_stride, V, v_stride, slots, n, Hkv, d, fmt, k_cache,
                                    v_cache, k_scales, v_scales, n_pages, page_size, stream))


def sa_paged_attn_workspace_size(R, H, Hkv, d) -> int:
    return int(_lib.sa_paged_attn_workspace_size(R, H, Hkv, d))


def sa_paged_attn(Q, q_stride, R, H, d, k_cache, v_cache, k_scales, v_scales, fmt, n_pages,
                  page_size, Hkv, block_table, max_pages, seq_lens, window, scale, out, lse,
                  workspace, ws_bytes, stream) -> int:
    return int(_lib.sa_paged_attn(Q, q_stride, R, H, d, k_cache, v_cache, k_scales, v_scales, fmt,
                                  n_pages, page_size, Hkv, block_table, max_pages, seq_lens,
                                  window, scale, out, lse, workspace, ws_bytes, stream))


def sa_sketch_get_device_status(workspace, stream) -> int:
    return int(_lib.sa_sketch_get_device_status(workspace, stream))


def sa_status_string(status: int) -> str:
    return _lib.sa_status_string(int(status)).decode()


def sa_sketch_debug_wait_timeout(workspace, budget_cycles: int, stream) -> int:
    return int(_lib.sa_sketch_debug_wait_timeout(workspace, int(budget_cycles), stream))


def sa_sketch_forward_noalloc(X, offsets, R, n_total, d, P, k, Wk, Wv, dt, sketch, mass, lse,
                              xsketch, device_status, stream) -> int:
    """Forward without a workspace (see include/sa_sketch.h). `device_status` is a host
    pointer (ctypes) or None."""
    return int(_lib.sa_sketch_forward_noalloc(X, offsets, R, n_total, d, P, k, Wk, Wv, dt, sketch,
                                              mass, lse, xsketch, device_status, stream))


def sa_sketch_profile_events(start_event, stop_event) -> int:
    return int(_lib.sa_sketch_profile_events(start_event, stop_event))


# ---------------------------------------------------------------- torch conveniences
def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _dt(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return SA_BF16
    if x.dtype == torch.float32:
        return SA_F32
    raise TypeError(f"X must be bfloat16 or float32, got {x.dtype}")


# the current stream's handle without a Stream object around it (0.1 us in place of 2.3)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device=None) -> int:
    if stream is None and _raw_stream is not None and device is not None and device.index is not None:
        return _raw_stream(device.index)
    s = torch.cuda.current_stream(device) if stream is None else stream
    return s.cuda_stream


def _used_on(stream, dev, *args) -> None:
    """For a call on a given stream: its tensors (in tuples and dictionaries too) that are dropped
    early stay allocated until that stream has passed the call, and its results, which come from
    that stream's pool, until the caller's stream has passed what it does with them."""
    if stream is None:
        return
    here = torch.cuda.current_stream(dev)
    for x in args:
        if isinstance(x, torch.Tensor):
            x.record_stream(stream)  # (nothing, for a tensor of the stream's own pool)
            x.record_stream(here)
        elif isinstance(x, (tuple, list, dict)):
            _used_on(stream, dev, *(x.values() if isinstance(x, dict) else x))


def _fail(where: str, what: str):
    raise SketchAttentionError(SA_ERR_INVALID_ARG, f"{where}: {what}")


def _require(cond: bool, where: str, what: str) -> None:
    if not cond:
        _fail(where, what)


_HERE = contextlib.nullcontext()


def _device(dev: torch.device):
    """Makes `dev` current for a call; nothing to do when it is (the guard costs microseconds)."""
    return _HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


@contextlib.contextmanager
def _on(where: str, dev: torch.device, stream):
    """The device and, if one is given, the stream of a call, current while it allocates and launches.
    A block of another stream's pool may still be in use by work queued there, which the given
    stream does not wait for."""
    if stream is None:
        with _device(dev):
            yield
        return
    _require(stream.device == dev, where, f"stream is on {stream.device}, the inputs on {dev}")
    with torch.cuda.stream(stream):
        yield


def _check_tensor(where: str, name: str, t: torch.Tensor | None, shape: tuple, dtype,
                  device=None, optional: bool = False) -> None:
    """The C ABI sees only a pointer: shape, dtype, memory layout and device are the
    caller's promise, so the torch conveniences check them here."""
    if t is None:
        _require(optional, where, f"{name} is required")
        return
    # the usual case first: the messages below cost more than a small call
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype and t.is_contiguous()
            and (device is None or t.device == device)):
        return
    _require(isinstance(t, torch.Tensor), where, f"{name} must be a tensor")
    _require(tuple(t.shape) == tuple(shape), where,
             f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    _require(t.dtype == dtype, where, f"{name} has dtype {t.dtype}, expected {dtype}")
    _require(t.is_contiguous(), where, f"{name} must be contiguous")
    if device is not None:
        _require(t.device == device, where, f"{name} is on {t.device}, expected {device}")


def _check_cuda(where: str, X: torch.Tensor) -> None:
    if not X.is_cuda:
        _fail(where, f"inputs are on {X.device}; the library runs on CUDA devices only")


def _check_ws(where: str, ws, dev) -> None:
    """A workspace that the caller gives: the library sees its pointer and its size, so those bytes
    have to be there, on the inputs' device (their number is the library's to check)."""
    if ws is not None and not (isinstance(ws, torch.Tensor) and ws.device == dev and ws.is_contiguous()):
        _fail(where, f"ws must be a contiguous tensor on {dev}")


def _check_forward_inputs(where, X, offsets, P, Wk, Wv):
    _require(isinstance(X, torch.Tensor) and X.dim() == 2, where, "X must be a 2-D tensor")
    _require(isinstance(P, torch.Tensor) and P.dim() == 2, where, "P must be a 2-D tensor")
    _require(isinstance(offsets, torch.Tensor) and offsets.dim() == 1 and offsets.numel() >= 1,
             where, "offsets must be a 1-D tensor with R + 1 entries")
    n_total, d = X.shape
    k = P.shape[0]
    _dt(X)
    dev = X.device
    _check_tensor(where, "X", X, (n_total, d), X.dtype, dev)
    _check_tensor(where, "offsets", offsets, (offsets.numel(),), torch.int64, dev)
    _check_tensor(where, "P", P, (k, d), X.dtype, dev)
    _check_tensor(where, "Wk", Wk, (d, d), X.dtype, dev)
    _check_tensor(where, "Wv", Wv, (d, d), X.dtype, dev)


def workspace(R: int, n_total: int, k: int, d: int, dtype: torch.dtype, backward: bool = False,
              device=None) -> torch.Tensor:
    """A workspace tensor large enough for one call with these sizes."""
    dt = SA_BF16 if dtype == torch.bfloat16 else SA_F32
    n = sa_sketch_workspace_size(R, n_total, k, d, dt, int(backward))
    if n == 0:
        raise SketchAttentionError(SA_ERR_UNSUPPORTED, "sa_sketch_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def forward(X: torch.Tensor, offsets: torch.Tensor, P: torch.Tensor, Wk: torch.Tensor,
            Wv: torch.Tensor, *, want_lse: bool = True, want_xsketch: bool = True,
            ws: torch.Tensor | None = None, out: dict | None = None, stream=None) -> dict:
    """Sketch Attention forward on the GPU. Returns sketch, mass (and lse, xsketch).

    X [n_total, d] bf16/fp32, offsets [R+1] int64, P [k, d], Wk, Wv [d, d] (same dtype
    as X), all contiguous on one CUDA device. `out`, if given, holds fp32 sketch [R, k, d]
    and mass [R, k], and optionally lse [n_total] and xsketch [R, k, d].
    """
    where = "forward"
    _check_forward_inputs(where, X, offsets, P, Wk, Wv)
    n_total, d = X.shape
    k = P.shape[0]
    R = offsets.shape[0] - 1
    dt = _dt(X)
    dev = X.device
    f32 = torch.float32
    _check_ws(where, ws, dev)
    if out is not None:
        _check_tensor(where, "sketch", out.get("sketch"), (R, k, d), f32, dev)
        _check_tensor(where, "mass", out.get("mass"), (R, k), f32, dev)
        _check_tensor(where, "lse", out.get("lse"), (n_total,), f32, dev, optional=True)
        _check_tensor(where, "xsketch", out.get("xsketch"), (R, k, d), f32, dev, optional=True)
    _check_cuda(where, X)
    with _on(where, dev, stream):
        if out is None:
            out = {"sketch": torch.empty(R, k, d, device=dev, dtype=f32),
                   "mass": torch.empty(R, k, device=dev, dtype=f32)}
            if want_lse:
                out["lse"] = torch.empty(n_total, device=dev, dtype=f32)
            if want_xsketch:
                out["xsketch"] = torch.empty(R, k, d, device=dev, dtype=f32)
        if ws is None:
            ws = workspace(R, n_total, k, d, X.dtype, False, dev)
        st = sa_sketch_forward(_ptr(X), _ptr(offsets), R, n_total, d, _ptr(P), k, _ptr(Wk),
                               _ptr(Wv), dt, _ptr(out["sketch"]), _ptr(out["mass"]),
                               _ptr(out.get("lse")), _ptr(out.get("xsketch")), _ptr(ws),
                               ws.nbytes, _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_sketch_forward")
    out["_ws"] = ws
    _used_on(stream, dev, X, offsets, P, Wk, Wv, out)
    return out


def backward(X, offsets, P, Wk, Wv, fwd: dict, dsketch: torch.Tensor, dmass=None, *,
             ws: torch.Tensor | None = None, stream=None) -> dict:
    """Gradients dX, dP, dWk, dWv given dL/dsketch (and optionally dL/dmass).

    `fwd` holds the forward's fp32 sketch [R, k, d], mass [R, k] and xsketch [R, k, d]
    (lse [n_total] optional); dsketch [R, k, d] and dmass [R, k] are fp32."""
    where = "backward"
    _check_forward_inputs(where, X, offsets, P, Wk, Wv)
    n_total, d = X.shape
    k = P.shape[0]
    R = offsets.shape[0] - 1
    dt = _dt(X)
    dev = X.device
    f32 = torch.float32
    _check_tensor(where, "sketch", fwd.get("sketch"), (R, k, d), f32, dev)
    _check_tensor(where, "mass", fwd.get("mass"), (R, k), f32, dev)
    _check_tensor(where, "xsketch", fwd.get("xsketch"), (R, k, d), f32, dev)
    _check_tensor(where, "lse", fwd.get("lse"), (n_total,), f32, dev, optional=True)
    _check_tensor(where, "dsketch", dsketch, (R, k, d), f32, dev)
    _check_tensor(where, "dmass", dmass, (R, k), f32, dev, optional=True)
    _check_ws(where, ws, dev)
    _check_cuda(where, X)
    with _on(where, dev, stream):
        out = {"dX": torch.empty(n_total, d, device=dev, dtype=f32),
               "dP": torch.empty(k, d, device=dev, dtype=f32),
               "dWk": torch.empty(d, d, device=dev, dtype=f32),
               "dWv": torch.empty(d, d, device=dev, dtype=f32)}
        if ws is None:
            ws = workspace(R, n_total, k, d, X.dtype, True, dev)
        st = sa_sketch_backward(_ptr(X), _ptr(offsets), R, n_total, d, _ptr(P), k, _ptr(Wk),
                                _ptr(Wv), dt, _ptr(fwd["sketch"]), _ptr(fwd["mass"]),
                                _ptr(fwd.get("lse")), _ptr(fwd["xsketch"]), _ptr(dsketch),
                                _ptr(dmass), _ptr(out["dX"]), _ptr(out["dP"]), _ptr(out["dWk"]),
                                _ptr(out["dWv"]), _ptr(ws), ws.nbytes, _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_sketch_backward")
    out["_ws"] = ws
    _used_on(stream, dev, X, offsets, P, Wk, Wv, fwd, dsketch, dmass, out)
    return out


def combine(xsketch: torch.Tensor, mass: torch.Tensor, Wv: torch.Tensor, *,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """sketch = (xsketch Wv) / mass for users whose partial xsketch and mass (from
    forward calls over parts of their tokens) have been summed. xsketch [R, k, d] and
    mass [R, k] fp32, Wv [d, d] bf16/fp32, all on one CUDA device."""
    where = "combine"
    _require(isinstance(xsketch, torch.Tensor) and xsketch.dim() == 3, where,
             "xsketch must be a 3-D tensor")
    R, k, d = xsketch.shape
    dev = xsketch.device
    f32 = torch.float32
    _check_tensor(where, "xsketch", xsketch, (R, k, d), f32, dev)
    _check_tensor(where, "mass", mass, (R, k), f32, dev)
    _require(isinstance(Wv, torch.Tensor), where, "Wv must be a tensor")
    _check_tensor(where, "Wv", Wv, (d, d), Wv.dtype, dev)
    dt = _dt(Wv)
    _check_tensor(where, "out", out, (R, k, d), f32, dev, optional=True)
    _check_cuda(where, xsketch)
    with _on(where, dev, stream):
        if out is None:
            out = torch.empty(R, k, d, device=dev, dtype=f32)
        st = sa_sketch_combine(_ptr(xsketch), _ptr(mass), R, k, d, _ptr(Wv), dt, _ptr(out),
                               _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_sketch_combine")
    _used_on(stream, dev, xsketch, mass, Wv, out)
    return out


def stca_forward(Q: torch.Tensor, cand_offsets: torch.Tensor, S: torch.Tensor, Wq: torch.Tensor,
                 WK: torch.Tensor, WV: torch.Tensor, *, want_lse: bool = True,
                 ws: torch.Tensor | None = None, stream=None) -> dict:
    """Candidate-to-sketch cross attention on the GPU: every candidate of user u attends
    over the k rows of u's sketch. Q [n_cand, d] bf16, cand_offsets [R+1] int64,
    S [R, k, d] fp32 (the forward's sketch), Wq, WK, WV [d, d] bf16, all contiguous on one
    CUDA device. Returns out [n_cand, d] fp32 (and lse [n_cand])."""
    where = "stca_forward"
    _require(isinstance(Q, torch.Tensor) and Q.dim() == 2, where, "Q must be a 2-D tensor")
    _require(isinstance(S, torch.Tensor) and S.dim() == 3, where, "S must be a 3-D tensor")
    _require(isinstance(cand_offsets, torch.Tensor) and cand_offsets.dim() == 1
             and cand_offsets.numel() >= 1, where, "cand_offsets must be a 1-D tensor with R + 1 entries")
    n_cand, d = Q.shape
    R, k = cand_offsets.numel() - 1, S.shape[1]
    dev = Q.device
    bf = torch.bfloat16
    _check_tensor(where, "Q", Q, (n_cand, d), bf, dev)
    _check_tensor(where, "cand_offsets", cand_offsets, (R + 1,), torch.int64, dev)
    _check_tensor(where, "S", S, (R, k, d), torch.float32, dev)
    for name, W in (("Wq", Wq), ("WK", WK), ("WV", WV)):
        _check_tensor(where, name, W, (d, d), bf, dev)
    _check_ws(where, ws, dev)
    _check_cuda(where, Q)
    with _on(where, dev, stream):
        out = {"out": torch.empty(n_cand, d, device=dev, dtype=torch.float32)}
        if want_lse:
            out["lse"] = torch.empty(n_cand, device=dev, dtype=torch.float32)
        if ws is None:
            nb = sa_stca_workspace_size(R, n_cand, k, d, 0)
            if nb == 0:
                raise SketchAttentionError(SA_ERR_UNSUPPORTED, "sa_stca_workspace_size")
            ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        st = sa_stca_forward(_ptr(Q), _ptr(cand_offsets), R, n_cand, d, _ptr(S), k, _ptr(Wq),
                             _ptr(WK), _ptr(WV), _ptr(out["out"]), _ptr(out.get("lse")),
                             _ptr(ws), ws.nbytes, _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_stca_forward")
    out["_ws"] = ws
    _used_on(stream, dev, Q, cand_offsets, S, Wq, WK, WV, out)
    return out


def stca_backward(Q: torch.Tensor, cand_offsets: torch.Tensor, S: torch.Tensor, Wq: torch.Tensor,
                  WK: torch.Tensor, WV: torch.Tensor, dout: torch.Tensor, *,
                  cand_offsets_host: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None) -> dict:
    """Gradients of stca_forward given dL/dout [n_cand, d] fp32: dQ, dS (into each
    user's sketch), dWq, dWK, dWV. Inputs as for stca_forward; cand_offsets_host, a CPU
    copy of cand_offsets, saves the device-to-host copy (and lets the call be captured
    into a CUDA graph)."""
    where = "stca_backward"
    _require(isinstance(Q, torch.Tensor) and Q.dim() == 2, where, "Q must be a 2-D tensor")
    _require(isinstance(S, torch.Tensor) and S.dim() == 3, where, "S must be a 3-D tensor")
    _require(isinstance(cand_offsets, torch.Tensor) and cand_offsets.dim() == 1
             and cand_offsets.numel() >= 1, where, "cand_offsets must be a 1-D tensor with R + 1 entries")
    n_cand, d = Q.shape
    R, k = cand_offsets.numel() - 1, S.shape[1]
    dev = Q.device
    bf, f32 = torch.bfloat16, torch.float32
    _check_tensor(where, "Q", Q, (n_cand, d), bf, dev)
    _check_tensor(where, "cand_offsets", cand_offsets, (R + 1,), torch.int64, dev)
    _check_tensor(where, "S", S, (R, k, d), f32, dev)
    for name, W in (("Wq", Wq), ("WK", WK), ("WV", WV)):
        _check_tensor(where, name, W, (d, d), bf, dev)
    _check_tensor(where, "dout", dout, (n_cand, d), f32, dev)
    _check_ws(where, ws, dev)
    _check_cuda(where, Q)
    if cand_offsets_host is None:
        coff_h = cand_offsets.cpu().contiguous()
    else:
        _check_tensor(where, "cand_offsets_host", cand_offsets_host, (R + 1,), torch.int64,
                      torch.device("cpu"))
        coff_h = cand_offsets_host
    with _on(where, dev, stream):
        out = {"dQ": torch.empty(n_cand, d, device=dev, dtype=f32),
               "dS": torch.empty(R, k, d, device=dev, dtype=f32),
               "dWq": torch.empty(d, d, device=dev, dtype=f32),
               "dWK": torch.empty(d, d, device=dev, dtype=f32),
               "dWV": torch.empty(d, d, device=dev, dtype=f32)}
        if ws is None:
            nb = sa_stca_workspace_size(R, n_cand, k, d, 1)
            if nb == 0:
                raise SketchAttentionError(SA_ERR_UNSUPPORTED, "sa_stca_workspace_size")
            ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        st = sa_stca_backward(_ptr(Q), _ptr(cand_offsets), _ptr(coff_h), R, n_cand, d, _ptr(S), k,
                              _ptr(Wq), _ptr(WK), _ptr(WV), _ptr(dout), _ptr(out["dQ"]),
                              _ptr(out["dS"]), _ptr(out["dWq"]), _ptr(out["dWK"]),
                              _ptr(out["dWV"]), _ptr(ws), ws.nbytes, _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_stca_backward")
    out["_ws"] = ws
    _used_on(stream, dev, Q, cand_offsets, S, Wq, WK, WV, dout, out)
    return out


def recent_ranges(offsets: torch.Tensor, L: int, *, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The recent branch's key ranges over a history laid out by `offsets` [R+1] (int64,
    CUDA): each user's last min(n_u, L) rows. Returns (key_begin, key_end), int64 [R]."""
    where = "recent_ranges"
    _require(isinstance(offsets, torch.Tensor) and offsets.dim() == 1 and offsets.numel() >= 1,
             where, "offsets must be a 1-D tensor with R + 1 entries")
    R = offsets.numel() - 1
    dev = offsets.device
    _check_tensor(where, "offsets", offsets, (R + 1,), torch.int64, dev)
    _check_cuda(where, offsets)
    with _on(where, dev, stream):
        kb = torch.empty(R, dtype=torch.int64, device=dev)
        ke = torch.empty(R, dtype=torch.int64, device=dev)
        st = sa_stca_recent_ranges(_ptr(offsets), R, int(L), _ptr(kb), _ptr(ke),
                                   _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_stca_recent_ranges")
    _used_on(stream, dev, offsets, kb, ke)
    return kb, ke


def _check_keys_inputs(where, Q, cand_offsets, Kx, key_begin, key_end, Wq, WK, WV, ws):
    _require(isinstance(Q, torch.Tensor) and Q.dim() == 2, where, "Q must be a 2-D tensor")
    _require(isinstance(Kx, torch.Tensor) and Kx.dim() == 2, where, "Kx must be a 2-D tensor")
    _require(isinstance(cand_offsets, torch.Tensor) and cand_offsets.dim() == 1
             and cand_offsets.numel() >= 1, where, "cand_offsets must be a 1-D tensor with R + 1 entries")
    n_cand, d = Q.shape
    R = cand_offsets.numel() - 1
    dev = Q.device
    bf = torch.bfloat16
    _check_tensor(where, "Q", Q, (n_cand, d), bf, dev)
    _check_tensor(where, "Kx", Kx, (Kx.shape[0], d), bf, dev)
    _check_tensor(where, "cand_offsets", cand_offsets, (R + 1,), torch.int64, dev)
    _check_tensor(where, "key_begin", key_begin, (R,), torch.int64, dev)
    _check_tensor(where, "key_end", key_end, (R,), torch.int64, dev)
    for name, W in (("Wq", Wq), ("WK", WK), ("WV", WV)):
        _check_tensor(where, name, W, (d, d), bf, dev)
    _check_ws(where, ws, dev)
    _check_cuda(where, Q)
    return n_cand, d, R, Kx.shape[0], dev


def stca_keys_forward(Q: torch.Tensor, cand_offsets: torch.Tensor, Kx: torch.Tensor,
                      key_begin: torch.Tensor, key_end: torch.Tensor, Wq: torch.Tensor,
                      WK: torch.Tensor, WV: torch.Tensor, *, want_lse: bool = True,
                      ws: torch.Tensor | None = None, stream=None) -> dict:
    """Cross attention from user u's candidates to the key rows Kx[key_begin[u]:key_end[u]]
    (the recent branch: Kx = the history X, ranges from recent_ranges). Q [n_cand, d] bf16,
    cand_offsets [R+1] int64, Kx [n_keys, d] bf16, key_begin / key_end [R] int64,
    Wq, WK, WV [d, d] bf16, all on one CUDA device. Returns out [n_cand, d] fp32 (and
    lse [n_cand])."""
    where = "stca_keys_forward"
    n_cand, d, R, n_keys, dev = _check_keys_inputs(where, Q, cand_offsets, Kx, key_begin, key_end,
                                                   Wq, WK, WV, ws)
    with _on(where, dev, stream):
        out = {"out": torch.empty(n_cand, d, device=dev, dtype=torch.float32)}
        if want_lse:
            out["lse"] = torch.empty(n_cand, device=dev, dtype=torch.float32)
        if ws is None:
            nb = sa_stca_keys_workspace_size(R, n_cand, d, 0)
            if nb == 0:
                raise SketchAttentionError(SA_ERR_UNSUPPORTED, "sa_stca_keys_workspace_size")
            ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        st = sa_stca_keys_forward(_ptr(Q), _ptr(cand_offsets), R, n_cand, d, _ptr(Kx), n_keys,
                                  _ptr(key_begin), _ptr(key_end), _ptr(Wq), _ptr(WK), _ptr(WV),
                                  _ptr(out["out"]), _ptr(out.get("lse")), _ptr(ws), ws.nbytes,
                                  _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_stca_keys_forward")
    out["_ws"] = ws
    _used_on(stream, dev, Q, cand_offsets, Kx, key_begin, key_end, Wq, WK, WV, out)
    return out


def stca_keys_backward(Q: torch.Tensor, cand_offsets: torch.Tensor, Kx: torch.Tensor,
                       key_begin: torch.Tensor, key_end: torch.Tensor, Wq: torch.Tensor,
                       WK: torch.Tensor, WV: torch.Tensor, dout: torch.Tensor, *,
                       dKx: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                       stream=None) -> dict:
    """Gradients of stca_keys_forward given dL/dout [n_cand, d] fp32: dQ, dKx [n_keys, d]
    (into the key rows), dWq, dWK, dWV. Inputs as for stca_keys_forward. With dKx given
    (fp32 [n_keys, d]), the key rows' gradient is added into it instead of a new tensor
    (for the recent branch: into the history gradient)."""
    where = "stca_keys_backward"
    n_cand, d, R, n_keys, dev = _check_keys_inputs(where, Q, cand_offsets, Kx, key_begin, key_end,
                                                   Wq, WK, WV, ws)
    f32 = torch.float32
    _check_tensor(where, "dout", dout, (n_cand, d), f32, dev)
    _check_tensor(where, "dKx", dKx, (n_keys, d), f32, dev, optional=True)
    accumulate = dKx is not None
    with _on(where, dev, stream):
        out = {"dQ": torch.empty(n_cand, d, device=dev, dtype=f32),
               "dKx": dKx if accumulate else torch.empty(n_keys, d, device=dev, dtype=f32),
               "dWq": torch.empty(d, d, device=dev, dtype=f32),
               "dWK": torch.empty(d, d, device=dev, dtype=f32),
               "dWV": torch.empty(d, d, device=dev, dtype=f32)}
        if ws is None:
            nb = sa_stca_keys_workspace_size(R, n_cand, d, 1)
            if nb == 0:
                raise SketchAttentionError(SA_ERR_UNSUPPORTED, "sa_stca_keys_workspace_size")
            ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        st = sa_stca_keys_backward(_ptr(Q), _ptr(cand_offsets), R, n_cand, d, _ptr(Kx), n_keys,
                                   _ptr(key_begin), _ptr(key_end), _ptr(Wq), _ptr(WK), _ptr(WV),
                                   _ptr(dout), _ptr(out["dQ"]), _ptr(out["dKx"]), accumulate,
                                   _ptr(out["dWq"]), _ptr(out["dWK"]), _ptr(out["dWV"]),
                                   _ptr(ws), ws.nbytes, _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_stca_keys_backward")
    out["_ws"] = ws
    _used_on(stream, dev, Q, cand_offsets, Kx, key_begin, key_end, Wq, WK, WV, dout, out)
    return out


def _rows_stride(where: str, name: str, x: torch.Tensor, heads: int, d: int) -> int:
    """Elements between consecutive rows of x [n, heads, d], whose heads are contiguous (a
    slice of a wider projection is fine)."""
    s0, s1, s2 = x.stride()
    if s2 != 1 or (s1 != d and heads != 1):
        _fail(where, f"{name}: a row's heads must be contiguous")
    return s0 if x.shape[0] > 1 else heads * d


def _check_heads(where: str, name: str, x, n, d, dev, heads=None) -> None:
    if not (isinstance(x, torch.Tensor) and x.dim() == 3):
        _fail(where, f"{name} must be [n, heads, d]")
    if x.dtype != torch.bfloat16:
        _fail(where, f"{name} has dtype {x.dtype}, expected torch.bfloat16")
    want = (n, x.shape[1] if heads is None else heads, d)
    if x.shape != want:
        _fail(where, f"{name} has shape {tuple(x.shape)}, expected {want}")
    if x.device != dev:
        _fail(where, f"{name} is on {x.device}, expected {dev}")


def _result(res, call: str) -> dict:
    """What _calls returned: a dictionary, or the status of a refused call."""
    if type(res) is dict:
        return res
    raise SketchAttentionError(res, call)


def _scale(scale, d: int) -> float:
    return float(d) ** -0.5 if scale is None else float(scale)


def _check_cross(where, Q, q_offsets, K, V, kv_offsets, key_mask, ws):
    _require(isinstance(Q, torch.Tensor) and Q.dim() == 3, where, "Q must be [n, heads, d]")
    _require(isinstance(K, torch.Tensor) and K.dim() == 3, where, "K must be [n, heads, d]")
    dev, (n_q, H, d), (n_kv, Hkv, _) = Q.device, Q.shape, K.shape
    _check_heads(where, "Q", Q, n_q, d, dev)
    _check_heads(where, "K", K, n_kv, d, dev)
    _check_heads(where, "V", V, n_kv, d, dev, Hkv)
    if Hkv < 1 or H < 1 or H % Hkv:
        _fail(where, f"{H} query heads cannot share {Hkv} key heads")
    _require(isinstance(q_offsets, torch.Tensor) and q_offsets.dim() == 1
             and q_offsets.numel() >= 1, where, "q_offsets must be a 1-D tensor with R + 1 entries")
    R = q_offsets.numel() - 1
    _check_tensor(where, "q_offsets", q_offsets, (R + 1,), torch.int64, dev)
    _check_tensor(where, "kv_offsets", kv_offsets, (R + 1,), torch.int64, dev)
    if key_mask is not None:
        _require(isinstance(key_mask, torch.Tensor) and key_mask.dtype in (torch.bool, torch.uint8),
                 where, "key_mask must be a bool or uint8 tensor")
        _check_tensor(where, "key_mask", key_mask, (n_kv,), key_mask.dtype, dev)
    _check_ws(where, ws, dev)
    _check_cuda(where, Q)
    strides = (_rows_stride(where, "Q", Q, H, d), _rows_stride(where, "K", K, Hkv, d),
               _rows_stride(where, "V", V, Hkv, d))
    return R, n_q, H, d, n_kv, Hkv, dev, strides


def cross_attention(Q: torch.Tensor, q_offsets: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
                    kv_offsets: torch.Tensor, *, key_mask: torch.Tensor | None = None,
                    scale: float | None = None, want_rest: bool = True, out: dict | None = None,
                    ws: torch.Tensor | None = None, stream=None) -> dict:
    """Multi-head cross attention from user u's query rows Q[q_offsets[u]:q_offsets[u+1]] to its
    key rows K, V[kv_offsets[u]:kv_offsets[u+1]] (sa_cross_attn_forward). Q [n_q, H, d], K and V
    [n_kv, Hkv, d] bf16 (rows may be strided, a row's heads contiguous), offsets [R + 1] int64,
    key_mask [n_kv] bool (False drops a key row), scale 1 / sqrt(d) by default. Returns out
    [n_q, H, d] bf16, lse [n_q, H] fp32 and, for the backward, what rounding took from out (rest,
    like out; want_rest=False leaves it away). They are written into `out` ({"out", "lse"} and,
    if wanted, "rest") when given."""
    if _calls is not None and out is None and stream is None:
        res = _calls.cross_forward(Q, q_offsets, K, V, kv_offsets, key_mask, scale, bool(want_rest), ws)
        if res is not None:
            return _result(res, "sa_cross_attn_forward")
    where = "cross_attention"
    R, n_q, H, d, n_kv, Hkv, dev, (qs, ks, vs) = _check_cross(where, Q, q_offsets, K, V, kv_offsets,
                                                              key_mask, ws)
    if out is not None:
        out = dict(out)
        _check_tensor(where, "out", out.get("out"), (n_q, H, d), torch.bfloat16, dev)
        _check_tensor(where, "rest", out.get("rest"), (n_q, H, d), torch.bfloat16, dev, optional=True)
        _check_tensor(where, "lse", out.get("lse"), (n_q, H), torch.float32, dev)
    with _on(where, dev, stream):
        if out is None:
            out = {"out": torch.empty(n_q, H, d, device=dev, dtype=torch.bfloat16),
                   "lse": torch.empty(n_q, H, device=dev, dtype=torch.float32)}
            if want_rest:
                out["rest"] = torch.empty(n_q, H, d, device=dev, dtype=torch.bfloat16)
        if ws is None:
            nb = sa_cross_attn_workspace_size(R, n_q, n_kv, H, Hkv, d, 0)
            if nb == 0:
                raise SketchAttentionError(SA_ERR_UNSUPPORTED, "sa_cross_attn_workspace_size")
            ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        st = sa_cross_attn_forward(_ptr(Q), qs, _ptr(q_offsets), R, n_q, H, d, _ptr(K), ks, _ptr(V),
                                   vs, _ptr(kv_offsets), n_kv, Hkv, _ptr(key_mask),
                                   _scale(scale, d), _ptr(out["out"]), _ptr(out.get("rest")),
                                   _ptr(out["lse"]), _ptr(ws), ws.nbytes, _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_cross_attn_forward")
    out["_ws"] = ws
    _used_on(stream, dev, Q, q_offsets, K, V, kv_offsets, key_mask, out)
    return out


def cross_attention_backward(Q: torch.Tensor, q_offsets: torch.Tensor, K: torch.Tensor,
                             V: torch.Tensor, kv_offsets: torch.Tensor, fwd: dict,
                             dout: torch.Tensor, *, key_mask: torch.Tensor | None = None,
                             scale: float | None = None, out: dict | None = None,
                             ws: torch.Tensor | None = None, stream=None) -> dict:
    """Gradients of cross_attention given its outputs `fwd` (out, lse, rest if it has one) and dout = dL/dout
    [n_q, H, d] bf16: dQ [n_q, H, d], dK and dV [n_kv, Hkv, d], bf16 (sa_cross_attn_backward),
    written into `out` ({"dQ", "dK", "dV"}) when given. Other arguments as passed to the
    forward."""
    if _calls is not None and out is None and stream is None:
        res = _calls.cross_backward(Q, q_offsets, K, V, kv_offsets, key_mask, scale, fwd.get("out"),
                                    fwd.get("lse"), fwd.get("rest"), dout, ws)
        if res is not None:
            return _result(res, "sa_cross_attn_backward")
    where = "cross_attention_backward"
    R, n_q, H, d, n_kv, Hkv, dev, (qs, ks, vs) = _check_cross(where, Q, q_offsets, K, V, kv_offsets,
                                                              key_mask, ws)
    bf = torch.bfloat16
    _check_tensor(where, "out", fwd.get("out"), (n_q, H, d), bf, dev)
    _check_tensor(where, "lse", fwd.get("lse"), (n_q, H), torch.float32, dev)
    _check_tensor(where, "rest", fwd.get("rest"), (n_q, H, d), bf, dev, optional=True)
    _check_tensor(where, "dout", dout, (n_q, H, d), bf, dev)
    if out is not None:
        out = dict(out)
        _check_tensor(where, "dQ", out.get("dQ"), (n_q, H, d), bf, dev)
        _check_tensor(where, "dK", out.get("dK"), (n_kv, Hkv, d), bf, dev)
        _check_tensor(where, "dV", out.get("dV"), (n_kv, Hkv, d), bf, dev)
    with _on(where, dev, stream):
        if out is None:
            out = {"dQ": torch.empty(n_q, H, d, device=dev, dtype=bf),
                   "dK": torch.empty(n_kv, Hkv, d, device=dev, dtype=bf),
                   "dV": torch.empty(n_kv, Hkv, d, device=dev, dtype=bf)}
        if ws is None:
            nb = sa_cross_attn_workspace_size(R, n_q, n_kv, H, Hkv, d, 1)
            if nb == 0:
                raise SketchAttentionError(SA_ERR_UNSUPPORTED, "sa_cross_attn_workspace_size")
            ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        st = sa_cross_attn_backward(_ptr(Q), qs, _ptr(q_offsets), R, n_q, H, d, _ptr(K), ks,
                                    _ptr(V), vs, _ptr(kv_offsets), n_kv, Hkv, _ptr(key_mask),
                                    _scale(scale, d), _ptr(fwd["out"]), _ptr(fwd.get("rest")),
                                    _ptr(fwd["lse"]), _ptr(dout), _ptr(out["dQ"]), _ptr(out["dK"]), _ptr(out["dV"]),
                                    _ptr(ws), ws.nbytes, _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_cross_attn_backward")
    out["_ws"] = ws
    _used_on(stream, dev, Q, q_offsets, K, V, kv_offsets, key_mask, fwd, dout, out)
    return out


def paged_cache(n_pages: int, Hkv: int, page_size: int, d: int, *, fmt: int = SA_CODEC_BF16,
                device="cuda") -> dict:
    """A paged key-value cache: K and V [n_pages, Hkv, page_size, d] (bfloat16, or
    float8_e4m3fn with k_scales and v_scales [n_pages, Hkv, page_size] fp32). The rows start
    unwritten."""
    where = "paged_cache"
    _require(fmt in (SA_CODEC_BF16, SA_CODEC_FP8), where, f"unknown format {fmt}")
    shape = (int(n_pages), int(Hkv), int(page_size), int(d))
    _require(min(shape) >= 0, where, f"negative size in {shape}")
    kind = torch.float8_e4m3fn if fmt == SA_CODEC_FP8 else torch.bfloat16
    cache = {n: torch.empty(shape, dtype=kind, device=device) for n in ("K", "V")}
    for n in ("k_scales", "v_scales"):
        cache[n] = (torch.empty(shape[:3], dtype=torch.float32, device=device)
                    if fmt == SA_CODEC_FP8 else None)
    return cache


def _check_cache(where: str, cache: dict, dev) -> tuple[int, int, int, int, int]:
    """(format, n_pages, Hkv, page_size, d) of a paged_cache."""
    K = cache.get("K") if isinstance(cache, dict) else None
    _require(isinstance(K, torch.Tensor) and K.dim() == 4, where,
             "cache must hold K [n_pages, Hkv, page_size, d]")
    fp8 = K.dtype == torch.float8_e4m3fn
    if not fp8 and K.dtype != torch.bfloat16:
        _fail(where, f"cache K has dtype {K.dtype}, expected torch.bfloat16 or torch.float8_e4m3fn")
    shape = tuple(K.shape)
    _check_tensor(where, "cache K", K, shape, K.dtype, dev)
    _check_tensor(where, "cache V", cache.get("V"), shape, K.dtype, dev)
    for n, name in (("k_scales", "cache k_scales"), ("v_scales", "cache v_scales")):
        if fp8:
            _check_tensor(where, name, cache.get(n), shape[:3], torch.float32, dev)
        elif cache.get(n) is not None:
            _fail(where, f"{name} belongs to an FP8 cache")
    return (SA_CODEC_FP8 if fp8 else SA_CODEC_BF16, *shape)


def page_tables(cached_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                block_table: torch.Tensor, page_size: int, n_slots: int, *,
                free_used: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                stream=None) -> dict:
    """Pages and slots for new_lens [R] new positions of requests that hold cached_lens [R]
    (int32; sa_page_tables): takes pages from free_pages (int32), from entry free_used (int64
    [1]; None: 0) on, and writes them into block_table [R, max_pages] (int32) in place. n_slots:
    room for the new positions (their number, or more: the rest is -1). Returns slots [n_slots]
    and new_offsets [R + 1] int64, seq_lens [R] int32, free_used [1] int64. Too few pages and
    the like are latched in the device status (device_status(result["_ws"])) and change
    nothing."""
    if _calls is not None and stream is None:
        res = _calls.page_tables(cached_lens, new_lens, free_pages, block_table, page_size, n_slots,
                                 free_used, ws)
        if res is not None:
            return _result(res, "sa_page_tables")
    where = "page_tables"
    _require(isinstance(cached_lens, torch.Tensor) and cached_lens.dim() == 1, where,
             "cached_lens must be a 1-D tensor")
    R, dev = cached_lens.numel(), cached_lens.device
    i32, i64 = torch.int32, torch.int64
    _check_tensor(where, "cached_lens", cached_lens, (R,), i32, dev)
    _check_tensor(where, "new_lens", new_lens, (R,), i32, dev)
    _require(isinstance(free_pages, torch.Tensor) and free_pages.dim() == 1, where,
             "free_pages must be a 1-D tensor")
    _check_tensor(where, "free_pages", free_pages, (free_pages.numel(),), i32, dev)
    _require(isinstance(block_table, torch.Tensor) and block_table.dim() == 2, where,
             "block_table must be [R, max_pages]")
    _check_tensor(where, "block_table", block_table, (R, block_table.shape[1]), i32, dev)
    _check_tensor(where, "free_used", free_used, (1,), i64, dev, optional=True)
    _check_ws(where, ws, dev)
    _check_cuda(where, cached_lens)
    _require(int(n_slots) >= 0, where, "n_slots must not be negative")
    with _on(where, dev, stream):
        out = {"slots": torch.empty(int(n_slots), dtype=i64, device=dev),
               "new_offsets": torch.empty(R + 1, dtype=i64, device=dev),
               "seq_lens": torch.empty(R, dtype=i32, device=dev),
               "free_used": torch.empty(1, dtype=i64, device=dev)}
        if ws is None:
            ws = torch.empty(256, dtype=torch.uint8, device=dev)
        st = sa_page_tables(_ptr(cached_lens), _ptr(new_lens), R, int(page_size), _ptr(free_pages),
                            free_pages.numel(), _ptr(free_used), _ptr(block_table),
                            block_table.shape[1], int(n_slots), _ptr(out["slots"]),
                            _ptr(out["new_offsets"]), _ptr(out["seq_lens"]), _ptr(out["free_used"]),
                            _ptr(ws), ws.nbytes, _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_page_tables")
    out["_ws"] = ws
    _used_on(stream, dev, cached_lens, new_lens, free_pages, block_table, free_used, out)
    return out


def paged_append(K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, cache: dict, *,
                 stream=None) -> None:
    """Writes rows K, V [n, Hkv, d] bf16 (rows may be strided) into the slots [n] int64 of a
    paged_cache, quantised for an FP8 cache (sa_paged_append). Slots outside the cache, such as
    the -1 of page_tables, are skipped; a slot must not be named twice."""
    if _calls is not None and stream is None and isinstance(cache, dict):
        res = _calls.paged_append(K, V, slots, cache.get("K"), cache.get("V"), cache.get("k_scales"),
                                  cache.get("v_scales"))
        if res == SA_OK:
            return
        if res is not None:
            raise SketchAttentionError(res, "sa_paged_append")
    where = "paged_append"
    _require(isinstance(K, torch.Tensor) and K.dim() == 3, where, "K must be [n, heads, d]")
    dev = K.device
    fmt, n_pages, Hkv, page_size, d = _check_cache(where, cache, dev)
    _check_heads(where, "K", K, K.shape[0], d, dev, Hkv)
    _check_heads(where, "V", V, K.shape[0], d, dev, Hkv)
    _check_tensor(where, "slots", slots, (K.shape[0],), torch.int64, dev)
    _check_cuda(where, K)
    ks, vs = _rows_stride(where, "K", K, Hkv, d), _rows_stride(where, "V", V, Hkv, d)
    with _on(where, dev, stream):
        st = sa_paged_append(_ptr(K), ks, _ptr(V), vs, _ptr(slots), K.shape[0], Hkv, d, fmt,
                             _ptr(cache["K"]), _ptr(cache["V"]), _ptr(cache.get("k_scales")),
                             _ptr(cache.get("v_scales")), n_pages, page_size, _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_paged_append")
    _used_on(stream, dev, K, V, slots, cache)


def paged_attention(Q: torch.Tensor, cache: dict, block_table: torch.Tensor,
                    seq_lens: torch.Tensor, *, window: int = 0, scale: float | None = None,
                    ws: torch.Tensor | None = None, stream=None) -> dict:
    """Attention of one new token per request, Q [R, H, d] bf16, over the last `window`
    positions (0: all) of its seq_lens [R] int32 in a paged_cache, through block_table
    [R, max_pages] int32 (sa_paged_attn). Returns out [R, H, d] bf16 and lse [R, H] fp32. Bad
    lengths and page ids are latched in the device status (device_status(result["_ws"]))."""
    if _calls is not None and stream is None and isinstance(cache, dict):
        res = _calls.paged_attention(Q, cache.get("K"), cache.get("V"), cache.get("k_scales"),
                                     cache.get("v_scales"), block_table, seq_lens, window, scale, ws)
        if res is not None:
            return _result(res, "sa_paged_attn")
    where = "paged_attention"
    _require(isinstance(Q, torch.Tensor) and Q.dim() == 3, where, "Q must be [n, heads, d]")
    dev, (R, H, d) = Q.device, Q.shape
    fmt, n_pages, Hkv, page_size, cd = _check_cache(where, cache, dev)
    _check_heads(where, "Q", Q, R, cd, dev)
    if Hkv < 1 or H < 1 or H % Hkv:
        _fail(where, f"{H} query heads cannot share {Hkv} key heads")
    _require(isinstance(block_table, torch.Tensor) and block_table.dim() == 2, where,
             "block_table must be [R, max_pages]")
    _check_tensor(where, "block_table", block_table, (R, block_table.shape[1]), torch.int32, dev)
    _check_tensor(where, "seq_lens", seq_lens, (R,), torch.int32, dev)
    _check_ws(where, ws, dev)
    _check_cuda(where, Q)
    qs = _rows_stride(where, "Q", Q, H, d)
    with _on(where, dev, stream):
        out = {"out": torch.empty(R, H, d, device=dev, dtype=torch.bfloat16),
               "lse": torch.empty(R, H, device=dev, dtype=torch.float32)}
        if ws is None:
            nb = sa_paged_attn_workspace_size(R, H, Hkv, d)
            if nb == 0:
                raise SketchAttentionError(SA_ERR_UNSUPPORTED, "sa_paged_attn_workspace_size")
            ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        st = sa_paged_attn(_ptr(Q), qs, R, H, d, _ptr(cache["K"]), _ptr(cache["V"]),
                           _ptr(cache.get("k_scales")), _ptr(cache.get("v_scales")), fmt, n_pages,
                           page_size, Hkv, _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
                           int(window), _scale(scale, d), _ptr(out["out"]), _ptr(out["lse"]),
                           _ptr(ws), ws.nbytes, _stream(stream, dev))
    if st != SA_OK:
        raise SketchAttentionError(st, "sa_paged_attn")
    out["_ws"] = ws
    _used_on(stream, dev, Q, cache, block_table, seq_lens, out)
    return out


def user_chunks(offsets_host: torch.Tensor, chunks: int) -> list[tuple[int, int]]:
    """The library's cut of users [0, R) into at most `chunks` consecutive parts of about
    equal token count (sa_sketch_host_parts). offsets_host: int64 [R + 1] on the host."""
    _require(isinstance(offsets_host, torch.Tensor) and offsets_host.dtype == torch.int64
             and offsets_host.device.type == "cpu" and offsets_host.dim() == 1,
             "user_chunks", "offsets_host must be a host int64 [R + 1] tensor")
    off = offsets_host.contiguous()
    R = off.numel() - 1
    bounds = (ctypes.c_int * (max(int(chunks), 1) + 1))()
    np_ = sa_sketch_host_parts(off.data_ptr(), R, int(chunks), ctypes.addressof(bounds))
    if np_ < 0:
        raise SketchAttentionError(-np_, "sa_sketch_host_parts")
    return [(bounds[i], bounds[i + 1]) for i in range(np_)]


def forward_from_host(Xh: torch.Tensor, offsets_h: torch.Tensor, P: torch.Tensor,
                      Wk: torch.Tensor, Wv: torch.Tensor, *, chunks: int = 4,
                      state: dict | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Forward from host X and offsets to host sketch and mass through
    sa_sketch_forward_host, which cuts the users into `chunks` parts and overlaps each
    part's copy to the device with the previous part's forward (the library owns the
    pipeline; this function only marshals). Xh and offsets_h should be pinned. P, Wk, Wv
    live on the device. `state` (a dict the caller keeps) holds the device buffer, the
    pinned outputs and the two copy streams between calls. The outputs are complete once
    the current stream reaches the end of this call's work; the returned host tensors are
    the state's staging, which the next call with the same `state` overwrites."""
    where = "forward_from_host"
    _require(isinstance(Xh, torch.Tensor) and Xh.dim() == 2 and Xh.device.type == "cpu"
             and Xh.is_contiguous(), where, "Xh must be a contiguous 2-D host tensor")
    _require(isinstance(offsets_h, torch.Tensor) and offsets_h.dim() == 1
             and offsets_h.numel() >= 1 and offsets_h.dtype == torch.int64
             and offsets_h.device.type == "cpu", where, "offsets_h must be host int64 [R + 1]")
    _require(isinstance(P, torch.Tensor) and P.is_cuda, where, "P, Wk, Wv must be on the GPU")
    _require(int(chunks) >= 1, where, "chunks must be at least 1")
    R = offsets_h.numel() - 1
    n_total, d = Xh.shape
    k = P.shape[0]
    dev = P.device
    dt = _dt(Xh)
    _check_tensor(where, "P", P, (k, d), Xh.dtype, dev)
    _check_tensor(where, "Wk", Wk, (d, d), Xh.dtype, dev)
    _check_tensor(where, "Wv", Wv, (d, d), Xh.dtype, dev)
    st = {} if state is None else state
    key = (R, n_total, k, d, Xh.dtype, int(chunks), dev)
    if st.get("key") != key:
        st.clear()
        with torch.cuda.device(dev):
            nb = sa_sketch_forward_host_buffer_size(R, n_total, k, d, dt, int(chunks))
            if nb == 0:
                raise SketchAttentionError(SA_ERR_UNSUPPORTED, "sa_sketch_forward_host_buffer_size")
            st.update(key=key, buf=torch.empty(nb, dtype=torch.uint8, device=dev),
                      sk_h=torch.empty(R, k, d, dtype=torch.float32).pin_memory(),
                      ms_h=torch.empty(R, k, dtype=torch.float32).pin_memory(),
                      s_h2d=torch.cuda.Stream(dev), s_d2h=torch.cuda.Stream(dev))
    off = offsets_h.contiguous()
    cur = torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        rc = sa_sketch_forward_host(_ptr(Xh), off.data_ptr(), R, n_total, d, _ptr(P), k, _ptr(Wk),
                                    _ptr(Wv), dt, _ptr(st["sk_h"]), _ptr(st["ms_h"]),
                                    _ptr(st["buf"]), st["buf"].nbytes, int(chunks),
                                    cur.cuda_stream, st["s_h2d"].cuda_stream,
                                    st["s_d2h"].cuda_stream)
    if rc != SA_OK:
        raise SketchAttentionError(rc, "sa_sketch_forward_host")
    return st["sk_h"], st["ms_h"]


def forward_from_host_status(state: dict, stream=None) -> int:
    """Device status of the last forward_from_host call made with `state` (synchronises)."""
    R, n_total, k, d, dtype, chunks, dev = state["key"]
    return sa_sketch_forward_host_status(_ptr(state["buf"]), R, n_total, k, d,
                                         SA_BF16 if dtype == torch.bfloat16 else SA_F32, chunks,
                                         _stream(stream, dev))


def device_status(ws: torch.Tensor, stream=None) -> int:
    return sa_sketch_get_device_status(_ptr(ws), _stream(stream))
