"""GB300-native OSCAR INT2 rotated paged KV cache: Python binding of liboscar.so.

The compute path is the CUDA library built from ``csrc/`` (see include/oscar.h
for the C ABI).  This module only marshals arguments: it exposes every C entry
point under the same name, raises :class:`OscarError` on a non-zero status, and
offers ``ptr()`` / ``stream_ptr()`` helpers for torch tensors and streams.
There is no fallback: importing the binding without a built library, or calling
a kernel entry point without a GPU, fails loudly.
"""
from __future__ import annotations

import array
import ctypes
import os
from typing import Optional, Sequence

from . import calibrate  # noqa: F401  (offline calibration tooling)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liboscar.so")

OK, ERR_INVALID, ERR_OOM, ERR_CUDA, ERR_DEVICE, ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5
DTYPE_F32, DTYPE_BF16 = 0, 1
DECODE_AUTO, DECODE_THREE_KERNELS, DECODE_ONE_LAUNCH = 0, 1, 2
DEV_BAD_PAGE, DEV_TIMEOUT, DEV_BAD_LEN, DEV_BAD_SLOT, DEV_BAD_VALUE = 1, 2, 4, 8, 16
KV8_INT8, KV8_E4M3 = 0, 1


class OscarError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"oscar status {status}: {message}")
        self.status = status


class oscar_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_layers", "n_q_heads", "n_kv_heads", "head_dim", "page_size", "group_size", "sink", "recent",
        "max_requests", "max_pages_per_req", "num_pages", "rotation_per_kv_head")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


def make_config(**kw) -> oscar_config:
    c = oscar_config()
    c.group_size = 32
    for k, v in kw.items():
        setattr(c, k, int(v))
    return c


_c_i32p = ctypes.POINTER(ctypes.c_int32)
_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_f32 = ctypes.c_float
_i64 = ctypes.c_int64
_szp = ctypes.POINTER(ctypes.c_size_t)
_cfgp = ctypes.POINTER(oscar_config)

# name -> (restype, argtypes); every entry point declared in include/oscar.h
_SIGS = {
    "oscar_last_error": (ctypes.c_char_p, []),
    "oscar_version": (ctypes.c_char_p, []),
    "oscar_int2_pool_bytes": (ctypes.c_size_t, [_cfgp]),
    "oscar_window_slab_bytes": (ctypes.c_size_t, [_cfgp]),
    "oscar_page_block_bytes": (ctypes.c_size_t, [_cfgp]),
    "oscar_create": (_i32, [_cfgp, _vp, _vp, ctypes.POINTER(_vp)]),
    "oscar_destroy": (_i32, [_vp]),
    "oscar_alloc_pages": (_i32, [_vp, _i32, _c_i32p]),
    "oscar_ref_pages": (_i32, [_vp, _c_i32p, _i32]),
    "oscar_unref_pages": (_i32, [_vp, _c_i32p, _i32]),
    "oscar_page_refcount": (_i32, [_vp, _i32, _c_i32p]),
    "oscar_free_page_count": (_i32, [_vp, _c_i32p]),
    "oscar_pages_needed": (_i32, [_cfgp, _i32]),
    "oscar_read_pages": (_i32, [_vp, _i32, _c_i32p, _i32, _vp]),
    "oscar_fork_prefix": (_i32, [_vp, _c_i32p, _c_i32p, _i32, _i32, _i32, _vp]),
    "oscar_write_kv": (_i32, [_vp, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _vp, _f32, _f32, _vp, _i32,
                              _vp, _vp]),
    "oscar_write_kv_hadamard": (_i32, [_vp, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _f32, _f32, _vp, _i32,
                                       _vp, _vp]),
    "oscar_set_layer_clip": (_i32, [_vp, _i32, _f32, _f32]),
    "oscar_append_step": (_i32, [_vp, _i32, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _f32, _f32, _vp, _i32, _vp, _vp]),
    "oscar_decode_workspace_size": (_i32, [_cfgp, _i32, _i32, ctypes.POINTER(ctypes.c_size_t)]),
    "oscar_decode_attn": (_i32, [_vp, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32,
                                 _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "oscar_decode_step": (_i32, [_vp, _i32, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32,
                                 _i32, _i32, _vp, _vp, _f32, _f32, _vp, ctypes.c_size_t, _vp]),
    "oscar_decode_attn_noalloc": (_i32, [_vp, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _i32,
                                         _i32, _vp, _vp, _vp]),
    "oscar_extend_workspace_size": (_i32, [_cfgp, _i32, ctypes.POINTER(ctypes.c_size_t)]),
    "oscar_extend_workspace_size_unpacked": (_i32, [_cfgp, _i32, _i32, _i32, _i32, ctypes.POINTER(ctypes.c_size_t)]),
    "oscar_extend_step": (_i32, [_vp, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _vp,
                                 _i32, _vp, _vp, _vp, _f32, _f32, _vp, ctypes.c_size_t, _vp]),
    "oscar_extend_attn": (_i32, [_vp, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _vp,
                                 _i32, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "oscar_bf16_decode_workspace_size": (_i32, [_cfgp, _i32, _i32, ctypes.POINTER(ctypes.c_size_t)]),
    "oscar_bf16_decode_attn": (_i32, [_vp, _i32, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _vp,
                                      ctypes.c_size_t, _vp]),
    "oscar_kv8_pool_bytes": (ctypes.c_size_t, [_cfgp]),
    "oscar_kv8_tail_bytes": (ctypes.c_size_t, [_cfgp]),
    "oscar_kv8_block_bytes": (ctypes.c_size_t, [_cfgp]),
    "oscar_kv8_pages_needed": (_i32, [_cfgp, _i32]),
    "oscar_kv8_bind": (_i32, [_vp, _i32, _vp, _vp]),
    "oscar_kv8_write": (_i32, [_vp, _i32, _vp, _i64, _vp, _i64, _i32, _vp, _vp, _i32, _i32, _vp, _i32, _vp, _vp]),
    "oscar_kv8_append": (_i32, [_vp, _i32, _vp, _i64, _vp, _i64, _i32, _vp, _i32, _vp, _i32, _vp, _vp]),
    "oscar_kv8_decode_workspace_size": (_i32, [_cfgp, _i32, _i32, _szp]),
    "oscar_kv8_decode_attn": (_i32, [_vp, _i32, _vp, _i64, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _vp,
                                     ctypes.c_size_t, _vp]),
    "oscar_kv8_select_workspace_size": (_i32, [_cfgp, _i32, _i32, _szp]),
    "oscar_kv8_select_pages": (_i32, [_vp, _i32, _vp, _i64, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _vp,
                                      _vp, ctypes.c_size_t, _vp]),
    "oscar_kv8_sparse_workspace_size": (_i32, [_cfgp, _i32, _i32, _szp]),
    "oscar_kv8_sparse_decode_attn": (_i32, [_vp, _i32, _vp, _i64, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp,
                                            _i32, _vp, ctypes.c_size_t, _vp]),
    "oscar_kv8_shared_workspace_size": (_i32, [_cfgp, _i32, _i32, _i32, _i32, _szp]),
    "oscar_kv8_shared_decode_attn": (_i32, [_vp, _i32, _vp, _i64, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _i32, _vp, _vp,
                                            _i32, _i32, _vp, ctypes.c_size_t, _vp]),
    "oscar_kv8_reorder": (_i32, [_vp, _vp, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "oscar_beam_select_workspace_size": (_i32, [_i32, _i32, _i32, _i32, _szp]),
    "oscar_beam_select": (_i32, [_vp, _vp, _i64, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                 ctypes.c_size_t, _vp]),
    "oscar_kv8_fork": (_i32, [_vp, _vp, _i32, _i32, _vp, _i32, _vp, _vp]),
    "oscar_compact_pages": (_i32, [_vp, _vp, _i32, _i32, _vp, _c_i32p, _vp]),
    "oscar_selftest_wait_timeout": (_i32, [_vp, _i32, _vp]),
    "oscar_check_status": (_i32, [_vp, _vp, _c_i32p]),
    "oscar_set_decode_form": (_i32, [_vp, _i32]),
    "oscar_set_timing": (_i32, [_vp, _i32]),
    "oscar_kernel_time": (_i32, [_vp, ctypes.c_char_p, ctypes.POINTER(ctypes.c_double), _c_i32p]),
    "oscar_reset_timing": (_i32, [_vp]),
    "oscar_launch_count": (ctypes.c_int64, [_vp]),
}

_lib: Optional[ctypes.CDLL] = None
_configs: dict = {}   # context -> its configuration, with the device of its 8-bit cache as .device (None: not bound)


def load() -> ctypes.CDLL:
    """Load liboscar.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OscarError(ERR_INVALID, f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                                          "python int2_rotated_paged_oscar_gb300/build.py")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(status: int) -> None:
    if status != OK:
        raise OscarError(status, load().oscar_last_error().decode())


def ptr(x) -> Optional[int]:
    """Device (or host) address of a torch tensor / int / None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def stream_ptr(stream=None) -> Optional[int]:
    if stream is None:
        return _current_raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_raw_stream = None


def _current_raw_stream() -> int:
    """Address of the current stream of the current device (torch's own shortcut where it has it: a Stream object
    costs 3 us)."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        torch.cuda.current_stream()   # initialises CUDA
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _raw_stream = (lambda: raw(device())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def _i32_array(seq: Sequence[int]):
    n = len(seq)
    try:
        return (ctypes.c_int32 * n).from_buffer(array.array("i", seq))   # integers that fit: the faster conversion
    except (TypeError, OverflowError, ValueError):
        pass
    return (ctypes.c_int32 * n)(*[int(v) for v in seq])


# ------------------------------------------------------------------ thin wrappers (same names as the C ABI)
def oscar_version() -> str:
    return load().oscar_version().decode()


def oscar_int2_pool_bytes(cfg: oscar_config) -> int:
    return load().oscar_int2_pool_bytes(ctypes.byref(cfg))


def oscar_window_slab_bytes(cfg: oscar_config) -> int:
    return load().oscar_window_slab_bytes(ctypes.byref(cfg))


def oscar_page_block_bytes(cfg: oscar_config) -> int:
    return load().oscar_page_block_bytes(ctypes.byref(cfg))


def oscar_create(cfg: oscar_config, int2_pool=None, window_slab=None) -> int:
    out = ctypes.c_void_p()
    _check(load().oscar_create(ctypes.byref(cfg), ptr(int2_pool), ptr(window_slab), ctypes.byref(out)))
    mine = oscar_config.from_buffer_copy(cfg)
    mine.device = None
    _configs[out.value] = mine
    return out.value


def oscar_destroy(ctx: int) -> None:
    _configs.pop(ctx, None)
    _check(load().oscar_destroy(ctx))


def oscar_alloc_pages(ctx: int, n: int):
    arr = (ctypes.c_int32 * max(n, 1))()
    _check(load().oscar_alloc_pages(ctx, n, arr))
    return arr[:n]


def oscar_ref_pages(ctx: int, ids: Sequence[int]) -> None:
    _check(load().oscar_ref_pages(ctx, _i32_array(ids), len(ids)))


def oscar_unref_pages(ctx: int, ids: Sequence[int]) -> None:
    _check(load().oscar_unref_pages(ctx, _i32_array(ids), len(ids)))


def oscar_page_refcount(ctx: int, page: int) -> int:
    out = ctypes.c_int32()
    _check(load().oscar_page_refcount(ctx, page, ctypes.byref(out)))
    return out.value


def oscar_free_page_count(ctx: int) -> int:
    out = ctypes.c_int32()
    _check(load().oscar_free_page_count(ctx, ctypes.byref(out)))
    return out.value


def oscar_pages_needed(cfg: oscar_config, seq_len: int) -> int:
    return load().oscar_pages_needed(ctypes.byref(cfg), seq_len)


def oscar_read_pages(ctx: int, cfg: oscar_config, layer: int, ids: Sequence[int]):
    """The INT2 blocks of pages ``ids`` of ``layer`` as a host uint8 array [len(ids), n_kv_heads, block bytes]
    (``cfg`` is the context's configuration; it gives the array's shape)."""
    import numpy as np
    bb = oscar_page_block_bytes(cfg)
    out = np.empty((len(ids), cfg.n_kv_heads, bb), np.uint8)
    _check(load().oscar_read_pages(ctx, layer, _i32_array(list(ids)), len(ids), out.ctypes.data))
    return out


def oscar_fork_prefix(ctx: int, src_bt: Sequence[int], n: int, src_slot: int, dst_slot: int, max_pages: int,
                      stream=0):
    dst = (ctypes.c_int32 * max_pages)()
    src = _i32_array(list(src_bt) + [-1] * (max_pages - len(src_bt)))
    _check(load().oscar_fork_prefix(ctx, src, dst, n, src_slot, dst_slot, stream_ptr(stream) if stream != 0 else None))
    return [dst[i] for i in range(max_pages)]


def oscar_write_kv(ctx, layer, K, V, dtype, cu_seqlens, start_pos, batch, total_tokens, R_K, R_V, clip_K, clip_V,
                   block_table, bt_stride, req_slot, stream=None) -> None:
    _check(load().oscar_write_kv(ctx, layer, ptr(K), ptr(V), dtype, ptr(cu_seqlens), ptr(start_pos), batch,
                                 total_tokens, ptr(R_K), ptr(R_V), float(clip_K), float(clip_V), ptr(block_table),
                                 bt_stride, ptr(req_slot), stream_ptr(stream)))


def oscar_write_kv_hadamard(ctx, layer, K, V, dtype, cu_seqlens, start_pos, batch, total_tokens, clip_K, clip_V,
                            block_table, bt_stride, req_slot, stream=None) -> None:
    _check(load().oscar_write_kv_hadamard(ctx, layer, ptr(K), ptr(V), dtype, ptr(cu_seqlens), ptr(start_pos), batch,
                                          total_tokens, float(clip_K), float(clip_V), ptr(block_table), bt_stride,
                                          ptr(req_slot), stream_ptr(stream)))


def oscar_append_step(ctx, layer, K_new, V_new, dtype, seq_lens_before, batch, R_K, R_V, clip_K, clip_V,
                      block_table, bt_stride, req_slot, stream=None) -> None:
    _check(load().oscar_append_step(ctx, layer, ptr(K_new), ptr(V_new), dtype, ptr(seq_lens_before), batch,
                                    ptr(R_K), ptr(R_V), float(clip_K), float(clip_V), ptr(block_table), bt_stride,
                                    ptr(req_slot), stream_ptr(stream)))


def oscar_set_layer_clip(ctx, layer, clip_K, clip_V) -> None:
    _check(load().oscar_set_layer_clip(ctx, layer, float(clip_K), float(clip_V)))


def oscar_decode_workspace_size(cfg: oscar_config, batch: int, max_seq: int) -> int:
    out = ctypes.c_size_t()
    _check(load().oscar_decode_workspace_size(ctypes.byref(cfg), batch, max_seq, ctypes.byref(out)))
    return out.value


def oscar_bf16_decode_workspace_size(cfg: oscar_config, batch: int, max_seq: int) -> int:
    out = ctypes.c_size_t()
    _check(load().oscar_bf16_decode_workspace_size(ctypes.byref(cfg), batch, max_seq, ctypes.byref(out)))
    return out.value


def oscar_decode_attn(ctx, layer, q, q_dtype, out, out_dtype, block_table, bt_stride, seq_lens, req_slot, batch,
                      max_seq, sink, recent, R_K, R_V, workspace, ws_bytes, stream=None) -> None:
    _check(load().oscar_decode_attn(ctx, layer, ptr(q), q_dtype, ptr(out), out_dtype, ptr(block_table), bt_stride,
                                    ptr(seq_lens), ptr(req_slot), batch, max_seq, sink, recent, ptr(R_K), ptr(R_V),
                                    ptr(workspace), ws_bytes, stream_ptr(stream)))


def oscar_decode_step(ctx, layer, K_new, V_new, kv_dtype, q, q_dtype, out, out_dtype, block_table, bt_stride,
                      seq_lens, req_slot, batch, max_seq, sink, recent, R_K, R_V, clip_K, clip_V, workspace, ws_bytes,
                      stream=None) -> None:
    _check(load().oscar_decode_step(ctx, layer, ptr(K_new), ptr(V_new), kv_dtype, ptr(q), q_dtype, ptr(out),
                                    out_dtype, ptr(block_table), bt_stride, ptr(seq_lens), ptr(req_slot), batch,
                                    max_seq, sink, recent, ptr(R_K), ptr(R_V), float(clip_K), float(clip_V),
                                    ptr(workspace), ws_bytes, stream_ptr(stream)))


def oscar_decode_attn_noalloc(ctx, layer, q, q_dtype, out, out_dtype, block_table, bt_stride, seq_lens, req_slot,
                              batch, max_seq, sink, recent, R_K, R_V, stream=None) -> None:
    """oscar_decode_attn without a workspace: scratch is the library's own 8 MiB device array (see oscar.h)."""
    _check(load().oscar_decode_attn_noalloc(ctx, layer, ptr(q), q_dtype, ptr(out), out_dtype, ptr(block_table),
                                            bt_stride, ptr(seq_lens), ptr(req_slot), batch, max_seq, sink, recent,
                                            ptr(R_K), ptr(R_V), stream_ptr(stream)))


def oscar_extend_workspace_size(cfg: oscar_config, total_tokens: int) -> int:
    out = ctypes.c_size_t()
    _check(load().oscar_extend_workspace_size(ctypes.byref(cfg), total_tokens, ctypes.byref(out)))
    return out.value


def oscar_extend_workspace_size_unpacked(cfg: oscar_config, total_tokens: int, batch: int, max_prefix: int,
                                         max_chunk: int) -> int:
    out = ctypes.c_size_t()
    _check(load().oscar_extend_workspace_size_unpacked(ctypes.byref(cfg), total_tokens, batch, max_prefix, max_chunk,
                                                       ctypes.byref(out)))
    return out.value


def oscar_extend_attn(ctx, layer, q, q_dtype, K_new, V_new, kv_dtype, out, out_dtype, cu_seqlens, prefix_lens, batch,
                      total_tokens, max_chunk, block_table, bt_stride, req_slot, R_K, R_V, workspace, ws_bytes,
                      stream=None) -> None:
    _check(load().oscar_extend_attn(ctx, layer, ptr(q), q_dtype, ptr(K_new), ptr(V_new), kv_dtype, ptr(out),
                                    out_dtype, ptr(cu_seqlens), ptr(prefix_lens), batch, total_tokens, max_chunk,
                                    ptr(block_table), bt_stride, ptr(req_slot), ptr(R_K), ptr(R_V), ptr(workspace),
                                    ws_bytes, stream_ptr(stream)))


def oscar_extend_step(ctx, layer, q, q_dtype, K_new, V_new, kv_dtype, out, out_dtype, cu_seqlens, prefix_lens, batch,
                      total_tokens, max_chunk, block_table, bt_stride, req_slot, R_K, R_V, clip_K, clip_V, workspace,
                      ws_bytes, stream=None) -> None:
    _check(load().oscar_extend_step(ctx, layer, ptr(q), q_dtype, ptr(K_new), ptr(V_new), kv_dtype, ptr(out),
                                    out_dtype, ptr(cu_seqlens), ptr(prefix_lens), batch, total_tokens, max_chunk,
                                    ptr(block_table), bt_stride, ptr(req_slot), ptr(R_K), ptr(R_V), float(clip_K),
                                    float(clip_V), ptr(workspace), ws_bytes, stream_ptr(stream)))


def oscar_bf16_decode_attn(ctx, layer, bf16_pool, q, q_dtype, out, out_dtype, block_table, bt_stride, seq_lens,
                           batch, max_seq, workspace, ws_bytes, stream=None) -> None:
    _check(load().oscar_bf16_decode_attn(ctx, layer, ptr(bf16_pool), ptr(q), q_dtype, ptr(out), out_dtype,
                                         ptr(block_table), bt_stride, ptr(seq_lens), batch, max_seq, ptr(workspace),
                                         ws_bytes, stream_ptr(stream)))


# ------------------------------------------------------------------ 8-bit cache
# These wrappers also check what the C ABI cannot see of a torch tensor: its device, element type, layout and size.
# A plain integer is passed on as an address, unchecked (rows then lie next to one another).
_torch_types: dict = {}


def _types() -> dict:
    """Element types by name and by DTYPE_* code (torch is imported on the first tensor argument)."""
    if not _torch_types:
        import torch
        _torch_types.update({"i32": torch.int32, DTYPE_F32: torch.float32, DTYPE_BF16: torch.bfloat16})
    return _torch_types


def _dense(x, name: str, device: Optional[int], count: int = 0, dtype="i32") -> Optional[int]:
    """Address of a dense tensor on the cache's device (None: on any CUDA device) of at least ``count`` elements of one
    type (dtype None: count bytes of any type)."""
    if count < 0:   # (a size that the library would take for a very large one)
        raise OscarError(ERR_INVALID, f"{name} cannot have {count} {'bytes' if dtype is None else 'elements'}")
    if x is None or isinstance(x, int):
        return x
    if (x.get_device() == device or device is None and x.is_cuda) and x.is_contiguous():
        if dtype is None:
            if x.numel() * x.element_size() >= count:
                return x.data_ptr()
        elif x.numel() >= count and x.dtype is (_torch_types or _types()).get(dtype, x.dtype):
            return x.data_ptr()
    raise OscarError(ERR_INVALID, f"{name} must be a contiguous tensor of at least {count} "
                                  f"{'bytes' if dtype is None else _types().get(dtype, 'elements')} on CUDA device "
                                  f"{'' if device is None else device}, not {x.dtype} "
                                  f"{tuple(x.shape)} on {x.device} with strides {tuple(x.stride())}")


def _rows(x, name: str, device: Optional[int], dtype: int, tokens: int, heads: int, d: int):
    """(address, elements between tokens) of [tokens][heads][d] rows; the tokens may lie further apart than their rows
    are long."""
    if x is None or isinstance(x, int):
        return x, 0
    shape = x.shape
    rows, hs, ds = shape if len(shape) == 3 else (-1, 0, 0)
    if rows < tokens or hs != heads or ds != d or x.dtype is not (_torch_types or _types()).get(dtype, x.dtype) \
            or not (x.get_device() == device or device is None and x.is_cuda):
        raise OscarError(ERR_INVALID, f"{name} must be a [{tokens}][{heads}][{d}] tensor of {_types().get(dtype)} on CUDA "
                                      f"device {'' if device is None else device}, not {x.dtype} {tuple(shape)} on {x.device}")
    t, h, c = x.stride()
    if c != 1 or (heads > 1 and h != d):
        raise OscarError(ERR_INVALID, f"the heads and channels of {name} must be adjacent, not strided {(t, h, c)}")
    if tokens > 1 and t < heads * d:   # (a broadcast row's stride of 0 would mean adjacent rows to the library)
        raise OscarError(ERR_INVALID, f"the tokens of {name} must lie at least {heads * d} elements apart, not {t}")
    return x.data_ptr(), t if tokens > 1 else 0


def _config(ctx) -> oscar_config:
    cfg = _configs.get(ctx)
    if cfg is None:
        raise OscarError(ERR_INVALID, "not a context of oscar_create")
    return cfg


def oscar_kv8_pool_bytes(cfg: oscar_config) -> int:
    return load().oscar_kv8_pool_bytes(ctypes.byref(cfg))


def oscar_kv8_tail_bytes(cfg: oscar_config) -> int:
    return load().oscar_kv8_tail_bytes(ctypes.byref(cfg))


def oscar_kv8_block_bytes(cfg: oscar_config) -> int:
    return load().oscar_kv8_block_bytes(ctypes.byref(cfg))


def oscar_kv8_pages_needed(cfg: oscar_config, seq_len: int) -> int:
    return load().oscar_kv8_pages_needed(ctypes.byref(cfg), seq_len)


def _current_device(*tensors) -> Optional[int]:
    """The current device, on which a context's buffers have to be; None where no argument is a CUDA tensor."""
    if any(getattr(x, "is_cuda", False) for x in tensors):
        import torch
        return torch.cuda.current_device()
    return None


def oscar_kv8_bind(ctx: int, fmt: int, pool, tail) -> None:
    """Bind an 8-bit cache: device buffers of oscar_kv8_pool_bytes and oscar_kv8_tail_bytes (any element type)."""
    cfg = _config(ctx)
    dev = _current_device(pool, tail)
    _check(load().oscar_kv8_bind(ctx, fmt, _dense(pool, "pool", dev, oscar_kv8_pool_bytes(cfg), None),
                                 _dense(tail, "tail", dev, oscar_kv8_tail_bytes(cfg), None)))
    cfg.device = dev


def oscar_kv8_write(ctx, layer, K, V, dtype, cu_seqlens, start_pos, batch, total_tokens, block_table, bt_stride,
                    req_slot, stream=None) -> None:
    cfg = _config(ctx)
    dev = cfg.device
    k, ks = _rows(K, "K", dev, dtype, total_tokens, cfg.n_kv_heads, cfg.head_dim)
    v, vs = _rows(V, "V", dev, dtype, total_tokens, cfg.n_kv_heads, cfg.head_dim)
    _check(load().oscar_kv8_write(ctx, layer, k, ks, v, vs, dtype, _dense(cu_seqlens, "cu_seqlens", dev, batch + 1),
                                  _dense(start_pos, "start_pos", dev, batch), batch, total_tokens,
                                  _dense(block_table, "block_table", dev, batch * bt_stride), bt_stride,
                                  _dense(req_slot, "req_slot", dev, batch), stream_ptr(stream)))


def oscar_kv8_append(ctx, layer, K_new, V_new, dtype, seq_lens_before, batch, block_table, bt_stride, req_slot,
                     stream=None) -> None:
    cfg = _config(ctx)
    dev = cfg.device
    k, ks = _rows(K_new, "K_new", dev, dtype, batch, cfg.n_kv_heads, cfg.head_dim)
    v, vs = _rows(V_new, "V_new", dev, dtype, batch, cfg.n_kv_heads, cfg.head_dim)
    _check(load().oscar_kv8_append(ctx, layer, k, ks, v, vs, dtype, _dense(seq_lens_before, "seq_lens_before", dev, batch),
                                   batch, _dense(block_table, "block_table", dev, batch * bt_stride), bt_stride,
                                   _dense(req_slot, "req_slot", dev, batch), stream_ptr(stream)))


def _size(fn, cfg, a: int, b: int) -> int:
    out = ctypes.c_size_t()
    _check(fn(ctypes.byref(cfg), a, b, ctypes.byref(out)))
    return out.value


def oscar_kv8_decode_workspace_size(cfg: oscar_config, batch: int, max_seq: int) -> int:
    return _size(load().oscar_kv8_decode_workspace_size, cfg, batch, max_seq)


def oscar_kv8_select_workspace_size(cfg: oscar_config, batch: int, max_seq: int) -> int:
    return _size(load().oscar_kv8_select_workspace_size, cfg, batch, max_seq)


def oscar_kv8_sparse_workspace_size(cfg: oscar_config, batch: int, n_select: int) -> int:
    return _size(load().oscar_kv8_sparse_workspace_size, cfg, batch, n_select)


def oscar_kv8_decode_attn(ctx, layer, q, q_dtype, out, out_dtype, block_table, bt_stride, seq_lens, req_slot, batch,
                          max_seq, workspace, ws_bytes, stream=None) -> None:
    cfg = _config(ctx)
    dev, hq, d = cfg.device, cfg.n_q_heads, cfg.head_dim
    qp, qs = _rows(q, "q", dev, q_dtype, batch, hq, d)
    _check(load().oscar_kv8_decode_attn(ctx, layer, qp, qs, q_dtype,
                                        _dense(out, "out", dev, batch * hq * d, out_dtype), out_dtype,
                                        _dense(block_table, "block_table", dev, batch * bt_stride), bt_stride,
                                        _dense(seq_lens, "seq_lens", dev, batch), _dense(req_slot, "req_slot", dev, batch), batch,
                                        max_seq, _dense(workspace, "workspace", dev, ws_bytes, None), ws_bytes,
                                        stream_ptr(stream)))


def oscar_kv8_select_pages(ctx, layer, q, q_dtype, block_table, bt_stride, seq_lens, batch, max_seq, keep_first,
                           keep_last, n_select, page_idx, workspace, ws_bytes, stream=None) -> None:
    cfg = _config(ctx)
    dev = cfg.device
    qp, qs = _rows(q, "q", dev, q_dtype, batch, cfg.n_q_heads, cfg.head_dim)
    _check(load().oscar_kv8_select_pages(ctx, layer, qp, qs, q_dtype,
                                         _dense(block_table, "block_table", dev, batch * bt_stride), bt_stride,
                                         _dense(seq_lens, "seq_lens", dev, batch), batch, max_seq, keep_first, keep_last,
                                         n_select, _dense(page_idx, "page_idx", dev, batch * cfg.n_kv_heads * n_select),
                                         _dense(workspace, "workspace", dev, ws_bytes, None), ws_bytes, stream_ptr(stream)))


def oscar_kv8_sparse_decode_attn(ctx, layer, q, q_dtype, out, out_dtype, page_idx, n_select, block_table, bt_stride,
                                 seq_lens, req_slot, batch, workspace, ws_bytes, stream=None) -> None:
    cfg = _config(ctx)
    dev, hq, d = cfg.device, cfg.n_q_heads, cfg.head_dim
    qp, qs = _rows(q, "q", dev, q_dtype, batch, hq, d)
    _check(load().oscar_kv8_sparse_decode_attn(ctx, layer, qp, qs, q_dtype,
                                               _dense(out, "out", dev, batch * hq * d, out_dtype),
                                               out_dtype,
                                               _dense(page_idx, "page_idx", dev, batch * cfg.n_kv_heads * n_select), n_select,
                                               _dense(block_table, "block_table", dev, batch * bt_stride), bt_stride,
                                               _dense(seq_lens, "seq_lens", dev, batch), _dense(req_slot, "req_slot", dev, batch),
                                               batch, _dense(workspace, "workspace", dev, ws_bytes, None), ws_bytes,
                                               stream_ptr(stream)))


def oscar_kv8_shared_workspace_size(cfg: oscar_config, batch: int, n_groups: int, max_shared: int, max_own: int) -> int:
    out = ctypes.c_size_t()
    _check(load().oscar_kv8_shared_workspace_size(ctypes.byref(cfg), batch, n_groups, max_shared, max_own, ctypes.byref(out)))
    return out.value


def oscar_kv8_shared_decode_attn(ctx, layer, q, q_dtype, out, out_dtype, group_starts, shared_pages, n_groups, max_shared,
                                 block_table, bt_stride, seq_lens, req_slot, batch, max_own, workspace, ws_bytes,
                                 stream=None) -> None:
    cfg = _config(ctx)
    dev, hq, d = cfg.device, cfg.n_q_heads, cfg.head_dim
    qp, qs = _rows(q, "q", dev, q_dtype, batch, hq, d)
    _check(load().oscar_kv8_shared_decode_attn(ctx, layer, qp, qs, q_dtype, _dense(out, "out", dev, batch * hq * d, out_dtype),
                                               out_dtype, _dense(group_starts, "group_starts", dev, n_groups + 1),
                                               _dense(shared_pages, "shared_pages", dev, n_groups), n_groups, max_shared,
                                               _dense(block_table, "block_table", dev, batch * bt_stride), bt_stride,
                                               _dense(seq_lens, "seq_lens", dev, batch), _dense(req_slot, "req_slot", dev, batch),
                                               batch, max_own, _dense(workspace, "workspace", dev, ws_bytes, None), ws_bytes,
                                               stream_ptr(stream)))


def oscar_kv8_reorder(ctx, parents, batch, beams, block_table, bt_stride, seq_lens, req_slot, new_block_table, new_seq_lens,
                      new_req_slot, stream=None) -> None:
    dev = _config(ctx).device
    rows = batch * beams
    _check(load().oscar_kv8_reorder(ctx, _dense(parents, "parents", dev, rows), batch, beams,
                                    _dense(block_table, "block_table", dev, rows * bt_stride), bt_stride,
                                    _dense(seq_lens, "seq_lens", dev, rows), _dense(req_slot, "req_slot", dev, rows),
                                    _dense(new_block_table, "new_block_table", dev, rows * bt_stride),
                                    _dense(new_seq_lens, "new_seq_lens", dev, rows),
                                    _dense(new_req_slot, "new_req_slot", dev, rows), stream_ptr(stream)))


def oscar_beam_select_workspace_size(batch: int, beams: int, vocab: int, n_out: int) -> int:
    out = ctypes.c_size_t()
    _check(load().oscar_beam_select_workspace_size(batch, beams, vocab, n_out, ctypes.byref(out)))
    return out.value


def _logits(x, device: Optional[int], dtype: int, batch: int, beams: int, vocab: int):
    """(address, elements between rows) of [batch][beams][vocab] or [batch * beams][vocab] logits."""
    if x is None or isinstance(x, int):
        return x, 0
    shape, stride = tuple(x.shape), tuple(x.stride())
    if len(shape) == 3 and shape[1] == beams and (shape[0] <= 1 or shape[1] <= 1 or stride[0] == shape[1] * stride[1]):
        step = stride[1] if shape[1] > 1 else stride[0]
        shape, stride = (shape[0] * shape[1], shape[2]), (step, stride[2])
    if len(shape) != 2 or shape[0] < batch * beams or shape[1] != vocab or x.dtype is not (_torch_types or _types()).get(dtype, x.dtype) \
            or not (x.get_device() == device or device is None and x.is_cuda):
        raise OscarError(ERR_INVALID, f"logits must be [{batch}][{beams}][{vocab}] of {_types().get(dtype)} in evenly spaced rows on "
                                      f"CUDA device {'' if device is None else device}, not {x.dtype} {tuple(x.shape)} on "
                                      f"{x.device} with strides {tuple(x.stride())}")
    if vocab > 1 and stride[1] != 1 or shape[0] > 1 and stride[0] < vocab:
        raise OscarError(ERR_INVALID, f"the logits of a row must be adjacent and rows at least {vocab} elements apart, not strided "
                                      f"{tuple(x.stride())}")
    return x.data_ptr(), stride[0] if shape[0] > 1 else 0


def oscar_beam_select(ctx, logits, dtype, scores, finished, pad_token, batch, beams, vocab, n_out, out_scores, out_tokens,
                      out_parents, workspace, ws_bytes, stream=None) -> None:
    """The next beams; finished is a uint8 or bool tensor of batch * beams elements, or None."""
    cfg = _config(ctx)
    dev = _current_device(logits, scores) if cfg.device is None else cfg.device
    lp, ls = _logits(logits, dev, dtype, batch, beams, vocab)
    if getattr(finished, "element_size", lambda: 1)() != 1:
        raise OscarError(ERR_INVALID, f"finished must have elements of one byte, not {finished.dtype}")
    _check(load().oscar_beam_select(ctx, lp, ls, dtype, _dense(scores, "scores", dev, batch * beams, DTYPE_F32),
                                    _dense(finished, "finished", dev, batch * beams, None), pad_token, batch, beams, vocab, n_out,
                                    _dense(out_scores, "out_scores", dev, batch * n_out, DTYPE_F32),
                                    _dense(out_tokens, "out_tokens", dev, batch * n_out),
                                    _dense(out_parents, "out_parents", dev, batch * n_out),
                                    _dense(workspace, "workspace", dev, ws_bytes, None), ws_bytes, stream_ptr(stream)))


def oscar_kv8_fork(ctx: int, src_bt: Sequence[int], n: int, src_slot: int, dst_slots: Sequence[int], max_pages: int,
                   stream=None):
    """The block tables of the forks, int32 [len(dst_slots)][max_pages]; max_pages is the configuration's
    max_pages_per_req.  A host-only context takes stream=0."""
    import numpy as np
    if max_pages != _config(ctx).max_pages_per_req:
        raise OscarError(ERR_INVALID, f"max_pages {max_pages} is not the configuration's max_pages_per_req")
    src = np.full(max_pages, -1, np.int32)
    mapped = np.asarray(src_bt, np.int32)[:max_pages]
    src[:len(mapped)] = mapped
    slots = np.ascontiguousarray(dst_slots, np.int32)
    dst = np.empty((len(slots), max_pages), np.int32)
    _check(load().oscar_kv8_fork(ctx, src.ctypes.data, n, src_slot, slots.ctypes.data, len(slots), dst.ctypes.data,
                                 stream_ptr(stream) if stream != 0 else None))
    return dst


def oscar_compact_pages(ctx: int, block_table, rows: int, bt_stride: int, num_pages: int, stream=None):
    """Compact the context's pages; returns (map, live): map int32 [num_pages] holds every page's new id, -1 for a free
    page.  num_pages is the configuration's.  block_table may be None (rows = 0); a host-only context takes stream=0."""
    import numpy as np
    cfg = _config(ctx)
    if num_pages != cfg.num_pages:
        raise OscarError(ERR_INVALID, f"num_pages {num_pages} is not the configuration's")
    dev = _current_device(block_table) if cfg.device is None else cfg.device
    table = np.empty(num_pages, np.int32)
    live = ctypes.c_int32()
    _check(load().oscar_compact_pages(ctx, _dense(block_table, "block_table", dev, rows * bt_stride), rows, bt_stride,
                                      table.ctypes.data, ctypes.byref(live), stream_ptr(stream) if stream != 0 else None))
    return table, live.value


def oscar_selftest_wait_timeout(ctx, limit_us: int, stream=None) -> None:
    _check(load().oscar_selftest_wait_timeout(ctx, int(limit_us), stream_ptr(stream)))


def oscar_check_status(ctx, stream=None) -> int:
    bits = ctypes.c_int32()
    st = load().oscar_check_status(ctx, stream_ptr(stream), ctypes.byref(bits))
    if st not in (OK, ERR_DEVICE):
        _check(st)
    return bits.value


def oscar_set_decode_form(ctx, form: int) -> None:
    _check(load().oscar_set_decode_form(ctx, int(form)))


def oscar_set_timing(ctx, enable: bool) -> None:
    _check(load().oscar_set_timing(ctx, 1 if enable else 0))


def oscar_kernel_time(ctx, name: str):
    ms = ctypes.c_double()
    n = ctypes.c_int32()
    _check(load().oscar_kernel_time(ctx, name.encode(), ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


def oscar_reset_timing(ctx) -> None:
    _check(load().oscar_reset_timing(ctx))


def oscar_launch_count(ctx) -> int:
    return load().oscar_launch_count(ctx)
