"""Python binding of the Delta-KV decode library (``include/dkv.h``).

Argument marshalling only: every step of the encode, append and decode path
runs in the library's CUDA kernels (``_lib/libdkv.so``, built for sm_100a).
PyTorch is used for device memory and streams.  If the shared library is
missing, every call raises -- there is no CPU fallback.

The functions carry the C names (``dkv_encode`` ...) and take either raw
integers (device pointers, a stream handle) or torch tensors / streams.
``Cache`` is a small convenience that allocates a cache with torch and keeps
its ``dkv_cache`` descriptor.
"""
from __future__ import annotations

import contextlib
import ctypes
from pathlib import Path

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "_lib" / "libdkv.so"
# the bounds-checked build (DKV_CHECKED=1, for tests): selected by setting
# DKV_LIBRARY=checked in the environment before the first load()
CHECKED_LIB_PATH = _PKG / "_lib" / "libdkv_checked.so"

DKV_OK, DKV_EINVAL, DKV_EALIGN, DKV_ECAPACITY, DKV_EUNSUPPORTED, DKV_ECUDA, DKV_EDEVICE = range(7)
DKV_FMT_FP16, DKV_FMT_Q4_0, DKV_FMT_DELTA = 0, 1, 2
DKV_F32, DKV_F16, DKV_BF16 = 0, 1, 2
DEV_BAD_SEQLEN, DEV_CAPACITY, DEV_TIMEOUT, DEV_BAD_HEADS, DEV_BAD_PAGE = 0x1, 0x2, 0x4, 0x8, 0x10
DEV_BOUNDS = 0x20
_I32_MAX = 2 ** 31 - 1      # ctypes drops what a C int32 has no room for
FORMATS = {"fp16": DKV_FMT_FP16, "q4": DKV_FMT_Q4_0, "delta": DKV_FMT_DELTA}


class DkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} ({status})")


class dkv_cache_desc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("kf", ctypes.c_int32),
                ("max_ctx", ctypes.c_int32), ("fmt", ctypes.c_int32)]


class dkv_lr_tensor(ctypes.Structure):
    _fields_ = [("ref", ctypes.c_void_p), ("ref_values", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("codes", ctypes.c_void_p)]


class dkv_cache(ctypes.Structure):
    _fields_ = [("desc", dkv_cache_desc), ("base", ctypes.c_void_p), ("bytes", ctypes.c_size_t),
                ("seq_stride", ctypes.c_size_t), ("rec_bytes", ctypes.c_size_t),
                ("n_groups", ctypes.c_int32), ("reserved0", ctypes.c_int32),
                ("off_data", ctypes.c_size_t), ("off_state", ctypes.c_size_t),
                ("off_seqlen", ctypes.c_size_t), ("off_header", ctypes.c_size_t),
                ("pool", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("page_bytes", ctypes.c_size_t), ("n_pages", ctypes.c_int64),
                ("page_groups", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class dkv_kv4_desc(ctypes.Structure):
    _fields_ = [("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("group", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class dkv_kv4_pool(ctypes.Structure):
    _fields_ = [("desc", dkv_kv4_desc), ("base", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_bytes", ctypes.c_size_t), ("status", ctypes.c_void_p)]


class dkv_kv4_batch(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("starts", ctypes.c_void_p)]


_lib = None
EXPORTS = ["dkv_abi_version", "dkv_cache_bytes", "dkv_cache_init", "dkv_encode", "dkv_append",
           "dkv_decode_workspace_bytes", "dkv_decode_attn", "dkv_decode_attn_split",
           "dkv_decode_attn_merge", "dkv_export_canonical", "dkv_dequantize",
           "dkv_get_device_status", "dkv_status_str", "dkv_decode_attn_noalloc",
           "dkv_debug_set_fault", "dkv_cache_meta_bytes", "dkv_page_bytes",
           "dkv_cache_init_paged", "dkv_decode_workspace_bytes_mq", "dkv_decode_attn_mq",
           "dkv_append_decode_attn", "dkv_append_decode_attn_split",
           "dkv_append_decode_attn_merge", "dkv_lr_encode", "dkv_lr_decode_workspace_bytes",
           "dkv_lr_decode_attn", "dkv_debug_division_check", "dkv_kv4_page_bytes",
           "dkv_kv4_init", "dkv_kv4_get_device_status", "dkv_kv4_append", "dkv_kv4_read",
           "dkv_kv4_decode_workspace_bytes", "dkv_kv4_decode_attn",
           "dkv_kv4_prompt_workspace_bytes", "dkv_kv4_prompt_attn"]


def load():
    """Load ``libdkv.so`` (raises if it has not been built), or the
    bounds-checked ``libdkv_checked.so`` when DKV_LIBRARY=checked."""
    global _lib
    if _lib is not None:
        return _lib
    import os
    path = CHECKED_LIB_PATH if os.environ.get("DKV_LIBRARY") == "checked" else LIB_PATH
    if not path.exists():
        raise RuntimeError(f"{path.name} not built ({path}); run __graft_entry__.build() "
                           "or python -m delta_quantized_kv_b200.build")
    lib = ctypes.CDLL(str(path))
    P, S, I, F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_float
    PC = ctypes.POINTER(dkv_cache)
    PD = ctypes.POINTER(dkv_cache_desc)
    L = ctypes.c_int64
    P4, B4, D4 = (ctypes.POINTER(t) for t in (dkv_kv4_pool, dkv_kv4_batch, dkv_kv4_desc))
    sig = {
        "dkv_abi_version": ([], I),
        "dkv_cache_bytes": ([PD], S),
        "dkv_cache_init": ([PD, P, S, PC, P], I),
        "dkv_encode": ([PC, P, P, I, P, I, P], I),
        "dkv_append": ([PC, P, P, I, I, P], I),
        "dkv_decode_workspace_bytes": ([PD, I], S),
        "dkv_decode_attn": ([PC, P, I, I, F, P, P, S, P], I),
        "dkv_decode_attn_split": ([PC, P, I, I, F, P, S, P], I),
        "dkv_decode_attn_merge": ([PC, I, P, P, S, P], I),
        "dkv_export_canonical": ([PC, P, P, P, P, P], I),
        "dkv_dequantize": ([PC, P, P], I),
        "dkv_get_device_status": ([PC, ctypes.POINTER(I), P], I),
        "dkv_status_str": ([I], ctypes.c_char_p),
        "dkv_decode_attn_noalloc": ([PC, P, I, I, F, P, P], I),
        "dkv_debug_set_fault": ([I], None),
        "dkv_cache_meta_bytes": ([PD], S),
        "dkv_page_bytes": ([PD, I], S),
        "dkv_cache_init_paged": ([PD, I, P, ctypes.c_int64, P, I, P, S, PC, P], I),
        "dkv_decode_workspace_bytes_mq": ([PD, I, I], S),
        "dkv_decode_attn_mq": ([PC, P, I, I, I, F, P, P, S, P], I),
        "dkv_append_decode_attn": ([PC, P, P, I, I, P, I, I, F, P, P, S, P], I),
        "dkv_append_decode_attn_split": ([PC, P, P, I, I, P, I, I, F, P, S, P], I),
        "dkv_append_decode_attn_merge": ([PC, I, I, P, P, S, P], I),
        "dkv_lr_encode": ([P, I, I, I, I, I, P, P, P, P, P, P], I),
        "dkv_lr_decode_workspace_bytes": ([I, I, I, I], S),
        "dkv_debug_division_check": ([P, I, P, P], I),
        "dkv_lr_decode_attn": ([ctypes.POINTER(dkv_lr_tensor), ctypes.POINTER(dkv_lr_tensor),
                                I, I, I, I, I, P, P, I, I, F, P, P, S, P], I),
        "dkv_kv4_page_bytes": ([D4], S),
        "dkv_kv4_init": ([D4, P, L, P, P4, P], I),
        "dkv_kv4_get_device_status": ([P4, ctypes.POINTER(I), P], I),
        "dkv_kv4_append": ([P4, B4, P, P, I, I, L, L, L, L, P], I),
        "dkv_kv4_read": ([P4, B4, P, P, I, I, P], I),
        "dkv_kv4_decode_workspace_bytes": ([D4, I, I, I, I], S),
        "dkv_kv4_prompt_workspace_bytes": ([D4, I, I, I, I, I], S),
        "dkv_kv4_prompt_attn": ([P4, B4, P, I, I, I, L, L, F, I, P, P, P, S, P], I),
        "dkv_kv4_decode_attn": ([P4, B4, P, I, I, I, L, L, F, I, P, P, P, S, P], I),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def status_str(s: int) -> str:
    return load().dkv_status_str(int(s)).decode()


def _ptr(x):
    """Device pointer of a tensor (or an int / None)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _on(stream, device):
    """A context in which torch allocates and launches on `stream` (None: as it does)."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device)
    return torch.cuda.stream(stream)


def _dtype_code(t) -> int:
    import torch
    return {torch.float32: DKV_F32, torch.float16: DKV_F16, torch.bfloat16: DKV_BF16}[t]


def _check(s: int, what: str):
    if s != DKV_OK:
        raise DkvError(s, what)


# ---------------------------------------------------------------------------
# the C functions, same names
# ---------------------------------------------------------------------------
def dkv_abi_version() -> int:
    return load().dkv_abi_version()


def dkv_cache_bytes(desc: dkv_cache_desc) -> int:
    return load().dkv_cache_bytes(ctypes.byref(desc))


def dkv_cache_init(desc: dkv_cache_desc, dev, nbytes: int, stream=None) -> dkv_cache:
    out = dkv_cache()
    _check(load().dkv_cache_init(ctypes.byref(desc), _ptr(dev), nbytes, ctypes.byref(out),
                                 _stream(stream)), "dkv_cache_init")
    return out


def dkv_cache_meta_bytes(desc: dkv_cache_desc) -> int:
    return load().dkv_cache_meta_bytes(ctypes.byref(desc))


def dkv_page_bytes(desc: dkv_cache_desc, page_groups: int) -> int:
    return load().dkv_page_bytes(ctypes.byref(desc), page_groups)


def dkv_cache_init_paged(desc: dkv_cache_desc, page_groups: int, pool, n_pages: int,
                         block_table, max_pages: int, meta, meta_bytes: int,
                         stream=None) -> dkv_cache:
    out = dkv_cache()
    _check(load().dkv_cache_init_paged(ctypes.byref(desc), page_groups, _ptr(pool), n_pages,
                                       _ptr(block_table), max_pages, _ptr(meta), meta_bytes,
                                       ctypes.byref(out), _stream(stream)),
           "dkv_cache_init_paged")
    return out


def dkv_encode(cache: dkv_cache, K, V, dtype=None, seq_lens=None, T=None, stream=None) -> None:
    dtype = _dtype_code(K.dtype) if dtype is None else dtype
    T = K.shape[2] if T is None else T
    _check(load().dkv_encode(ctypes.byref(cache), _ptr(K), _ptr(V), dtype, _ptr(seq_lens), T,
                             _stream(stream)), "dkv_encode")


def dkv_append(cache: dkv_cache, K_new, V_new, dtype=None, n_new=None, stream=None) -> None:
    dtype = _dtype_code(K_new.dtype) if dtype is None else dtype
    n_new = K_new.shape[2] if n_new is None else n_new
    _check(load().dkv_append(ctypes.byref(cache), _ptr(K_new), _ptr(V_new), dtype, n_new,
                             _stream(stream)), "dkv_append")


def dkv_decode_workspace_bytes(desc: dkv_cache_desc, n_q_heads: int) -> int:
    return load().dkv_decode_workspace_bytes(ctypes.byref(desc), n_q_heads)


def dkv_decode_attn(cache: dkv_cache, Q, q_dtype, n_q_heads, softmax_scale, out, workspace,
                    ws_bytes, stream=None) -> None:
    _check(load().dkv_decode_attn(ctypes.byref(cache), _ptr(Q), q_dtype, n_q_heads,
                                  softmax_scale, _ptr(out), _ptr(workspace), ws_bytes,
                                  _stream(stream)), "dkv_decode_attn")


def dkv_decode_workspace_bytes_mq(desc: dkv_cache_desc, n_q_heads: int, n_queries: int) -> int:
    return load().dkv_decode_workspace_bytes_mq(ctypes.byref(desc), n_q_heads, n_queries)


def dkv_decode_attn_mq(cache: dkv_cache, Q, q_dtype, n_q_heads, n_queries, softmax_scale, out,
                       workspace, ws_bytes, stream=None) -> None:
    _check(load().dkv_decode_attn_mq(ctypes.byref(cache), _ptr(Q), q_dtype, n_q_heads, n_queries,
                                     softmax_scale, _ptr(out), _ptr(workspace), ws_bytes,
                                     _stream(stream)), "dkv_decode_attn_mq")


def dkv_append_decode_attn(cache: dkv_cache, K_new, V_new, kv_dtype, n_new, Q, q_dtype,
                           n_q_heads, softmax_scale, out, workspace, ws_bytes,
                           stream=None) -> None:
    _check(load().dkv_append_decode_attn(ctypes.byref(cache), _ptr(K_new), _ptr(V_new), kv_dtype,
                                         n_new, _ptr(Q), q_dtype, n_q_heads, softmax_scale,
                                         _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)),
           "dkv_append_decode_attn")


def dkv_append_decode_attn_split(cache: dkv_cache, K_new, V_new, kv_dtype, n_new, Q, q_dtype,
                                 n_q_heads, softmax_scale, workspace, ws_bytes,
                                 stream=None) -> None:
    _check(load().dkv_append_decode_attn_split(ctypes.byref(cache), _ptr(K_new), _ptr(V_new),
                                               kv_dtype, n_new, _ptr(Q), q_dtype, n_q_heads,
                                               softmax_scale, _ptr(workspace), ws_bytes,
                                               _stream(stream)), "dkv_append_decode_attn_split")


def dkv_append_decode_attn_merge(cache: dkv_cache, n_new, n_q_heads, out, workspace, ws_bytes,
                                 stream=None) -> None:
    _check(load().dkv_append_decode_attn_merge(ctypes.byref(cache), n_new, n_q_heads, _ptr(out),
                                               _ptr(workspace), ws_bytes, _stream(stream)),
           "dkv_append_decode_attn_merge")


def lr_encode(X, stride: int, n_refs: int, stream=None) -> dict:
    """Long-range reference encoding (dkv_lr_encode) of X [n_seq, T, 128] on
    the GPU -> dict of device tensors ref, ref_values, scales, codes, xhat in
    the canonical layouts."""
    import torch
    if X.dim() != 3 or X.shape[2] != 128:
        raise ValueError("lr_encode takes X of shape [n_seq, T, 128]")
    n_seq, T, Dh = X.shape
    if stride < 1 or not 1 <= n_refs <= 8:
        raise DkvError(DKV_EINVAL, "dkv_lr_encode")
    ng = -(-T // stride)
    dev = X.device
    out = {"ref": torch.empty((n_seq, T, n_refs), dtype=torch.int32, device=dev),
           "ref_values": torch.empty((n_seq, ng, Dh), dtype=torch.int16, device=dev),
           "scales": torch.empty((n_seq, T, Dh // 32), dtype=torch.int16, device=dev),
           "codes": torch.empty((n_seq, T, Dh), dtype=torch.uint8, device=dev),
           "xhat": torch.empty((n_seq, T, Dh), dtype=torch.float32, device=dev)}
    X = X.contiguous()
    _check(load().dkv_lr_encode(_ptr(X), _dtype_code(X.dtype), n_seq, T, stride, n_refs,
                                _ptr(out["ref"]), _ptr(out["ref_values"]), _ptr(out["scales"]),
                                _ptr(out["codes"]), _ptr(out["xhat"]), _stream(stream)),
           "dkv_lr_encode")
    return out


def dkv_lr_decode_workspace_bytes(batch: int, n_kv_heads: int, T: int, stride: int) -> int:
    return load().dkv_lr_decode_workspace_bytes(batch, n_kv_heads, T, stride)


def _lr_view(enc) -> dkv_lr_tensor:
    return dkv_lr_tensor(_ptr(enc["ref"]), _ptr(enc["ref_values"]), _ptr(enc["scales"]),
                         _ptr(enc["codes"]))


def lr_decode_attn(enc_k: dict, enc_v: dict, Q, softmax_scale: float, stride: int,
                   n_kv_heads: int, lens=None, out=None, workspace=None, stream=None):
    """Decode attention over long-range reference encodings (dkv_lr_decode_attn).
    enc_k, enc_v: the dicts `lr_encode` returns for K and V, each encoding
    [B * n_kv_heads, T, 128] sequences (sequence = batch entry * n_kv_heads +
    kv head) with the same stride and n_refs; Q [B, n_q_heads, 128];
    lens: device int32 [B] or None.  Returns fp32 [B, n_q_heads, 128]."""
    import torch
    n_seq, T, n_refs = enc_k["ref"].shape
    B = n_seq // n_kv_heads
    Hq = Q.shape[1]
    if out is None:
        out = torch.empty((B, Hq, 128), dtype=torch.float32, device=Q.device)
    nb = dkv_lr_decode_workspace_bytes(B, n_kv_heads, T, stride)
    if workspace is None:
        workspace = torch.empty(nb // 4 + 64, dtype=torch.float32, device=Q.device)
    kv, vv = _lr_view(enc_k), _lr_view(enc_v)
    Q = Q.contiguous()
    _check(load().dkv_lr_decode_attn(ctypes.byref(kv), ctypes.byref(vv), B, n_kv_heads, T, stride,
                                     n_refs, _ptr(lens), _ptr(Q), _dtype_code(Q.dtype), Hq,
                                     softmax_scale, _ptr(out), _ptr(workspace),
                                     workspace.numel() * 4, _stream(stream)),
           "dkv_lr_decode_attn")
    return out


def dkv_decode_attn_split(cache: dkv_cache, Q, q_dtype, n_q_heads, softmax_scale, workspace,
                          ws_bytes, stream=None) -> None:
    _check(load().dkv_decode_attn_split(ctypes.byref(cache), _ptr(Q), q_dtype, n_q_heads,
                                        softmax_scale, _ptr(workspace), ws_bytes,
                                        _stream(stream)), "dkv_decode_attn_split")


def dkv_decode_attn_merge(cache: dkv_cache, n_q_heads, out, workspace, ws_bytes,
                          stream=None) -> None:
    _check(load().dkv_decode_attn_merge(ctypes.byref(cache), n_q_heads, _ptr(out),
                                        _ptr(workspace), ws_bytes, _stream(stream)),
           "dkv_decode_attn_merge")


def dkv_decode_attn_noalloc(cache: dkv_cache, Q, q_dtype, n_q_heads, softmax_scale, out,
                            stream=None) -> None:
    """Decode step that needs no workspace: the partial records go to a fixed
    16 MiB array the library keeps on each GPU (for callers that cannot
    allocate device memory when they decode, e.g. under graph capture).
    Calls overlapping on the GPU race on that array."""
    _check(load().dkv_decode_attn_noalloc(ctypes.byref(cache), _ptr(Q), q_dtype, n_q_heads,
                                          softmax_scale, _ptr(out), _stream(stream)),
           "dkv_decode_attn_noalloc")


def dkv_export_canonical(cache: dkv_cache, codes=None, scales=None, keyframes=None, state=None,
                         stream=None) -> None:
    _check(load().dkv_export_canonical(ctypes.byref(cache), _ptr(codes), _ptr(scales),
                                       _ptr(keyframes), _ptr(state), _stream(stream)),
           "dkv_export_canonical")


def dkv_dequantize(cache: dkv_cache, out, stream=None) -> None:
    _check(load().dkv_dequantize(ctypes.byref(cache), _ptr(out), _stream(stream)),
           "dkv_dequantize")


def dkv_debug_set_fault(mode: int) -> None:
    """Test support: mode 1 makes later split launches time out by design."""
    load().dkv_debug_set_fault(int(mode))


def dkv_debug_division_check(u, mismatches, stream=None) -> None:
    """Test support: count (into the device uint64 `mismatches`) the encoder
    quotients that differ from IEEE division, over every fp16 divisor and the
    dividends RN(u_i b) and their neighbours (u: device fp32)."""
    _check(load().dkv_debug_division_check(_ptr(u), u.numel(), _ptr(mismatches),
                                           _stream(stream)), "dkv_debug_division_check")


def dkv_kv4_page_bytes(desc: dkv_kv4_desc) -> int:
    return load().dkv_kv4_page_bytes(ctypes.byref(desc))


def dkv_kv4_init(desc: dkv_kv4_desc, pool, n_pages: int, status, stream=None) -> dkv_kv4_pool:
    out = dkv_kv4_pool()
    _check(load().dkv_kv4_init(ctypes.byref(desc), _ptr(pool), n_pages, _ptr(status),
                               ctypes.byref(out), _stream(stream)), "dkv_kv4_init")
    return out


def dkv_kv4_get_device_status(pool: dkv_kv4_pool, stream=None) -> int:
    word = ctypes.c_int32(0)
    s = load().dkv_kv4_get_device_status(ctypes.byref(pool), ctypes.byref(word), _stream(stream))
    if s not in (DKV_OK, DKV_EDEVICE):
        raise DkvError(s, "dkv_kv4_get_device_status")
    return word.value


def dkv_kv4_append(pool: dkv_kv4_pool, seqs: dkv_kv4_batch, K, V, dtype, n_rows, k_row_stride,
                   k_head_stride, v_row_stride, v_head_stride, stream=None) -> None:
    _check(load().dkv_kv4_append(ctypes.byref(pool), ctypes.byref(seqs), _ptr(K), _ptr(V), dtype,
                                 n_rows, k_row_stride, k_head_stride, v_row_stride,
                                 v_head_stride, _stream(stream)), "dkv_kv4_append")


def dkv_kv4_read(pool: dkv_kv4_pool, seqs: dkv_kv4_batch, K_out, V_out, dtype, n_rows,
                 stream=None) -> None:
    _check(load().dkv_kv4_read(ctypes.byref(pool), ctypes.byref(seqs), _ptr(K_out), _ptr(V_out),
                               dtype, n_rows, _stream(stream)), "dkv_kv4_read")


def dkv_kv4_decode_workspace_bytes(desc: dkv_kv4_desc, batch: int, max_pages: int,
                                   n_q_heads: int, n_queries: int) -> int:
    return load().dkv_kv4_decode_workspace_bytes(ctypes.byref(desc), batch, max_pages, n_q_heads,
                                                 n_queries)


def dkv_kv4_decode_attn(pool: dkv_kv4_pool, seqs: dkv_kv4_batch, Q, q_dtype, n_q_heads, n_queries,
                        q_row_stride, q_head_stride, softmax_scale, window, out, lse, workspace,
                        ws_bytes, stream=None) -> None:
    _check(load().dkv_kv4_decode_attn(ctypes.byref(pool), ctypes.byref(seqs), _ptr(Q), q_dtype,
                                      n_q_heads, n_queries, q_row_stride, q_head_stride,
                                      softmax_scale, window, _ptr(out), _ptr(lse),
                                      _ptr(workspace), ws_bytes, _stream(stream)),
           "dkv_kv4_decode_attn")


def dkv_kv4_prompt_workspace_bytes(desc: dkv_kv4_desc, batch: int, max_pages: int,
                                   n_q_heads: int, n_rows: int, ragged: bool) -> int:
    return load().dkv_kv4_prompt_workspace_bytes(ctypes.byref(desc), batch, max_pages, n_q_heads,
                                                 n_rows, int(ragged))


def dkv_kv4_prompt_attn(pool: dkv_kv4_pool, seqs: dkv_kv4_batch, Q, q_dtype, n_q_heads, n_rows,
                        q_row_stride, q_head_stride, softmax_scale, window, out, lse, workspace,
                        ws_bytes, stream=None) -> None:
    _check(load().dkv_kv4_prompt_attn(ctypes.byref(pool), ctypes.byref(seqs), _ptr(Q), q_dtype,
                                      n_q_heads, n_rows, q_row_stride, q_head_stride,
                                      softmax_scale, window, _ptr(out), _ptr(lse),
                                      _ptr(workspace), ws_bytes, _stream(stream)),
           "dkv_kv4_prompt_attn")


def dkv_get_device_status(cache: dkv_cache, stream=None) -> int:
    word = ctypes.c_int32(0)
    s = load().dkv_get_device_status(ctypes.byref(cache), ctypes.byref(word), _stream(stream))
    if s not in (DKV_OK, DKV_EDEVICE):
        raise DkvError(s, "dkv_get_device_status")
    return word.value


# ---------------------------------------------------------------------------
# convenience wrapper (torch allocations)
# ---------------------------------------------------------------------------
class Cache:
    """A Delta-KV (or comparator) cache in torch-allocated device memory."""

    def __init__(self, batch, n_kv_heads, max_ctx, fmt="delta", kf=32, head_dim=128,
                 device="cuda", stream=None, page_groups=None, n_pages=None,
                 block_table=None, page_seed=0):
        """page_groups: a paged cache (delta format) with pages of page_groups
        keyframe groups; the pool holds n_pages pages (default: exactly the
        pages every sequence needs at max_ctx) and block_table ([batch,
        max_pages] int32, default: a seeded random assignment of distinct
        pages) maps each sequence's groups to pages."""
        import torch
        self.desc = dkv_cache_desc(batch, n_kv_heads, head_dim, kf, max_ctx,
                                   FORMATS[fmt] if isinstance(fmt, str) else fmt)
        if page_groups:
            mb = dkv_cache_meta_bytes(self.desc)
            pb = dkv_page_bytes(self.desc, page_groups)
            if mb == 0 or pb == 0:
                raise DkvError(DKV_EINVAL, "dkv_cache_meta_bytes / dkv_page_bytes")
            n_groups = -(-max_ctx // kf)
            max_pages = -(-n_groups // page_groups)
            if n_pages is None:
                n_pages = batch * max_pages
            if block_table is None:
                g = torch.Generator().manual_seed(page_seed)
                perm = torch.randperm(n_pages, generator=g)[:batch * max_pages]
                block_table = perm.view(batch, max_pages).to(torch.int32)
            self.block_table = block_table.to(device=device, dtype=torch.int32).contiguous()
        else:
            nbytes = dkv_cache_bytes(self.desc)
            if nbytes == 0:
                raise DkvError(DKV_EINVAL, "dkv_cache_bytes")
        # the memory is taken on the stream that initialises it: a block that comes
        # back from work still queued on another one would be written under it
        with _on(stream, device):
            self.buf = torch.empty((mb if page_groups else nbytes) + 256, dtype=torch.uint8,
                                   device=device)
            base = (self.buf.data_ptr() + 255) // 256 * 256
            if page_groups:
                self.pool = torch.empty(n_pages * pb + 256, dtype=torch.uint8, device=device)
                pool = (self.pool.data_ptr() + 255) // 256 * 256
                self.c = dkv_cache_init_paged(self.desc, page_groups, pool, n_pages,
                                              self.block_table, max_pages, base, mb)
            else:
                self.c = dkv_cache_init(self.desc, base, nbytes)
        self._ws = None
        self._ws_heads = None
        self.device = device

    @property
    def fmt(self):
        return self.desc.fmt

    def encode(self, K, V, seq_lens=None, stream=None):
        dkv_encode(self.c, K, V, seq_lens=seq_lens, stream=stream)

    def append(self, K_new, V_new, stream=None):
        dkv_append(self.c, K_new, V_new, stream=stream)

    def workspace(self, n_q_heads):
        import torch
        if self._ws is None or self._ws_heads != n_q_heads:
            nb = dkv_decode_workspace_bytes(self.desc, n_q_heads)
            if nb == 0:
                raise DkvError(DKV_ECUDA, "dkv_decode_workspace_bytes")
            self._ws = torch.zeros(nb // 4 + 64, dtype=torch.float32, device=self.device)
            self._ws_heads = n_q_heads
        return self._ws

    def decode_attn(self, Q, softmax_scale, out=None, stream=None):
        import torch
        B, Hq, Dh = Q.shape
        if out is None:
            out = torch.empty((B, Hq, Dh), dtype=torch.float32, device=Q.device)
        ws = self.workspace(Hq)
        dkv_decode_attn(self.c, Q, _dtype_code(Q.dtype), Hq, softmax_scale, out, ws,
                        ws.numel() * 4, stream)
        return out

    def workspace_mq(self, n_q_heads, n_queries):
        import torch
        key = ("mq", n_q_heads, n_queries)
        ws = getattr(self, "_ws_mq", {}).get(key)
        if ws is None:
            nb = dkv_decode_workspace_bytes_mq(self.desc, n_q_heads, n_queries)
            if nb == 0:
                raise DkvError(DKV_EINVAL, "dkv_decode_workspace_bytes_mq")
            ws = torch.zeros(nb // 4 + 64, dtype=torch.float32, device=self.device)
            self._ws_mq = {key: ws}
        return ws

    def decode_attn_mq(self, Q, softmax_scale, out=None, stream=None):
        """Q: [B, n_queries, Hq, D]; query t attends causally (see
        dkv_decode_attn_mq).  Returns fp32 [B, n_queries, Hq, D]."""
        import torch
        B, nq, Hq, Dh = Q.shape
        if out is None:
            out = torch.empty((B, nq, Hq, Dh), dtype=torch.float32, device=Q.device)
        ws = self.workspace_mq(Hq, nq)
        dkv_decode_attn_mq(self.c, Q.contiguous(), _dtype_code(Q.dtype), Hq, nq, softmax_scale,
                           out, ws, ws.numel() * 4, stream)
        return out

    def append_decode_attn(self, K_new, V_new, Q, softmax_scale, out=None, stream=None):
        """Fused append + decode (dkv_append_decode_attn): K_new, V_new
        [B, Hkv, n_new, D]; Q [B, Hq, D] (n_new = 1) or [B, n_new, Hq, D].
        Returns fp32 of Q's shape."""
        import torch
        n_new = K_new.shape[2]
        Hq = Q.shape[-2]
        if Q.dim() == 3 and n_new != 1:
            raise ValueError("Q of shape [B, Hq, D] takes one new token per sequence")
        if Q.dim() == 4 and Q.shape[1] != n_new:
            raise ValueError("Q must hold one query per new token")
        if out is None:
            out = torch.empty(Q.shape, dtype=torch.float32, device=Q.device)
        ws = self.workspace_mq(Hq, n_new)
        dkv_append_decode_attn(self.c, K_new, V_new, _dtype_code(K_new.dtype), n_new,
                               Q.contiguous(), _dtype_code(Q.dtype), Hq, softmax_scale, out, ws,
                               ws.numel() * 4, stream)
        return out

    def seq_lens(self):
        import torch
        n = self.desc.batch
        base = self.c.base + self.c.off_seqlen
        off = base - self.buf.data_ptr()
        return self.buf[off:off + 4 * n].view(torch.int32).clone()

    def export(self, stream=None):
        """Canonical fields as torch tensors (codes, scales, keyframes, state)."""
        import torch
        d = self.desc
        B, H, cap = d.batch, d.n_kv_heads, d.max_ctx
        dev = self.device
        out = {}
        if d.fmt in (DKV_FMT_DELTA, DKV_FMT_Q4_0):
            out["codes"] = torch.zeros((B, H, 2, cap, 128), dtype=torch.uint8, device=dev)
            out["scales"] = torch.zeros((B, H, 2, cap, 4), dtype=torch.int16, device=dev)
        if d.fmt == DKV_FMT_DELTA:
            out["keyframes"] = torch.zeros((B, H, 2, self.c.n_groups, 128), dtype=torch.int16,
                                           device=dev)
            out["state"] = torch.zeros((B, H, 2, 128), dtype=torch.float32, device=dev)
        if d.fmt == DKV_FMT_FP16:
            out["keyframes"] = torch.zeros((B, H, 2, cap, 128), dtype=torch.int16, device=dev)
        dkv_export_canonical(self.c, out.get("codes"), out.get("scales"), out.get("keyframes"),
                             out.get("state"), stream)
        return out

    def dequantize(self, stream=None):
        import torch
        d = self.desc
        out = torch.zeros((d.batch, d.n_kv_heads, 2, d.max_ctx, 128), dtype=torch.float32,
                          device=self.device)
        dkv_dequantize(self.c, out, stream)
        return out

    def device_status(self, stream=None) -> int:
        return dkv_get_device_status(self.c, stream)


class Kv4Cache:
    """A paged 4-bit cache (dkv_kv4_*) in torch-allocated device memory.

    The pages hold keys and values in 4 bits, `group` channels a block; the
    caller owns the block table (device int32 [batch, max_pages]), the lengths
    (device int32 [batch], the call's own tokens included) and, for ragged
    calls, the first row of each sequence (`starts`, device int32 [batch + 1];
    None: the same number of rows for each).  Row i of a sequence's n rows
    stands for position seq_len - n + i.  Every call, the constructor too,
    launches on `stream` (default: the current stream of the cache's device)
    and takes its memory from torch's allocator on that stream, so calls may be
    captured into graphs and run on several streams at once.  As everywhere in
    torch, streams that share tensors (the pages among them) are put in order by
    the caller.
    """

    def __init__(self, n_pages, n_kv_heads, head_dim=128, page_size=64, group=32, device="cuda",
                 stream=None):
        import torch
        given = (n_kv_heads, head_dim, group, page_size)
        self.desc = dkv_kv4_desc(*given)
        pb = dkv_kv4_page_bytes(self.desc)
        kept = tuple(getattr(self.desc, name) for name, _ in self.desc._fields_)
        if pb == 0 or n_pages < 1 or kept != given:
            raise DkvError(DKV_EINVAL, "dkv_kv4_page_bytes")
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("a Kv4Cache lives on a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        # what every call needs at hand: a decode step's calls take microseconds
        self._torch, self._lib, self._index = torch, load(), self.device.index
        # the memory is taken where it is zeroed: a block that comes back from work
        # still queued on another stream would be written under the zeroes
        with self._elsewhere(stream) or contextlib.nullcontext():
            self.pool = torch.empty(n_pages * pb + 256, dtype=torch.uint8, device=self.device)
            self.status = torch.empty(1, dtype=torch.int32, device=self.device)
            base = (self.pool.data_ptr() + 255) // 256 * 256
            self.c = dkv_kv4_init(self.desc, base, n_pages, self.status)
        self._desc, self._pool = ctypes.byref(self.desc), ctypes.byref(self.c)
        self._codes = {torch.float32: DKV_F32, torch.float16: DKV_F16, torch.bfloat16: DKV_BF16}
        self._stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda i: torch.cuda.current_stream(i).cuda_stream)

    # -- argument checks ----------------------------------------------------
    def _tensor(self, x, name, dims=None):
        if x.device != self.device:
            raise ValueError(f"{name} is on {x.device}, the cache on {self.device}")
        if dims is not None and x.dim() != dims:
            raise ValueError(f"{name} has {x.dim()} dimensions, not {dims}")
        return x

    def _batch(self, block_table, seq_lens, starts):
        i32, dev = self._torch.int32, self._index
        for name, x, dims in (("block_table", block_table, 2), ("seq_lens", seq_lens, 1),
                              ("starts", starts, 1)):
            if x is None:
                if name == "starts":
                    continue
                raise ValueError(f"{name} is missing")
            if x.get_device() != dev or x.dim() != dims or x.dtype is not i32 \
                    or not x.is_contiguous():
                self._tensor(x, name, dims)
                raise ValueError(f"{name} must be contiguous int32")
        (B,), (rows, width) = seq_lens.shape, block_table.shape
        if width > _I32_MAX:
            raise ValueError(f"block_table has {width} columns")
        if rows != B or (starts is not None and starts.shape[0] != B + 1):
            raise ValueError("block_table, seq_lens and starts disagree about the batch")
        return dkv_kv4_batch(B, width, block_table.data_ptr(), seq_lens.data_ptr(),
                             None if starts is None else starts.data_ptr())

    def _rows(self, x, name, heads=None):
        """[rows, heads, head_dim] with contiguous channels: shape, row and head
        strides (a dimension of one has none that matters) and type code."""
        if x.get_device() != self._index or x.dim() != 3:
            self._tensor(x, name, 3)
        shape, (row, head, one) = x.shape, x.stride()
        if shape[2] != self.desc.head_dim or (heads is not None and shape[1] != heads) \
                or shape[0] > _I32_MAX:
            raise ValueError(f"{name} has shape {tuple(shape)}")
        if one != 1:
            raise ValueError(f"{name} must have contiguous channels")
        code = self._codes.get(x.dtype)
        if code is None:
            raise ValueError(f"{name} is {x.dtype}")
        return shape, row if shape[0] > 1 else 0, head if shape[1] > 1 else 0, code

    def _elsewhere(self, stream):
        """None where calls go to the current stream of the current device;
        otherwise a context that makes it so."""
        torch = self._torch
        if stream is None:
            if torch.cuda.current_device() == self._index:
                return None
            return torch.cuda.device(self.device)
        if not isinstance(stream, int) and stream.device != self.device:
            raise ValueError(f"the stream is of {stream.device}, the cache on {self.device}")
        return _on(stream, self.device)

    # -- the operators ------------------------------------------------------
    def append(self, K_new, V_new, block_table, seq_lens, starts=None, stream=None):
        """Quantise the rows K_new, V_new [rows, n_kv_heads, head_dim] (fp32,
        fp16 or bf16; views with row and head strides) into their sequences'
        pages (dkv_kv4_append)."""
        ctx = self._elsewhere(stream)
        if ctx is not None:
            with ctx:
                return self.append(K_new, V_new, block_table, seq_lens, starts)
        H = self.desc.n_kv_heads
        shape, k_row, k_head, code = self._rows(K_new, "K_new", H)
        v_shape, v_row, v_head, v_code = self._rows(V_new, "V_new", H)
        if shape != v_shape or code != v_code:
            raise ValueError("K_new and V_new differ in shape or dtype")
        seqs = self._batch(block_table, seq_lens, starts)
        if shape[0]:
            _check(self._lib.dkv_kv4_append(
                self._pool, ctypes.byref(seqs), K_new.data_ptr(), V_new.data_ptr(), code, shape[0],
                k_row, k_head, v_row, v_head, self._stream(self._index)), "dkv_kv4_append")

    def read(self, n_rows, block_table, seq_lens, starts=None, dtype=None, out=None, stream=None):
        """The values held at the rows' positions (dkv_kv4_read): (K, V), each
        [n_rows, n_kv_heads, head_dim] of dtype (default fp16).  out: a pair of
        contiguous tensors to write instead; padding rows are left as they are."""
        ctx = self._elsewhere(stream)
        if ctx is not None:
            with ctx:
                return self.read(n_rows, block_table, seq_lens, starts, dtype, out)
        torch = self._torch
        shape = (n_rows, self.desc.n_kv_heads, self.desc.head_dim)
        seqs = self._batch(block_table, seq_lens, starts)
        if dtype is None:
            dtype = torch.float16 if out is None else out[0].dtype
        if dtype not in self._codes:
            raise ValueError(f"dtype is {dtype}, not fp32, fp16 or bf16")
        if out is None:
            k = self.status.new_empty(shape, dtype=dtype)
            out = (k, torch.empty_like(k))
        else:
            for x in out:
                self._tensor(x, "out")
                if tuple(x.shape) != shape or not x.is_contiguous() or x.dtype != dtype:
                    raise ValueError("out must be two contiguous tensors [n_rows, n_kv_heads, "
                                     "head_dim] of dtype")
        k, v = out
        if n_rows:
            _check(self._lib.dkv_kv4_read(self._pool, ctypes.byref(seqs), k.data_ptr(),
                                          v.data_ptr(), self._codes[k.dtype], n_rows,
                                          self._stream(self._index)), "dkv_kv4_read")
        return out

    def _attn(self, what, rows, Q, sizes, n_queries, seqs, softmax_scale, window, out, return_lse):
        """The rest of an attention call.  rows: Q as [rows, n_q_heads, D];
        sizes: what its workspace depends on."""
        torch = self._torch
        shape, row, head, code = self._rows(rows, "Q")
        # (like tensors that are at hand: half of torch.empty's time on the host)
        if out is None:
            out = torch.empty_like(Q, memory_format=torch.contiguous_format)
        else:
            if out.shape != Q.shape or out.dtype != Q.dtype or not out.is_contiguous():
                raise ValueError("out must be contiguous, of Q's shape and dtype")
            self._tensor(out, "out")
        lse = Q.new_empty(Q.shape[:-1], dtype=torch.float32) if return_lse else None
        if shape[0]:
            lib = self._lib
            size, call = (lib.dkv_kv4_decode_workspace_bytes, lib.dkv_kv4_decode_attn) \
                if what == "decode" else (lib.dkv_kv4_prompt_workspace_bytes, lib.dkv_kv4_prompt_attn)
            nb = size(self._desc, *sizes)
            # a window past every position counts as none: it need not fit 32 bits
            window = max(-1, min(window, _I32_MAX))
            ws = self.status.new_empty(nb // 4 + 4)
            _check(call(self._pool, ctypes.byref(seqs), rows.data_ptr(), code, shape[1], n_queries,
                     row, head, softmax_scale, window, out.data_ptr(),
                     None if lse is None else lse.data_ptr(), ws.data_ptr(), nb,
                     self._stream(self._index)), f"dkv_kv4_{what}_attn")
        return (out, lse) if return_lse else out

    def decode_attn(self, Q, softmax_scale, block_table, seq_lens, window=0, out=None,
                    return_lse=False, stream=None):
        """Decode attention (dkv_kv4_decode_attn).  Q [batch, n_q_heads, D], or
        [batch, n_queries, n_q_heads, D] for the n_queries newest positions;
        fp16 or bf16.  Returns Q's shape and dtype (and the log-sum-exp, fp32)."""
        ctx = self._elsewhere(stream)
        if ctx is not None:
            with ctx:
                return self.decode_attn(Q, softmax_scale, block_table, seq_lens, window, out,
                                        return_lse)
        shape = Q.shape
        if len(shape) not in (3, 4):
            raise ValueError("Q has shape [batch, n_q_heads, D] or [batch, n_queries, n_q_heads, D]")
        seqs = self._batch(block_table, seq_lens, None)
        if shape[0] != seqs.batch:
            raise ValueError("Q and seq_lens disagree about the batch")
        nq, rows = 1, Q
        if len(shape) == 4:
            # one row stride: a copy only where the batch is no plain view
            nq, rows = shape[1], Q.reshape(-1, shape[2], shape[3])
        return self._attn("decode", rows, Q, (seqs.batch, seqs.max_pages, shape[-2], nq), nq, seqs,
                          softmax_scale, window, out, return_lse)

    def prompt_attn(self, Q, softmax_scale, block_table, seq_lens, starts=None, window=0,
                    out=None, return_lse=False, stream=None):
        """Prompt attention (dkv_kv4_prompt_attn): Q [rows, n_q_heads, D] (fp16
        or bf16), the rows of `starts`, whose keys and values are in the cache.
        Returns Q's shape and dtype (and the log-sum-exp, fp32); padding rows
        of `out` are left as they are (undefined in a new one)."""
        ctx = self._elsewhere(stream)
        if ctx is not None:
            with ctx:
                return self.prompt_attn(Q, softmax_scale, block_table, seq_lens, starts, window,
                                        out, return_lse)
        if Q.dim() != 3:
            self._tensor(Q, "Q", 3)
        seqs = self._batch(block_table, seq_lens, starts)
        n, Hq = Q.shape[:2]
        return self._attn("prompt", Q, Q, (seqs.batch, seqs.max_pages, Hq, n, int(starts is not None)),
                          n, seqs, softmax_scale, window, out, return_lse)

    def device_status(self, stream=None) -> int:
        """Read the pool's status word and clear what was read (synchronises)."""
        ctx = self._elsewhere(stream)
        if ctx is not None:
            with ctx:
                return self.device_status()
        return dkv_kv4_get_device_status(self.c, self._stream(self._index))
