"""ctypes binding of libmha_gb300.so (include/mha.h).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the cudaStream_t, and status codes become exceptions.  Every
step of the computation runs in the library's CUDA kernels; there is no CPU
or PyTorch fallback, and a missing library is an error.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

MHA_OK = 0
MHA_ERR_INVALID_ARG = 1
MHA_ERR_UNSUPPORTED = 2
MHA_ERR_CUDA = 3
MHA_ERR_OOM = 4
MHA_ERR_TIMEOUT = 5
MHA_ERR_DEVICE = 6

MHA_F32 = 0
MHA_BF16 = 1
MHA_E4M3 = 2

MASK_NONE = 0
MASK_CAUSAL = 1
MASK_KEY_PADDING = 2
MASK_CAUSAL_BOTTOM_RIGHT = 4

ROPE_INTERLEAVED = 0
ROPE_HALF = 1

LIB_PATH = _build.LIB

_lock = threading.Lock()
_lib = None


ENCODER_PARAM_NAMES = ("Wq", "Wk", "Wv", "Wo", "bq", "bk", "bv", "bo", "ln1_gamma",
                       "ln1_beta", "W1", "b1", "W2", "b2", "ln2_gamma", "ln2_beta")


class EncoderParams(ctypes.Structure):
    """mha_encoder_params of include/mha.h (device pointers)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ENCODER_PARAM_NAMES]


class KvPages(ctypes.Structure):
    """mha_kv_pages of include/mha.h."""
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("d", ctypes.c_int), ("layers", ctypes.c_int),
                ("page_stride", ctypes.c_int64), ("layer_stride", ctypes.c_int64),
                ("page_table", ctypes.c_void_p), ("kv_lengths", ctypes.c_void_p),
                ("B", ctypes.c_int), ("table_cols", ctypes.c_int)]


class KvScales(ctypes.Structure):
    """mha_kv_scales of include/mha.h."""
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p)]


class MhaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def _declare(lib):
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.sdpa_forward.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp,
                                 i32, i32, vp]
    lib.sdpa_forward.restype = i32
    lib.sdpa_decode.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp, i32, i32,
                                vp]
    lib.sdpa_decode.restype = i32
    lib.sdpa_forward_lse.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp,
                                     i32, vp]
    lib.sdpa_forward_lse.restype = i32
    lib.sdpa_backward_workspace_bytes.argtypes = [i32, i32, i32]
    lib.sdpa_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.sdpa_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                  f32, i32, vp, i32, vp, ctypes.c_size_t, vp]
    lib.sdpa_backward.restype = i32
    lib.sdpa_forward_host_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.sdpa_forward_host_workspace_bytes.restype = ctypes.c_size_t
    lib.sdpa_forward_host.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp, i32,
                                      i32, vp, ctypes.c_size_t, vp]
    lib.sdpa_forward_host.restype = i32
    lib.sinusoidal_pe.argtypes = [vp, i32, i32, i32, vp]
    lib.sinusoidal_pe.restype = i32
    lib.embed_pe_forward.argtypes = [vp, vp, i32, vp, i32, vp, i32, i32, i32, i32, f32, i32, vp]
    lib.embed_pe_forward.restype = i32
    lib.sdpa_decode_splits.argtypes = [i32, i32, i32, i32]
    lib.sdpa_decode_splits.restype = i32
    i64 = ctypes.c_int64
    kvp = ctypes.POINTER(KvPages)
    lib.sdpa_paged.argtypes = [vp, i64, kvp, i32, vp, vp, i32, i32, i32, f32, i32, i32, i32, vp]
    lib.sdpa_paged.restype = i32
    lib.qk_norm_rope_forward.argtypes = [vp, i64, vp, i64, vp, vp, vp, i32, i32, i32, vp, vp, i32,
                                         i32, i32, i32, i32, i32, vp, f32, i32, vp]
    lib.qk_norm_rope_forward.restype = i32
    lib.qk_norm_rope_backward.argtypes = [vp, i64, vp, i64, vp, vp, vp, i32, i32, i32, vp, vp, vp,
                                          i64, vp, i64, vp, vp, i32, i32, i32, i32, i32, i32, vp,
                                          f32, i32, i32, i32, vp, ctypes.c_size_t, vp]
    lib.qk_norm_rope_backward.restype = i32
    lib.qk_norm_rope_backward_workspace_bytes.argtypes = [i32]
    lib.qk_norm_rope_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.qk_norm_rope_paged.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, vp, i32, i32, i32, vp,
                                       kvp, i32, vp, i32, i32, f32, vp]
    lib.qk_norm_rope_paged.restype = i32
    lib.kv_pages_fork.argtypes = [kvp, vp, vp, vp, i32, vp]
    lib.kv_pages_fork.restype = i32
    lib.kv_pages_compact_workspace_bytes.argtypes = [i32]
    lib.kv_pages_compact_workspace_bytes.restype = ctypes.c_size_t
    lib.kv_pages_compact.argtypes = [kvp, kvp, vp, vp, ctypes.c_size_t, vp]
    lib.kv_pages_compact.restype = i32
    scp, sz = ctypes.POINTER(KvScales), ctypes.c_size_t
    lib.sdpa_paged_e4m3.argtypes = [vp, i64, kvp, scp, i32, vp, vp, i32, i32, i32, f32, i32, i32,
                                    i32, vp]
    lib.sdpa_paged_e4m3.restype = i32
    lib.qk_norm_rope_paged_e4m3.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, vp, i32, i32, i32, vp,
                                            kvp, scp, i32, vp, i32, i32, f32, vp]
    lib.qk_norm_rope_paged_e4m3.restype = i32
    lib.kv_pages_fork_e4m3.argtypes = [kvp, scp, vp, vp, vp, i32, vp]
    lib.kv_pages_fork_e4m3.restype = i32
    lib.kv_pages_compact_e4m3.argtypes = [kvp, scp, kvp, scp, vp, vp, sz, vp]
    lib.kv_pages_compact_e4m3.restype = i32
    lib.kv_pages_bounds.argtypes = [kvp, scp, i32, vp, i32, vp, vp, vp]
    lib.kv_pages_bounds.restype = i32
    lib.kv_pages_select_workspace_bytes.argtypes = [i32, i32, i32]
    lib.kv_pages_select_workspace_bytes.restype = sz
    lib.kv_pages_select.argtypes = [vp, i64, kvp, i32, vp, vp, vp, i32, i32, i32, vp, vp, vp, sz, vp]
    lib.kv_pages_select.restype = i32
    lib.sdpa_paged_selected.argtypes = [vp, i64, kvp, scp, i32, vp, vp, i32, vp, i32, i32, f32, i32,
                                        i32, vp]
    lib.sdpa_paged_selected.restype = i32
    lib.sdpa_forward_float_mask.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32,
                                            vp, vp, i64, i64, i32, i32, vp]
    lib.sdpa_forward_float_mask.restype = i32
    lib.encoder_create.argtypes = [ctypes.POINTER(vp), i32, i32, i32, i32, i32, i32]
    lib.encoder_create.restype = i32
    lib.encoder_forward.argtypes = [vp, vp, ctypes.POINTER(EncoderParams), i32, i32, i32, vp,
                                    f32, vp, i32, vp]
    lib.encoder_forward.restype = i32
    lib.encoder_destroy.argtypes = [vp]
    lib.encoder_destroy.restype = i32
    lib.mha_create.argtypes = [ctypes.POINTER(vp), i32, i32, i32, i32, i32]
    lib.mha_create.restype = i32
    lib.mha_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]
    lib.mha_forward.restype = i32
    lib.mha_check.argtypes = [vp]
    lib.mha_check.restype = i32
    lib.mha_destroy.argtypes = [vp]
    lib.mha_destroy.restype = i32
    lib.mha_status_string.argtypes = [i32]
    lib.mha_status_string.restype = ctypes.c_char_p
    lib.mha_set_wait_limit_ms.argtypes = [i32]
    lib.mha_set_wait_limit_ms.restype = i32
    lib.mha_selftest_wait_timeout.argtypes = [i32, vp]
    lib.mha_selftest_wait_timeout.restype = i32
    return lib


def lib():
    """The loaded library.  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"CUDA library {LIB_PATH} is missing; build it with "
                    "transformer_head_scaled_03_gb300.build.build()")
            _lib = _declare(ctypes.CDLL(LIB_PATH))
    return _lib


def status_string(status: int) -> str:
    return lib().mha_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != MHA_OK:
        raise MhaError(status, what)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return MHA_BF16
    if t == torch.float32:
        return MHA_F32
    raise TypeError(f"unsupported dtype {t}")


def _dev_ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr()) if t.numel() else None


def _stream(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _mask_strides(add_mask, B, H, Lq, Lk):
    """Batch and head strides (elements, 0 = broadcast) of a float32 mask
    broadcastable to [B, H, Lq, Lk] whose [Lq, Lk] rows are contiguous."""
    if add_mask.dtype != torch.float32 or not add_mask.is_cuda:
        raise ValueError("add_mask must be a float32 CUDA tensor")
    m = add_mask
    while m.dim() < 4:
        m = m.unsqueeze(0)
    if m.dim() != 4 or tuple(m.shape[2:]) != (Lq, Lk) or m.shape[0] not in (1, B) \
            or m.shape[1] not in (1, H):
        raise ValueError("add_mask must broadcast to [B, H, Lq, Lk]")
    if Lk > 1 and m.stride(3) != 1 or Lq > 1 and m.stride(2) != Lk:
        raise ValueError("add_mask rows must be contiguous")
    sb = m.stride(0) if m.shape[0] > 1 else 0
    sh = m.stride(1) if m.shape[1] > 1 else 0
    return sb, sh


def sdpa_forward(Q, K, V, scale: float | None = None, mask_kind: int = MASK_NONE,
                 key_lengths=None, out_dtype: torch.dtype | None = None, out=None,
                 stream=None, add_mask=None):
    """O = softmax(Q K^T * scale + mask) V for Q [B,H,Lq,d], K/V [B,H,Lk,d].

    ``add_mask``: optional float32 tensor broadcastable to [B,H,Lq,Lk], added
    to the scaled scores (-inf blocks a key)."""
    B, H, Lq, d = Q.shape
    Lk = K.shape[2]
    if K.shape != (B, H, Lk, d) or V.shape != (B, H, Lk, d):
        raise ValueError("Q/K/V shapes disagree")
    if K.dtype != Q.dtype or V.dtype != Q.dtype:
        raise ValueError("Q/K/V dtypes disagree")
    odt = out_dtype or Q.dtype
    if out is None:
        out = torch.empty((B, H, Lq, d), dtype=odt, device=Q.device)
    elif out.shape != (B, H, Lq, d) or out.dtype != odt:
        raise ValueError("out has the wrong shape or dtype")
    if key_lengths is not None and key_lengths.dtype != torch.int32:
        raise ValueError("key_lengths must be int32")
    if add_mask is not None:
        sb, sh = _mask_strides(add_mask, B, H, Lq, Lk)
        st = lib().sdpa_forward_float_mask(
            _dev_ptr(Q), _dev_ptr(K), _dev_ptr(V), _dev_ptr(out), B, H, Lq, Lk, d,
            float(scale or 0.0), int(mask_kind), _dev_ptr(key_lengths),
            ctypes.c_void_p(add_mask.data_ptr()), sb, sh, _dtype_code(Q.dtype),
            _dtype_code(odt), _stream(stream))
        _check(st, "sdpa_forward_float_mask")
        return out
    st = lib().sdpa_forward(_dev_ptr(Q), _dev_ptr(K), _dev_ptr(V), _dev_ptr(out), B, H, Lq, Lk,
                            d, float(scale or 0.0), int(mask_kind), _dev_ptr(key_lengths),
                            _dtype_code(Q.dtype), _dtype_code(odt), _stream(stream))
    _check(st, "sdpa_forward")
    return out


def sdpa_decode(Q, K_cache, V_cache, kv_lengths=None, causal: bool = True,
                scale: float | None = None, out_dtype: torch.dtype | None = None,
                num_splits: int = 0, out=None, stream=None):
    """Decode-shape attention: Q [B,H,Lq<=16,d] (the newest Lq positions)
    against caches K/V [B,H,Lk,d] holding kv_lengths[b] tokens (all Lk when
    None); bottom-right causal unless ``causal`` is False."""
    B, H, Lq, d = Q.shape
    Lk = K_cache.shape[2]
    if K_cache.shape != (B, H, Lk, d) or V_cache.shape != (B, H, Lk, d):
        raise ValueError("Q/cache shapes disagree")
    if K_cache.dtype != Q.dtype or V_cache.dtype != Q.dtype:
        raise ValueError("Q/cache dtypes disagree")
    odt = out_dtype or Q.dtype
    if out is None:
        out = torch.empty((B, H, Lq, d), dtype=odt, device=Q.device)
    elif out.shape != (B, H, Lq, d) or out.dtype != odt:
        raise ValueError("out has the wrong shape or dtype")
    mask = MASK_CAUSAL_BOTTOM_RIGHT if causal else MASK_NONE
    if kv_lengths is not None:
        if kv_lengths.dtype != torch.int32:
            raise ValueError("kv_lengths must be int32")
        mask |= MASK_KEY_PADDING
    st = lib().sdpa_decode(_dev_ptr(Q), _dev_ptr(K_cache), _dev_ptr(V_cache), _dev_ptr(out), B, H,
                           Lq, Lk, d, float(scale or 0.0), mask, _dev_ptr(kv_lengths),
                           _dtype_code(odt), int(num_splits), _stream(stream))
    _check(st, "sdpa_decode")
    return out


def decode_splits(B: int, H: int, Lk: int, d: int) -> int:
    """The split count sdpa_decode picks by default."""
    return int(lib().sdpa_decode_splits(B, H, Lk, d))


def sdpa_forward_lse(Q, K, V, scale: float | None = None, mask_kind: int = MASK_NONE,
                     key_lengths=None, out=None, lse=None, stream=None):
    """bf16 forward that also returns the base-2 row log-sum-exp [B,H,Lq]."""
    B, H, Lq, d = Q.shape
    Lk = K.shape[2]
    if Q.dtype != torch.bfloat16 or K.dtype != Q.dtype or V.dtype != Q.dtype:
        raise ValueError("bf16 Q/K/V required")
    if out is None:
        out = torch.empty_like(Q)
    if lse is None:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=Q.device)
    st = lib().sdpa_forward_lse(_dev_ptr(Q), _dev_ptr(K), _dev_ptr(V), _dev_ptr(out),
                                _dev_ptr(lse), B, H, Lq, Lk, d, float(scale or 0.0),
                                int(mask_kind), _dev_ptr(key_lengths), _dtype_code(out.dtype),
                                _stream(stream))
    _check(st, "sdpa_forward_lse")
    return out, lse


def sdpa_backward(Q, K, V, O, dO, lse, scale: float | None = None, mask_kind: int = MASK_NONE,
                  key_lengths=None, grad_dtype: torch.dtype = torch.bfloat16, workspace=None,
                  stream=None):
    """(dQ fp32, dK, dV) of scaled dot-product attention for upstream dO."""
    B, H, Lq, d = Q.shape
    Lk = K.shape[2]
    dQ = torch.empty((B, H, Lq, d), dtype=torch.float32, device=Q.device)
    dK = torch.empty((B, H, Lk, d), dtype=grad_dtype, device=Q.device)
    dV = torch.empty((B, H, Lk, d), dtype=grad_dtype, device=Q.device)
    need = int(lib().sdpa_backward_workspace_bytes(B, H, Lq))
    if workspace is None:
        workspace = torch.empty(max(16, (need + 15) // 16 * 16), dtype=torch.uint8,
                                device=Q.device)
    st = lib().sdpa_backward(_dev_ptr(Q), _dev_ptr(K), _dev_ptr(V), _dev_ptr(O), _dev_ptr(dO),
                             _dev_ptr(lse), _dev_ptr(dQ), _dev_ptr(dK), _dev_ptr(dV), B, H, Lq, Lk,
                             d, float(scale or 0.0), int(mask_kind), _dev_ptr(key_lengths),
                             _dtype_code(grad_dtype), _dev_ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "sdpa_backward")
    return dQ, dK, dV


def sinusoidal_pe(n_pos: int, d_model: int, first_pos: int = 0, out=None, stream=None,
                  device=None):
    """The positional-encoding table, fp32 [n_pos, d_model] on the device."""
    if out is None:
        out = torch.empty((n_pos, d_model), dtype=torch.float32,
                          device=device if device is not None else "cuda")
    elif out.shape != (n_pos, d_model) or out.dtype != torch.float32:
        raise ValueError("out has the wrong shape or dtype")
    _check(lib().sinusoidal_pe(_dev_ptr(out), int(first_pos), int(n_pos), int(d_model),
                               _stream(stream)), "sinusoidal_pe")
    return out


def embed_pe(ids, table, pe, pos_offset: int = 0, scale: float | None = None, out=None,
             stream=None):
    """x [B, L, D] = table[ids] * scale (default sqrt(D)) + pe[pos_offset + l]."""
    B, L = ids.shape
    vocab, D = table.shape
    if ids.dtype != torch.int32:
        raise ValueError("ids must be int32")
    if pe.dtype != torch.float32 or pe.dim() != 2 or pe.shape[1] != D:
        raise ValueError("pe must be float32 [rows, D]")
    if out is None:
        out = torch.empty((B, L, D), dtype=table.dtype, device=table.device)
    elif out.shape != (B, L, D) or out.dtype != table.dtype:
        raise ValueError("out has the wrong shape or dtype")
    st = lib().embed_pe_forward(_dev_ptr(ids), _dev_ptr(table), vocab, _dev_ptr(pe), pe.shape[0],
                                _dev_ptr(out), B, L, D, int(pos_offset), float(scale or 0.0),
                                _dtype_code(table.dtype), _stream(stream))
    _check(st, "embed_pe_forward")
    return out


def _int32(name, t, *shape):
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)}")


def _c_int(name, v):
    """v as a C int (ctypes drops the bits above 32 without a word)."""
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} out of range")
    return v


def _launch_on(stream, *tensors):
    """Check that every tensor is on the current device, where the library
    launches; the raw stream to launch on.  (The paged calls take tens of
    microseconds or less, so what the host does for each of them counts.)"""
    if not tensors[0].is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    here = torch._C._cuda_getDevice()
    for t in tensors:
        if t.get_device() != here:
            raise ValueError(f"tensors must be on the current CUDA device (cuda:{here})")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(here)
    if stream.device_index != here:
        raise ValueError(f"stream must be on the current device (cuda:{here})")
    return stream.cuda_stream


def _given(*tensors):
    return [t for t in tensors if t is not None]


def _new(stream, shape, dtype, device):
    """A tensor that `stream` (the current one when None) may use; the caching
    allocator keeps its memory until that stream is past it."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None and stream != torch.cuda.current_stream():
        # what freed this memory ran on the current stream, so the kernels
        # start behind that
        stream.wait_stream(torch.cuda.current_stream())
        t.record_stream(stream)
    return t


def _check_workspace(workspace):
    """A given workspace's size is counted from its elements."""
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _kv_pools(K_pages, V_pages):
    """What an mha_kv_pages says of pools [P, Hkv, page, d] or [layers, P, Hkv,
    page, d] (pages and layers at any stride, a page itself contiguous)."""
    shape = K_pages.shape
    if len(shape) not in (4, 5) or V_pages.shape != shape or V_pages.dtype != K_pages.dtype:
        raise ValueError("K_pages and V_pages must be alike, [P, Hkv, page, d] or "
                         "[layers, P, Hkv, page, d]")
    P, Hkv, ps, d = shape[-4:]
    layers = shape[0] if len(shape) == 5 else 1
    strides = K_pages.stride()
    if V_pages.stride() != strides or strides[-3:] != (ps * d, d, 1) or P == 1:
        # a size of 1 has any stride: 0, as good as dense, stands for it
        strides, other = (
            (s[0] if layers > 1 else 0, s[-4] if P > 1 else 0, s[-3] if Hkv > 1 else ps * d, *s[-2:])
            for s in (strides, V_pages.stride()))
        if strides[-3:] != (ps * d, d, 1) or other != strides:
            raise ValueError("a page must be contiguous, and K_pages and V_pages laid out alike")
    # the library reads a stride of 0 as "dense"
    if P > 1 and strides[-4] == 0 or layers > 1 and strides[0] == 0:
        raise ValueError("pages and layers must not be broadcast")
    dtype = MHA_E4M3 if K_pages.dtype is _E4M3 else _dtype_code(K_pages.dtype)
    return (K_pages.data_ptr(), V_pages.data_ptr(), dtype, P, ps, Hkv, d, layers, strides[-4],
            strides[0] if layers > 1 else 0)


def _kv_pages(K_pages, V_pages, page_table, kv_lengths):
    """The mha_kv_pages of a cache."""
    pools = _kv_pools(K_pages, V_pages)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, pages per sequence]")
    B, cols = page_table.shape
    _int32("page_table", page_table, B, cols)
    _int32("kv_lengths", kv_lengths, B)
    return KvPages(*pools, page_table.data_ptr(), kv_lengths.data_ptr(), B, cols)


_E4M3 = torch.float8_e4m3fn


def _kv_scales(K_pages, K_scale, V_scale):
    """The mha_kv_scales of pools in 8 bits, None for others."""
    if K_pages.dtype is not _E4M3:
        if K_scale is not None or V_scale is not None:
            raise ValueError("K_scale and V_scale are for pages in 8 bits (float8_e4m3fn)")
        return None
    if K_scale is None or V_scale is None:
        raise ValueError("pages in 8 bits need K_scale and V_scale")
    want = K_pages.shape[:-2]
    for name, s in (("K_scale", K_scale), ("V_scale", V_scale)):
        if s.dtype is not torch.float32 or s.shape != want or not s.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 tensor of shape {list(want)}")
    return KvScales(K_scale.data_ptr(), V_scale.data_ptr())


def _packed(name, x, heads, d, dtype):
    """Token stride of packed rows [T, heads, d] (a slice of a wider tensor's
    last dimension will do)."""
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or x.dtype != dtype:
        raise ValueError(f"{name} must be [T, {heads}, {d}] {dtype}")
    st, sh, sc = x.stride()
    if sc != 1 or (heads > 1 and sh != d):
        raise ValueError(f"{name}'s heads must be contiguous")
    if shape[0] <= 1:
        return heads * d
    if st == 0:     # a broadcast: the library reads 0 as "dense"
        raise ValueError(f"{name}'s tokens must be evenly spaced, a row or more apart")
    return st


def sdpa_paged(Q, K_pages, V_pages, page_table, kv_lengths, q_offsets, max_new: int | None = None,
               causal: bool = True, scale: float | None = None,
               out_dtype: torch.dtype | None = None, layer: int = 0, num_splits: int = 0, out=None,
               stream=None, K_scale=None, V_scale=None):
    """O [T, H, d] = attention of packed new tokens Q [T, H, d] (sequence b's
    are q_offsets[b]..q_offsets[b+1], the newest of its kv_lengths[b] tokens)
    over a paged cache K_pages, V_pages [P, Hkv, page, d] (or with a leading
    layer dimension); bottom-right causal unless ``causal`` is False.
    ``max_new`` bounds the new tokens of one sequence (default: T, which costs
    a batch of single tokens a sixth to a third more than ``max_new=1``).
    Pages in 8 bits (float8_e4m3fn, Q in bf16) come with ``K_scale`` and
    ``V_scale`` float32 [P, Hkv] (or [layers, P, Hkv])."""
    pages = _kv_pages(K_pages, V_pages, page_table, kv_lengths)
    scales = _kv_scales(K_pages, K_scale, V_scale)
    if Q.dim() != 3 or Q.dtype != (K_pages.dtype if scales is None else torch.bfloat16):
        raise ValueError("Q must be [T, H, d] of the cache's dtype, or bf16 over pages in 8 bits")
    T, H, d = Q.shape
    q_ts = _packed("Q", Q, H, pages.d, Q.dtype)
    _int32("q_offsets", q_offsets, pages.B + 1)
    odt = out_dtype or Q.dtype
    layer, num_splits = _c_int("layer", layer), _c_int("num_splits", num_splits)
    # a bound above T says no more than T
    max_new = max(1, T) if max_new is None else min(int(max_new), max(1, T))
    max_new = _c_int("max_new", max_new)
    on = _launch_on(stream, Q, K_pages, V_pages, page_table, kv_lengths, q_offsets,
                    Q if out is None else out, *_given(K_scale, V_scale))
    if out is None:
        out = _new(stream, (T, H, d), odt, Q.device)
    elif out.shape != (T, H, d) or out.dtype != odt or not out.is_contiguous():
        raise ValueError("out has the wrong shape, dtype or layout")
    rest = (layer, q_offsets.data_ptr(), out.data_ptr(), T, H, max_new, float(scale or 0.0),
            MASK_CAUSAL_BOTTOM_RIGHT if causal else MASK_NONE, _dtype_code(odt), num_splits, on)
    dev = _lib or lib()
    if scales is None:
        _check(dev.sdpa_paged(Q.data_ptr(), q_ts, pages, *rest), "sdpa_paged")
    else:
        _check(dev.sdpa_paged_e4m3(Q.data_ptr(), q_ts, pages, scales, *rest), "sdpa_paged_e4m3")
    return out


def _token_rows(name, x, B, L, d, dtype):
    """Heads and token stride of rows [B, L, heads, d] whose tokens are evenly
    spaced (a dense tensor, or a slice of a projection's output)."""
    shape = x.shape
    if len(shape) != 4 or shape[0] != B or shape[1] != L or shape[3] != d or x.dtype is not dtype:
        raise ValueError(f"{name} must be [{B}, {L}, heads, {d}] {dtype}")
    heads, (sb, sl, sh, sc) = shape[2], x.stride()
    ts = sl if L > 1 else sb if B > 1 else heads * d
    # a stride of 0 is a broadcast, which the library would read as "dense"
    if (sc != 1 and d > 1 or heads > 1 and sh != d or B > 1 and L > 1 and sb != L * ts
            or ts == 0) and x.numel():
        raise ValueError(f"{name}'s tokens must be evenly spaced and its heads contiguous")
    return heads, ts


def _rope_args(Q, K, gamma_q, gamma_k, pe, positions):
    if Q.dim() != 4:
        raise ValueError("Q and K must be [B, L, heads, d]")
    B, L, _, d = Q.shape
    H, q_ts = _token_rows("Q", Q, B, L, d, Q.dtype)
    Hkv, k_ts = _token_rows("K", K, B, L, d, Q.dtype)
    _gammas(gamma_q, gamma_k, pe, d, Q.dtype)
    if positions is not None:
        _int32("positions", positions, B, L)
    return B, L, H, Hkv, d, q_ts, k_ts


def _gammas(gamma_q, gamma_k, pe, d, dtype):
    for g in (gamma_q, gamma_k):
        if g.numel() != d or g.dim() != 1 or g.dtype is not dtype or not g.is_contiguous():
            raise ValueError("gamma_q and gamma_k must be contiguous [d] of the rows' dtype")
    if pe.dtype is not torch.float32 or pe.dim() != 2 or not pe.is_contiguous():
        raise ValueError("pe must be contiguous float32 [rows, rope_dim]")


def qk_norm_rope(Q, K, gamma_q, gamma_k, pe, pos_offset: int = 0, positions=None,
                 pairing: int = ROPE_INTERLEAVED, eps: float = 1e-6, out=None, stream=None):
    """(Q' [B, H, L, d], K' [B, Hkv, L, d]): every head of Q [B, L, H, d] and
    K [B, L, Hkv, d] divided by its root mean square, times gamma [d], its
    first pe.shape[1] columns rotated by the token's position (a row of pe, a
    ``sinusoidal_pe`` table): ``positions`` int32 [B, L], or pos_offset + l."""
    B, L, H, Hkv, d, q_ts, k_ts = _rope_args(Q, K, gamma_q, gamma_k, pe, positions)
    pos_offset, pairing = _c_int("pos_offset", pos_offset), _c_int("pairing", pairing)
    on = _launch_on(stream, Q, K, gamma_q, gamma_k, pe, Q if positions is None else positions,
                    *(() if out is None else out))
    want = ((B, H, L, d), (B, Hkv, L, d))
    if out is None:
        out = (_new(stream, want[0], Q.dtype, Q.device), _new(stream, want[1], Q.dtype, Q.device))
    else:
        for o, s in zip(out, want):
            if o.shape != s or o.dtype != Q.dtype or not o.is_contiguous():
                raise ValueError("out has the wrong shapes, dtype or layout")
    rows, r = pe.shape
    st = (_lib or lib()).qk_norm_rope_forward(
        Q.data_ptr(), q_ts, K.data_ptr(), k_ts, gamma_q.data_ptr(), gamma_k.data_ptr(),
        pe.data_ptr(), rows, r, pairing, out[0].data_ptr(), out[1].data_ptr(), B, L, H, Hkv,
        d, pos_offset, None if positions is None else positions.data_ptr(), float(eps),
        _dtype_code(Q.dtype), on)
    _check(st, "qk_norm_rope_forward")
    return out


def qk_norm_rope_backward(Q, K, gamma_q, gamma_k, pe, dQo, dKo, pos_offset: int = 0,
                          positions=None, pairing: int = ROPE_INTERLEAVED, eps: float = 1e-6,
                          out=None, workspace=None, stream=None):
    """(dQ [B, L, H, d], dK [B, L, Hkv, d], dgamma_q, dgamma_k fp32 [d]) of
    qk_norm_rope for upstream dQo [B, H, L, d], dKo [B, Hkv, L, d] (bf16 or
    fp32 each, as ``sdpa_backward`` returns them).  ``out``: (dQ, dK) to fill,
    laid out as Q and K may be."""
    B, L, H, Hkv, d, q_ts, k_ts = _rope_args(Q, K, gamma_q, gamma_k, pe, positions)
    pos_offset, pairing = _c_int("pos_offset", pos_offset), _c_int("pairing", pairing)
    if dQo.shape != (B, H, L, d) or dKo.shape != (B, Hkv, L, d) \
            or not dQo.is_contiguous() or not dKo.is_contiguous():
        raise ValueError("dQo and dKo must be contiguous [B, heads, L, d]")
    _check_workspace(workspace)
    on = _launch_on(stream, Q, K, gamma_q, gamma_k, pe, dQo, dKo,
                    Q if positions is None else positions, Q if workspace is None else workspace,
                    *(() if out is None else out))
    if out is None:
        out = (_new(stream, (B, L, H, d), Q.dtype, Q.device),
               _new(stream, (B, L, Hkv, d), Q.dtype, Q.device))
        dq_ts, dk_ts = H * d, Hkv * d
    else:
        (h0, dq_ts), (h1, dk_ts) = (_token_rows("out", o, B, L, d, Q.dtype) for o in out)
        if h0 != H or h1 != Hkv:
            raise ValueError("out has the wrong shapes")
    # each gamma's gradient starts on 16 bytes
    dgamma_q, dgamma_k = _new(stream, (2, d + -d % 4), torch.float32, Q.device).unbind(0)
    if d % 4:
        dgamma_q, dgamma_k = dgamma_q[:d], dgamma_k[:d]
    dev = _lib or lib()
    if workspace is None:
        workspace = _new(stream, (dev.qk_norm_rope_backward_workspace_bytes(d) or 16,),
                         torch.uint8, Q.device)
    rows, r = pe.shape
    st = dev.qk_norm_rope_backward(
        Q.data_ptr(), q_ts, K.data_ptr(), k_ts, gamma_q.data_ptr(), gamma_k.data_ptr(),
        pe.data_ptr(), rows, r, pairing, dQo.data_ptr(), dKo.data_ptr(), out[0].data_ptr(),
        dq_ts, out[1].data_ptr(), dk_ts, dgamma_q.data_ptr(), dgamma_k.data_ptr(), B, L, H, Hkv,
        d, pos_offset, None if positions is None else positions.data_ptr(), float(eps),
        _dtype_code(Q.dtype), _dtype_code(dQo.dtype), _dtype_code(dKo.dtype),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), on)
    _check(st, "qk_norm_rope_backward")
    return out[0], out[1], dgamma_q, dgamma_k


def qk_norm_rope_paged(Q, K, V, gamma_q, gamma_k, pe, K_pages, V_pages, page_table, kv_lengths,
                       q_offsets, pairing: int = ROPE_INTERLEAVED, eps: float = 1e-6,
                       layer: int = 0, out=None, stream=None, K_scale=None, V_scale=None):
    """Q' [T, H, d] for ``sdpa_paged``; the normed, rotated keys and the values
    of the T packed new tokens go into their pages (``kv_lengths`` already
    counts them).  Pages in 8 bits (float8_e4m3fn; the rows stay bf16) come
    with ``K_scale`` and ``V_scale``, which are updated."""
    pages = _kv_pages(K_pages, V_pages, page_table, kv_lengths)
    scales = _kv_scales(K_pages, K_scale, V_scale)
    if Q.dim() != 3:
        raise ValueError("Q must be [T, H, d]")
    T, H, d = Q.shape
    dt = K_pages.dtype if scales is None else torch.bfloat16
    q_ts = _packed("Q", Q, H, pages.d, dt)
    k_ts = _packed("K", K, pages.kv_heads, d, dt)
    v_ts = _packed("V", V, pages.kv_heads, d, dt)
    if K.shape[0] != T or V.shape[0] != T:
        raise ValueError("Q, K and V must hold the same tokens")
    _gammas(gamma_q, gamma_k, pe, d, dt)
    layer, pairing = _c_int("layer", layer), _c_int("pairing", pairing)
    _int32("q_offsets", q_offsets, pages.B + 1)
    on = _launch_on(stream, Q, K, V, gamma_q, gamma_k, pe, K_pages, V_pages, page_table, kv_lengths,
                    q_offsets, Q if out is None else out, *_given(K_scale, V_scale))
    if out is None:
        out = _new(stream, (T, H, d), dt, Q.device)
    elif out.shape != (T, H, d) or out.dtype != dt or not out.is_contiguous():
        raise ValueError("out has the wrong shape, dtype or layout")
    rows = (Q.data_ptr(), q_ts, K.data_ptr(), k_ts, V.data_ptr(), v_ts, gamma_q.data_ptr(),
            gamma_k.data_ptr(), pe.data_ptr(), pe.shape[0], pe.shape[1], pairing, out.data_ptr())
    rest = (layer, q_offsets.data_ptr(), T, H, float(eps), on)
    dev = _lib or lib()
    if scales is None:
        _check(dev.qk_norm_rope_paged(*rows, pages, *rest), "qk_norm_rope_paged")
    else:
        _check(dev.qk_norm_rope_paged_e4m3(*rows, pages, scales, *rest), "qk_norm_rope_paged_e4m3")
    return out


def kv_pages_fork(K_pages, V_pages, page_table, kv_lengths, parents, children, fresh, stream=None,
                  K_scale=None, V_scale=None):
    """Sequences children[i] continue parents[i]: full pages shared, the last
    partly filled one copied into page fresh[i] (every layer; of pages in 8
    bits with its ``K_scale`` and ``V_scale``); page_table and kv_lengths are
    updated in place."""
    pages = _kv_pages(K_pages, V_pages, page_table, kv_lengths)
    scales = _kv_scales(K_pages, K_scale, V_scale)
    n = parents.numel()
    for name, t in (("parents", parents), ("children", children), ("fresh", fresh)):
        _int32(name, t, n)
    on = _launch_on(stream, K_pages, V_pages, page_table, kv_lengths, parents, children, fresh,
                    *_given(K_scale, V_scale))
    dev, pairs = _lib or lib(), (parents.data_ptr(), children.data_ptr(), fresh.data_ptr(), n, on)
    if scales is None:
        _check(dev.kv_pages_fork(pages, *pairs), "kv_pages_fork")
    else:
        _check(dev.kv_pages_fork_e4m3(pages, scales, *pairs), "kv_pages_fork_e4m3")


def kv_pages_compact(K_pages, V_pages, page_table, kv_lengths, K_out, V_out, table_out,
                     workspace=None, stream=None, K_scale=None, V_scale=None, K_scale_out=None,
                     V_scale_out=None):
    """The pages that some sequence holds become pages 0..n-1 of K_out, V_out,
    in order; table_out is the renumbered page table.  Returns n (int32 [1]).
    Of pages in 8 bits the scales move to ``K_scale_out``, ``V_scale_out``."""
    src = _kv_pages(K_pages, V_pages, page_table, kv_lengths)
    dst = _kv_pages(K_out, V_out, table_out, kv_lengths)
    scales = _kv_scales(K_pages, K_scale, V_scale)
    scales_out = _kv_scales(K_out, K_scale_out, V_scale_out)
    _check_workspace(workspace)
    on = _launch_on(stream, K_pages, V_pages, page_table, kv_lengths, K_out, V_out, table_out,
                    K_pages if workspace is None else workspace,
                    *_given(K_scale, V_scale, K_scale_out, V_scale_out))
    dev = _lib or lib()
    need = dev.kv_pages_compact_workspace_bytes(src.num_pages)
    # n, and the workspace 16 bytes behind it
    own = 0 if workspace is not None else need // 4
    count = _new(stream, (4 + own,), torch.int32, K_pages.device)
    if workspace is None:
        at, size = count.data_ptr() + 16, need
    else:
        at, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if scales is None and scales_out is None:
        _check(dev.kv_pages_compact(src, dst, count.data_ptr(), at, size, on), "kv_pages_compact")
    else:
        _check(dev.kv_pages_compact_e4m3(src, scales, dst, scales_out, count.data_ptr(), at, size, on),
               "kv_pages_compact_e4m3")
    return count[:1]


def _bounds_of(K_pages, bounds, bound_scale):
    lead, d = K_pages.shape[:-2], K_pages.shape[-1]
    if bounds.dtype is not torch.int8 or bounds.shape != (*lead, 2, d) or not bounds.is_contiguous():
        raise ValueError(f"bounds must be a contiguous int8 tensor of shape {[*lead, 2, d]}")
    if bound_scale.dtype is not torch.float32 or bound_scale.shape != lead \
            or not bound_scale.is_contiguous():
        raise ValueError(f"bound_scale must be a contiguous float32 tensor of shape {list(lead)}")


def kv_pages_bounds(K_pages, V_pages, page_table, kv_lengths, q_offsets, bounds, bound_scale, T: int,
                    layer: int = 0, stream=None, K_scale=None, V_scale=None):
    """Fill in, for every full page among those that hold one of the newest T
    packed tokens, the bounds of its keys: ``bounds`` int8 [P, Hkv, 2, d] (lo,
    hi by columns) and ``bound_scale`` float32 [P, Hkv] (both with a leading
    layer dimension if the pools have one), lo * scale <= key <= hi * scale."""
    pages = _kv_pages(K_pages, V_pages, page_table, kv_lengths)
    scales = _kv_scales(K_pages, K_scale, V_scale)
    _int32("q_offsets", q_offsets, pages.B + 1)
    _bounds_of(K_pages, bounds, bound_scale)
    layer, T = _c_int("layer", layer), _c_int("T", T)
    on = _launch_on(stream, K_pages, V_pages, page_table, kv_lengths, q_offsets, bounds, bound_scale,
                    *_given(K_scale, V_scale))
    _check((_lib or lib()).kv_pages_bounds(pages, scales, layer, q_offsets.data_ptr(), T,
                                           bounds.data_ptr(), bound_scale.data_ptr(), on),
           "kv_pages_bounds")


_SMALL_WORKSPACE = 8 << 20   # an allocation more costs a call 4 us


def kv_pages_select(Q, K_pages, V_pages, page_table, kv_lengths, q_offsets, bounds, bound_scale,
                    n_select: int, layer: int = 0, out=None, workspace=None, stream=None,
                    K_scale=None, V_scale=None):
    """(selected int32 [T, Hkv, n_select], lengths int32 [T]) for
    ``sdpa_paged_selected``: for every packed new token Q [T, H, d] and kv head
    its newest page and the full pages before it whose bounds (from
    ``kv_pages_bounds``) admit the largest scores, in order of position, -1
    behind the last; and the rows the token sees in them.  ``out``: the two to
    fill."""
    pages = _kv_pages(K_pages, V_pages, page_table, kv_lengths)
    if _given(K_scale, V_scale):
        _kv_scales(K_pages, K_scale, V_scale)    # the pages themselves are not read
    if Q.dim() != 3 or Q.dtype is not torch.bfloat16:
        raise ValueError("Q must be bf16 [T, H, d]")
    T, H, d = Q.shape
    q_ts = _packed("Q", Q, H, pages.d, Q.dtype)
    _int32("q_offsets", q_offsets, pages.B + 1)
    _bounds_of(K_pages, bounds, bound_scale)
    layer, n_select = _c_int("layer", layer), _c_int("n_select", n_select)
    if n_select < 1:
        raise ValueError("n_select must be at least 1")
    _check_workspace(workspace)
    on = _launch_on(stream, Q, K_pages, V_pages, page_table, kv_lengths, q_offsets, bounds, bound_scale,
                    *_given(K_scale, V_scale, workspace), *(() if out is None else out))
    dev, Hkv = _lib or lib(), pages.kv_heads
    n = T * Hkv * n_select
    need = dev.kv_pages_select_workspace_bytes(T, Hkv, pages.table_cols) if workspace is None else 0
    if out is None:
        # one allocation: the two tables, and a small workspace behind them (a large
        # one would be held as long as they are)
        small = need if need <= _SMALL_WORKSPACE else 0
        at = -(-(n + T) // 4) * 4
        own = _new(stream, (at + small // 4,), torch.int32, Q.device)
        out = own.as_strided((T, Hkv, n_select), (Hkv * n_select, n_select, 1)), own.narrow(0, n, T)
        ws, size = own.data_ptr() + 4 * at, need
    else:
        small = 0
        _int32("selected", out[0], T, Hkv, n_select)
        _int32("lengths", out[1], T)
    if workspace is None and not small:
        own = _new(stream, (need or 16,), torch.uint8, Q.device)
        ws, size = own.data_ptr(), need
    if workspace is not None:
        ws, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = dev.kv_pages_select(Q.data_ptr(), q_ts, pages, layer, q_offsets.data_ptr(), bounds.data_ptr(),
                             bound_scale.data_ptr(), T, H, n_select, out[0].data_ptr(),
                             out[1].data_ptr(), ws, size, on)
    _check(st, "kv_pages_select")
    return out


def sdpa_paged_selected(Q, K_pages, V_pages, selected, lengths, scale: float | None = None,
                        out_dtype: torch.dtype | None = None, layer: int = 0, num_splits: int = 0,
                        out=None, stream=None, K_scale=None, V_scale=None):
    """O [T, H, d] = attention of each token Q [T, H, d] over the first
    lengths[t] rows of its own pages selected[t, g, :] (int32 [T, Hkv, n]) per
    kv head, as ``kv_pages_select`` gives them.  A token of length 0 is passed
    over."""
    pools = _kv_pools(K_pages, V_pages)
    scales = _kv_scales(K_pages, K_scale, V_scale)
    Hkv, pd = pools[5], pools[6]
    if Q.dim() != 3 or Q.dtype != (K_pages.dtype if scales is None else torch.bfloat16):
        raise ValueError("Q must be [T, H, d] of the cache's dtype, or bf16 over pages in 8 bits")
    T, H, d = Q.shape
    q_ts = _packed("Q", Q, H, pd, Q.dtype)
    if selected.dim() != 3:
        raise ValueError("selected must be [T, Hkv, pages]")
    n = selected.shape[2]
    _int32("selected", selected, T, Hkv, n)
    _int32("lengths", lengths, T)
    odt = out_dtype or Q.dtype
    layer, num_splits = _c_int("layer", layer), _c_int("num_splits", num_splits)
    on = _launch_on(stream, Q, K_pages, V_pages, selected, lengths, Q if out is None else out,
                    *_given(K_scale, V_scale))
    if out is None:
        out = _new(stream, (T, H, d), odt, Q.device)
    elif out.shape != (T, H, d) or out.dtype != odt or not out.is_contiguous():
        raise ValueError("out has the wrong shape, dtype or layout")
    st = (_lib or lib()).sdpa_paged_selected(
        Q.data_ptr(), q_ts, KvPages(*pools, None, None, 0, 1), scales, layer, selected.data_ptr(),
        lengths.data_ptr(), n, out.data_ptr(), T, H, float(scale or 0.0), _dtype_code(odt), num_splits,
        on)
    _check(st, "sdpa_paged_selected")
    return out


class MhaHandle:
    """Owner of an ``mha_create`` handle (destroyed with ``close``)."""

    def __init__(self, d_model: int, dtype: torch.dtype, max_batch: int, max_lq: int,
                 max_lk: int):
        h = ctypes.c_void_p()
        _check(lib().mha_create(ctypes.byref(h), d_model, _dtype_code(dtype), max_batch, max_lq,
                                max_lk), "mha_create")
        self._h = h
        self.d_model, self.dtype = d_model, dtype

    @property
    def raw(self):
        if self._h is None:
            raise RuntimeError("handle destroyed")
        return self._h

    def close(self):
        if self._h is not None:
            _check(lib().mha_destroy(self._h), "mha_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def mha_create(d_model: int, dtype: torch.dtype, max_batch: int, max_lq: int,
               max_lk: int) -> MhaHandle:
    return MhaHandle(d_model, dtype, max_batch, max_lq, max_lk)


def mha_forward(handle: MhaHandle, x_q, x_kv, Wq, Wk, Wv, Wo, h: int,
                mask_kind: int = MASK_NONE, key_lengths=None, out=None, stream=None):
    """out = Concat(head_1..head_h) Wo, head_i = Attention(x_q Wq_i, x_kv Wk_i, x_kv Wv_i)."""
    B, Lq, D = x_q.shape
    Lk = x_kv.shape[1]
    if x_kv.shape != (B, Lk, D):
        raise ValueError("x_kv shape")
    for W in (Wq, Wk, Wv, Wo):
        if W.shape != (D, D) or W.dtype != x_q.dtype:
            raise ValueError("weights must be [D, D] of the activations' dtype")
    if out is None:
        out = torch.empty((B, Lq, D), dtype=x_q.dtype, device=x_q.device)
    st = lib().mha_forward(handle.raw, _dev_ptr(x_q), _dev_ptr(x_kv), _dev_ptr(Wq),
                           _dev_ptr(Wk), _dev_ptr(Wv), _dev_ptr(Wo), B, Lq, Lk, int(h),
                           int(mask_kind), _dev_ptr(key_lengths), _dev_ptr(out),
                           _stream(stream))
    _check(st, "mha_forward")
    return out


class EncoderLayer:
    """One post-norm encoder layer on the library (encoder_create /
    encoder_forward / encoder_destroy).  ``params`` maps the names in
    ENCODER_PARAM_NAMES to device tensors of the layer's dtype."""

    def __init__(self, d_model: int, heads: int, d_ff: int, dtype: torch.dtype,
                 max_batch: int, max_len: int):
        h = ctypes.c_void_p()
        _check(lib().encoder_create(ctypes.byref(h), d_model, heads, d_ff, _dtype_code(dtype),
                                    max_batch, max_len), "encoder_create")
        self._h = h
        self.d_model, self.heads, self.d_ff, self.dtype = d_model, heads, d_ff, dtype

    def forward(self, x, params: dict, mask_kind: int = MASK_NONE, key_lengths=None,
                ln_eps: float = 1e-5, out=None, stream=None, out_dtype=None):
        """``out_dtype``: the layer's dtype (default), or torch.float32 for a
        bf16 layer to keep the final LayerNorm's output unrounded."""
        if self._h is None:
            raise RuntimeError("encoder destroyed")
        B, L, D = x.shape
        if D != self.d_model or x.dtype != self.dtype:
            raise ValueError("x does not match the layer")
        shapes = {"W1": (D, self.d_ff), "b1": (self.d_ff,), "W2": (self.d_ff, D)}
        for n in ENCODER_PARAM_NAMES:
            t = params[n]
            want = shapes.get(n, (D, D) if n.startswith("W") else (D,))
            if tuple(t.shape) != want or t.dtype != self.dtype:
                raise ValueError(f"parameter {n} must be {want} {self.dtype}")
        p = EncoderParams(*[_dev_ptr(params[n]) for n in ENCODER_PARAM_NAMES])
        odt = self.dtype if out_dtype is None else out_dtype
        if out is None:
            out = torch.empty(x.shape, dtype=odt, device=x.device)
        if out.dtype != odt or tuple(out.shape) != tuple(x.shape):
            raise ValueError("out does not match the output dtype and shape")
        st = lib().encoder_forward(self._h, _dev_ptr(x), ctypes.byref(p), B, L, int(mask_kind),
                                   _dev_ptr(key_lengths), float(ln_eps), _dev_ptr(out),
                                   _dtype_code(odt), _stream(stream))
        _check(st, "encoder_forward")
        return out

    def close(self):
        if self._h is not None:
            _check(lib().encoder_destroy(self._h), "encoder_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def mha_check(handle: MhaHandle | None = None) -> int:
    """Synchronise and return (then clear) the device error status code."""
    return int(lib().mha_check(handle.raw if handle is not None else None))


def mha_destroy(handle: MhaHandle):
    handle.close()


def selftest_wait_timeout(limit_ms: int = 100, stream=None):
    """Launch the bounded-wait self-test (see include/mha.h); mha_check() then
    reports MHA_ERR_TIMEOUT."""
    _check(lib().mha_selftest_wait_timeout(int(limit_ms), _stream(stream)),
           "mha_selftest_wait_timeout")


def set_wait_limit_ms(ms: int) -> int:
    return int(lib().mha_set_wait_limit_ms(int(ms)))


def sdpa_forward_host(Qh, Kh, Vh, scale=None, mask_kind=MASK_NONE, lengths_h=None,
                      out_dtype=None, device="cuda", bufs=None, stream=None):
    """End-to-end call from host (pinned) tensors through the library's
    sdpa_forward_host: copies in, attention and copies out overlap chunk by
    chunk on the device.  Returns the pinned output; it is complete once
    ``stream`` (the current stream by default) has been synchronised.

    ``bufs`` (a dict) keeps the device workspace and the pinned output
    between calls."""
    bufs = {} if bufs is None else bufs
    B, H, Lq, d = Qh.shape
    Lk = Kh.shape[2]
    odt = out_dtype or Qh.dtype
    need = int(lib().sdpa_forward_host_workspace_bytes(B, H, Lq, Lk, d, _dtype_code(Qh.dtype),
                                                       _dtype_code(odt)))
    ws = bufs.get("ws")
    if ws is None or ws.numel() < need:
        ws = bufs["ws"] = torch.empty(max(256, need), dtype=torch.uint8, device=device)
    Oh = bufs.get("Oh")
    if Oh is None or Oh.shape != Qh.shape or Oh.dtype != odt:
        Oh = bufs["Oh"] = torch.empty(Qh.shape, dtype=odt, pin_memory=True)
    lp = ctypes.c_void_p(lengths_h.data_ptr()) if lengths_h is not None else None
    st = lib().sdpa_forward_host(ctypes.c_void_p(Qh.data_ptr()), ctypes.c_void_p(Kh.data_ptr()),
                                 ctypes.c_void_p(Vh.data_ptr()), ctypes.c_void_p(Oh.data_ptr()),
                                 B, H, Lq, Lk, d, float(scale or 0.0), int(mask_kind), lp,
                                 _dtype_code(Qh.dtype), _dtype_code(odt), _dev_ptr(ws),
                                 ws.numel(), _stream(stream))
    _check(st, "sdpa_forward_host")
    return Oh
