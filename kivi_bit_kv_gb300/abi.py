"""ctypes binding of libkivi (include/kivi.h), one Python function per C entry point.

Argument marshalling only: tensors are checked for dtype, device, shape and
contiguity, their device pointers and the current CUDA stream are passed to the
C library, and a non-zero status raises :class:`KiviError`.  Every step of the
method runs in the library's CUDA kernels; there is no Python or CPU fallback,
and a missing library is an error.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# KIVI_LIB selects another in-tree build of the library (the bounds-checked
# one, libkivi_checked.so); by default libkivi.so next to this file.
LIB_PATH = os.environ.get("KIVI_LIB") or os.path.join(HERE, "libkivi.so")

KIVI_OK = 0
KIVI_EINVAL = 1
KIVI_ECAPACITY = 2
KIVI_ECUDA = 3
KIVI_ETIMEOUT = 4
KIVI_EWORKSPACE = 5
KIVI_ECHECK = 6

(KIVI_BUF_KQ, KIVI_BUF_KSCALE, KIVI_BUF_KZERO, KIVI_BUF_VQ, KIVI_BUF_VSCALE, KIVI_BUF_VZERO,
 KIVI_BUF_KRES, KIVI_BUF_VRES, KIVI_BUF_LEN) = range(9)

# Every symbol include/kivi.h declares.
EXPORTS = (
    "kivi_abi_version", "kivi_status_string", "kivi_last_error", "kivi_cache_validate",
    "kivi_buffer_bytes", "kivi_cache_bytes", "kivi_quant_keys", "kivi_quant_values",
    "kivi_dequant", "kivi_append_token", "kivi_decode_qk", "kivi_decode_pv",
    "kivi_workspace_bytes", "kivi_decode_pv_noalloc", "kivi_decode_attention",
    "kivi_codec_fingerprint", "kivi_payload_bytes", "kivi_export", "kivi_import",
    "kivi_check_status", "kivi_block_select", "kivi_sparse_attention", "kivi_tree_attention",
    "kivi_attend_workspace_bytes", "kivi_append_path", "kivi_norm_rope", "kivi_token_probs",
    "kivi_verify_tree",
)

KIVI_PAYLOAD_MAGIC = 0x5056494B
KIVI_PAYLOAD_VERSION = 1
KIVI_PAYLOAD_HEADER_BYTES = 64

KIVI_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024

KIVI_MAX_DRAFT = 256
KIVI_MAX_AXES = 8
KIVI_MAX_VOCAB = 1 << 20

KIVI_F16, KIVI_BF16, KIVI_F32 = range(3)
_DTYPES = {torch.float16: KIVI_F16, torch.bfloat16: KIVI_BF16, torch.float32: KIVI_F32}


class KiviError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: {message} (status {status})")
        self.status = status


class kivi_cache(C.Structure):
    """Mirror of the C struct ``kivi_cache``."""
    _fields_ = [
        ("B", C.c_int32), ("H", C.c_int32), ("D", C.c_int32),
        ("bits_k", C.c_int32), ("bits_v", C.c_int32),
        ("G", C.c_int32), ("R", C.c_int32), ("Tmax", C.c_int32),
        ("kq", C.c_void_p), ("kscale", C.c_void_p), ("kzero", C.c_void_p),
        ("vq", C.c_void_p), ("vscale", C.c_void_p), ("vzero", C.c_void_p),
        ("kres", C.c_void_p), ("vres", C.c_void_p), ("len", C.c_void_p),
    ]


# The C struct kivi_heads: Hq, N, dtype, rot, interleaved, n_axes, eps, reserved; the
# inputs; nine strides; q_weight, k_weight, inv_freq, axis, pos, base, n_tok; the outputs.
_HEADS = struct.Struct("=6ifi3Q9q7Q3Q")


_LIB = None


def load(path: str | None = None):
    """Load libkivi.so (built in-tree by ``kivi_bit_kv_gb300.build``)."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"{p} is missing: build it with kivi_bit_kv_gb300.build.build(); "
                          "there is no fallback path")
    L = C.CDLL(p)
    vp, i32, f32, sz = C.c_void_p, C.c_int32, C.c_float, C.c_size_t
    cp = C.POINTER(kivi_cache)
    sig = {
        "kivi_abi_version": ([], i32),
        "kivi_status_string": ([i32], C.c_char_p),
        "kivi_last_error": ([], C.c_char_p),
        "kivi_cache_validate": ([cp], i32),
        "kivi_buffer_bytes": ([cp, i32], sz),
        "kivi_cache_bytes": ([i32] * 6, sz),
        "kivi_quant_keys": ([cp, vp, i32, vp, vp], i32),
        "kivi_quant_values": ([cp, vp, i32, vp, vp], i32),
        "kivi_dequant": ([cp, i32, vp, i32, vp], i32),
        "kivi_append_token": ([cp, vp, vp, vp, vp], i32),
        "kivi_decode_qk": ([cp, vp, i32, f32, vp, i32, vp], i32),
        "kivi_decode_pv": ([cp, vp, i32, i32, vp, vp, sz, vp], i32),
        "kivi_workspace_bytes": ([cp, i32], sz),
        "kivi_decode_pv_noalloc": ([cp, vp, i32, i32, vp, vp], i32),
        "kivi_decode_attention": ([cp, vp, i32, f32, vp, vp, sz, vp], i32),
        "kivi_codec_fingerprint": ([cp], C.c_uint64),
        "kivi_payload_bytes": ([cp, vp], sz),
        "kivi_export": ([cp, vp, sz, vp, vp], i32),
        "kivi_import": ([cp, vp, sz, vp, vp], i32),
        "kivi_check_status": ([C.POINTER(i32)], i32),
        "kivi_block_select": ([cp, vp, i32, vp, i32, vp, vp], i32),
        "kivi_sparse_attention": ([cp, vp, i32, f32, vp, i32, vp, vp, sz, vp], i32),
        "kivi_tree_attention": ([cp, vp, i32, i32, vp, vp, vp, vp, f32, vp, vp, sz, vp], i32),
        "kivi_attend_workspace_bytes": ([cp, i32, i32], sz),
        "kivi_append_path": ([cp, vp, vp, i32, vp, i32, vp, vp, vp], i32),
        "kivi_norm_rope": ([cp, vp, vp], i32),
        "kivi_token_probs": ([vp, i32, i32, i32, i32, C.c_int64, C.c_int64, vp, vp, vp, vp], i32),
        "kivi_verify_tree": ([i32, i32, i32] + [vp] * 10, i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _LIB = L
    return L


def _check(status: int, where: str):
    if status != KIVI_OK:
        L = load()
        msg = L.kivi_last_error().decode() or L.kivi_status_string(status).decode()
        raise KiviError(status, where, msg)


def _stream(stream, device) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, dtype, name: str, device=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, cache is on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# ------------------------------------------------------------ host-only ---

def kivi_abi_version() -> int:
    return int(load().kivi_abi_version())


def kivi_status_string(status: int) -> str:
    return load().kivi_status_string(status).decode()


def kivi_last_error() -> str:
    return load().kivi_last_error().decode()


def kivi_cache_validate(desc: kivi_cache) -> int:
    return int(load().kivi_cache_validate(C.byref(desc)))


def kivi_buffer_bytes(desc: kivi_cache, buffer: int) -> int:
    return int(load().kivi_buffer_bytes(C.byref(desc), buffer))


def kivi_cache_bytes(T: int, D: int, bits: int, G: int, R: int, which: int) -> int:
    return int(load().kivi_cache_bytes(T, D, bits, G, R, which))


def kivi_codec_fingerprint(desc: kivi_cache) -> int:
    """FNV-1a 64 fingerprint of the codec (D, bits, G, R) of a descriptor."""
    return int(load().kivi_codec_fingerprint(C.byref(desc)))


def kivi_payload_bytes(desc: kivi_cache, lens) -> int:
    """Bytes of the compact payload when sequence b holds lens[b] tokens."""
    arr = (C.c_int32 * desc.B)(*[int(x) for x in lens])
    return int(load().kivi_payload_bytes(C.byref(desc), C.cast(arr, C.c_void_p)))


def kivi_workspace_bytes(cache, Hq: int) -> int:
    return int(load().kivi_workspace_bytes(C.byref(cache.desc), Hq))


def kivi_attend_workspace_bytes(cache, Hq: int, N: int = 1) -> int:
    return int(load().kivi_attend_workspace_bytes(C.byref(cache.desc), Hq, N))


# ---------------------------------------------------------- device calls ---

def kivi_quant_keys(cache, K: torch.Tensor, seq_lens: torch.Tensor | None = None, stream=None):
    """Prefix-encode keys K fp16 [B, H, T, D] into ``cache``."""
    B, H, T, D = K.shape
    if (B, H, D) != (cache.B, cache.H, cache.D):
        raise ValueError(f"K shape {tuple(K.shape)} does not match cache (B, H, D)="
                         f"{(cache.B, cache.H, cache.D)}")
    kp = _dev(K, torch.float16, "K", cache.device)
    lp = None if seq_lens is None else _dev(seq_lens, torch.int32, "seq_lens", cache.device)
    _check(load().kivi_quant_keys(C.byref(cache.desc), kp, T, lp, _stream(stream, cache.device)),
           "kivi_quant_keys")


def kivi_quant_values(cache, V: torch.Tensor, seq_lens: torch.Tensor | None = None, stream=None):
    """Prefix-encode values V fp16 [B, H, T, D] into ``cache``."""
    B, H, T, D = V.shape
    if (B, H, D) != (cache.B, cache.H, cache.D):
        raise ValueError(f"V shape {tuple(V.shape)} does not match cache (B, H, D)="
                         f"{(cache.B, cache.H, cache.D)}")
    vp = _dev(V, torch.float16, "V", cache.device)
    lp = None if seq_lens is None else _dev(seq_lens, torch.int32, "seq_lens", cache.device)
    _check(load().kivi_quant_values(C.byref(cache.desc), vp, T, lp, _stream(stream, cache.device)),
           "kivi_quant_values")


def kivi_dequant(cache, which: int, out: torch.Tensor, stream=None):
    """Materialize keys (which=0) or values (which=1) into out fp16 [B, H, T_out, D]."""
    B, H, T_out, D = out.shape
    if (B, H, D) != (cache.B, cache.H, cache.D):
        raise ValueError(f"out shape {tuple(out.shape)} does not match cache")
    op = _dev(out, torch.float16, "out", cache.device)
    _check(load().kivi_dequant(C.byref(cache.desc), which, op, T_out, _stream(stream, cache.device)),
           "kivi_dequant")


def kivi_append_token(cache, k: torch.Tensor, v: torch.Tensor, status: torch.Tensor, stream=None):
    """Append one token k, v fp16 [B, H, D] (or [B, H, 1, D]) to every sequence."""
    shape = (cache.B, cache.H, cache.D)
    for name, t in (("k", k), ("v", v)):
        if tuple(t.shape) not in (shape, (cache.B, cache.H, 1, cache.D)):
            raise ValueError(f"{name} shape {tuple(t.shape)}; expected {shape}")
    if status.numel() < 1:
        raise ValueError("status must hold one int32")
    _check(load().kivi_append_token(C.byref(cache.desc), _dev(k, torch.float16, "k", cache.device),
                                    _dev(v, torch.float16, "v", cache.device),
                                    _dev(status, torch.int32, "status", cache.device),
                                    _stream(stream, cache.device)), "kivi_append_token")


def kivi_decode_qk(cache, q: torch.Tensor, logits: torch.Tensor, sm_scale: float | None = None,
                   stream=None):
    """logits fp32 [B, Hq, ld] <- sm_scale * q . K_hat^T for q fp16 [B, Hq, D] (or [B, Hq, 1, D])."""
    B, Hq = q.shape[0], q.shape[1]
    if B != cache.B or q.shape[-1] != cache.D or q.numel() != B * Hq * cache.D:
        raise ValueError(f"q shape {tuple(q.shape)} does not match cache")
    if logits.dim() != 3 or tuple(logits.shape[:2]) != (B, Hq):
        raise ValueError(f"logits must be [B, Hq, ld], got {tuple(logits.shape)}")
    sm = float(cache.D ** -0.5) if sm_scale is None else float(sm_scale)
    _check(load().kivi_decode_qk(C.byref(cache.desc), _dev(q, torch.float16, "q", cache.device), Hq,
                                 sm, _dev(logits, torch.float32, "logits", cache.device),
                                 logits.shape[2], _stream(stream, cache.device)), "kivi_decode_qk")


def kivi_decode_pv(cache, logits: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, stream=None):
    """out fp32 [B, Hq, D] <- softmax(logits) . V_hat, with ws a device workspace."""
    B, Hq, ld = logits.shape
    if tuple(out.shape) not in ((B, Hq, cache.D), (B, Hq, 1, cache.D)):
        raise ValueError(f"out shape {tuple(out.shape)}; expected {(B, Hq, cache.D)}")
    wp = _dev(ws, ws.dtype, "ws", cache.device)
    _check(load().kivi_decode_pv(C.byref(cache.desc), _dev(logits, torch.float32, "logits", cache.device),
                                 ld, Hq, _dev(out, torch.float32, "out", cache.device), wp,
                                 ws.numel() * ws.element_size(), _stream(stream, cache.device)),
           "kivi_decode_pv")


def kivi_decode_pv_noalloc(cache, logits: torch.Tensor, out: torch.Tensor, stream=None):
    """kivi_decode_pv without a workspace argument, for callers that cannot
    allocate device memory: the library's fixed 16 MiB per-device scratch
    holds the partial results.  Calls sharing a device must not overlap on
    the GPU (order them on one stream); the first call on a device should
    come before any stream capture."""
    B, Hq, ld = logits.shape
    if tuple(out.shape) not in ((B, Hq, cache.D), (B, Hq, 1, cache.D)):
        raise ValueError(f"out shape {tuple(out.shape)}; expected {(B, Hq, cache.D)}")
    _check(load().kivi_decode_pv_noalloc(C.byref(cache.desc),
                                         _dev(logits, torch.float32, "logits", cache.device), ld, Hq,
                                         _dev(out, torch.float32, "out", cache.device),
                                         _stream(stream, cache.device)), "kivi_decode_pv_noalloc")


def kivi_decode_attention(cache, q: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                          sm_scale: float | None = None, stream=None):
    """out fp32 [B, Hq, D] <- softmax(sm_scale q . K_hat^T) . V_hat in one fused
    pass (logits stay on chip); q fp16 [B, Hq, D] (or [B, Hq, 1, D]), ws a
    device workspace of at least kivi_workspace_bytes(cache, Hq) bytes."""
    B, Hq = q.shape[0], q.shape[1]
    if B != cache.B or q.shape[-1] != cache.D or q.numel() != B * Hq * cache.D:
        raise ValueError(f"q shape {tuple(q.shape)} does not match cache")
    if tuple(out.shape) not in ((B, Hq, cache.D), (B, Hq, 1, cache.D)):
        raise ValueError(f"out shape {tuple(out.shape)}; expected {(B, Hq, cache.D)}")
    sm = float(cache.D ** -0.5) if sm_scale is None else float(sm_scale)
    wp = _dev(ws, ws.dtype, "ws", cache.device)
    _check(load().kivi_decode_attention(C.byref(cache.desc), _dev(q, torch.float16, "q", cache.device),
                                        Hq, sm, _dev(out, torch.float32, "out", cache.device), wp,
                                        ws.numel() * ws.element_size(), _stream(stream, cache.device)),
           "kivi_decode_attention")


# The calls of a decode step are a few microseconds of GPU work, so the checks
# below cost little when they pass: shapes compare as tuples, a tensor's other
# properties in one expression (_dev says which one is wrong), and the current
# stream is asked for as a raw handle.

def _bad_shape(t, name: str, *shapes):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    raise ValueError(f"{name} shape {tuple(t.shape)}; expected {' or '.join(map(str, shapes))}")


def _ptr(t: torch.Tensor, dtype, name: str, device) -> int:
    if t.dtype is dtype and t.get_device() == device.index and t.is_contiguous():
        return t.data_ptr()
    return _dev(t, dtype, name, device)


def _raw_stream(stream, device) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return _stream(stream, device)


def _call(fn, where: str, device, *args):
    """fn(*args) with the cache's device current, as the library requires."""
    if torch._C._cuda_getDevice() == device.index:
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st != KIVI_OK:
        _check(st, where)


def kivi_block_select(cache, q: torch.Tensor, blocks: torch.Tensor, scores: torch.Tensor, stream=None):
    """blocks int32 [B, H, n_keep] <- the quantized key groups of largest score,
    ascending and padded with -1; scores fp32 [B, H, Tmax/G] <- the scores, an
    upper bound of q . k over each group up to rounding; q fp16 [B, Hq, D] (or [B, Hq, 1, D])."""
    B, H, D, dev = cache.B, cache.H, cache.D, cache.device
    Hq = q.shape[1] if q.dim() > 1 else 0
    if q.shape != (B, Hq, D) and q.shape != (B, Hq, 1, D):
        _bad_shape(q, "q", (B, Hq, D), (B, Hq, 1, D))
    n_keep = blocks.shape[-1] if blocks.dim() else 0
    if blocks.shape != (B, H, n_keep):
        _bad_shape(blocks, "blocks", (B, H, n_keep))
    if scores.shape != (B, H, cache.Tmax // cache.G):
        _bad_shape(scores, "scores", (B, H, cache.Tmax // cache.G))
    _call(load().kivi_block_select, "kivi_block_select", dev, C.byref(cache.desc),
          _ptr(q, torch.float16, "q", dev), Hq, _ptr(blocks, torch.int32, "blocks", dev), n_keep,
          _ptr(scores, torch.float32, "scores", dev), _raw_stream(stream, dev))


def kivi_sparse_attention(cache, q: torch.Tensor, blocks: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                          sm_scale: float | None = None, stream=None):
    """out fp32 [B, Hq, D] <- decode attention of q fp16 [B, Hq, D] (or
    [B, Hq, 1, D]) over the key groups blocks int32 [B, H, n_keep] lists and
    the fp16 residual; ws of at least kivi_attend_workspace_bytes(cache, Hq)."""
    B, H, D, dev = cache.B, cache.H, cache.D, cache.device
    Hq = q.shape[1] if q.dim() > 1 else 0
    if q.shape != (B, Hq, D) and q.shape != (B, Hq, 1, D):
        _bad_shape(q, "q", (B, Hq, D), (B, Hq, 1, D))
    n_keep = blocks.shape[-1] if blocks.dim() else 0
    if blocks.shape != (B, H, n_keep):
        _bad_shape(blocks, "blocks", (B, H, n_keep))
    if out.shape != (B, Hq, D) and out.shape != (B, Hq, 1, D):
        _bad_shape(out, "out", (B, Hq, D), (B, Hq, 1, D))
    _call(load().kivi_sparse_attention, "kivi_sparse_attention", dev, C.byref(cache.desc),
          _ptr(q, torch.float16, "q", dev), Hq, D ** -0.5 if sm_scale is None else float(sm_scale),
          _ptr(blocks, torch.int32, "blocks", dev), n_keep, _ptr(out, torch.float32, "out", dev),
          _ptr(ws, ws.dtype, "ws", dev), ws.numel() * ws.element_size(), _raw_stream(stream, dev))


def kivi_tree_attention(cache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, mask: torch.Tensor,
                        out: torch.Tensor, ws: torch.Tensor, n_draft: torch.Tensor | None = None,
                        sm_scale: float | None = None, stream=None):
    """out fp32 [B, Hq, N, D] <- attention of N drafted tokens q fp16
    [B, Hq, N, D] over the cache and the drafts k, v fp16 [B, H, N, D] that
    mask int64 [B, N, ceil(N/64)] allows (bit j % 64 of word j // 64 of row i:
    token i attends token j).  n_draft int32 [B]: tokens each sequence drafted
    (rows from there on keep their contents); ws of at least
    kivi_attend_workspace_bytes(cache, Hq, N)."""
    B, H, D, dev = cache.B, cache.H, cache.D, cache.device
    Hq, N = (q.shape[1], q.shape[2]) if q.dim() == 4 else (0, 0)
    if q.shape != (B, Hq, N, D):
        _bad_shape(q, "q", (B, Hq, N, D))
    if k.shape != (B, H, N, D):
        _bad_shape(k, "k", (B, H, N, D))
    if v.shape != (B, H, N, D):
        _bad_shape(v, "v", (B, H, N, D))
    if mask.shape != (B, N, (N + 63) // 64):
        _bad_shape(mask, "mask", (B, N, (N + 63) // 64))
    if out.shape != (B, Hq, N, D):
        _bad_shape(out, "out", (B, Hq, N, D))
    if n_draft is not None and n_draft.shape != (B,):
        _bad_shape(n_draft, "n_draft", (B,))
    _call(load().kivi_tree_attention, "kivi_tree_attention", dev, C.byref(cache.desc),
          _ptr(q, torch.float16, "q", dev), Hq, N, _ptr(k, torch.float16, "k", dev),
          _ptr(v, torch.float16, "v", dev), _ptr(mask, torch.int64, "mask", dev),
          None if n_draft is None else _ptr(n_draft, torch.int32, "n_draft", dev),
          D ** -0.5 if sm_scale is None else float(sm_scale), _ptr(out, torch.float32, "out", dev),
          _ptr(ws, ws.dtype, "ws", dev), ws.numel() * ws.element_size(), _raw_stream(stream, dev))


def kivi_append_path(cache, k: torch.Tensor, v: torch.Tensor, path: torch.Tensor, counts: torch.Tensor,
                     status: torch.Tensor, stream=None):
    """Append the drafted tokens path[b, :counts[b]] (path int32 [B, P], counts
    int32 [B]) of k, v fp16 [B, H, N, D] to every sequence.  A sequence with a
    bad count or path entry, or without room, is left as it was and status[0]
    set on the device (KIVI_EINVAL, KIVI_ECAPACITY)."""
    B, H, D, dev = cache.B, cache.H, cache.D, cache.device
    N = k.shape[2] if k.dim() == 4 else 0
    if k.shape != (B, H, N, D):
        _bad_shape(k, "k", (B, H, N, D))
    if v.shape != (B, H, N, D):
        _bad_shape(v, "v", (B, H, N, D))
    P = path.shape[-1] if path.dim() else 0
    if path.shape != (B, P):
        _bad_shape(path, "path", (B, P))
    if counts.shape != (B,):
        _bad_shape(counts, "counts", (B,))
    if status.numel() < 1:
        raise ValueError("status must hold one int32")
    _call(load().kivi_append_path, "kivi_append_path", dev, C.byref(cache.desc), _ptr(k, torch.float16, "k", dev),
          _ptr(v, torch.float16, "v", dev), N, _ptr(path, torch.int32, "path", dev), P,
          _ptr(counts, torch.int32, "counts", dev), _ptr(status, torch.int32, "status", dev),
          _raw_stream(stream, dev))


def _rows_ptr(t: torch.Tensor, dtype, name: str, device) -> int:
    """Pointer of an input whose last dimension is contiguous (any other strides)."""
    if t.dtype is dtype and t.get_device() == device.index:
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} is on {t.device}, expected {device}")


def _projection(x, y, name: str, shape, out_shape, dtype, device):
    """Pointer and strides of the projection x, pointer of its output y; zeros for none."""
    if x is None or y is None:
        if x is not y:
            raise ValueError(f"{name}_in and {name} are given together or not at all")
        return 0, (0, 0, 0), 0
    if x.shape != shape:
        _bad_shape(x, name + "_in", shape)
    if y.shape != out_shape:
        _bad_shape(y, name, out_shape)
    st = x.stride()
    if st[3] != 1:
        raise ValueError(f"{name}_in must have contiguous channels")
    return _rows_ptr(x, dtype, name + "_in", device), st[:3], _ptr(y, torch.float16, name, device)


def _vector(t, n: int, dtype, name: str, device) -> int:
    """Pointer of an optional vector of n entries; 0 for None."""
    if t is None:
        return 0
    if t.shape != (n,):
        _bad_shape(t, name, (n,))
    return _ptr(t, dtype, name, device)


def kivi_norm_rope(cache, q_in: torch.Tensor | None, k_in: torch.Tensor | None, v_in: torch.Tensor | None,
                   q: torch.Tensor | None, k: torch.Tensor | None, v: torch.Tensor | None,
                   inv_freq: torch.Tensor | None, pos: torch.Tensor | None = None, base: torch.Tensor | None = None,
                   axis: torch.Tensor | None = None, interleaved: bool = False, q_weight: torch.Tensor | None = None,
                   k_weight: torch.Tensor | None = None, eps: float = 1e-6, n_tok: torch.Tensor | None = None,
                   stream=None):
    """q fp16 [B, Hq, N, D], k, v fp16 [B, H, N, D] <- the projections q_in
    [B, N, Hq, D], k_in, v_in [B, N, H, D] (fp16, bf16 or fp32; any strides of 16
    bytes but contiguous channels, so views of one fused projection will do):
    heads of q and k with a weight fp32 [D] are RMS-normalized, then the first
    2 len(inv_freq) channels rotated by position * inv_freq (fp32 [rot/2]; None
    rotates nothing).  Positions: pos int32 [B, N] or [n_axes, B, N] (None: the
    token's index) plus base int32 [B]; axis int32 [rot/2] picks a pair's axis.
    interleaved pairs channels 2j and 2j + 1 instead of j and j + rot/2.  n_tok
    int32 [B]: tokens of each sequence (rows from there on keep their
    contents).  An input and its output may both be None."""
    B, H, D, dev = cache.B, cache.H, cache.D, cache.device
    first = q_in if q_in is not None else k_in if k_in is not None else v_in
    if first is None:
        raise ValueError("q_in, k_in and v_in are all None")
    if first.dim() != 4:
        _bad_shape(first, "q_in, k_in, v_in", (B, "N", "heads", D))
    N, dtype = first.shape[1], first.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"projections must be fp16, bf16 or fp32, got {dtype}")
    Hq = q_in.shape[2] if q_in is not None and q_in.dim() == 4 else H
    shape, out_shape = (B, N, H, D), (B, H, N, D)
    qp, qs, qo = _projection(q_in, q, "q", (B, N, Hq, D), (B, Hq, N, D), dtype, dev)
    kp, ks, ko = _projection(k_in, k, "k", shape, out_shape, dtype, dev)
    vp, vs, vo = _projection(v_in, v, "v", shape, out_shape, dtype, dev)
    half, fp = 0, 0
    if inv_freq is not None:
        half = inv_freq.numel()
        fp = _vector(inv_freq, half, torch.float32, "inv_freq", dev) if half else 0
    n_axes, pp = 1, 0
    if pos is not None:
        n_axes = pos.shape[0] if pos.dim() == 3 else 1
        if pos.shape != (B, N) and pos.shape != (n_axes, B, N):
            _bad_shape(pos, "pos", (B, N), ("n_axes", B, N))
        pp = _ptr(pos, torch.int32, "pos", dev)
    i32, f32 = torch.int32, torch.float32
    args = _HEADS.pack(
        Hq, N, _DTYPES[dtype], 2 * half, 1 if interleaved else 0, n_axes, eps, 0, qp, kp, vp, *qs, *ks, *vs,
        _vector(q_weight, D, f32, "q_weight", dev), _vector(k_weight, D, f32, "k_weight", dev), fp,
        _vector(axis, half, i32, "axis", dev) if half else 0, pp, _vector(base, B, i32, "base", dev),
        _vector(n_tok, B, i32, "n_tok", dev), qo, ko, vo)
    _call(load().kivi_norm_rope, "kivi_norm_rope", dev, C.byref(cache.desc), args, _raw_stream(stream, dev))


def kivi_token_probs(logits: torch.Tensor, probs: torch.Tensor, temperature: torch.Tensor | None = None,
                     n_rows: torch.Tensor | None = None, stream=None):
    """probs fp32 [B, N, V] <- softmax of logits [B, N, V] (fp16, bf16 or fp32;
    contiguous rows, any other strides) over temperature fp32 [B] (None: 1; 0: all
    on the first of the largest).  n_rows int32 [B]: rows of each sequence (rows from
    there on are left as they were)."""
    if logits.dim() != 3:
        _bad_shape(logits, "logits", ("B", "N", "V"))
    B, N, V = logits.shape
    dev = probs.device
    if probs.shape != (B, N, V):
        _bad_shape(probs, "probs", (B, N, V))
    if temperature is not None and temperature.shape != (B,):
        _bad_shape(temperature, "temperature", (B,))
    if n_rows is not None and n_rows.shape != (B,):
        _bad_shape(n_rows, "n_rows", (B,))
    dtype = logits.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"logits must be fp16, bf16 or fp32, got {dtype}")
    sb, sn, sv = logits.stride()
    if sv != 1 and V > 1:
        raise ValueError("logits must have contiguous rows")
    pp = _ptr(probs, torch.float32, "probs", dev)
    _call(load().kivi_token_probs, "kivi_token_probs", dev, _rows_ptr(logits, dtype, "logits", dev), _DTYPES[dtype],
          B, N, V, sb, sn, None if temperature is None else _ptr(temperature, torch.float32, "temperature", dev),
          None if n_rows is None else _ptr(n_rows, torch.int32, "n_rows", dev), pp, _raw_stream(stream, dev))


def kivi_verify_tree(tokens: torch.Tensor, parent: torch.Tensor, u: torch.Tensor, target: torch.Tensor,
                     draft: torch.Tensor | None, path: torch.Tensor, counts: torch.Tensor, next: torch.Tensor,
                     n_draft: torch.Tensor | None = None, stream=None):
    """path int32 [B, N], counts int32 [B] (as kivi_append_path takes them) and next
    int32 [B] <- the accepted nodes of each tree and the token after them, from the
    target's probabilities fp32 [B, N, V] after each node, the draft's fp32
    [B, N, V] from which a node's children were drawn (None: not drawn), tokens,
    parent int32 [B, N] (node 0: the pending token; parents have lower indices) and
    uniform numbers u fp32 [B, N] (u[:, 0] draws the next token).  n_draft int32
    [B]: nodes of each tree."""
    if target.dim() != 3:
        _bad_shape(target, "target", ("B", "N", "V"))
    B, N, V = target.shape
    dev = target.device
    for name, t in (("tokens", tokens), ("parent", parent), ("u", u), ("path", path)):
        if t.shape != (B, N):
            _bad_shape(t, name, (B, N))
    for name, t in (("counts", counts), ("next", next), ("n_draft", n_draft)):
        if t is not None and t.shape != (B,):
            _bad_shape(t, name, (B,))
    if draft is not None and draft.shape != (B, N, V):
        _bad_shape(draft, "draft", (B, N, V))
    i32, tp = torch.int32, _ptr(target, torch.float32, "target", dev)
    _call(load().kivi_verify_tree, "kivi_verify_tree", dev, B, N, V, _ptr(tokens, i32, "tokens", dev),
          _ptr(parent, i32, "parent", dev), None if n_draft is None else _ptr(n_draft, i32, "n_draft", dev),
          _ptr(u, torch.float32, "u", dev), tp, None if draft is None else _ptr(draft, torch.float32, "draft", dev),
          _ptr(path, i32, "path", dev), _ptr(counts, i32, "counts", dev), _ptr(next, i32, "next", dev),
          _raw_stream(stream, dev))


def _payload_buf(t: torch.Tensor, name: str, device) -> int:
    """A uint8 payload buffer: a CUDA tensor on the cache's device or a pinned
    CPU tensor (read and written by the kernels over the CPU-GPU link)."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
        raise TypeError(f"{name} must be a torch.uint8 tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.is_cuda:
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, cache is on {device}")
    elif not t.is_pinned():
        raise ValueError(f"{name} must be a CUDA tensor or pinned host memory (pin_memory=True)")
    return t.data_ptr()


def kivi_export(cache, dst: torch.Tensor, status: torch.Tensor, stream=None):
    """Write the cache's compact payload (include/kivi.h) into dst (uint8,
    CUDA or pinned host).  A payload larger than dst sets status[0] to
    KIVI_EWORKSPACE on the device and writes nothing."""
    _check(load().kivi_export(C.byref(cache.desc), _payload_buf(dst, "dst", cache.device), dst.numel(),
                              _dev(status, torch.int32, "status", cache.device),
                              _stream(stream, cache.device)), "kivi_export")


def kivi_import(cache, src: torch.Tensor, status: torch.Tensor, stream=None):
    """Read a compact payload from src (uint8, CUDA or pinned host) into the
    cache.  A header that does not match the cache's codec sets status[0] to
    KIVI_EINVAL on the device (KIVI_ECAPACITY for a sequence longer than
    Tmax, KIVI_EWORKSPACE for a truncated payload) and the cache is left as
    it was."""
    _check(load().kivi_import(C.byref(cache.desc), _payload_buf(src, "src", cache.device), src.numel(),
                              _dev(status, torch.int32, "status", cache.device),
                              _stream(stream, cache.device)), "kivi_import")


def kivi_check_status() -> int:
    """Status of the first failed device bounds check since the previous call
    (KIVI_ECHECK) or KIVI_OK; always KIVI_OK in a library built without
    KIVI_CHECKS.  Synchronizes the device."""
    out = C.c_int32(-1)
    _check(load().kivi_check_status(C.byref(out)), "kivi_check_status")
    return int(out.value)
