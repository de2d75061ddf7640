"""The key/value cache in 4 bits: binding of the ``magi_bca_kv4_*`` entry points.

As the rest of the package this only marshals arguments; ``include/magi_bca.h``
describes the format and each operation.  Lengths and positions are int32
tensors on the device, so a decoding step can be captured in a CUDA graph and
replayed while the history grows.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple

__all__ = ["Kv4Cache", "magi_bca_kv4_cache", "magi_bca_kv4_append", "magi_bca_kv4_read", "magi_bca_kv4_fwd",
           "magi_bca_kv4_weights", "magi_bca_kv4_evict", "magi_bca_kv4_fwd_workspace_size",
           "magi_bca_kv4_weights_workspace_size"]


# magi_bca_kv4_cache and magi_bca_kv4_query as the C compiler lays them out.
# A call is some microseconds of host time, so the structs go over as bytes.
_CACHE = struct.Struct("=4Q4i")    # k_codes, k_scales, v_codes, v_scales; batch, heads_kv, head_dim, capacity
_QUERY = struct.Struct("=2i2fq")   # seqlen_q, heads_q; softmax_scale, rms_eps; rope_batch_stride


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the entry points (called once, when the library is loaded)."""
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    cp = qp = ctypes.c_char_p
    lib.magi_bca_kv4_append.argtypes = [vp, vp, cp, vp, vp, i32, vp, i64, f32, vp]
    lib.magi_bca_kv4_read.argtypes = [cp, vp, i32, vp, vp, vp]
    lib.magi_bca_kv4_fwd.argtypes = [vp, cp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, qp, vp]
    lib.magi_bca_kv4_weights.argtypes = [vp, cp, vp, vp, vp, vp, vp, vp, f32, vp, sz, qp, vp]
    lib.magi_bca_kv4_evict.argtypes = [cp, vp, vp, i32, i32, cp, vp, vp, vp, vp]
    for name in ("append", "read", "fwd", "weights", "evict"):
        getattr(lib, "magi_bca_kv4_" + name).restype = ctypes.c_int
    for name in ("fwd", "weights"):
        f = getattr(lib, f"magi_bca_kv4_{name}_workspace_size")
        f.argtypes, f.restype = [cp, qp], sz


class Kv4Cache(NamedTuple):
    """The four uint8 tensors of a cache (any 4-tuple of them will do):
    k_codes [B, Hkv, capacity, D/2], k_scales [B, Hkv, capacity, D/16],
    v_codes [B, Hkv, capacity/2, D], v_scales [B, Hkv, capacity/2, D/16, 2]."""
    k_codes: "torch.Tensor"   # noqa: F821
    k_scales: "torch.Tensor"  # noqa: F821
    v_codes: "torch.Tensor"   # noqa: F821
    v_scales: "torch.Tensor"  # noqa: F821


def magi_bca_kv4_cache(batch: int, heads_kv: int, head_dim: int, capacity: int, device="cuda") -> Kv4Cache:
    """A zeroed cache; capacity is rounded up to a multiple of 128 slots."""
    import torch
    if head_dim not in (64, 128):
        raise ValueError(f"head_dim must be 64 or 128 (got {head_dim})")
    if min(batch, heads_kv, capacity) < 1:
        raise ValueError("batch, heads_kv and capacity must be positive")
    cap = -(-int(capacity) // 128) * 128
    z = lambda *s: torch.zeros(*s, device=device, dtype=torch.uint8)  # noqa: E731
    return Kv4Cache(z(batch, heads_kv, cap, head_dim // 2), z(batch, heads_kv, cap, head_dim // 16),
                    z(batch, heads_kv, cap // 2, head_dim), z(batch, heads_kv, cap // 2, head_dim // 16, 2))


# The checks are written for the good case: one expression a tensor, and the
# reason looked for only where it fails.  torch and the library are loaded by the
# first call.
torch = None
_lib = None


def _load():
    global torch, _lib, _u8, _bf16, _f32, _i32
    import torch as t
    from . import library
    _u8, _bf16, _f32, _i32 = t.uint8, t.bfloat16, t.float32, t.int32
    _lib, torch = library(), t


def _refuse(name, t, dtype, shape, index):
    """Says what is wrong with an argument (never returns)."""
    kind = str(dtype)[6:]
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {kind} CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{index}")


def _check(name, t, dtype, shape, index):
    """The tensor's address, if it is a contiguous one of this type and shape on device `index`."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(name, t, dtype, shape, index)


def _cache(cache, index, name="cache"):
    """Checks a cache's tensors: (the C struct's bytes, batch, heads, head_dim, capacity)."""
    kc, ks, vc, vs = cache
    if not isinstance(kc, torch.Tensor) or kc.dim() != 4:
        raise TypeError(f"{name}.k_codes must be a uint8 CUDA tensor [batch, heads_kv, capacity, head_dim/2]")
    shape = kc.shape
    B, H, cap, half = shape
    D = 2 * half
    n = D // 16
    return _CACHE.pack(_check(name + ".k_codes", kc, _u8, shape, index), _check(name + ".k_scales", ks, _u8, (B, H, cap, n), index),
                       _check(name + ".v_codes", vc, _u8, (B, H, cap // 2, D), index),
                       _check(name + ".v_scales", vs, _u8, (B, H, cap // 2, n, 2), index), B, H, D, cap), B, H, D, cap


def _check_rope(name, t, batch, n, half, index):
    """(pointer, batch stride in elements) of an angle table [n, D/2] or [B, n, D/2]."""
    if t is None:
        return None, 0
    if isinstance(t, torch.Tensor) and t.dim() == 3:
        return _check(name, t, _f32, (batch, n, half), index), n * half
    return _check(name, t, _f32, (n, half), index), 0


def _device_of(name, t):
    """The device index a call runs on: that of its first tensor."""
    if torch is None:
        _load()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != 4:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected 4 dimensions")
    return t.get_device()


def _run(f, index, stream, *args):
    """Calls the entry point f on device `index`; the stream goes last."""
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        st = f(*args, handle)
    else:
        with torch.cuda.device(index):
            st = f(*args, handle)
    if st != 0:
        from . import MagiBcaError
        raise MagiBcaError(st, f.__name__)


def magi_bca_kv4_append(cache, k, v, start, counts=None, rope_k=None, rms_eps: float = 1e-6, stream=None) -> None:
    """Quantises k, v [B, n, Hkv, D] bf16 into the slots start[b] .. of each
    batch element (start: int32 [B] on the device).  counts: int32 [B], how many
    of the n tokens are real (None: all).  rope_k: fp32 angles [n, D/2] or
    [B, n, D/2] applied to k before its norm."""
    dev = _device_of("k", k)
    shape = k.shape
    B, n, H, D = shape
    c, cB, cH, cD, _ = _cache(cache, dev)
    if cB != B or cH != H or cD != D:
        raise ValueError(f"k has shape {tuple(shape)}, the cache holds batch {cB}, {cH} heads of {cD}")
    if n < 1:
        return
    rp, rs = _check_rope("rope_k", rope_k, B, n, D // 2, dev)
    _run(_lib.magi_bca_kv4_append, dev, stream, _check("k", k, _bf16, shape, dev), _check("v", v, _bf16, shape, dev), c,
         _check("start", start, _i32, (B,), dev), None if counts is None else _check("counts", counts, _i32, (B,), dev),
         n, rp, rs, rms_eps)


def magi_bca_kv4_read(cache, start, n: int, k=None, v=None, stream=None):
    """The values of the slots start[b] .. start[b] + n - 1 (start None: from
    slot 0) as bf16 (k, v) [B, n, Hkv, D]; the keys are normalised and rotated."""
    dev = _device_of("cache.k_codes", cache[0])
    c, B, H, D, _ = _cache(cache, dev)
    n = int(n)
    shape = (B, n, H, D)
    k = cache[0].new_empty(shape, dtype=_bf16) if k is None else k
    v = torch.empty_like(k) if v is None else v
    kp, vp = _check("k", k, _bf16, shape, dev), _check("v", v, _bf16, shape, dev)
    sp = None if start is None else _check("start", start, _i32, (B,), dev)
    if n > 0:
        _run(_lib.magi_bca_kv4_read, dev, stream, c, sp, n, kp, vp)
    return k, v


def _query(q, cache, gamma_q, gamma_k, rope_q, softmax_scale, rms_eps):
    """Checks the query side and the cache; returns what the two calls share."""
    dev = _device_of("q", q)
    c, cB, cH, cD, cap = _cache(cache, dev)
    shape = q.shape
    B, Sq, Hq, D = shape
    if cB != B or cD != D:
        raise ValueError(f"q has shape {tuple(shape)}, the cache holds batch {cB}, heads of {cD}")
    if Sq < 1:
        raise ValueError("q has no tokens")
    rp, rs = _check_rope("rope_q", rope_q, B, Sq, D // 2, dev)
    return (dev, c, _QUERY.pack(Sq, Hq, softmax_scale, rms_eps, rs), _check("q", q, _bf16, shape, dev),
            _check("gamma_q", gamma_q, _f32, (D,), dev), _check("gamma_k", gamma_k, _f32, (D,), dev), rp, (B, cH, cap))


def _workspace(size_fn, c, query, workspace, q, stream):
    """(pointer, bytes, tensor) of the caller's workspace or a new one."""
    if workspace is None:
        n = size_fn(c, query)
        if n == 0:
            return None, 0, None
        workspace = q.new_empty(n, dtype=_u8)
        return workspace.data_ptr(), n, workspace
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA tensor")
    if workspace.device != q.device:
        raise ValueError(f"workspace is on {workspace.device}, the call runs on {q.device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), None


def _keep(made, stream):
    """A workspace made here (on the current stream) and used on another one must
    not be handed out again before that stream is done with it."""
    if made is not None and stream is not None and not torch.cuda.is_current_stream_capturing():
        made.record_stream(stream)


def magi_bca_kv4_fwd(q, cache, lengths, gamma_q, gamma_k, rope_q=None, base_out=None, base_lse=None, out=None,
                     lse=None, softmax_scale: float = 0.0, rms_eps: float = 1e-6, want_lse: bool = True,
                     workspace=None, stream=None):
    """Attention of q [B, Sq, Hq, D] over the first lengths[b] (int32 [B] on the
    device) tokens of the cache.  rope_q: angles [Sq, D/2] or [B, Sq, D/2].
    base_out / base_lse: the same queries' attention over other keys, as
    ``magi_bca_fwd`` returns it, to be joined.  Returns (out, lse)."""
    dev, c, query, qp, gq, gk, rp, _ = _query(q, cache, gamma_q, gamma_k, rope_q, softmax_scale, rms_eps)
    shape = q.shape
    rows = (shape[0], shape[2], shape[1])
    if (base_out is None) != (base_lse is None):
        raise ValueError("base_out and base_lse go together")
    bo = bl = lp = None
    if base_out is not None:
        bo, bl = _check("base_out", base_out, _bf16, shape, dev), _check("base_lse", base_lse, _f32, rows, dev)
    ln = _check("lengths", lengths, _i32, rows[:1], dev)
    out = torch.empty_like(q) if out is None else out
    if lse is None and want_lse:
        lse = gamma_q.new_empty(rows)
    if lse is not None:
        lp = _check("lse", lse, _f32, rows, dev)
    wp, wb, made = _workspace(_lib.magi_bca_kv4_fwd_workspace_size, c, query, workspace, q, stream)
    _run(_lib.magi_bca_kv4_fwd, dev, stream, qp, c, ln, gq, gk, rp, bo, bl, _check("out", out, _bf16, shape, dev), lp, wp,
         wb, query)
    if made is not None:
        _keep(made, stream)
    return out, lse


def magi_bca_kv4_weights(q, cache, lengths, lse, gamma_q, gamma_k, weights, rope_q=None, decay: float = 1.0,
                         softmax_scale: float = 0.0, rms_eps: float = 1e-6, workspace=None, stream=None):
    """weights[b, h, j] = decay * weights[b, h, j] + the attention weight key j
    (j < lengths[b]) receives from q, given the rows' lse [B, Hq, Sq].  weights:
    fp32 [B, Hkv, capacity], changed in place and returned."""
    dev, c, query, qp, gq, gk, rp, wshape = _query(q, cache, gamma_q, gamma_k, rope_q, softmax_scale, rms_eps)
    B, Sq, Hq, _ = q.shape
    lp = _check("lse", lse, _f32, (B, Hq, Sq), dev)
    w = _check("weights", weights, _f32, wshape, dev)
    ln = _check("lengths", lengths, _i32, (B,), dev)
    wp, wb, made = _workspace(_lib.magi_bca_kv4_weights_workspace_size, c, query, workspace, q, stream)
    _run(_lib.magi_bca_kv4_weights, dev, stream, qp, c, ln, lp, gq, gk, rp, w, decay, wp, wb, query)
    if made is not None:
        _keep(made, stream)
    return weights


def magi_bca_kv4_evict(cache, weights, lengths, keep: int, recent: int, dst_cache, dst_weights, dst_lengths=None,
                       index=None, stream=None):
    """Moves to dst_cache the last `recent` tokens of each (batch element, head)
    and those with the largest weight, min(keep, length) in all, in their order;
    dst_weights [B, Hkv, dst capacity] gets their weights.  Returns (dst_lengths
    int32 [B], index int32 [B, Hkv, keep]: the slot each token came from, -1
    behind the last)."""
    dev = _device_of("cache.k_codes", cache[0])
    c, B, H, D, cap = _cache(cache, dev)
    d, dB, dH, dD, dcap = _cache(dst_cache, dev, "dst_cache")
    if dB != B or dH != H or dD != D:
        raise ValueError("dst_cache must have the cache's batch, heads and head_dim")
    keep, recent = int(keep), int(recent)
    if not (1 <= keep <= dcap and 0 <= recent <= keep):
        raise ValueError(f"need 1 <= keep <= {dcap} and 0 <= recent <= keep (got {keep}, {recent})")
    w = _check("weights", weights, _f32, (B, H, cap), dev)
    dw = _check("dst_weights", dst_weights, _f32, (B, H, dcap), dev)
    ln = _check("lengths", lengths, _i32, (B,), dev)
    dst_lengths = torch.empty_like(lengths) if dst_lengths is None else dst_lengths
    index = lengths.new_empty((B, H, keep)) if index is None else index
    _run(_lib.magi_bca_kv4_evict, dev, stream, c, w, ln, keep, recent, d, dw, _check("dst_lengths", dst_lengths, _i32, (B,), dev),
         _check("index", index, _i32, (B, H, keep), dev))
    return dst_lengths, index


def _size(name, cache, seqlen_q, heads_q):
    c = _cache(cache, _device_of("cache.k_codes", cache[0]))[0]
    return int(getattr(_lib, name)(c, _QUERY.pack(seqlen_q, heads_q, 0.0, 0.0, 0)))


def magi_bca_kv4_fwd_workspace_size(cache, seqlen_q: int, heads_q: int) -> int:
    """Bytes of workspace ``magi_bca_kv4_fwd`` needs for a cache of this shape."""
    return _size("magi_bca_kv4_fwd_workspace_size", cache, seqlen_q, heads_q)


def magi_bca_kv4_weights_workspace_size(cache, seqlen_q: int, heads_q: int) -> int:
    """Bytes of workspace ``magi_bca_kv4_weights`` needs for a cache of this shape."""
    return _size("magi_bca_kv4_weights_workspace_size", cache, seqlen_q, heads_q)
