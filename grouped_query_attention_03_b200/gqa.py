"""ctypes binding of the C ABI in ``include/gqa.h`` (argument marshalling only).

Every computation runs in the CUDA library ``libgqa_b200.so``; this module
checks tensor dtypes, devices and contiguity, passes raw device pointers and
the current CUDA stream, and turns a non-zero ``gqa_status`` into
``GQAError``.  There is no fallback: if the library is missing, every call
raises.  PyTorch provides device memory and streams, nothing else.
"""
import ctypes
import os

import torch

from . import build as _build

LIB_PATH = _build.LIB

GQA_F32, GQA_BF16 = 0, 1
NO_WINDOW = -1

STATUS_NAMES = {
    0: "GQA_OK", 1: "GQA_ERR_NULL", 2: "GQA_ERR_SHAPE", 3: "GQA_ERR_GROUPS",
    4: "GQA_ERR_WINDOW", 5: "GQA_ERR_CAPACITY", 6: "GQA_ERR_OVERFLOW",
    7: "GQA_ERR_UNSUPPORTED", 8: "GQA_ERR_WORKSPACE", 9: "GQA_ERR_CUDA",
    10: "GQA_ERR_DEVICE", 11: "GQA_ERR_TIMEOUT", 12: "GQA_ERR_SEGMENT",
    13: "GQA_ERR_TREE",
}

# Every symbol include/gqa.h declares.
EXPORTS = ("gqa_prefill", "gqa_prefill_packed", "gqa_decode", "gqa_decode_workspace_bytes",
           "gqa_decode_append", "gqa_decode_multi", "gqa_decode_noalloc", "gqa_cache_append", "gqa_cache_bytes",
           "gqa_ring_append", "gqa_ring_decode_append", "gqa_kv_head_for_query", "gqa_window_start", "gqa_prefill_kernel", "gqa_status_string",
           "gqa_version", "gqa_selftest_wait_timeout", "gqa_qk_norm_rope", "gqa_decode_tree",
           "gqa_decode_tree_workspace_bytes", "gqa_tree_commit", "gqa_decode_scored",
           "gqa_decode_scored_workspace_bytes", "gqa_cache_evict")

NOALLOC_SCRATCH_BYTES = 8 << 20  # GQA_NOALLOC_SCRATCH_BYTES in include/gqa.h
MAX_TREE = 128  # GQA_MAX_TREE in include/gqa.h
WORKSPACE_ZERO_BYTES = 4352  # GQA_WORKSPACE_ZERO_BYTES in include/gqa.h


class GQAError(RuntimeError):
    def __init__(self, status, what):
        self.status = int(status)
        name = STATUS_NAMES.get(self.status, str(status))
        super().__init__(f"{what}: {name} ({_status_string(self.status)})")


_lib = None


def lib():
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"CUDA library {LIB_PATH} is missing; build it with "
                "grouped_query_attention_03_b200.build.build()")
        _lib = _declare(ctypes.CDLL(LIB_PATH))
    return _lib


def _declare(L):
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    sz, i64 = ctypes.c_size_t, ctypes.c_int64
    L.gqa_prefill.argtypes = [i32, vp, vp, vp, vp, vp] + [i32] * 6 + [f32, vp, vp]
    L.gqa_prefill.restype = i32
    L.gqa_prefill_packed.argtypes = [i32, vp, vp, vp, vp, vp, vp] + [i32] * 6 + [f32, vp, vp]
    L.gqa_prefill_packed.restype = i32
    L.gqa_decode.argtypes = [i32, vp, vp, vp, vp, vp] + [i32] * 6 + [f32, vp, sz, vp, vp]
    L.gqa_decode.restype = i32
    L.gqa_decode_append.argtypes = [i32] + [vp] * 7 + [i32] * 6 + [f32, vp, sz, vp, vp]
    L.gqa_decode_append.restype = i32
    L.gqa_decode_multi.argtypes = [i32, vp, vp, vp, vp, vp] + [i32] * 7 + [f32, vp, vp]
    L.gqa_decode_multi.restype = i32
    L.gqa_decode_noalloc.argtypes = [i32, vp, vp, vp, vp, vp] + [i32] * 6 + [f32, vp, vp]
    L.gqa_decode_noalloc.restype = i32
    L.gqa_decode_workspace_bytes.argtypes = [i32] * 6
    L.gqa_decode_workspace_bytes.restype = sz
    L.gqa_cache_append.argtypes = [i32, vp, vp, vp, vp, vp] + [i32] * 5 + [vp, vp]
    L.gqa_cache_append.restype = i32
    L.gqa_ring_append.argtypes = [i32, vp, vp, vp, vp, vp] + [i32] * 5 + [vp, vp]
    L.gqa_ring_append.restype = i32
    L.gqa_ring_decode_append.argtypes = [i32] + [vp] * 7 + [i32] * 5 + [f32, vp, sz, vp, vp]
    L.gqa_ring_decode_append.restype = i32
    L.gqa_cache_bytes.argtypes = [i64] * 6
    L.gqa_cache_bytes.restype = ctypes.c_uint64
    L.gqa_kv_head_for_query.argtypes = [i32] * 3
    L.gqa_kv_head_for_query.restype = i32
    L.gqa_prefill_kernel.argtypes = [i32] * 7
    L.gqa_prefill_kernel.restype = i32
    L.gqa_window_start.argtypes = [i32, i32]
    L.gqa_window_start.restype = i32
    L.gqa_status_string.argtypes = [i32]
    L.gqa_status_string.restype = ctypes.c_char_p
    L.gqa_version.argtypes = []
    L.gqa_version.restype = ctypes.c_char_p
    L.gqa_selftest_wait_timeout.argtypes = [i64, i32, vp, vp, vp]
    L.gqa_selftest_wait_timeout.restype = i32
    L.gqa_qk_norm_rope.argtypes = [i32, vp, i64, i64, vp, vp, f32, vp, i32, i32, vp, i32,
                                   vp, vp, vp, vp] + [i32] * 5 + [vp]
    L.gqa_qk_norm_rope.restype = i32
    L.gqa_decode_tree.argtypes = [i32] + [vp] * 8 + [i32] * 7 + [f32, vp, sz, vp, vp]
    L.gqa_decode_tree.restype = i32
    L.gqa_tree_commit.argtypes = [i32] + [vp] * 8 + [i32] * 6 + [vp, vp]
    L.gqa_tree_commit.restype = i32
    L.gqa_decode_scored.argtypes = [i32] + [vp] * 6 + [i32] * 6 + [f32, vp, sz, vp, vp]
    L.gqa_decode_scored.restype = i32
    for f in (L.gqa_decode_tree_workspace_bytes, L.gqa_decode_scored_workspace_bytes):
        f.argtypes = [i32] * 7
        f.restype = sz
    L.gqa_cache_evict.argtypes = [i32] + [vp] * 9 + [i32] * 7 + [vp, vp]
    L.gqa_cache_evict.restype = i32
    return L


def _status_string(s):
    try:
        return lib().gqa_status_string(int(s)).decode()
    except Exception:  # pragma: no cover - only while reporting another error
        return "?"


def _check(status, what):
    if status != 0:
        raise GQAError(status, what)


def _run(dev, what, fn, *args):
    """Call a C entry point with `dev` (the tensors' device) current: the
    library looks up per-device state (SM count, fixed scratch address) on
    the current device."""
    if dev.index == _current_device():
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status:
        raise GQAError(status, what)


_DTYPE_CODES = {torch.float32: GQA_F32, torch.bfloat16: GQA_BF16}


def _dtype_code(t):
    code = _DTYPE_CODES.get(t.dtype)
    if code is not None:
        return code
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _ptr(t, name, dtype=None, device=None):
    if t is None:
        return None
    try:  # the usual case first: a decode step is called often
        if t.dtype is dtype and t.get_device() == device.index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:  # not a tensor, or no device given
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live in CUDA device memory")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# The current stream's handle without building a torch.cuda.Stream around it
# (2 us of a small call), and the current device without the check that CUDA
# has been initialised (a tensor on it exists), where this torch has them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream, device):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _alloc(stream, make, *args):
    """make(*args): what a call allocates itself.  On another stream than the
    current one its memory has to be that stream's, so that it is cleared, and
    used again, in the order of the call."""
    if stream is None:
        return make(*args)
    with torch.cuda.stream(stream):
        return make(*args)


def _empty_as(q):
    return torch.empty_like(q, memory_format=torch.contiguous_format)


def _check_lens(lens, B):
    if lens.shape != (B,):
        raise ValueError(f"lengths must be [{B}]")


def _window(window):
    return NO_WINDOW if window is None else int(window)


def ring_append(k_ring, v_ring, k_new, v_new, seq_lens, *, status=None, stream=None):
    """Rolling buffer of W slots (k_ring [B,Hkv,W,d]): write positions
    [len_b, len_b + t_new) at slots p mod W (the last W of them survive) and
    advance seq_lens in place."""
    B, Hkv, W, d = k_ring.shape
    t_new = k_new.shape[2]
    if k_new.shape != (B, Hkv, t_new, d) or v_new.shape != k_new.shape:
        raise ValueError("new K/V shape mismatch")
    dev = k_ring.device
    st = _alloc(stream, new_status, dev) if status is None else status
    _run(dev, "gqa_ring_append", lib().gqa_ring_append,
         _dtype_code(k_ring), _ptr(k_ring, "k_ring"), _ptr(v_ring, "v_ring", k_ring.dtype, dev),
         _ptr(k_new, "k_new", k_ring.dtype, dev), _ptr(v_new, "v_new", k_ring.dtype, dev),
         _ptr(seq_lens, "seq_lens", torch.int32, dev), B, Hkv, W, d, t_new,
         _ptr(st, "status", torch.int32, dev), _stream(stream, dev))


def ring_decode_append(q, k_ring, v_ring, k_new, v_new, seq_lens, *, scale=None, out=None,
                       workspace=None, status=None, stream=None):
    """The decode step against a rolling buffer of W slots, the step's row
    appended in the same call: the query at position len_b reads the last W
    positions; seq_lens (positions before the step) grows by one."""
    B, Hq, d = q.shape
    Hkv, W = k_ring.shape[1], k_ring.shape[2]
    if k_ring.shape != (B, Hkv, W, d) or v_ring.shape != k_ring.shape:
        raise ValueError("ring shape mismatch")
    if k_new.shape != (B, Hkv, 1, d) or v_new.shape != k_new.shape:
        raise ValueError("new K/V must be [B,Hkv,1,d]")
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _alloc(stream, torch.empty_like, q)
    dev = q.device
    if workspace is None:
        workspace = _alloc(stream, decode_workspace, q, k_ring)
    st = _alloc(stream, new_status, dev) if status is None else status
    _run(dev, "gqa_ring_decode_append", lib().gqa_ring_decode_append,
         _dtype_code(q), _ptr(q, "q"), _ptr(k_ring, "k_ring", q.dtype, dev),
         _ptr(v_ring, "v_ring", q.dtype, dev), _ptr(k_new, "k_new", q.dtype, dev),
         _ptr(v_new, "v_new", q.dtype, dev), _ptr(out, "out", q.dtype, dev),
         _ptr(seq_lens, "seq_lens", torch.int32, dev), B, Hq, Hkv, W, d, float(scale),
         _ptr(workspace, "workspace", torch.uint8, dev), workspace.numel(),
         _ptr(st, "status", torch.int32, dev), _stream(stream, dev))
    return out


def new_status(device):
    """A zeroed device int32 status word."""
    return torch.zeros(1, dtype=torch.int32, device=device)


def prefill(q, k, v, *, window=None, scale=None, seq_lens=None, out=None,
            status=None, stream=None):
    """o = GQA(q, k, v) over whole prompts.  q [B,Hq,T,d], k/v [B,Hkv,T,d]."""
    B, Hq, T, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (B, Hkv, T, d) or v.shape != k.shape:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _alloc(stream, torch.empty_like, q)
    dev = q.device
    st = status
    _run(dev, "gqa_prefill", lib().gqa_prefill,
         _dtype_code(q), _ptr(q, "q"), _ptr(k, "k", q.dtype, dev), _ptr(v, "v", q.dtype, dev),
         _ptr(out, "out", q.dtype, dev), _ptr(seq_lens, "seq_lens", torch.int32, dev),
         B, Hq, Hkv, T, d, _window(window), float(scale),
         _ptr(st, "status", torch.int32, dev), _stream(stream, dev))
    return out


def prefill_packed(q, k, v, seg_start, *, window=None, scale=None, seq_lens=None,
                   out=None, status=None, stream=None):
    """prefill() over packed sequences: seg_start [B,T] int32 holds each
    cell's segment start; cell t attends [max(seg_start, t-(w-1)), t]."""
    B, Hq, T, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (B, Hkv, T, d) or v.shape != k.shape:
        raise ValueError("shape mismatch")
    if tuple(seg_start.shape) != (B, T):
        raise ValueError("seg_start must be [B, T]")
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _alloc(stream, torch.empty_like, q)
    dev = q.device
    st = _alloc(stream, new_status, dev) if status is None else status
    _run(dev, "gqa_prefill_packed", lib().gqa_prefill_packed,
         _dtype_code(q), _ptr(q, "q"), _ptr(k, "k", q.dtype, dev), _ptr(v, "v", q.dtype, dev),
         _ptr(out, "out", q.dtype, dev), _ptr(seq_lens, "seq_lens", torch.int32, dev),
         _ptr(seg_start, "seg_start", torch.int32, dev),
         B, Hq, Hkv, T, d, _window(window), float(scale), _ptr(st, "status", torch.int32, dev),
         _stream(stream, dev))
    return out


def decode_workspace_bytes(dtype, B, Hq, Hkv, C, d):
    code = GQA_BF16 if dtype == torch.bfloat16 else GQA_F32
    return int(lib().gqa_decode_workspace_bytes(code, B, Hq, Hkv, C, d))


def decode_workspace(q, k_cache):
    """A zero-filled device workspace large enough for decode on these
    shapes (reusable by later calls of any shape that fits)."""
    B, Hq, d = q.shape
    Hkv, C = k_cache.shape[1], k_cache.shape[2]
    n = decode_workspace_bytes(q.dtype, B, Hq, Hkv, C, d)
    # zero-filled once; every completed call leaves it ready for the next
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=q.device)


def decode(q, k_cache, v_cache, seq_lens, *, window=None, scale=None, out=None,
           workspace=None, status=None, stream=None):
    """One new token per sequence: q [B,Hq,d], caches [B,Hkv,C,d],
    seq_lens [B] int32 counting the cached cells including the new token."""
    B, Hq, d = q.shape
    Hkv, C = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != (B, Hkv, C, d) or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape mismatch")
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _alloc(stream, torch.empty_like, q)
    dev = q.device
    if workspace is None:
        workspace = _alloc(stream, decode_workspace, q, k_cache)
    st = _alloc(stream, new_status, dev) if status is None else status
    _run(dev, "gqa_decode", lib().gqa_decode,
         _dtype_code(q), _ptr(q, "q"), _ptr(k_cache, "k_cache", q.dtype, dev),
         _ptr(v_cache, "v_cache", q.dtype, dev), _ptr(out, "out", q.dtype, dev),
         _ptr(seq_lens, "seq_lens", torch.int32, dev), B, Hq, Hkv, C, d,
         _window(window), float(scale), _ptr(workspace, "workspace", torch.uint8, dev),
         workspace.numel(), _ptr(st, "status", torch.int32, dev), _stream(stream, dev))
    return out


def decode_append(q, k_cache, v_cache, k_new, v_new, seq_lens, *, window=None, scale=None,
                  out=None, workspace=None, status=None, stream=None):
    """The decode step with its cache append fused in: seq_lens [B] int32
    counts the cells cached BEFORE the step; k_new/v_new [B,Hkv,1,d] are the
    step's key and value rows.  Attends over the cached cells plus the new
    row, writes the new row at cell seq_lens[b] and advances seq_lens in
    place (all-or-nothing on the device)."""
    B, Hq, d = q.shape
    Hkv, C = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != (B, Hkv, C, d) or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape mismatch")
    if k_new.shape != (B, Hkv, 1, d) or v_new.shape != k_new.shape:
        raise ValueError("new K/V must be [B,Hkv,1,d]")
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _alloc(stream, torch.empty_like, q)
    dev = q.device
    if workspace is None:
        workspace = _alloc(stream, decode_workspace, q, k_cache)
    st = _alloc(stream, new_status, dev) if status is None else status
    _run(dev, "gqa_decode_append", lib().gqa_decode_append,
         _dtype_code(q), _ptr(q, "q"), _ptr(k_cache, "k_cache", q.dtype, dev),
         _ptr(v_cache, "v_cache", q.dtype, dev), _ptr(k_new, "k_new", q.dtype, dev),
         _ptr(v_new, "v_new", q.dtype, dev), _ptr(out, "out", q.dtype, dev),
         _ptr(seq_lens, "seq_lens", torch.int32, dev), B, Hq, Hkv, C, d,
         _window(window), float(scale), _ptr(workspace, "workspace", torch.uint8, dev),
         workspace.numel(), _ptr(st, "status", torch.int32, dev), _stream(stream, dev))
    return out


def decode_multi(q, k_cache, v_cache, seq_lens, *, window=None, scale=None, out=None,
                 status=None, stream=None):
    """t_new new query rows per sequence against the cache: q [B,Hq,t_new,d],
    caches [B,Hkv,C,d], seq_lens [B] int32 counting the cached cells
    including the t_new new ones (query row i sits at cell n_b - t_new + i)."""
    B, Hq, t_new, d = q.shape
    Hkv, C = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != (B, Hkv, C, d) or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape mismatch")
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _alloc(stream, torch.empty_like, q)
    dev = q.device
    st = _alloc(stream, new_status, dev) if status is None else status
    _run(dev, "gqa_decode_multi", lib().gqa_decode_multi,
         _dtype_code(q), _ptr(q, "q"), _ptr(k_cache, "k_cache", q.dtype, dev),
         _ptr(v_cache, "v_cache", q.dtype, dev), _ptr(out, "out", q.dtype, dev),
         _ptr(seq_lens, "seq_lens", torch.int32, dev), B, Hq, Hkv, C, d, t_new,
         _window(window), float(scale), _ptr(st, "status", torch.int32, dev),
         _stream(stream, dev))
    return out


def decode_noalloc(q, k_cache, v_cache, seq_lens, *, window=None, scale=None, out=None,
                   status=None, stream=None):
    """decode() without a workspace argument, for callers that cannot
    allocate device memory: the library's fixed device array serves as the
    workspace (see gqa_decode_noalloc in include/gqa.h)."""
    B, Hq, d = q.shape
    Hkv, C = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != (B, Hkv, C, d) or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape mismatch")
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _alloc(stream, torch.empty_like, q)
    dev = q.device
    st = _alloc(stream, new_status, dev) if status is None else status
    _run(dev, "gqa_decode_noalloc", lib().gqa_decode_noalloc,
         _dtype_code(q), _ptr(q, "q"), _ptr(k_cache, "k_cache", q.dtype, dev),
         _ptr(v_cache, "v_cache", q.dtype, dev), _ptr(out, "out", q.dtype, dev),
         _ptr(seq_lens, "seq_lens", torch.int32, dev), B, Hq, Hkv, C, d,
         _window(window), float(scale), _ptr(st, "status", torch.int32, dev),
         _stream(stream, dev))
    return out


def cache_append(k_cache, v_cache, k_new, v_new, seq_lens, *, status=None, stream=None):
    """Write k_new/v_new [B,Hkv,t_new,d] at cells [len_b, len_b+t_new) and
    advance seq_lens in place (all-or-nothing on the device)."""
    B, Hkv, C, d = k_cache.shape
    t_new = k_new.shape[2]
    if k_new.shape != (B, Hkv, t_new, d) or v_new.shape != k_new.shape:
        raise ValueError("new K/V shape mismatch")
    dev = k_cache.device
    st = _alloc(stream, new_status, dev) if status is None else status
    _run(dev, "gqa_cache_append", lib().gqa_cache_append,
         _dtype_code(k_cache), _ptr(k_cache, "k_cache"), _ptr(v_cache, "v_cache", k_cache.dtype, dev),
         _ptr(k_new, "k_new", k_cache.dtype, dev), _ptr(v_new, "v_new", k_cache.dtype, dev),
         _ptr(seq_lens, "seq_lens", torch.int32, dev), B, Hkv, C, d, t_new,
         _ptr(st, "status", torch.int32, dev), _stream(stream, dev))
    return st


def qk_norm_rope(qkv, Hq, Hkv, d, *, q_weight=None, k_weight=None, eps=1e-6, inv_freq=None,
                 interleaved=False, positions=None, axes=None, out=None, stream=None):
    """The rows of one QKV projection, qkv [B,T,>=(Hq+2*Hkv)*d] (rows may be
    strided), as normalised, position-rotated q [B,Hq,T,d], k and v
    [B,Hkv,T,d].  q_weight/k_weight [d]: RMS norm of each query (key) head;
    inv_freq [rot/2] float32: rotation of the first rot elements, pairs
    (i, i + rot/2) or (interleaved) (2i, 2i + 1); positions int32 [B,T] or
    [A,B,T] (None: 0..T-1), axes: the axis of each pair (a list of rot/2
    numbers below A; None: all 0)."""
    if qkv.dim() != 3 or (qkv.stride(2) != 1 and qkv.shape[2] > 1):
        raise ValueError("qkv must be [B,T,width] with contiguous rows")
    B, T, width = qkv.shape
    if width < (Hq + 2 * Hkv) * d:
        raise ValueError(f"qkv rows of {width} elements do not hold {Hq} + 2 * {Hkv} heads of {d}")
    dev, dt = qkv.device, qkv.dtype
    half = 0 if inv_freq is None else inv_freq.numel()
    if positions is None:
        naxes = 1
    else:
        at = positions.shape
        naxes = at[0] if len(at) == 3 else 1
        if at != (B, T) and at != (naxes, B, T):
            raise ValueError("positions must be [B,T] or [axes,B,T]")
    pair_axis = None
    if axes is not None:
        if len(axes) != half:
            raise ValueError(f"axes must name the axis of each of the {half} pairs")
        if naxes > 1 or any(axes):  # one axis: nothing to say
            pair_axis = (ctypes.c_int32 * half)(*axes)
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None and w.numel() != d:
            raise ValueError(f"{name} must have {d} elements")
    if out is None:
        out = _alloc(stream, lambda: tuple(torch.empty((B, h, T, d), dtype=dt, device=dev)
                                           for h in (Hq, Hkv, Hkv)))
    q, k, v = out
    rows = (B, Hkv, T, d)
    if q.shape != (B, Hq, T, d) or k.shape != rows or v.shape != rows:
        raise ValueError("out must be q [B,Hq,T,d], k and v [B,Hkv,T,d]")
    if not qkv.is_cuda:
        raise ValueError("qkv must live in CUDA device memory")
    # a dimension of one row has no meaningful stride
    row_stride = qkv.stride(1) if T > 1 else width
    batch_stride = qkv.stride(0) if B > 1 else 0
    _run(dev, "gqa_qk_norm_rope", lib().gqa_qk_norm_rope,
         _dtype_code(qkv), qkv.data_ptr(), batch_stride, row_stride,
         _ptr(q_weight, "q_weight", dt, dev), _ptr(k_weight, "k_weight", dt, dev), float(eps),
         _ptr(inv_freq, "inv_freq", torch.float32, dev), 2 * half, 1 if interleaved else 0,
         _ptr(positions, "positions", torch.int32, dev), naxes, pair_axis,
         _ptr(q, "q", dt, dev), _ptr(k, "k", dt, dev), _ptr(v, "v", dt, dev),
         B, Hq, Hkv, T, d, _stream(stream, dev))
    return q, k, v


def _workspace(n, device):
    """n bytes, ready for a first call: zero-filled where they must be.  (A few
    MB cost less to clear than the slice does.)"""
    if n <= 1 << 22:
        return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:WORKSPACE_ZERO_BYTES].zero_()
    return ws


def decode_tree_workspace(q, k_cache):
    """A device workspace for decode_tree on these shapes, ready for its first
    use (and for later calls of any shape that fits)."""
    B, Hq, t, d = q.shape
    code = _dtype_code(q)
    n = lib().gqa_decode_tree_workspace_bytes(code, B, Hq, k_cache.shape[1], k_cache.shape[2], d, t)
    return _workspace(n, q.device)  # every completed call leaves it ready for the next


def decode_tree(q, k_cache, v_cache, k_draft, v_draft, parents, seq_lens, *, window=None,
                scale=None, out=None, workspace=None, status=None, stream=None):
    """Attention for a tree of drafted tokens: q [B,Hq,t,d] the nodes'
    queries, caches [B,Hkv,C,d] of seq_lens [B] int32 committed cells,
    k_draft/v_draft [B,Hkv,t,d] the nodes' rows (not in the cache yet).  Node
    i reads the committed cells and its own line in the tree; parents [B,t]
    int32: -1 a root, -2 padding, None a chain."""
    B, Hq, t, d = shape = q.shape
    cells, drafts = k_cache.shape, k_draft.shape
    Hkv, C = cells[1], cells[2]
    if cells != (B, Hkv, C, d) or v_cache.shape != cells:
        raise ValueError("cache shape mismatch")
    if drafts != (B, Hkv, t, d) or v_draft.shape != drafts:
        raise ValueError("drafted K/V must be [B,Hkv,t,d]")
    if parents is not None and parents.shape != (B, t):
        raise ValueError("parents must be [B, t]")
    _check_lens(seq_lens, B)
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _alloc(stream, _empty_as, q)
    elif out.shape != shape:
        raise ValueError("out must have the shape of q")
    dev, dt = q.device, q.dtype
    if workspace is None:
        workspace = _alloc(stream, decode_tree_workspace, q, k_cache)
    st = _alloc(stream, new_status, dev) if status is None else status
    _run(dev, "gqa_decode_tree", lib().gqa_decode_tree,
         _dtype_code(q), _ptr(q, "q"), _ptr(k_cache, "k_cache", dt, dev),
         _ptr(v_cache, "v_cache", dt, dev), _ptr(k_draft, "k_draft", dt, dev),
         _ptr(v_draft, "v_draft", dt, dev), _ptr(parents, "parents", torch.int32, dev),
         _ptr(out, "out", dt, dev), _ptr(seq_lens, "seq_lens", torch.int32, dev),
         B, Hq, Hkv, C, d, t, _window(window), float(scale),
         _ptr(workspace, "workspace", torch.uint8, dev), workspace.numel(),
         _ptr(st, "status", torch.int32, dev), _stream(stream, dev))
    return out


def tree_commit(k_cache, v_cache, k_draft, v_draft, path, path_lens, seq_lens, *, lens_out=None,
                status=None, stream=None):
    """The accepted path enters the cache: rows path[b, :path_lens[b]] (int32
    [B,P], ascending nodes) of k_draft/v_draft [B,Hkv,t,d] go to cells
    seq_lens[b] on, and lens_out (default: seq_lens itself) becomes seq_lens
    + path_lens (all-or-nothing on the device).  Returns the status word."""
    B, Hkv, C, d = cells = k_cache.shape
    drafts, steps = k_draft.shape, path.shape
    t = drafts[2]
    if v_cache.shape != cells:
        raise ValueError("cache shape mismatch")
    if drafts != (B, Hkv, t, d) or v_draft.shape != drafts:
        raise ValueError("drafted K/V must be [B,Hkv,t,d]")
    if len(steps) != 2 or steps[0] != B or path_lens.shape != (B,):
        raise ValueError("path must be [B,P] and path_lens [B]")
    _check_lens(seq_lens, B)
    if lens_out is None:
        lens_out = seq_lens
    else:
        _check_lens(lens_out, B)
    dev, dt = k_cache.device, k_cache.dtype
    st = _alloc(stream, new_status, dev) if status is None else status
    _run(dev, "gqa_tree_commit", lib().gqa_tree_commit,
         _dtype_code(k_cache), _ptr(k_cache, "k_cache"), _ptr(v_cache, "v_cache", dt, dev),
         _ptr(k_draft, "k_draft", dt, dev), _ptr(v_draft, "v_draft", dt, dev),
         _ptr(path, "path", torch.int32, dev), _ptr(path_lens, "path_lens", torch.int32, dev),
         _ptr(seq_lens, "seq_lens", torch.int32, dev), _ptr(lens_out, "lens_out", torch.int32, dev),
         B, Hkv, C, d, t, steps[1], _ptr(st, "status", torch.int32, dev), _stream(stream, dev))
    return st


def _scored_shape(q):
    shape = q.shape
    if len(shape) == 3:
        return shape[0], shape[1], 1, shape[2]
    if len(shape) != 4:
        raise ValueError("q must be [B,Hq,d] or [B,Hq,t,d]")
    return shape


def decode_scored_workspace(q, k_cache):
    """A device workspace for decode_scored on these shapes, ready for its first
    use (and for later calls of any shape that fits)."""
    B, Hq, t, d = _scored_shape(q)
    code = _dtype_code(q)
    n = lib().gqa_decode_scored_workspace_bytes(code, B, Hq, k_cache.shape[1], k_cache.shape[2], d, t)
    return _workspace(n, q.device)  # every completed call leaves it ready for the next


def decode_scored(q, k_cache, v_cache, weights, seq_lens, *, scale=None, out=None, workspace=None,
                  status=None, stream=None):
    """decode() (q [B,Hq,d]) or decode_multi() (q [B,Hq,t,d]) that also adds
    to weights [B,Hkv,C] float32 the softmax weights each cell received."""
    shape, cells = q.shape, k_cache.shape
    B, Hq, t, d = _scored_shape(q)
    Hkv, C = cells[1], cells[2]
    if cells != (B, Hkv, C, d) or v_cache.shape != cells:
        raise ValueError("cache shape mismatch")
    if weights.shape != (B, Hkv, C):
        raise ValueError("weights must be [B,Hkv,C]")
    _check_lens(seq_lens, B)
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _alloc(stream, _empty_as, q)
    elif out.shape != shape:
        raise ValueError("out must have the shape of q")
    dev, dt = q.device, q.dtype
    if workspace is None:
        workspace = _alloc(stream, decode_scored_workspace, q, k_cache)
    st = _alloc(stream, new_status, dev) if status is None else status
    _run(dev, "gqa_decode_scored", lib().gqa_decode_scored,
         _dtype_code(q), _ptr(q, "q"), _ptr(k_cache, "k_cache", dt, dev),
         _ptr(v_cache, "v_cache", dt, dev), _ptr(out, "out", dt, dev),
         _ptr(weights, "weights", torch.float32, dev), _ptr(seq_lens, "seq_lens", torch.int32, dev),
         B, Hq, Hkv, C, d, t, float(scale), _ptr(workspace, "workspace", torch.uint8, dev),
         workspace.numel(), _ptr(st, "status", torch.int32, dev), _stream(stream, dev))
    return out


def cache_evict(k_cache, v_cache, weights, seq_lens, budget, recent, *, k_out=None, v_out=None,
                weights_out=None, lens_out=None, kept=None, status=None, stream=None):
    """Lanes of more than `budget` cells keep their last `recent` and, of the
    others, the budget - recent with the largest weights [B,Hkv,C] float32,
    in their order: in place, or into k_out/v_out [B,Hkv,C_out,d] and
    weights_out [B,Hkv,C_out].  lens_out (default: seq_lens itself) becomes
    min(seq_lens, budget).  Returns kept [B,Hkv,budget] int32, the cell that
    each kept row came from (-1 behind them)."""
    B, Hkv, C, d = cells = k_cache.shape
    if v_cache.shape != cells or weights.shape != (B, Hkv, C):
        raise ValueError("cache and weights shape mismatch")
    C_out = C
    if k_out is None and v_out is None and weights_out is None:
        k_out, v_out, weights_out = k_cache, v_cache, weights
    elif k_out is None or v_out is None or weights_out is None:
        raise ValueError("k_out, v_out and weights_out come together")
    else:
        new_cells = k_out.shape
        C_out = new_cells[2]
        if new_cells != (B, Hkv, C_out, d) or v_out.shape != new_cells or \
                weights_out.shape != (B, Hkv, C_out):
            raise ValueError("output shape mismatch")
    _check_lens(seq_lens, B)
    if lens_out is None:
        lens_out = seq_lens
    else:
        _check_lens(lens_out, B)
    dev, dt = k_cache.device, k_cache.dtype
    if kept is None:
        kept = _alloc(stream, lambda: torch.empty((B, Hkv, max(budget, 0)), dtype=torch.int32, device=dev))
    elif kept.shape != (B, Hkv, budget):
        raise ValueError("kept must be [B,Hkv,budget]")
    st = _alloc(stream, new_status, dev) if status is None else status
    _run(dev, "gqa_cache_evict", lib().gqa_cache_evict,
         _dtype_code(k_cache), _ptr(k_cache, "k_cache"), _ptr(v_cache, "v_cache", dt, dev),
         _ptr(weights, "weights", torch.float32, dev), _ptr(seq_lens, "seq_lens", torch.int32, dev),
         _ptr(k_out, "k_out", dt, dev), _ptr(v_out, "v_out", dt, dev),
         _ptr(weights_out, "weights_out", torch.float32, dev),
         _ptr(lens_out, "lens_out", torch.int32, dev), _ptr(kept, "kept", torch.int32, dev),
         B, Hkv, C, C_out, d, int(budget), int(recent), _ptr(st, "status", torch.int32, dev),
         _stream(stream, dev))
    return kept


def cache_bytes(L, B, T, Hkv, d, elem_bytes):
    return int(lib().gqa_cache_bytes(L, B, T, Hkv, d, elem_bytes))


def prefill_kernel(B, Hq, Hkv, T, d, window=None, sms=None):
    """Which kernel gqa_prefill runs for a bf16 prompt of this shape: "pair"
    (two heads of a KV group per CTA), "split" (one head per CTA) or "simt"
    (CUDA cores).  `sms` defaults to the current device's SM count."""
    if sms is None:
        sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    r = lib().gqa_prefill_kernel(B, Hq, Hkv, T, d, -1 if window is None else window, sms)
    if r < 0:
        raise ValueError(f"prefill_kernel: invalid arguments {(B, Hq, Hkv, T, d, window, sms)}")
    return ("simt", "pair", "split")[r]


def kv_head_for_query(h, Hq, Hkv):
    g = lib().gqa_kv_head_for_query(h, Hq, Hkv)
    return None if g < 0 else g


def window_start(t, window):
    s = lib().gqa_window_start(t, _window(window))
    return None if s < 0 else s


def version():
    return lib().gqa_version().decode()


def selftest_wait_timeout(limit_us, *, arrive=False, device=None, status=None, stream=None):
    """Run the kernels' two bounded wait routines on mbarriers nobody
    arrives on (arrive=False: both give up after limit_us and the kernel
    records GQA_ERR_TIMEOUT) or that one thread completes first (arrive=True:
    both succeed).  Returns (status, gave_up) device tensors."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    st = _alloc(stream, new_status, dev) if status is None else status
    gave_up = _alloc(stream, lambda: torch.zeros(2, dtype=torch.int32, device=dev))
    _run(dev, "gqa_selftest_wait_timeout", lib().gqa_selftest_wait_timeout,
         int(limit_us), 1 if arrive else 0, _ptr(st, "status", torch.int32, dev),
         _ptr(gave_up, "gave_up", torch.int32, dev), _stream(stream, dev))
    return st, gave_up
