"""ctypes binding of librkv.so (C ABI in include/rkv.h), same names as the C calls.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of librkv.so.  Tensors are torch CUDA tensors used for device memory
and streams; they are passed to the library as raw pointers and row strides.
There is no CPU fallback: importing this module raises ImportError when the
library has not been built.
"""

import ctypes
import math
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "librkv.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"librkv.so not found at {LIB_PATH}; build it with "
        "`python -m rolling_kv_cache_rope_b200.build` (nvcc, sm_100a). There is no CPU fallback.")

_lib = ctypes.CDLL(LIB_PATH)

RKV_OK, RKV_ERR_INVALID_ARG, RKV_ERR_UNSUPPORTED, RKV_ERR_CUDA, RKV_ERR_TIMEOUT, RKV_ERR_DEVICE_CHECK = 0, 1, 2, 3, 4, 5
RKV_ROPE_Q, RKV_ROPE_K = 1, 2
RKV_MAX_SEQS = 16
STATUS_NAMES = {0: "RKV_OK", 1: "RKV_ERR_INVALID_ARG", 2: "RKV_ERR_UNSUPPORTED", 3: "RKV_ERR_CUDA",
                4: "RKV_ERR_TIMEOUT", 5: "RKV_ERR_DEVICE_CHECK"}


class rkv_rope3d(ctypes.Structure):
    _fields_ = [("grid_h", ctypes.c_int32), ("grid_w", ctypes.c_int32), ("pairs_t", ctypes.c_int32),
                ("pairs_h", ctypes.c_int32), ("pairs_w", ctypes.c_int32), ("theta", ctypes.c_float),
                ("theta_h", ctypes.c_float), ("theta_w", ctypes.c_float), ("layout", ctypes.c_int32)]


RKV_ROPE_ADJACENT, RKV_ROPE_HALF = 0, 1
RKV_ROPE_BATCH_MAX = 8


class rkv_rope_tensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("L", ctypes.c_int64),
                ("x_row_stride", ctypes.c_int64), ("y_row_stride", ctypes.c_int64), ("t0", ctypes.c_int32)]


class rkv_attn_seq(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("o", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("o_stride", ctypes.c_int64), ("Lq", ctypes.c_int32), ("Lk", ctypes.c_int32),
                ("q_t0", ctypes.c_int32), ("k_t0", ctypes.c_int32), ("q_frame_offset", ctypes.c_int32),
                ("block_frames", ctypes.c_int32), ("flags", ctypes.c_uint32), ("reserved", ctypes.c_int32)]


class rkv_attn_debug(ctypes.Structure):
    _fields_ = [("row_stats", ctypes.c_void_p), ("stall", ctypes.c_uint32), ("timeout_us", ctypes.c_uint32)]


class rkv_ring_debug(ctypes.Structure):
    _fields_ = [("stall", ctypes.c_uint32), ("timeout_us", ctypes.c_uint32)]


RKV_DEBUG_STALL_NONE, RKV_DEBUG_STALL_V_READY, RKV_DEBUG_STALL_K_READY, RKV_DEBUG_STALL_P_FULL = 0, 1, 2, 3
RKV_DEBUG_STALL_BULK_LOAD = 1


class rkv_attn_window(ctypes.Structure):
    _fields_ = [("window_blocks", ctypes.c_int32), ("sink_blocks", ctypes.c_int32)]


class rkv_paged_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("n_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("H", ctypes.c_int32),
                ("D", ctypes.c_int32), ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("status", ctypes.c_void_p)]


RKV_DECODE_MAX_LQ = 64


class rkv_ring(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("slots", ctypes.c_int32),
                ("tokens_per_frame", ctypes.c_int32), ("H", ctypes.c_int32), ("D", ctypes.c_int32),
                ("head", ctypes.c_int32), ("count", ctypes.c_int32), ("pinned", ctypes.c_int32)]


_c = ctypes
_lib.rope3d_apply.restype = _c.c_int
_lib.rope3d_apply.argtypes = [_c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int32, _c.c_int32, _c.c_int64, _c.c_int64,
                              _c.c_int32, _c.POINTER(rkv_rope3d), _c.c_void_p]
_lib.rope3d_apply_batch.restype = _c.c_int
_lib.rope3d_apply_batch.argtypes = [_c.POINTER(rkv_rope_tensor), _c.c_int32, _c.c_int32, _c.c_int32,
                                    _c.POINTER(rkv_rope3d), _c.c_void_p]
_lib.attn_fwd_varlen_workspace_size.restype = _c.c_size_t
_lib.attn_fwd_varlen_workspace_size.argtypes = [_c.POINTER(rkv_attn_seq), _c.c_int32, _c.c_int32, _c.c_int32]
_lib.attn_fwd_varlen.restype = _c.c_int
_lib.attn_fwd_varlen.argtypes = [_c.POINTER(rkv_attn_seq), _c.c_int32, _c.c_int32, _c.c_int32, _c.c_float,
                                 _c.POINTER(rkv_rope3d), _c.c_void_p, _c.c_size_t, _c.c_void_p]
_lib.rkv_attn_status.restype = _c.c_int
_lib.rkv_attn_status.argtypes = [_c.c_void_p, _c.c_void_p]
_lib.attn_fwd_varlen_debug.restype = _c.c_int
_lib.attn_fwd_varlen_debug.argtypes = [_c.POINTER(rkv_attn_seq), _c.c_int32, _c.c_int32, _c.c_int32, _c.c_float,
                                       _c.POINTER(rkv_rope3d), _c.c_void_p, _c.c_size_t, _c.POINTER(rkv_attn_debug),
                                       _c.c_void_p]
_lib.attn_fwd_varlen_noalloc.restype = _c.c_int
_lib.attn_fwd_varlen_noalloc.argtypes = [_c.POINTER(rkv_attn_seq), _c.c_int32, _c.c_int32, _c.c_int32, _c.c_float,
                                         _c.POINTER(rkv_rope3d), _c.c_void_p]
_lib.rkv_attn_noalloc_status.restype = _c.c_int
_lib.rkv_attn_noalloc_status.argtypes = [_c.c_void_p]
_lib.rkv_attn_mask_rows.restype = _c.c_int
_lib.rkv_attn_mask_rows.argtypes = [_c.POINTER(rkv_attn_seq), _c.c_int32, _c.c_int32, _c.POINTER(rkv_rope3d),
                                    _c.POINTER(_c.c_int64), _c.POINTER(_c.c_int32), _c.POINTER(_c.c_int64)]
_lib.kvcache_ring_update.restype = _c.c_int
_lib.kvcache_ring_update.argtypes = [_c.POINTER(rkv_ring), _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int32,
                                     _c.POINTER(_c.c_int32), _c.c_void_p]
_lib.kvcache_ring_update_rope.restype = _c.c_int
_lib.kvcache_ring_update_rope.argtypes = [_c.POINTER(rkv_ring), _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int32,
                                          _c.c_int32, _c.POINTER(rkv_rope3d), _c.POINTER(_c.c_int32), _c.c_void_p]
_lib.kvcache_ring_update_debug.restype = _c.c_int
_lib.kvcache_ring_update_debug.argtypes = [_c.POINTER(rkv_ring), _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int32,
                                           _c.POINTER(_c.c_int32), _c.POINTER(rkv_ring_debug), _c.c_void_p]
_lib.attn_fwd_window.restype = _c.c_int
_lib.attn_fwd_window.argtypes = [_c.POINTER(rkv_attn_seq), _c.POINTER(rkv_attn_window), _c.c_int32, _c.c_int32,
                                 _c.c_int32, _c.c_int32, _c.c_float, _c.POINTER(rkv_rope3d), _c.c_void_p, _c.c_size_t,
                                 _c.c_void_p]
_lib.rkv_attn_window_rows.restype = _c.c_int
_lib.rkv_attn_window_rows.argtypes = [_c.POINTER(rkv_attn_seq), _c.POINTER(rkv_attn_window), _c.c_int32, _c.c_int32,
                                      _c.c_int32, _c.POINTER(rkv_rope3d), _c.POINTER(_c.c_int64), _c.POINTER(_c.c_int64),
                                      _c.POINTER(_c.c_int64), _c.POINTER(_c.c_int32), _c.POINTER(_c.c_int64)]
_lib.kvcache_paged_insert.restype = _c.c_int
_lib.kvcache_paged_insert.argtypes = [_c.POINTER(rkv_paged_cache), _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int32,
                                      _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p]
_lib.attn_decode_paged_workspace_size.restype = _c.c_size_t
_lib.attn_decode_paged_workspace_size.argtypes = [_c.POINTER(rkv_paged_cache), _c.c_int32, _c.c_int32, _c.c_int32]
_lib.attn_decode_paged.restype = _c.c_int
_lib.attn_decode_paged.argtypes = [_c.POINTER(rkv_paged_cache), _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64,
                                   _c.c_int32, _c.c_int32, _c.c_void_p, _c.c_float, _c.c_int32, _c.c_int32,
                                   _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]
_lib.kvcache_paged_evict_workspace_size.restype = _c.c_size_t
_lib.kvcache_paged_evict_workspace_size.argtypes = [_c.POINTER(rkv_paged_cache), _c.c_int32]
_lib.kvcache_paged_evict.restype = _c.c_int
_lib.kvcache_paged_evict.argtypes = [_c.POINTER(rkv_paged_cache), _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                     _c.c_int32, _c.c_int32, _c.c_int32, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                     _c.c_void_p, _c.c_size_t, _c.c_void_p]
_lib.rkv_paged_status.restype = _c.c_int
_lib.rkv_paged_status.argtypes = [_c.POINTER(rkv_paged_cache), _c.c_void_p]
_lib.rkv_ring_status.restype = _c.c_int
_lib.rkv_ring_status.argtypes = [_c.c_void_p]
_lib.rkv_ring_slot.restype = _c.c_int32
_lib.rkv_ring_slot.argtypes = [_c.POINTER(rkv_ring), _c.c_int32]
_lib.rkv_last_error_string.restype = _c.c_char_p
_lib.rkv_last_error_string.argtypes = []
_lib.rkv_version.restype = _c.c_int32
_lib.rkv_version.argtypes = []


def lib():
    """The raw ctypes library (tests use it to drive the C ABI directly)."""
    return _lib


class RkvError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def rkv_last_error_string():
    return _lib.rkv_last_error_string().decode()


def rkv_version():
    return int(_lib.rkv_version())


def _check(status):
    if status != RKV_OK:
        raise RkvError(status, rkv_last_error_string())


def make_rope(grid_h, grid_w, pairs=(22, 21, 21), theta=10000.0, layout="adjacent"):
    """RoPE parameters.  ``theta``: one frequency base or a (t, h, w) triple;
    ``layout``: "adjacent" (pairs 2j, 2j+1) or "half" (pairs j, j + D/2)."""
    th = tuple(float(v) for v in theta) if isinstance(theta, (tuple, list)) else (float(theta),) * 3
    if layout not in ("adjacent", "half"):
        raise ValueError("layout must be 'adjacent' or 'half'")
    return rkv_rope3d(int(grid_h), int(grid_w), int(pairs[0]), int(pairs[1]), int(pairs[2]), th[0], th[1], th[2],
                      RKV_ROPE_HALF if layout == "half" else RKV_ROPE_ADJACENT)


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _rows(t, name):
    """Check a [L, H, D] bf16 CUDA view with contiguous rows; return its row stride."""
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 3:
        raise ValueError(f"{name} must be a bf16 CUDA tensor of shape [L, H, D]")
    return _stride_of_rows(t, t.shape, name)


def _stride_of_rows(t, shape, name):
    """Row stride of t, [L, H, D] with contiguous rows.  Over a dimension of one
    a stride says nothing: a single row's is H*D."""
    s = t.stride()
    if s[2] != 1 or (s[1] != shape[2] and shape[1] != 1):
        raise ValueError(f"{name}: each row must hold H*D contiguous values")
    return s[0] if shape[0] > 1 else shape[1] * shape[2]


def rope3d_apply(x, y=None, t0=0, rope=None, stream=None):
    """y = RoPE3D(x); x, y bf16 [L, H, 128] CUDA tensors (y=None -> new tensor,
    y=x -> in place).  Returns y."""
    import torch
    if y is None:
        y = torch.empty_like(x)
    xs, ys = _rows(x, "x"), _rows(y, "y")
    if tuple(x.shape) != tuple(y.shape):
        raise ValueError("x and y shapes differ")
    L, H, D = x.shape
    _check(_lib.rope3d_apply(x.data_ptr(), y.data_ptr(), L, H, D, xs, ys, int(t0), ctypes.byref(rope),
                             _stream(stream)))
    return y


def rope3d_apply_batch(items, rope=None, stream=None):
    """rope3d_apply on several tensors in one launch.  items: sequence of
    (x, y, t0) with x, y bf16 [L, H, 128] CUDA tensors of the same H (y=None ->
    new tensor, y=x -> in place).  Returns the list of y."""
    import torch
    outs = []
    arr = (rkv_rope_tensor * max(1, len(items)))()
    H = None
    for i, (x, y, t0) in enumerate(items):
        if y is None:
            y = torch.empty_like(x)
        xs, ys = _rows(x, "x"), _rows(y, "y")
        if tuple(x.shape) != tuple(y.shape):
            raise ValueError("x and y shapes differ")
        if H is None:
            H = x.shape[1]
        elif x.shape[1] != H:
            raise ValueError("all tensors of a batch must have the same number of heads")
        arr[i] = rkv_rope_tensor(x.data_ptr(), y.data_ptr(), x.shape[0], xs, ys, int(t0))
        outs.append(y)
    _check(_lib.rope3d_apply_batch(arr, len(items), H or 1, 128, ctypes.byref(rope), _stream(stream)))
    return outs


class AttnSeq:
    """One sequence of a batched attention launch (see rkv_attn_seq)."""

    def __init__(self, q, k, v, o, q_t0=0, k_t0=0, rope_q=True, rope_k=True, block_frames=0, q_frame_offset=0):
        self.q, self.k, self.v, self.o = q, k, v, o
        self.q_t0, self.k_t0 = int(q_t0), int(k_t0)
        self.flags = (RKV_ROPE_Q if rope_q else 0) | (RKV_ROPE_K if rope_k else 0)
        self.block_frames = int(block_frames)
        self.q_frame_offset = int(q_frame_offset)

    def to_c(self):
        qs, ks, vs, os_ = _rows(self.q, "q"), _rows(self.k, "k"), _rows(self.v, "v"), _rows(self.o, "o")
        if self.k.shape[0] != self.v.shape[0] or self.q.shape[0] != self.o.shape[0]:
            raise ValueError("k/v or q/o row counts differ")
        return rkv_attn_seq(self.q.data_ptr(), self.k.data_ptr(), self.v.data_ptr(), self.o.data_ptr(),
                            qs, ks, vs, os_, self.q.shape[0], self.k.shape[0], self.q_t0, self.k_t0,
                            self.q_frame_offset, self.block_frames, self.flags, 0)


def attn_fwd_varlen_workspace_size(n_seqs=1, H=12, D=128):
    return int(_lib.attn_fwd_varlen_workspace_size(None, n_seqs, H, D))


def attn_fwd_varlen(seqs, rope, softmax_scale=None, workspace=None, stream=None):
    """Run every AttnSeq in ONE kernel launch; outputs are written to each seq.o.
    ``workspace`` is a uint8 CUDA tensor of attn_fwd_varlen_workspace_size()
    bytes (allocated here when None)."""
    import torch
    if not seqs:
        raise ValueError("need at least one sequence")
    H, D = seqs[0].q.shape[1], seqs[0].q.shape[2]
    arr = (rkv_attn_seq * len(seqs))(*[s.to_c() for s in seqs])
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    size = attn_fwd_varlen_workspace_size(len(seqs), H, D)
    if workspace is None:
        workspace = torch.empty(size, dtype=torch.uint8, device=seqs[0].q.device)
    _check(_lib.attn_fwd_varlen(arr, len(seqs), H, D, float(softmax_scale), ctypes.byref(rope),
                                workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return workspace


def rkv_attn_status(workspace, stream=None):
    """Synchronise and raise RkvError if the last launch on ``workspace`` timed out."""
    _check(_lib.rkv_attn_status(workspace.data_ptr(), _stream(stream)))


def attn_fwd_varlen_debug(seqs, rope, row_stats=None, stall=RKV_DEBUG_STALL_NONE, timeout_us=0, softmax_scale=None,
                          workspace=None, stream=None):
    """attn_fwd_varlen with test and debug aids (see rkv.h): ``row_stats`` an
    int32 CUDA tensor of sum(Lq) * H * 4 elements that receives the per-row
    mask record; ``stall`` one of RKV_DEBUG_STALL_*; ``timeout_us`` the limit
    of every device-side wait (0 = default).  Returns the workspace."""
    import torch
    if not seqs:
        raise ValueError("need at least one sequence")
    H, D = seqs[0].q.shape[1], seqs[0].q.shape[2]
    arr = (rkv_attn_seq * len(seqs))(*[s.to_c() for s in seqs])
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if workspace is None:
        workspace = torch.empty(attn_fwd_varlen_workspace_size(len(seqs), H, D), dtype=torch.uint8,
                                device=seqs[0].q.device)
    ptr = None
    if row_stats is not None:
        rows = sum(int(s.q.shape[0]) for s in seqs)
        if row_stats.dtype != torch.int32 or not row_stats.is_cuda or not row_stats.is_contiguous() \
                or row_stats.numel() < rows * H * 4:
            raise ValueError(f"row_stats must be a contiguous int32 CUDA tensor of >= {rows * H * 4} elements")
        ptr = row_stats.data_ptr()
    dbg = rkv_attn_debug(ptr, int(stall), int(timeout_us))
    _check(_lib.attn_fwd_varlen_debug(arr, len(seqs), H, D, float(softmax_scale), ctypes.byref(rope),
                                      workspace.data_ptr(), workspace.numel(), ctypes.byref(dbg), _stream(stream)))
    return workspace


def attn_fwd_varlen_noalloc(seqs, rope, softmax_scale=None, stream=None):
    """attn_fwd_varlen without a caller workspace (the library's fixed scratch)."""
    if not seqs:
        raise ValueError("need at least one sequence")
    H, D = seqs[0].q.shape[1], seqs[0].q.shape[2]
    arr = (rkv_attn_seq * len(seqs))(*[s.to_c() for s in seqs])
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    _check(_lib.attn_fwd_varlen_noalloc(arr, len(seqs), H, D, float(softmax_scale), ctypes.byref(rope),
                                        _stream(stream)))


def rkv_attn_noalloc_status(stream=None):
    """Synchronise and raise RkvError if the last no-alloc launch on this GPU timed out."""
    _check(_lib.rkv_attn_noalloc_status(_stream(stream)))


def attn_mask_rows(seqs, H, rope):
    """The mask and key-tile plan attn_fwd_varlen uses for ``seqs``, evaluated
    on the host by the kernel's own code (no GPU needed).  ``seqs``: AttnSeq
    objects or dicts with Lq, Lk and optional q_frame_offset, block_frames.
    Returns (limits, units): limits[i][r] = keys visible to query row r of
    sequence i (a prefix); units = int32 [n_units, 4] rows of (sequence,
    head, 512-row query block, 128-key tiles processed), in launch order."""
    import numpy as np
    descs = []
    for s in seqs:
        if isinstance(s, dict):
            descs.append(rkv_attn_seq(Lq=int(s["Lq"]), Lk=int(s["Lk"]), q_frame_offset=int(s.get("q_frame_offset", 0)),
                                      block_frames=int(s.get("block_frames", 0))))
        else:
            descs.append(rkv_attn_seq(Lq=int(s.q.shape[0]), Lk=int(s.k.shape[0]), q_frame_offset=s.q_frame_offset,
                                      block_frames=s.block_frames))
    if not descs:
        raise ValueError("need at least one sequence")
    arr = (rkv_attn_seq * len(descs))(*descs)
    lq = [d.Lq for d in descs]
    limits = np.zeros(max(1, sum(lq)), dtype=np.int64)
    n_units = sum(int(H) * ((x + 511) // 512) for x in lq)
    units = np.zeros((max(1, n_units), 4), dtype=np.int32)
    got = ctypes.c_int64(0)
    _check(_lib.rkv_attn_mask_rows(arr, len(descs), int(H), ctypes.byref(rope),
                                   limits.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                   units.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), ctypes.byref(got)))
    if got.value != n_units:
        raise RuntimeError(f"unit count {got.value} != {n_units}")
    out, at = [], 0
    for x in lq:
        out.append(limits[at:at + x].copy())
        at += x
    return out, units[:n_units]


def rkv_ring_status(stream=None):
    """Synchronise and raise RkvError if a ring insert on this GPU gave up on
    a bounded device-side wait since the last call."""
    _check(_lib.rkv_ring_status(_stream(stream)))


def _ring_buffer(t, shape, name):
    """Check a caller-supplied ring buffer: the kernels write
    slots * tokens_per_frame * H * D contiguous bf16 values from its start, so
    anything smaller, strided or on the host is refused here (the C side
    cannot see a buffer's size)."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16:
        raise ValueError(f"ring {name} must be a bf16 tensor")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"ring {name} must be a contiguous tensor of shape {tuple(shape)} "
                         f"(got {tuple(t.shape)}, contiguous={t.is_contiguous()})")
    if not t.is_cuda:
        raise ValueError(f"ring {name} must be in CUDA device memory")
    return t


class KVRing:
    """A per-layer ring of frame slots for K and V (device bf16
    [slots][tokens_per_frame][H][D] each) plus its head/count state; the
    first ``pinned`` slots keep the first frames ever inserted."""

    def __init__(self, slots, tokens_per_frame, H, D=128, device="cuda", k=None, v=None, pinned=0):
        import torch
        if not 0 <= pinned < slots:
            raise ValueError(f"pinned ({pinned}) must be in [0, slots={slots})")
        shape = (slots, tokens_per_frame, H, D)
        self.k = torch.empty(shape, dtype=torch.bfloat16, device=device) if k is None else _ring_buffer(k, shape, "k")
        self.v = torch.empty(shape, dtype=torch.bfloat16, device=device) if v is None else _ring_buffer(v, shape, "v")
        self.c = rkv_ring(self.k.data_ptr(), self.v.data_ptr(), slots, tokens_per_frame, H, D, pinned, 0, pinned)

    @property
    def head(self):
        return self.c.head

    @property
    def count(self):
        return self.c.count

    @property
    def slots(self):
        return self.c.slots

    @property
    def pinned(self):
        return self.c.pinned

    def slot(self, j):
        return int(_lib.rkv_ring_slot(ctypes.byref(self.c), int(j)))

    def valid_rows(self):
        """Number of valid key rows when the valid slots are the prefix [0, count)
        (a ring filled from empty, or a full ring)."""
        return self.c.count * self.c.tokens_per_frame


def _ring_insert_args(ring, k_new, v_new, n_frames):
    ks, vs = _rows(k_new, "k_new"), _rows(v_new, "v_new")
    if ks != vs:
        raise ValueError("k_new and v_new must share a row stride")
    F = ring.c.tokens_per_frame
    if n_frames is None:
        n_frames = k_new.shape[0] // F
    if k_new.shape[0] < n_frames * F or v_new.shape[0] < n_frames * F:
        raise ValueError("k_new/v_new hold fewer than n_frames frames")
    return ks, int(n_frames)


def kvcache_ring_update(ring, k_new, v_new, n_frames=None, stream=None):
    """Insert n_frames frames ([n*F, H, D] bf16 CUDA tensors) into ``ring``;
    returns the number of frames evicted."""
    ks, n_frames = _ring_insert_args(ring, k_new, v_new, n_frames)
    ev = ctypes.c_int32(0)
    _check(_lib.kvcache_ring_update(ctypes.byref(ring.c), k_new.data_ptr(), v_new.data_ptr(), ks, n_frames,
                                    ctypes.byref(ev), _stream(stream)))
    return ev.value


def kvcache_ring_update_debug(ring, k_new, v_new, n_frames=None, stall=RKV_DEBUG_STALL_BULK_LOAD, timeout_us=0,
                              stream=None):
    """kvcache_ring_update with stall injection (see rkv.h); returns the
    number of frames evicted."""
    ks, n_frames = _ring_insert_args(ring, k_new, v_new, n_frames)
    ev = ctypes.c_int32(0)
    dbg = rkv_ring_debug(int(stall), int(timeout_us))
    _check(_lib.kvcache_ring_update_debug(ctypes.byref(ring.c), k_new.data_ptr(), v_new.data_ptr(), ks, n_frames,
                                          ctypes.byref(ev), ctypes.byref(dbg), _stream(stream)))
    return ev.value


def kvcache_ring_update_rope(ring, k_new, v_new, t0, rope, n_frames=None, stream=None):
    """Insert n_frames frames like kvcache_ring_update, rotating the raw keys
    k_new by RoPE3D on the way in (frame i at time t0 + i); returns the
    number of frames evicted."""
    ks, n_frames = _ring_insert_args(ring, k_new, v_new, n_frames)
    ev = ctypes.c_int32(0)
    _check(_lib.kvcache_ring_update_rope(ctypes.byref(ring.c), k_new.data_ptr(), v_new.data_ptr(), ks, n_frames,
                                         int(t0), ctypes.byref(rope), ctypes.byref(ev), _stream(stream)))
    return ev.value


def attn_fwd_window(seqs, windows, rope, softmax_scale=None, workspace=None, stream=None):
    """Run every AttnSeq (block_frames >= 1 each) in one launch with a sliding
    window and first blocks that stay visible; ``windows``: one
    (window_blocks, sink_blocks) per sequence, window_blocks = 0 for none.
    k and v may have fewer heads than q (grouped heads).  Returns the
    workspace (attn_fwd_varlen_workspace_size() bytes, allocated here when
    None; rkv_attn_status reads it)."""
    import torch
    if not seqs:
        raise ValueError("need at least one sequence")
    if len(windows) != len(seqs):
        raise ValueError("need one (window_blocks, sink_blocks) per sequence")
    index = seqs[0].q.get_device()
    if any(x.get_device() != index for s in seqs for x in (s.q, s.k, s.v, s.o)):
        raise ValueError("the sequences of one launch must be on one device")
    if index >= 0 and _elsewhere(index, stream):
        with _on(seqs[0].q, stream):
            return attn_fwd_window(seqs, windows, rope, softmax_scale, workspace)
    H, D, H_kv = seqs[0].q.shape[1], seqs[0].q.shape[2], seqs[0].k.shape[1]
    for s in seqs:
        if tuple(s.q.shape[1:]) != (H, D) or tuple(s.o.shape[1:]) != (H, D) or tuple(s.k.shape[1:]) != (H_kv, D) \
                or tuple(s.v.shape[1:]) != (H_kv, D):
            raise ValueError("the sequences of one launch share the numbers of query and key heads")
    arr = (rkv_attn_seq * len(seqs))(*[s.to_c() for s in seqs])
    win = (rkv_attn_window * len(seqs))(*[rkv_attn_window(_i32(w), _i32(k)) for w, k in windows])
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if workspace is None:
        workspace = torch.empty(attn_fwd_varlen_workspace_size(len(seqs), H, D), dtype=torch.uint8,
                                device=seqs[0].q.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the sequences' device")
    _check(_lib.attn_fwd_window(arr, win, len(seqs), H, H_kv, D, float(softmax_scale), ctypes.byref(rope),
                                workspace.data_ptr(), workspace.nbytes, _raw_stream(index)))
    return workspace


def attn_window_rows(seqs, windows, H, rope, H_kv=None):
    """The mask and key-tile plan attn_fwd_window uses, evaluated on the host
    by the kernel's own code (no GPU needed).  ``seqs``: dicts with Lq, Lk,
    block_frames and optional q_frame_offset.  Returns (sink, begin, limit,
    units): lists per sequence of per-row key ranges [0, sink) and [begin,
    limit), and int32 [n_units, 4] rows of (sequence, first head, first query
    row, 128-key tiles processed)."""
    import numpy as np
    arr = (rkv_attn_seq * len(seqs))(*[
        rkv_attn_seq(Lq=int(s["Lq"]), Lk=int(s["Lk"]), q_frame_offset=int(s.get("q_frame_offset", 0)),
                     block_frames=int(s["block_frames"])) for s in seqs])
    win = (rkv_attn_window * len(seqs))(*[rkv_attn_window(_i32(w), _i32(k)) for w, k in windows])
    lq = [int(s["Lq"]) for s in seqs]
    got = [np.zeros(max(1, sum(lq)), dtype=np.int64) for _ in range(3)]
    units = np.zeros((max(1, sum(int(H) * ((x + 511) // 512) for x in lq)), 4), dtype=np.int32)
    n = ctypes.c_int64(0)
    p64 = ctypes.POINTER(ctypes.c_int64)
    _check(_lib.rkv_attn_window_rows(arr, win, len(seqs), int(H), int(H if H_kv is None else H_kv), ctypes.byref(rope),
                                     *[g.ctypes.data_as(p64) for g in got],
                                     units.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), ctypes.byref(n)))
    at = np.cumsum([0] + lq)
    return (*[[g[at[i]:at[i + 1]].copy() for i in range(len(lq))] for g in got], units[:n.value])


class _on:
    """Makes t's device current for a call on a stream that is not its current
    one, and that stream too, so that what the call allocates belongs to the
    stream it runs on."""

    def __init__(self, t, stream):
        import torch
        if stream is not None and stream.device != t.device:
            raise ValueError("the stream and the tensors are on different devices")
        self.guard = torch.cuda.device(t.device) if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        self.guard.__enter__()

    def __exit__(self, *exc):
        return self.guard.__exit__(*exc)


def _elsewhere(index, stream):
    """Whether a call on tensors of device ``index`` has to be made under _on."""
    import torch
    return stream is not None or torch._C._cuda_getDevice() != index


def _i32(x):
    """A count as int32 takes it: one past its range means as much as the
    largest (ctypes would keep the low 32 bits)."""
    return max(-1, min(int(x), 0x7FFFFFFF))


def _raw_stream(index):
    """Handle of the current stream of device ``index``."""
    import torch
    return torch._C._cuda_getCurrentRawStream(index)


def _row_stride(t, name, shape, index):
    """Row stride of a bf16 tensor [L, H, D] of the given shape on device
    ``index`` whose rows are contiguous."""
    import torch
    if t.dtype is not torch.bfloat16 or t.get_device() != index or t.shape != shape:
        raise ValueError(f"{name} must be a bf16 CUDA tensor of shape {tuple(shape)} on the cache's device")
    return _stride_of_rows(t, shape, name)


def _check_table(t, device):
    """Row stride of a page table, int32 [n_seqs, max_pages] on ``device``."""
    import torch
    if t.dtype != torch.int32 or t.dim() != 2 or t.device != device or 0 in t.shape \
            or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("page_table must be int32 [n_seqs, max_pages] (at least one of each) with contiguous rows, on "
                         "the device of k")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


class PagedKVCache:
    """A paged cache of several token streams over caller tensors (see
    rkv_paged_cache): ``k``, ``v`` bf16 CUDA [n_pages, page_tokens, H, 128]
    (each page contiguous; the buffers of a KVRing are one), ``page_table``
    int32 CUDA [n_seqs, max_pages].  ``status`` is the word device-side checks
    record in (rkv_paged_status)."""

    def __init__(self, k, v, page_table):
        import torch
        if k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16 or k.dim() != 4 or not k.is_cuda or not v.is_cuda:
            raise ValueError("k and v must be bf16 CUDA tensors of shape [n_pages, page_tokens, H, D]")
        n_pages, P, H, D = k.shape
        # (over a dimension of one a stride says nothing)
        of = lambda t: [x for n, x in zip(t.shape, t.stride()) if n > 1]  # noqa: E731
        if v.shape != k.shape or of(v) != of(k) or v.device != k.device:
            raise ValueError("k and v must share shape, strides and device")
        if any(n > 1 and x != w for n, x, w in zip(k.shape[1:], k.stride()[1:], (H * D, D, 1))):
            raise ValueError("a page must be contiguous")
        table_stride = _check_table(page_table, k.device)
        self.k, self.v, self.page_table = k, v, page_table
        self.status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self.n_seqs, self.max_pages = page_table.shape
        self.H, self.capacity, self.index = H, self.max_pages * P, k.get_device()
        self._per_seq = torch.Size((self.n_seqs,))
        self._per_token = torch.Size((self.n_seqs, H, self.capacity))
        stride = k.stride(0) if n_pages > 1 else P * H * D
        self.c = rkv_paged_cache(k.data_ptr(), v.data_ptr(), stride, n_pages, P, H, D, page_table.data_ptr(),
                                 table_stride, self.n_seqs, self.max_pages, self.status.data_ptr())
        self.ref = ctypes.byref(self.c)
        # calls on other streams wait for the zeros of the status word (a capture
        # runs when it is replayed; what is made in one belongs to it)
        self._made_on, self._zeroed = _raw_stream(self.index), None
        with torch.cuda.device(k.device):
            if not torch.cuda.is_current_stream_capturing():
                self._zeroed = torch.cuda.Event()
                self._zeroed.record()

    def _stream(self):
        """Handle of the current stream, on which the status word is zeroed."""
        handle = _raw_stream(self.index)
        if handle != self._made_on and self._zeroed is not None:
            self._after_zeros()
        return handle

    def _after_zeros(self):
        import torch
        if torch.cuda.is_current_stream_capturing():
            return
        if self._zeroed.query():
            self._zeroed = None
        else:
            torch.cuda.current_stream(self.k.device).wait_event(self._zeroed)

    def _ints(self, t, name):
        """Device pointer of an int32 [n_seqs] tensor."""
        import torch
        if t.dtype is not torch.int32 or t.shape != self._per_seq or t.get_device() != self.index \
                or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 [n_seqs={self.n_seqs}] tensor on the cache's device")
        return t.data_ptr()

    def _scores(self, t, name, dtype):
        """Device pointer of a [n_seqs, H, capacity] tensor, or NULL for None."""
        if t is None:
            return None
        if t.dtype is not dtype or t.shape != self._per_token or t.get_device() != self.index \
                or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(self._per_token)} on the "
                             "cache's device")
        return t.data_ptr()

    def _workspace(self, t, size):
        """A workspace tensor, allocated here when None, and its bytes."""
        import torch
        if t is None:
            t = torch.empty(max(16, size), dtype=torch.uint8, device=self.k.device)
        elif t.get_device() != self.index or not t.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the cache's device")
        return t, t.nbytes


def kvcache_paged_insert(cache, k_new, v_new, seq_lens, next_pos=None, pos=None, weight=None, stream=None):
    """Write the newest tokens of every sequence, k_new and v_new bf16
    [n_seqs * n_new, H, 128] sequence by sequence; ``seq_lens`` (int32 CUDA
    [n_seqs]) counts them already.  ``pos`` (with ``next_pos``) and ``weight``:
    the scores of the new tokens (see rkv.h)."""
    import torch
    if _elsewhere(cache.index, stream):
        with _on(cache.k, stream):
            return kvcache_paged_insert(cache, k_new, v_new, seq_lens, next_pos, pos, weight)
    shape = k_new.shape
    if len(shape) != 3 or shape[1] != cache.H or shape[2] != 128 or shape[0] % cache.n_seqs:
        raise ValueError(f"k_new and v_new must be [n_seqs * n_new, {cache.H}, 128] with n_seqs = {cache.n_seqs}")
    ks = _row_stride(k_new, "k_new", shape, cache.index)
    if ks != _row_stride(v_new, "v_new", shape, cache.index):
        raise ValueError("k_new and v_new must share a row stride")
    _check(_lib.kvcache_paged_insert(cache.ref, k_new.data_ptr(), v_new.data_ptr(), ks, shape[0] // cache.n_seqs,
                                     cache._ints(seq_lens, "seq_lens"),
                                     None if next_pos is None else cache._ints(next_pos, "next_pos"),
                                     cache._scores(pos, "pos", torch.int32),
                                     cache._scores(weight, "weight", torch.float32), cache._stream()))


def attn_decode_paged_workspace_size(cache, Hq, Lq=1, weights=False):
    return int(_lib.attn_decode_paged_workspace_size(cache.ref, int(Hq), int(Lq), 1 if weights else 0))


def attn_decode_paged(q, cache, seq_lens, o=None, window=0, sinks=0, softmax_scale=None, weight_in=None,
                      weight_out=None, workspace=None, stream=None):
    """Attention of the newest Lq tokens of every sequence over its pages: q
    bf16 [n_seqs * Lq, Hq, 128], sequence by sequence; ``seq_lens`` counts
    them.  ``window`` / ``sinks``: a token sees the last ``window`` tokens and
    the first ``sinks`` (0 = all), by index in the cache (not for an evicted
    one, whose order is no longer the stream's).  ``weight_out`` = ``weight_in`` + the
    attention weight each cached token received (may be the same tensor).
    Returns o (allocated here when None)."""
    import torch
    if _elsewhere(cache.index, stream):
        with _on(cache.k, stream):
            return attn_decode_paged(q, cache, seq_lens, o, window, sinks, softmax_scale, weight_in, weight_out,
                                     workspace)
    shape = q.shape
    if len(shape) != 3 or shape[2] != 128 or shape[0] % cache.n_seqs:
        raise ValueError(f"q must be [n_seqs * Lq, Hq, 128] with n_seqs = {cache.n_seqs}")
    qs = _row_stride(q, "q", shape, cache.index)
    if o is None:
        o = torch.empty(shape, dtype=q.dtype, device=q.device)
    os_ = _row_stride(o, "o", shape, cache.index)
    Lq, Hq = shape[0] // cache.n_seqs, shape[1]
    size = 0 if workspace is not None else attn_decode_paged_workspace_size(cache, Hq, Lq, weight_out is not None)
    workspace, size = cache._workspace(workspace, size)
    _check(_lib.attn_decode_paged(cache.ref, q.data_ptr(), o.data_ptr(), qs, os_, Hq, Lq,
                                  cache._ints(seq_lens, "seq_lens"),
                                  _SCALE if softmax_scale is None else softmax_scale, _i32(window), _i32(sinks),
                                  cache._scores(weight_in, "weight_in", torch.float32),
                                  cache._scores(weight_out, "weight_out", torch.float32), workspace.data_ptr(), size,
                                  cache._stream()))
    return o


_SCALE = 1.0 / math.sqrt(128)


def kvcache_paged_evict_workspace_size(cache, budget):
    return int(_lib.kvcache_paged_evict_workspace_size(cache.ref, _i32(budget)))


def kvcache_paged_evict(cache, seq_lens, weight, pos, next_pos, budget, sinks=0, recent=0, seq_lens_out=None,
                        weight_out=None, pos_out=None, workspace=None, stream=None):
    """Cut every sequence to ``budget`` tokens per key head, dropping those of
    the least accumulated weight (see rkv.h); what is left is in no particular
    order, so it is attended without a window.  The outputs default to their
    inputs (in place)."""
    import torch
    if _elsewhere(cache.index, stream):
        with _on(cache.k, stream):
            return kvcache_paged_evict(cache, seq_lens, weight, pos, next_pos, budget, sinks, recent, seq_lens_out,
                                       weight_out, pos_out, workspace)
    if (weight_out is None) != (pos_out is None):
        raise ValueError("weight_out and pos_out go together")
    lens_in, w_in = cache._ints(seq_lens, "seq_lens"), cache._scores(weight, "weight", torch.float32)
    p_in = cache._scores(pos, "pos", torch.int32)
    size = 0 if workspace is not None else kvcache_paged_evict_workspace_size(cache, budget)
    workspace, size = cache._workspace(workspace, size)
    _check(_lib.kvcache_paged_evict(
        cache.ref, lens_in, w_in, p_in, cache._ints(next_pos, "next_pos"), _i32(budget), _i32(sinks), _i32(recent),
        lens_in if seq_lens_out is None else cache._ints(seq_lens_out, "seq_lens_out"),
        w_in if weight_out is None else cache._scores(weight_out, "weight_out", torch.float32),
        p_in if pos_out is None else cache._scores(pos_out, "pos_out", torch.int32), workspace.data_ptr(), size,
        cache._stream()))


def rkv_paged_status(cache, stream=None):
    """Synchronise and raise RkvError if a call on ``cache`` met a length or a
    page out of range since the last report."""
    if _elsewhere(cache.index, stream):
        with _on(cache.k, stream):
            return rkv_paged_status(cache)
    _check(_lib.rkv_paged_status(cache.ref, cache._stream()))
