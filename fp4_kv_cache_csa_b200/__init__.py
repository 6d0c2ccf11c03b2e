"""Python binding of libcsa: CSA / HCA / window attention over an MXFP4 KV cache on B200.

Argument marshalling only. Every step of the method runs in the CUDA kernels of
libcsa.so (built in-tree by ``python -m fp4_kv_cache_csa_b200.build``); PyTorch
is used for device memory and streams. Importing this module does not load the
library; the first call does, and raises ``CsaError`` if it is missing -- there
is no CPU fallback.

The function names mirror the C ABI in include/csa.h:
    csa_compress_quantize, csa_index_topk, csa_decode_attend, hca_decode_attend,
    csa_read_device_status (+ the workspace-size queries),
    hca_shared_attend, csa_cache_copy, csa_rotary, csa_rotary_frequencies.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa.so")

CSA_IDX_BF16 = 0
CSA_IDX_E4M3 = 1
CSA_IDX_MXFP4 = 2

CSA_SCALE_E8M0_32 = 0  # one E8M0 scale byte per 32 elements (OCP MXFP4)
CSA_SCALE_E4M3_16 = 1  # one E4M3 scale byte per 16 elements

CSA_BF16 = 0
CSA_F32 = 1
CSA_ROPE_PAIRS = 0  # channels 2p, 2p + 1 turn together
CSA_ROPE_HALF = 1   # channels p, p + rot_dim / 2 turn together
CSA_ROPE_SCALE_NONE = 0
CSA_ROPE_SCALE_LINEAR = 1
CSA_ROPE_SCALE_BASE = 2
CSA_ROPE_SCALE_PARTS = 3

CSA_DEV_TOKEN_COUNT = 0x1
CSA_DEV_CAPACITY = 0x2
CSA_DEV_BAD_INDEX = 0x4
CSA_DEV_BAD_WINDOW = 0x8
CSA_DEV_TIMEOUT = 0x10

EXPORTED = (
    "csa_status_string", "csa_version", "csa_compress_quantize", "csa_index_topk_workspace", "csa_index_topk",
    "csa_attend_workspace", "csa_decode_attend", "hca_decode_attend", "csa_read_device_status",
    "csa_index_topk_noalloc", "csa_index_pool_workspace", "csa_index_topk_pool", "csa_index_reindex_workspace",
    "csa_index_topk_reindex", "csa_index_reindex_layers_workspace", "csa_index_topk_reindex_layers",
    "csa_probe_mxf4_mma", "csa_rotary", "csa_rotary_frequencies",
    "csa_cache_copy_workspace", "csa_cache_copy", "hca_shared_attend_workspace", "hca_shared_attend",
)


class CsaError(RuntimeError):
    pass


class _CCache(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("dim", ctypes.c_int32), ("block", ctypes.c_int32), ("capacity", ctypes.c_int32),
        ("fp4", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("idx_key", ctypes.c_void_p),
        ("idx_dim", ctypes.c_int32), ("idx_dtype", ctypes.c_int32),
        ("n_blocks", ctypes.c_void_p), ("status", ctypes.c_void_p), ("scale_fmt", ctypes.c_int32),
        ("idx_key_scale", ctypes.c_void_p),
    ]


class _CVectors(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _CRope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_begin", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("mscale", ctypes.c_float)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libcsa.so and declare the C signatures. Raises CsaError if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise CsaError(f"libcsa.so not found at {path}: build it with `python -m fp4_kv_cache_csa_b200.build`")
    _lib = declare(ctypes.CDLL(path))
    return _lib


def declare(lib):
    """Declare the C signatures of a loaded libcsa (the library itself or a test variant of it)."""
    P, I, S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    CP = ctypes.POINTER(_CCache)
    lib.csa_status_string.argtypes = [I]
    lib.csa_status_string.restype = ctypes.c_char_p
    lib.csa_version.argtypes = []
    lib.csa_version.restype = I
    lib.csa_compress_quantize.argtypes = [CP, P, P, P, P, I, P]
    lib.csa_compress_quantize.restype = I
    lib.csa_index_topk_workspace.argtypes = [CP, I, I]
    lib.csa_index_topk_workspace.restype = S
    lib.csa_index_topk.argtypes = [CP, P, P, I, I, P, P, I, P, P, S, P]
    lib.csa_index_topk.restype = I
    lib.csa_index_topk_noalloc.argtypes = [CP, P, P, I, I, P, P, I, P, P]
    lib.csa_index_topk_noalloc.restype = I
    lib.csa_index_pool_workspace.argtypes = [CP, I, I, I, I]
    lib.csa_index_pool_workspace.restype = S
    lib.csa_index_topk_pool.argtypes = [CP, P, P, I, I, P, P, I, P, I, I, P, P, S, P]
    lib.csa_index_topk_pool.restype = I
    lib.csa_index_reindex_workspace.argtypes = [CP, I, I, I]
    lib.csa_index_reindex_workspace.restype = S
    lib.csa_index_topk_reindex.argtypes = [CP, P, P, I, I, P, P, I, P, I, I, P, P, S, P]
    lib.csa_index_topk_reindex.restype = I
    lib.csa_index_reindex_layers_workspace.argtypes = [CP, I, I, I, I]
    lib.csa_index_reindex_layers_workspace.restype = S
    lib.csa_index_topk_reindex_layers.argtypes = [CP, P, P, I, I, I, P, P, I, P, I, I, P, P, S, P]
    lib.csa_index_topk_reindex_layers.restype = I
    lib.csa_attend_workspace.argtypes = [CP, I, I]
    lib.csa_attend_workspace.restype = S
    lib.csa_decode_attend.argtypes = [CP, P, I, I, P, P, I, P, P, P, I, ctypes.c_float, P, P, P, S, P]
    lib.csa_decode_attend.restype = I
    lib.hca_decode_attend.argtypes = [CP, P, I, I, P, P, P, P, P, I, ctypes.c_float, P, P, P, S, P]
    lib.hca_decode_attend.restype = I
    lib.csa_read_device_status.argtypes = [CP, P, ctypes.POINTER(I)]
    lib.csa_read_device_status.restype = I
    lib.csa_probe_mxf4_mma.argtypes = [I, P, P, ctypes.POINTER(ctypes.c_int64)]
    lib.csa_probe_mxf4_mma.restype = I
    lib.hca_shared_attend_workspace.argtypes = [CP, I, I]
    lib.hca_shared_attend_workspace.restype = S
    lib.hca_shared_attend.argtypes = [CP, P, I, I, P, P, P, P, ctypes.c_float, P, P, P, S, P]
    lib.hca_shared_attend.restype = I
    lib.csa_cache_copy_workspace.argtypes = [CP, I, I]
    lib.csa_cache_copy_workspace.restype = S
    lib.csa_cache_copy.argtypes = [CP, CP, I, P, P, P, I, P, P, S, P]
    lib.csa_cache_copy.restype = I
    VP, D = ctypes.POINTER(_CVectors), ctypes.c_double
    lib.csa_rotary.argtypes = [VP, VP, I, I, I, ctypes.POINTER(_CRope), P, I, P]
    lib.csa_rotary.restype = I
    lib.csa_rotary_frequencies.argtypes = [I, D, I, D, I, D, D, P, P]
    lib.csa_rotary_frequencies.restype = I
    return lib


def _check(status: int, what: str):
    if status != 0:
        msg = load_library().csa_status_string(status).decode()
        raise CsaError(f"{what}: {msg} (status {status})")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _on(device, stream, call):
    """call(raw stream) with the tensors' device current, on `stream` or that device's current one. What
    the call allocates then belongs to that stream."""
    import torch

    if device.type != "cuda":
        raise CsaError(f"tensors must be on a CUDA device, not {device}")
    if stream is not None and stream.device != device:
        raise CsaError(f"stream is of {stream.device}, tensors are on {device}")
    if stream is None and device.index == torch.cuda.current_device():
        return call(_raw_stream(device.index))
    with torch.cuda.device(device) if stream is None else torch.cuda.stream(stream):
        return call(torch.cuda.current_stream().cuda_stream)


def _raw_stream(index):
    """The handle of a device's current stream (without a stream object where PyTorch offers that: 3 us less)."""
    import torch

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _expect(what, name, t, at, dtype, shape):
    """One tensor of a call: on device number `at` (-1: the host), of `dtype`, dense, of this shape."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != at or not t.is_contiguous():
        raise CsaError(f"{what}: {name} must be a dense {dtype} tensor {list(shape)} on {f'cuda:{at}' if at >= 0 else 'cpu'}, "
                       f"not {t.dtype} {list(t.shape)}{'' if t.is_contiguous() else ' (strided)'} on {t.device}")


def _expect_cache(what, c, at, int32):
    """A cache of a call whose tensors are on device number `at`: dense planes whose sizes belong together, and int32
    counts beside them (with others a kernel would read and write elsewhere)."""
    n, fp4, scale, key = c.n_blocks, c.fp4, c.scale, c.idx_key
    if (fp4.get_device() != at or n.get_device() != at or n.dtype is not int32 or n.numel() < fp4.shape[0]
            or not n.is_contiguous()
            or scale.numel() * (16 if c.scale_fmt == CSA_SCALE_E8M0_32 else 8) != fp4.numel()  # (codes: two a byte)
            or not fp4.is_contiguous() or not scale.is_contiguous() or (key is not None and not key.is_contiguous())):
        raise CsaError(f"{what}: a cache's planes must be dense tensors [batch, capacity, row] on the call's device, with "
                       "rows of its scale format, and n_blocks int32 [batch]")


def _expect_workspace(what, ws, device):
    """A caller's workspace: dense, and on `device` (the library checks its size)."""
    if ws is not None and (ws.device != device or not ws.is_contiguous()):
        raise CsaError(f"{what}: workspace must be a dense tensor on {device}, not on {ws.device}")


@dataclass
class Cache:
    """One compressed cache (one layer): device tensors owned by the caller (see include/csa.h).

    fp4 [B, cap, D/2] uint8, scale [B, cap, D/32] uint8 (E8M0) or [B, cap, D/16] uint8 (E4M3),
    idx_key [B, cap, dI] bf16 / uint8 (e4m3) or [B, cap, dI/2] uint8 (MXFP4 codes, with
    idx_key_scale [B, cap, dI/32] uint8) or None, n_blocks [B] int32, status [1] int32 or None.
    """
    fp4: object
    scale: object
    n_blocks: object
    block: int
    idx_key: object = None
    idx_dtype: int = CSA_IDX_BF16
    status: object = None
    scale_fmt: int = CSA_SCALE_E8M0_32
    idx_key_scale: object = None

    @property
    def batch(self) -> int:
        return self.fp4.shape[0]

    @property
    def capacity(self) -> int:
        return self.fp4.shape[1]

    @property
    def dim(self) -> int:
        return self.fp4.shape[2] * 2

    @property
    def idx_dim(self) -> int:
        if self.idx_key is None:
            return 0
        return self.idx_key.shape[2] * (2 if self.idx_dtype == CSA_IDX_MXFP4 else 1)

    def c_struct(self) -> _CCache:
        batch, capacity, half = self.fp4.shape
        key, key_scale, status = self.idx_key, self.idx_key_scale, self.status
        return _CCache(batch, 2 * half, self.block, capacity, self.fp4.data_ptr(), _ptr(self.scale),
                       None if key is None else key.data_ptr(), 0 if key is None else self.idx_dim, self.idx_dtype,
                       _ptr(self.n_blocks), None if status is None else status.data_ptr(), self.scale_fmt,
                       None if key_scale is None else key_scale.data_ptr())

    @staticmethod
    def allocate(batch: int, capacity: int, dim: int, block: int, idx_dim: int = 0, idx_dtype: int = CSA_IDX_BF16,
                 device="cuda", scale_fmt: int = CSA_SCALE_E8M0_32):
        """Zero-filled cache tensors on `device` (torch allocation; the library allocates nothing)."""
        import torch

        idx = idx_scale = None
        if idx_dim and idx_dtype == CSA_IDX_MXFP4:
            idx = torch.zeros(batch, capacity, idx_dim // 2, dtype=torch.uint8, device=device)
            idx_scale = torch.zeros(batch, capacity, idx_dim // 32, dtype=torch.uint8, device=device)
        elif idx_dim:
            dt = torch.bfloat16 if idx_dtype == CSA_IDX_BF16 else torch.uint8
            idx = torch.zeros(batch, capacity, idx_dim, dtype=dt, device=device)
        return Cache(fp4=torch.zeros(batch, capacity, dim // 2, dtype=torch.uint8, device=device),
                     scale=torch.zeros(batch, capacity, dim // (32 if scale_fmt == CSA_SCALE_E8M0_32 else 16),
                                       dtype=torch.uint8, device=device),
                     n_blocks=torch.zeros(batch, dtype=torch.int32, device=device), block=block,
                     idx_key=idx, idx_dtype=idx_dtype, status=torch.zeros(1, dtype=torch.int32, device=device),
                     scale_fmt=scale_fmt, idx_key_scale=idx_scale)


def csa_version() -> int:
    return load_library().csa_version()


def csa_compress_quantize(cache: Cache, kv_tok, idx_tok, gate_w, tok_offsets, stream=None):
    """Rows a1+a2: pool every m new tokens of each request into one block and store it (FP4 + indexer key)."""
    lib = load_library()
    c = cache.c_struct()
    _check(lib.csa_compress_quantize(ctypes.byref(c), _ptr(kv_tok), _ptr(idx_tok), _ptr(gate_w), _ptr(tok_offsets),
                                     int(kv_tok.shape[0]), _stream(stream)), "csa_compress_quantize")


def csa_index_topk_workspace(cache: Cache, n_queries: int, topk: int) -> int:
    return int(load_library().csa_index_topk_workspace(ctypes.byref(cache.c_struct()), n_queries, topk))


def csa_index_topk_noalloc(cache: Cache, q_idx, w, q_offsets, q_pos, topk: int, sel_idx, stream=None):
    """csa_index_topk with the library's fixed 32 MiB device scratch instead of a workspace, for
    callers that cannot allocate device memory (see include/csa.h). sel_idx must be passed in."""
    lib = load_library()
    c = cache.c_struct()
    _check(lib.csa_index_topk_noalloc(ctypes.byref(c), _ptr(q_idx), _ptr(w), int(q_idx.shape[0]),
                                      int(q_idx.shape[1]), _ptr(q_offsets), _ptr(q_pos), topk, _ptr(sel_idx),
                                      _stream(stream)), "csa_index_topk_noalloc")
    return sel_idx


def csa_attend_workspace(cache: Cache, n_queries: int, heads: int) -> int:
    return int(load_library().csa_attend_workspace(ctypes.byref(cache.c_struct()), n_queries, heads))


def _workspace(nbytes: int, workspace, device):
    import torch

    if workspace is not None:
        return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def csa_index_topk(cache: Cache, q_idx, w, q_offsets, q_pos, topk: int, sel_idx=None, workspace=None, stream=None):
    """Rows a3+a4: indexer scores of every visible block and the top-k blocks per query (ascending, -1 padded)."""
    import torch

    lib = load_library()
    n_queries, idx_heads = int(q_idx.shape[0]), int(q_idx.shape[1])
    if sel_idx is None:
        sel_idx = torch.empty(n_queries, topk, dtype=torch.int32, device=q_idx.device)
    need = csa_index_topk_workspace(cache, n_queries, topk)
    workspace = _workspace(need, workspace, q_idx.device)
    c = cache.c_struct()
    _check(lib.csa_index_topk(ctypes.byref(c), _ptr(q_idx), _ptr(w), n_queries, idx_heads, _ptr(q_offsets),
                              _ptr(q_pos), topk, _ptr(sel_idx), _ptr(workspace), workspace.numel(), _stream(stream)),
           "csa_index_topk")
    return sel_idx


def csa_index_pool_workspace(cache: Cache, n_queries: int, topk: int, pool_group: int = 8,
                             pool_blocks: int = 2000) -> int:
    return int(load_library().csa_index_pool_workspace(ctypes.byref(cache.c_struct()), n_queries, topk, pool_group,
                                                       pool_blocks))


def csa_index_reindex_workspace(cache: Cache, n_queries: int, pool_group: int = 8, pool_blocks: int = 2000) -> int:
    return int(load_library().csa_index_reindex_workspace(ctypes.byref(cache.c_struct()), n_queries, pool_group,
                                                          pool_blocks))


def csa_index_topk_pool(cache: Cache, q_idx, w, q_offsets, q_pos, topk: int, pool_group: int = 8,
                        pool_blocks: int = 2000, sel_idx=None, pool_blk=None, workspace=None, stream=None):
    """A Full-mode layer's indexer: its top-k (as csa_index_topk) and the candidate pool of the
    hierarchical indexer (the pool_blocks best groups of pool_group blocks by their best score)."""
    import torch

    lib = load_library()
    n_queries, idx_heads = int(q_idx.shape[0]), int(q_idx.shape[1])
    if sel_idx is None:
        sel_idx = torch.empty(n_queries, topk, dtype=torch.int32, device=q_idx.device)
    if pool_blk is None:
        pool_blk = torch.empty(n_queries, pool_blocks, dtype=torch.int32, device=q_idx.device)
    need = csa_index_pool_workspace(cache, n_queries, topk, pool_group, pool_blocks)
    workspace = _workspace(need, workspace, q_idx.device)
    c = cache.c_struct()
    _check(lib.csa_index_topk_pool(ctypes.byref(c), _ptr(q_idx), _ptr(w), n_queries, idx_heads, _ptr(q_offsets),
                                   _ptr(q_pos), topk, _ptr(sel_idx), pool_group, pool_blocks, _ptr(pool_blk),
                                   _ptr(workspace), workspace.numel(), _stream(stream)), "csa_index_topk_pool")
    return sel_idx, pool_blk


def csa_index_topk_reindex(cache: Cache, q_idx, w, q_offsets, q_pos, topk: int, pool_blk, pool_group: int = 8,
                           sel_idx=None, workspace=None, stream=None):
    """A Reindex-mode layer's indexer: its own query scored only against the pool's blocks."""
    import torch

    lib = load_library()
    n_queries, idx_heads = int(q_idx.shape[0]), int(q_idx.shape[1])
    pool_blocks = int(pool_blk.shape[1])
    if sel_idx is None:
        sel_idx = torch.empty(n_queries, topk, dtype=torch.int32, device=q_idx.device)
    need = csa_index_reindex_workspace(cache, n_queries, pool_group, pool_blocks)
    workspace = _workspace(need, workspace, q_idx.device)
    c = cache.c_struct()
    _check(lib.csa_index_topk_reindex(ctypes.byref(c), _ptr(q_idx), _ptr(w), n_queries, idx_heads, _ptr(q_offsets),
                                      _ptr(q_pos), topk, _ptr(sel_idx), pool_group, pool_blocks, _ptr(pool_blk),
                                      _ptr(workspace), workspace.numel(), _stream(stream)), "csa_index_topk_reindex")
    return sel_idx


def csa_index_reindex_layers_workspace(cache: Cache, n_queries: int, n_layers: int, pool_group: int,
                                       pool_blocks: int) -> int:
    return int(load_library().csa_index_reindex_layers_workspace(ctypes.byref(cache.c_struct()), n_queries, n_layers,
                                                                 pool_group, pool_blocks))


def csa_index_topk_reindex_layers(cache: Cache, q_idx, w, q_offsets, q_pos, topk: int, pool_blk, pool_group: int = 8,
                                  sel_idx=None, workspace=None, stream=None):
    """Several Reindex-mode layers over one pool in one call. q_idx [Nq, L, H_I, dI] bf16,
    w [Nq, L, H_I] float32; returns sel_idx [Nq, L, topk]."""
    import torch

    lib = load_library()
    n_queries, n_layers, idx_heads = (int(x) for x in q_idx.shape[:3])
    pool_blocks = int(pool_blk.shape[1])
    if sel_idx is None:
        sel_idx = torch.empty(n_queries, n_layers, topk, dtype=torch.int32, device=q_idx.device)
    need = csa_index_reindex_layers_workspace(cache, n_queries, n_layers, pool_group, pool_blocks)
    workspace = _workspace(need, workspace, q_idx.device)
    c = cache.c_struct()
    _check(lib.csa_index_topk_reindex_layers(ctypes.byref(c), _ptr(q_idx), _ptr(w), n_queries, n_layers, idx_heads,
                                             _ptr(q_offsets), _ptr(q_pos), topk, _ptr(sel_idx), pool_group,
                                             pool_blocks, _ptr(pool_blk), _ptr(workspace), workspace.numel(),
                                             _stream(stream)), "csa_index_topk_reindex_layers")
    return sel_idx


def csa_decode_attend(cache: Cache, q, q_offsets, sel_idx, win_kv=None, win_start=None, win_len=None,
                      max_win: int = 128, softmax_scale: Optional[float] = None, out=None, lse=None,
                      workspace=None, stream=None):
    """Rows a5+a6+a8: joint softmax attention over the selected compressed entries and the window."""
    import torch

    lib = load_library()
    n_queries, heads, D = (int(x) for x in q.shape)
    if softmax_scale is None:
        softmax_scale = D ** -0.5
    if out is None:
        out = torch.empty(n_queries, heads, D, dtype=torch.float32, device=q.device)
    need = csa_attend_workspace(cache, n_queries, heads)
    workspace = _workspace(need, workspace, q.device)
    c = cache.c_struct()
    _check(lib.csa_decode_attend(ctypes.byref(c), _ptr(q), n_queries, heads, _ptr(q_offsets), _ptr(sel_idx),
                                 int(sel_idx.shape[1]), _ptr(win_kv), _ptr(win_start), _ptr(win_len), max_win,
                                 float(softmax_scale), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                                 _stream(stream)), "csa_decode_attend")
    return out


def hca_decode_attend(cache: Cache, q, q_offsets, q_pos, win_kv=None, win_start=None, win_len=None,
                      max_win: int = 128, softmax_scale: Optional[float] = None, out=None, lse=None,
                      workspace=None, stream=None):
    """Row a7 (+a8): dense attention over every visible compressed entry and the window."""
    import torch

    lib = load_library()
    n_queries, heads, D = (int(x) for x in q.shape)
    if softmax_scale is None:
        softmax_scale = D ** -0.5
    if out is None:
        out = torch.empty(n_queries, heads, D, dtype=torch.float32, device=q.device)
    need = csa_attend_workspace(cache, n_queries, heads)
    workspace = _workspace(need, workspace, q.device)
    c = cache.c_struct()
    _check(lib.hca_decode_attend(ctypes.byref(c), _ptr(q), n_queries, heads, _ptr(q_offsets), _ptr(q_pos),
                                 _ptr(win_kv), _ptr(win_start), _ptr(win_len), max_win, float(softmax_scale),
                                 _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)),
           "hca_decode_attend")
    return out


def hca_shared_attend_workspace(cache: Cache, n_queries: int, heads: int) -> int:
    return int(load_library().hca_shared_attend_workspace(ctypes.byref(cache.c_struct()), n_queries, heads))


def hca_shared_attend(cache: Cache, q, q_offsets, q_pos=None, join_out=None, join_lse=None,
                      softmax_scale: Optional[float] = None, out=None, lse=None, workspace=None, stream=None):
    """Dense attention of many queries over one slot's blocks (a prompt that continuations share, a prefill
    chunk), each tile dequantized once for 64 // H queries; joined with (join_out, join_lse), the
    float32 result of a query's own part, as one softmax. Without q_pos every query sees all blocks of its
    slot. q [Nq, H, D] bf16; returns out [Nq, H, D] bf16, and fills lse [Nq, H] float32 if given. No gradient
    is recorded."""
    import torch

    lib, what = load_library(), "hca_shared_attend"
    device, f32, i32 = q.device, torch.float32, torch.int32
    if q.dim() != 3:
        raise CsaError(f"{what}: q must be [queries, heads, dim], not {list(q.shape)}")
    n, heads, D = q.shape
    at = q.get_device()
    batch, _, codes = cache.fp4.shape
    _expect(what, "q", q, at, torch.bfloat16, (n, heads, 2 * codes))
    _expect_cache(what, cache, at, i32)
    _expect(what, "q_offsets", q_offsets, at, i32, (batch + 1,))
    if q_pos is not None:
        _expect(what, "q_pos", q_pos, at, i32, (n,))
    if join_out is not None:
        _expect(what, "join_out", join_out, at, f32, (n, heads, D))
    if join_lse is not None:
        _expect(what, "join_lse", join_lse, at, f32, (n, heads))
    if out is not None:
        _expect(what, "out", out, at, torch.bfloat16, (n, heads, D))
    if lse is not None:
        _expect(what, "lse", lse, at, f32, (n, heads))
    _expect_workspace(what, workspace, device)
    c = ctypes.byref(cache.c_struct())

    def call(s):
        to = torch.empty_like(q) if out is None else out
        ws = _workspace(lib.hca_shared_attend_workspace(c, n, heads), workspace, device)
        _check(lib.hca_shared_attend(c, q.data_ptr(), n, heads, q_offsets.data_ptr(), _ptr(q_pos), _ptr(join_out),
                                     _ptr(join_lse), D ** -0.5 if softmax_scale is None else softmax_scale,
                                     to.data_ptr(), _ptr(lse), ws.data_ptr(), ws.nbytes, s), what)
        for t in (out, lse):
            if t is not None:
                torch.autograd.graph.increment_version(t)  # as in csa_rotary
        return to

    return _on(device, stream, call)


def csa_cache_copy_workspace(dst: Cache, n_jobs: int, keep_cols: int = 0) -> int:
    return int(load_library().csa_cache_copy_workspace(ctypes.byref(dst.c_struct()), n_jobs, keep_cols))


def csa_cache_copy(src: Cache, dst: Cache, src_slot, dst_slot, keep=None, max_blocks=None, workspace=None,
                   stream=None):
    """Fork, move, cut, compact or free cache slots: slot dst_slot[i] of dst becomes the blocks of slot
    src_slot[i] of src (-1: none) -- all of them, the first max_blocks[i], or those listed in keep [n, cols]
    (ascending, -1 behind the last, as the indexer returns them). Slots and limits are int32 tensors;
    src may be dst, and a slot its own source (in place)."""
    import torch

    lib, what = load_library(), "csa_cache_copy"
    device, n, i32 = src.fp4.device, src_slot.shape[0] if src_slot.dim() else -1, torch.int32
    at = src.fp4.get_device()
    _expect_cache(what, src, at, i32)
    if dst is not src:
        _expect_cache(what, dst, at, i32)
    _expect(what, "src_slot", src_slot, at, i32, (n,))
    _expect(what, "dst_slot", dst_slot, at, i32, (n,))
    cols = 0
    if keep is not None:
        cols = keep.shape[-1] if keep.dim() else 0
        _expect(what, "keep", keep, at, i32, (n, cols))
        if cols == 0:
            raise CsaError(f"{what}: keep needs a column (-1 in it keeps nothing)")
    if max_blocks is not None:
        _expect(what, "max_blocks", max_blocks, at, i32, (n,))
    _expect_workspace(what, workspace, device)
    cs = src.c_struct()
    cd = cs if dst is src else dst.c_struct()

    def call(s):
        ws = _workspace(lib.csa_cache_copy_workspace(ctypes.byref(cd), n, cols), workspace, device)
        _check(lib.csa_cache_copy(ctypes.byref(cs), ctypes.byref(cd), n, src_slot.data_ptr(), dst_slot.data_ptr(),
                                  _ptr(keep), cols, _ptr(max_blocks), ws.data_ptr(), ws.nbytes, s), what)

    _on(device, stream, call)


def _vectors(what, name, t):
    import torch

    kind = CSA_BF16 if t.dtype is torch.bfloat16 else CSA_F32
    if kind == CSA_F32 and t.dtype is not torch.float32:
        raise CsaError(f"{what}: {name} must be bfloat16 or float32, not {t.dtype}")
    step = t.stride()
    if len(step) not in (2, 3) or (step[-1] != 1 and t.shape[-1] > 1):
        raise CsaError(f"{what}: {name} must be [rows, (heads,) dim] with adjacent channels")
    return _CVectors(t.data_ptr(), kind, step[0], step[1] if len(step) == 3 else 0)


def csa_rotary(x, pos, inv_freq, out=None, rot_begin: Optional[int] = None, layout: int = CSA_ROPE_PAIRS,
               inverse: bool = False, mscale: float = 1.0, out_dtype=None, stream=None):
    """Rotary positions: x [rows, (heads,) dim] bf16 or float32 (any strides, channels adjacent) with the
    channels [rot_begin, rot_begin + 2 len(inv_freq)) turned by pos [rows] int32 * inv_freq float32
    (rot_begin: the last ones by default). Returns `out`: x itself turns it in place; by default a new
    tensor of out_dtype (x's type). inverse=True turns back, and is the gradient of x: the backward pass of a
    caller's autograd function. The call itself records none, and refuses tensors that require one."""
    import torch

    lib, what = load_library(), "csa_rotary"
    cx = _vectors(what, "x", x)
    rows, dim = x.shape[0], x.shape[-1]
    heads = x.shape[1] if x.dim() == 3 else 1
    if out is not None and (out.shape != x.shape or out.device != x.device or
                            (out_dtype is not None and out.dtype != out_dtype)):
        raise CsaError(f"{what}: out must match x's shape and device, and out_dtype")
    if torch.is_grad_enabled() and (x.requires_grad or inv_freq.requires_grad or
                                    (out is not None and out.requires_grad)):
        raise CsaError(f"{what} records no gradient: call it on detached tensors or under torch.no_grad(); the "
                       "gradient of x is csa_rotary(dy, ..., inverse=True)")
    rot = 2 * inv_freq.shape[0] if inv_freq.dim() else 0
    at = x.get_device()
    _expect(what, "pos", pos, at, torch.int32, (rows,))
    _expect(what, "inv_freq", inv_freq, at, torch.float32, (rot // 2,))
    rope = _CRope(inv_freq.data_ptr(), dim - rot if rot_begin is None else rot_begin, rot, layout, mscale)

    def call(s):
        # (empty_like takes a third of empty's time)
        to = torch.empty_like(x, dtype=out_dtype, memory_format=torch.contiguous_format) if out is None else out
        co = cx if to is x else _vectors(what, "out", to)
        _check(lib.csa_rotary(ctypes.byref(cx), ctypes.byref(co), rows, heads, dim, ctypes.byref(rope), pos.data_ptr(),
                              int(inverse), s), what)
        if out is not None:
            torch.autograd.graph.increment_version(out)  # who kept it for a backward pass finds it changed
        return to

    return _on(x.device, stream, call)


def csa_rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: int = CSA_ROPE_SCALE_NONE,
                           factor: float = 1.0, original_len: int = 1, beta_fast: float = 32.0,
                           beta_slow: float = 1.0):
    """(inv_freq, mscale) for csa_rotary: float32 [rot_dim / 2] on the host, and the scale of its
    outputs (1 but for CSA_ROPE_SCALE_PARTS). See include/csa.h for the scalings."""
    import torch

    inv = torch.empty(max(rot_dim, 0) // 2, dtype=torch.float32)
    m = ctypes.c_float(1.0)
    _check(load_library().csa_rotary_frequencies(rot_dim, base, scaling, factor, original_len, beta_fast, beta_slow,
                                                 inv.data_ptr() or None, ctypes.byref(m)), "csa_rotary_frequencies")
    return inv, float(m.value)


def csa_probe_mxf4_mma(iters: int, status, stream=None) -> int:
    """Launch the block-scaled MXFP4 MMA probe (one CTA per SM); returns its dense FLOPs.
    `status` is a device int32 tensor that receives CSA_DEV_TIMEOUT if completion is not seen."""
    lib = load_library()
    flops = ctypes.c_int64(0)
    _check(lib.csa_probe_mxf4_mma(int(iters), _ptr(status), _stream(stream), ctypes.byref(flops)), "csa_probe_mxf4_mma")
    return int(flops.value)


def csa_read_device_status(cache: Cache, stream=None) -> int:
    """Synchronize, return and clear the device status bits (CSA_DEV_*)."""
    lib = load_library()
    v = ctypes.c_int32(0)
    c = cache.c_struct()
    _check(lib.csa_read_device_status(ctypes.byref(c), _stream(stream), ctypes.byref(v)), "csa_read_device_status")
    return int(v.value)
