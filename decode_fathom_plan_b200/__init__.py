"""Python binding of libfathom.so, the sm_100a Fathom read-depth key scan and
the decode step around it.

Argument marshalling only (ctypes; for the calls on a paged cache a small
native module): every step of the path (pack, plan, scan, select, norm and
rotation, append, attention) runs in the library's CUDA kernels.  PyTorch
supplies device memory, pinned host memory and streams.  There is no CPU
fallback: if the library is missing or no GPU is present, the calls raise.

The entry points carry the C names of include/fathom.h and take torch
tensors (or raw addresses) where the C call takes pointers.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfathom.so")

FATHOM_OK = 0
FATHOM_ERR_INVALID_ARG = 1
FATHOM_ERR_CUDA = 2
FATHOM_ERR_NONFINITE = 3
FATHOM_ERR_TIMEOUT = 4
FATHOM_ERR_WORKSPACE = 5
FATHOM_ERR_UNIMPLEMENTED = 6

FATHOM_RES_DEVICE = 0
FATHOM_RES_HOST_MAPPED = 1

FATHOM_SCAN_DEFAULT = 0
FATHOM_SCAN_FORCE_EXACT = 1
FATHOM_SCAN_PROFILE = 2

FATHOM_F32 = 0
FATHOM_BF16 = 1
FATHOM_F16 = 2

FATHOM_ROTARY_PLAIN = 0
FATHOM_ROTARY_LINEAR = 1
FATHOM_ROTARY_NTK = 2
FATHOM_ROTARY_YARN = 3
FATHOM_ROTARY_YARN_INDEX = 4

EXPORTED = (
    "fathom_n_words", "fathom_status_str", "fathom_pack_workspace_bytes", "fathom_pack_keys",
    "fathom_plan", "fathom_fixed_plan", "fathom_scan_workspace_bytes", "fathom_scan_topk",
    "fathom_scan_batched_workspace_bytes", "fathom_scan_topk_batched",
    "fathom_last_device_status", "fathom_launch_count", "fathom_set_wait_limit", "fathom_profile_read",
    "fathom_scan_topk_static", "fathom_link_probe", "fathom_append_keys",
    "fathom_sparse_attention_workspace_bytes", "fathom_sparse_attention", "fathom_plan_marginal",
    "fathom_merge_topk",
    "fathom_rotary_turns", "fathom_qk_norm_rope", "fathom_append_kv",
    "fathom_paged_attention_workspace_bytes", "fathom_paged_attention",
    "fathom_sparse_attention_paged_workspace_bytes", "fathom_sparse_attention_paged",
)


class FathomError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} (status {status})")


class fathom_index(ctypes.Structure):
    """Mirror of the C fathom_index descriptor."""
    _fields_ = [
        ("n_kv_heads", ctypes.c_int32), ("group", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("n_keys", ctypes.c_int32),
        ("n_words", ctypes.c_int32), ("residency", ctypes.c_int32),
        ("planes", ctypes.c_void_p), ("mn", ctypes.c_void_p), ("scale", ctypes.c_void_p),
        ("sigma2", ctypes.c_void_p), ("sum_code", ctypes.c_void_p),
        ("sum_code2", ctypes.c_void_p), ("bits", ctypes.c_int32),
        ("block_keys", ctypes.c_int32),
    ]


class fathom_rows(ctypes.Structure):
    """Mirror of the C fathom_rows view."""
    _fields_ = [
        ("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64), ("n_heads", ctypes.c_int32), ("dtype", ctypes.c_int32),
    ]


class fathom_rotary(ctypes.Structure):
    """Mirror of the C fathom_rotary descriptor."""
    _fields_ = [
        ("turns", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32), ("magnitude", ctypes.c_float),
    ]


class fathom_kv_cache(ctypes.Structure):
    """Mirror of the C fathom_kv_cache descriptor."""
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
        ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
    ]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libfathom.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python decode_fathom_plan_b200/build.py` (nvcc, sm_100a)")
    lib = ctypes.CDLL(path)
    P, I32, SZ, U32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_uint32
    IX = ctypes.POINTER(fathom_index)
    RW, RO = ctypes.POINTER(fathom_rows), ctypes.POINTER(fathom_rotary)
    KV, F32, F64, I64 = (ctypes.POINTER(fathom_kv_cache), ctypes.c_float, ctypes.c_double,
                         ctypes.c_int64)
    sig = {
        "fathom_n_words": ([I32], I32),
        "fathom_status_str": ([ctypes.c_int], ctypes.c_char_p),
        "fathom_pack_workspace_bytes": ([IX], SZ),
        "fathom_pack_keys": ([P, IX, P, SZ, P], ctypes.c_int),
        "fathom_append_keys": ([IX, P, I32, P, P], ctypes.c_int),
        "fathom_sparse_attention_workspace_bytes": ([I32, I32, I32], SZ),
        "fathom_sparse_attention": ([P, P, I32, I32, I32, I32, P, P, I32, ctypes.c_float, P, P,
                                     SZ, P], ctypes.c_int),
        "fathom_plan": ([IX, P, P, P, P, P, P], ctypes.c_int),
        "fathom_fixed_plan": ([IX, P, I32, P, P, P, P], ctypes.c_int),
        "fathom_plan_marginal": ([IX, P, P, P, P, P, P], ctypes.c_int),
        "fathom_merge_topk": ([P, P, P, I32, I32, I32, I32, P, P, P], ctypes.c_int),
        "fathom_scan_workspace_bytes": ([IX, I32], SZ),
        "fathom_scan_topk": ([IX, P, P, P, I32, P, P, P, SZ, U32, P], ctypes.c_int),
        "fathom_scan_topk_static": ([IX, P, P, P, I32, P, P, U32, P], ctypes.c_int),
        "fathom_scan_batched_workspace_bytes": ([IX, I32, I32], SZ),
        "fathom_scan_topk_batched": ([IX, I32, P, P, P, I32, P, P, P, SZ, U32, P], ctypes.c_int),
        "fathom_last_device_status": ([P], ctypes.c_int),
        "fathom_launch_count": ([], ctypes.c_uint64),
        "fathom_set_wait_limit": ([ctypes.c_uint64], ctypes.c_uint64),
        "fathom_link_probe": ([P, SZ, P, P], ctypes.c_int),
        "fathom_profile_read": ([ctypes.POINTER(ctypes.c_double),
                                 ctypes.POINTER(ctypes.c_uint64)], ctypes.c_int),
        "fathom_rotary_turns": ([P, P, I32, F64, I32, F64, I64, F64, F64], ctypes.c_int),
        "fathom_qk_norm_rope": ([I32, I32, P, RO, P, P, F32, RW, RW, RW, RW, P], ctypes.c_int),
        "fathom_append_kv": ([KV, I32, RW, RW, P, P, P, I32, I32, RO, P, F32, P], ctypes.c_int),
        "fathom_paged_attention_workspace_bytes": ([KV, I32, I32, I32, I32], SZ),
        "fathom_paged_attention": ([KV, RW, P, I32, P, I32, I32, I32, F32, F32, P, RW, P, SZ, P],
                                   ctypes.c_int),
        "fathom_sparse_attention_paged_workspace_bytes": ([I32, I32, I32, I32], SZ),
        "fathom_sparse_attention_paged": ([KV, RW, P, I32, P, I32, P, I32, F32, F32, P, RW, P, SZ,
                                           P], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _ptr(x) -> int:
    """Address of a torch tensor (or pass through an int / None)."""
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, what: str):
    if rc != FATHOM_OK:
        raise FathomError(rc, what)


def status_str(status: int) -> str:
    return load_library().fathom_status_str(int(status)).decode()


# --------------------------------------------------------------- C entry points
def fathom_n_words(n_keys: int) -> int:
    return int(load_library().fathom_n_words(int(n_keys)))


def fathom_status_str(status: int) -> str:
    return status_str(status)


def fathom_pack_workspace_bytes(index: fathom_index) -> int:
    return int(load_library().fathom_pack_workspace_bytes(ctypes.byref(index)))


def fathom_pack_keys(keys, index: fathom_index, workspace, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load_library().fathom_pack_keys(_ptr(keys), ctypes.byref(index), _ptr(workspace),
                                           ws_bytes, _stream(stream)), "fathom_pack_keys")


def fathom_append_keys(keys, index: fathom_index, m: int, clamped=None, stream=None):
    """Append m keys (device float32 [H][m][d]) to the index; index.n_keys
    grows by m.  clamped: optional device uint32 [H][d] drift counters."""
    _check(load_library().fathom_append_keys(ctypes.byref(index), _ptr(keys), int(m),
                                             None if clamped is None else _ptr(clamped),
                                             _stream(stream)), "fathom_append_keys")


def fathom_plan(index: fathom_index, q_bf16, budget, t, t_union, nbytes, stream=None):
    _check(load_library().fathom_plan(ctypes.byref(index), _ptr(q_bf16), _ptr(budget), _ptr(t),
                                      _ptr(t_union), _ptr(nbytes), _stream(stream)),
           "fathom_plan")


def fathom_plan_marginal(index: fathom_index, q_bf16, budget, t, t_union, nbytes, stream=None):
    _check(load_library().fathom_plan_marginal(ctypes.byref(index), _ptr(q_bf16), _ptr(budget),
                                               _ptr(t), _ptr(t_union), _ptr(nbytes),
                                               _stream(stream)), "fathom_plan_marginal")


def fathom_fixed_plan(index: fathom_index, q_bf16, r: int, t, t_union, nbytes, stream=None):
    _check(load_library().fathom_fixed_plan(ctypes.byref(index), _ptr(q_bf16), int(r), _ptr(t),
                                            _ptr(t_union), _ptr(nbytes), _stream(stream)),
           "fathom_fixed_plan")


def fathom_scan_workspace_bytes(index: fathom_index, k: int) -> int:
    return int(load_library().fathom_scan_workspace_bytes(ctypes.byref(index), int(k)))


def fathom_scan_topk(index: fathom_index, q_bf16, t, t_union, k: int, out_idx, out_score,
                     workspace, flags: int = 0, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load_library().fathom_scan_topk(ctypes.byref(index), _ptr(q_bf16), _ptr(t),
                                           _ptr(t_union), int(k), _ptr(out_idx), _ptr(out_score),
                                           _ptr(workspace), ws_bytes, int(flags),
                                           _stream(stream)), "fathom_scan_topk")


def fathom_scan_topk_static(index: fathom_index, q_bf16, t, t_union, k: int, out_idx,
                            out_score, flags: int = 0, stream=None):
    """fathom_scan_topk without a workspace argument, for callers that cannot
    allocate device memory: runs on the library's fixed 8 MiB per-GPU scratch
    array (see include/fathom.h for the limits and the sharing rule)."""
    _check(load_library().fathom_scan_topk_static(ctypes.byref(index), _ptr(q_bf16), _ptr(t),
                                                  _ptr(t_union), int(k), _ptr(out_idx),
                                                  _ptr(out_score), int(flags), _stream(stream)),
           "fathom_scan_topk_static")


def _index_array(sessions: Sequence[fathom_index]):
    arr = (fathom_index * len(sessions))()
    for i, s in enumerate(sessions):
        arr[i] = s
    return arr


def fathom_scan_batched_workspace_bytes(sessions: Sequence[fathom_index], k: int) -> int:
    arr = _index_array(sessions)
    return int(load_library().fathom_scan_batched_workspace_bytes(arr, len(sessions), int(k)))


def fathom_scan_topk_batched(sessions: Sequence[fathom_index], q_bf16, t, t_union, k: int,
                             out_idx, out_score, workspace, flags: int = 0, stream=None):
    n = len(sessions)
    arr = _index_array(sessions)
    vp = ctypes.c_void_p * n
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load_library().fathom_scan_topk_batched(
        arr, n, vp(*[_ptr(x) for x in q_bf16]), vp(*[_ptr(x) for x in t]),
        vp(*[_ptr(x) for x in t_union]), int(k), vp(*[_ptr(x) for x in out_idx]),
        vp(*[_ptr(x) for x in out_score]), _ptr(workspace), ws_bytes, int(flags),
        _stream(stream)), "fathom_scan_topk_batched")


def fathom_sparse_attention_workspace_bytes(n_queries: int, head_dim: int, k: int) -> int:
    return int(load_library().fathom_sparse_attention_workspace_bytes(int(n_queries),
                                                                       int(head_dim), int(k)))


def fathom_sparse_attention(keys, values, n_kv_heads: int, group: int, head_dim: int,
                            n_keys: int, q_bf16, idx, k: int, softmax_scale: float, out,
                            workspace, stream=None):
    """Softmax attention of each query over its k selected keys (fp32)."""
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load_library().fathom_sparse_attention(
        _ptr(keys), _ptr(values), int(n_kv_heads), int(group), int(head_dim), int(n_keys),
        _ptr(q_bf16), _ptr(idx), int(k), float(softmax_scale), _ptr(out), _ptr(workspace),
        ws_bytes, _stream(stream)), "fathom_sparse_attention")


def fathom_merge_topk(shard_idx, shard_score, shard_offset, k: int, out_idx, out_score,
                      stream=None):
    """Exact top-k over S shard lists ([S][Q][k_shard] device tensors) of key
    ranges starting at shard_offset (S ints, ascending)."""
    S, Q, k_s = shard_idx.shape
    offs = (ctypes.c_int64 * S)(*[int(o) for o in shard_offset])
    _check(load_library().fathom_merge_topk(_ptr(shard_idx), _ptr(shard_score), offs, S, Q, k_s,
                                            int(k), _ptr(out_idx), _ptr(out_score),
                                            _stream(stream)), "fathom_merge_topk")


# ------------------------------------------------- calls on a paged cache
# These take tensors, whose addresses, shapes and strides _binding.so passes on
# (csrc/binding.cpp).  A tensor that the C call would misread (wrong type,
# layout or device) raises ValueError.  A call runs on the tensors' device, on
# `stream` (a stream, its address or None) or that device's current one.
_native = None


def _load_binding():
    global _native
    if _native is None:
        load_library()
        import torch  # noqa: F401  (its libraries are loaded before the module's)
        try:
            from . import _binding
        except ImportError as e:
            raise ImportError(f"{PKG}/_binding.so is missing or does not load: build it with "
                              "`python decode_fathom_plan_b200/build.py`") from e
        _native = _binding
    return _native


_DTYPES = {}


def _dtype_code(dtype) -> int:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: FATHOM_F32, torch.bfloat16: FATHOM_BF16,
                        torch.float16: FATHOM_F16})
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"float32, bfloat16 or float16 is wanted, not {dtype}")
    return code


def fathom_rotary_turns(rotary_dim: int, base: float = 10000.0, scaling: int = FATHOM_ROTARY_PLAIN,
                        factor: float = 1.0, original_len: int = 1, beta_fast: float = 32.0,
                        beta_slow: float = 1.0):
    """-> (turns per position, a host float64 tensor [rotary_dim/2]; magnitude)."""
    import torch
    turns = torch.empty(max(1, int(rotary_dim) // 2), dtype=torch.float64)
    magnitude = ctypes.c_float()
    _check(load_library().fathom_rotary_turns(turns.data_ptr(), ctypes.byref(magnitude),
                                              int(rotary_dim), float(base), int(scaling),
                                              float(factor), int(original_len), float(beta_fast),
                                              float(beta_slow)), "fathom_rotary_turns")
    return turns, magnitude.value


def fathom_qk_norm_rope(q, k, pos, q_out, k_out, rotary=None, q_weight=None, k_weight=None,
                        eps: float = 1e-6, stream=None):
    """Norm (where a weight is given) and rotation (where a RotaryTable is
    given) of query rows q [T][Hq][d] and key rows k [T][Hk][d] at positions
    pos (int32 [T]) into q_out and k_out; q and q_out, or k and k_out, may be
    None."""
    table, where = (None, None) if rotary is None else (rotary.desc, rotary.device_index)
    rc = (_native or _load_binding()).qk_norm_rope(q, k, pos, q_out, k_out, table, where, q_weight,
                                                   k_weight, eps, stream)
    if rc:
        raise FathomError(rc, "fathom_qk_norm_rope")


def fathom_append_kv(cache: fathom_kv_cache, k, v, seq, pos, page_table, rotary=None,
                     k_weight=None, eps: float = 1e-6, stream=None):
    """Write key rows k and value rows v [T][H][d] to positions pos (int32 [T])
    of sequences seq (int32 [T], negative: padding) of a paged cache, each key
    normed and rotated on the way; page_table int32 [n_seqs][pages]."""
    table, where = (None, None) if rotary is None else (rotary.desc, rotary.device_index)
    rc = (_native or _load_binding()).append_kv(cache, k, v, seq, pos, page_table, table, where,
                                                k_weight, eps, stream)
    if rc:
        raise FathomError(rc, "fathom_append_kv")


def fathom_paged_attention_workspace_bytes(cache: fathom_kv_cache, n_seqs: int, group: int,
                                           max_len: int, prefix_len: int = 0) -> int:
    return int(load_library().fathom_paged_attention_workspace_bytes(
        ctypes.byref(cache), int(n_seqs), int(group), int(max_len), int(prefix_len)))


def fathom_paged_attention(cache: fathom_kv_cache, q, page_table, seq_lens, max_len: int, out,
                           workspace, softmax_scale: float, prefix_len: int = 0,
                           softcap: float = 0.0, slopes=None, stream=None):
    """Attention of one query token per sequence, q [n_seqs][Hq][d], over all
    seq_lens[b] <= max_len keys of its pages; the first prefix_len keys are the
    same pages in every row of page_table."""
    rc = (_native or _load_binding()).paged_attention(cache, q, page_table, seq_lens, max_len, out,
                                                      workspace, softmax_scale, prefix_len, softcap,
                                                      slopes, stream)
    if rc:
        raise FathomError(rc, "fathom_paged_attention")


def fathom_sparse_attention_paged_workspace_bytes(n_seqs: int, n_heads: int, head_dim: int,
                                                  k: int) -> int:
    return int(load_library().fathom_sparse_attention_paged_workspace_bytes(
        int(n_seqs), int(n_heads), int(head_dim), int(k)))


def fathom_sparse_attention_paged(cache: fathom_kv_cache, q, idx, page_table, seq_lens, out,
                                  workspace, softmax_scale: float, softcap: float = 0.0,
                                  slopes=None, stream=None):
    """Attention of each query head of q [n_seqs][Hq][d] over the keys that
    idx (int32 [n_seqs][Hq][k], -1: no key) lists of its sequence's pages."""
    rc = (_native or _load_binding()).sparse_attention_paged(cache, q, idx, page_table, seq_lens,
                                                             out, workspace, softmax_scale, softcap,
                                                             slopes, stream)
    if rc:
        raise FathomError(rc, "fathom_sparse_attention_paged")


def fathom_last_device_status(stream=None) -> int:
    return int(load_library().fathom_last_device_status(_stream(stream)))


def fathom_link_probe(buffer, nbytes: int, sink, stream=None):
    """Zero-copy read of `nbytes` of a pinned host (or device) buffer."""
    _check(load_library().fathom_link_probe(_ptr(buffer), int(nbytes), _ptr(sink),
                                            _stream(stream)), "fathom_link_probe")


def fathom_launch_count() -> int:
    return int(load_library().fathom_launch_count())


def fathom_set_wait_limit(ns: int) -> int:
    """Limit of the waits inside kernels, in nanoseconds; returns the one before."""
    return int(load_library().fathom_set_wait_limit(int(ns)))


def fathom_profile_read():
    """-> (summed milliseconds of profiled main-scan launches, launches)."""
    ms = ctypes.c_double(0.0)
    n = ctypes.c_uint64(0)
    _check(load_library().fathom_profile_read(ctypes.byref(ms), ctypes.byref(n)),
           "fathom_profile_read")
    return ms.value, n.value


# ---------------------------------------------------------- memory plumbing
class KeyIndex:
    """Owns the torch buffers of one packed K index and its C descriptor.

    residency "device" keeps the planes in HBM; "host_mapped" keeps them in
    pinned host memory read zero-copy by the scan.  Statistics stay on the
    device either way.  bits: 4 (the 4-bit K cache) or 8 (the 8-plane
    variant for an 8-bit K cache).  block_keys: 0 for one scale per channel,
    or grouped per-token-block scales over blocks of that many tokens (a
    multiple of 2048); mn, scale, sum_code and sum_code2 are then
    [H][n_blocks][d] with n_blocks counted over the capacity."""

    def __init__(self, n_kv_heads: int, group: int, n_keys: int, head_dim: int = 128,
                 residency: str = "device", device: Optional[int] = None,
                 capacity: Optional[int] = None, bits: int = 4, block_keys: int = 0):
        import torch
        if bits not in (4, 8):
            raise ValueError(f"bits must be 4 or 8, not {bits}")
        if block_keys < 0 or block_keys % 2048:
            raise ValueError(f"block_keys must be 0 or a multiple of 2048, not {block_keys}")
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
        self.n_words = fathom_n_words(max(n_keys, capacity or n_keys))
        H, d = n_kv_heads, head_dim
        shape = (H, d, bits, self.n_words)
        if residency == "device":
            self.planes = torch.empty(shape, dtype=torch.int32, device=dev)
            res = FATHOM_RES_DEVICE
        elif residency == "host_mapped":
            self.planes = torch.empty(shape, dtype=torch.int32, pin_memory=True)
            res = FATHOM_RES_HOST_MAPPED
        else:
            raise ValueError(f"unknown residency {residency!r}")
        stat = (H, d)
        if block_keys:
            stat = (H, -(-32 * self.n_words // block_keys), d)
        self.mn = torch.empty(stat, dtype=torch.float32, device=dev)
        self.scale = torch.empty_like(self.mn)
        self.sigma2 = torch.empty((H, d), dtype=torch.float32, device=dev)
        self.sum_code = torch.empty(stat, dtype=torch.int64, device=dev)
        self.sum_code2 = torch.empty_like(self.sum_code)
        self.residency = residency
        self.desc = fathom_index(H, group, d, n_keys, self.n_words, res,
                                 self.planes.data_ptr(), self.mn.data_ptr(),
                                 self.scale.data_ptr(), self.sigma2.data_ptr(),
                                 self.sum_code.data_ptr(), self.sum_code2.data_ptr(), bits,
                                 block_keys)
        self.device = dev

    @property
    def n_kv_heads(self):
        return self.desc.n_kv_heads

    @property
    def group(self):
        return self.desc.group

    @property
    def head_dim(self):
        return self.desc.head_dim

    @property
    def n_keys(self):
        return self.desc.n_keys

    @property
    def bits(self):
        return self.desc.bits

    @property
    def block_keys(self):
        return self.desc.block_keys

    @property
    def capacity(self):
        return 32 * self.n_words

    def append(self, keys, clamped=None, stream=None):
        """Append device float32 keys [H][m][d] (decode-step keys) to this
        index; clamped: optional device uint32 [H][d] drift counters."""
        fathom_append_keys(keys, self.desc, keys.shape[1], clamped, stream)
        return self

    def pack(self, keys, stream=None):
        """Quantise and pack device float32 keys [H][n][d] into this index."""
        import torch
        ws = torch.empty(max(16, fathom_pack_workspace_bytes(self.desc)), dtype=torch.uint8,
                         device=self.device)
        fathom_pack_keys(keys, self.desc, ws, stream)
        return self


class ScanBuffers:
    """Device outputs and workspace for planning and scanning one session."""

    def __init__(self, index: KeyIndex, k: int):
        import torch
        dev = index.device
        Q, H, d = index.n_kv_heads * index.group, index.n_kv_heads, index.head_dim
        self.k = k
        self.t = torch.empty((Q, d), dtype=torch.uint8, device=dev)
        self.t_union = torch.empty((H, d), dtype=torch.uint8, device=dev)
        self.nbytes = torch.empty((Q + H,), dtype=torch.int64, device=dev)
        self.idx = torch.empty((Q, k), dtype=torch.int32, device=dev)
        self.score = torch.empty((Q, k), dtype=torch.float32, device=dev)
        self.workspace = torch.empty(max(16, fathom_scan_workspace_bytes(index.desc, k)),
                                     dtype=torch.uint8, device=dev)


def plan_and_scan(index: KeyIndex, q_bf16, budget, buf: ScanBuffers, flags: int = 0,
                  stream=None, fixed_r: Optional[int] = None):
    """One decode-step scan of a layer: plan (or fixed plan) then scan+top-k."""
    if fixed_r is None:
        fathom_plan(index.desc, q_bf16, budget, buf.t, buf.t_union, buf.nbytes, stream)
    else:
        fathom_fixed_plan(index.desc, q_bf16, fixed_r, buf.t, buf.t_union, buf.nbytes, stream)
    fathom_scan_topk(index.desc, q_bf16, buf.t, buf.t_union, buf.k, buf.idx, buf.score,
                     buf.workspace, flags, stream)
    return buf


class RotaryTable:
    """Owns the device table of a position rotation and its C descriptor.

    rotary_dim: channels of a head that are rotated (default: all of
    head_dim).  interleaved: pairs are (2i, 2i + 1) instead of (i, i +
    rotary_dim/2).  scaling: "none", "linear", "ntk", "yarn" or "yarn_index",
    stretched by factor (include/fathom.h gives the formulas).  "yarn" is the
    paper's, whose ramp runs over the turns of a pair; "yarn_index", whose ramp
    runs over the pairs' numbers, is what checkpoints with beta_fast, beta_slow
    and an original length in their configuration are trained with."""

    _SCALINGS = {"none": FATHOM_ROTARY_PLAIN, "linear": FATHOM_ROTARY_LINEAR,
                 "ntk": FATHOM_ROTARY_NTK, "yarn": FATHOM_ROTARY_YARN,
                 "yarn_index": FATHOM_ROTARY_YARN_INDEX}

    def __init__(self, head_dim: int, rotary_dim: Optional[int] = None, base: float = 10000.0,
                 interleaved: bool = False, scaling: str = "none", factor: float = 1.0,
                 original_len: int = 1, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 device: Optional[int] = None):
        import torch
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        if rotary_dim > head_dim:
            raise ValueError(f"rotary_dim {rotary_dim} of a head of {head_dim} channels")
        if scaling not in self._SCALINGS:
            raise ValueError(f"scaling is one of {', '.join(self._SCALINGS)}, not {scaling!r}")
        turns, magnitude = fathom_rotary_turns(rotary_dim, base, self._SCALINGS[scaling], factor,
                                               original_len, beta_fast, beta_slow)
        self._set(turns, interleaved, magnitude, device)

    @classmethod
    def from_frequencies(cls, frequencies, head_dim: int, interleaved: bool = False,
                         magnitude: float = 1.0, device: Optional[int] = None):
        """A table of given frequencies, radians per position of each pair
        (numbers or a tensor [rotary_dim/2], kept in float64), for scalings
        that fathom_rotary_turns does not have."""
        import math

        import torch
        f = torch.as_tensor(frequencies, dtype=torch.float64).detach().cpu()
        if f.dim() != 1 or not 1 <= f.numel() <= head_dim // 2:
            raise ValueError(f"1 to {head_dim // 2} frequencies are wanted for a head of {head_dim} "
                             f"channels, not {list(f.shape)}")
        if not torch.isfinite(f).all() or not math.isfinite(magnitude):
            raise ValueError("finite frequencies and magnitude are wanted")
        self = cls.__new__(cls)
        self._set(f / (2 * math.pi), interleaved, float(magnitude), device)
        return self

    def _set(self, turns, interleaved, magnitude, device):
        import torch
        self.device = torch.device("cuda", torch.cuda.current_device() if device is None
                                   else device)
        self.turns = turns.to(self.device)
        self.magnitude = magnitude
        self.device_index = self.device.index
        self.desc = fathom_rotary(self.turns.data_ptr(), 2 * turns.numel(), int(interleaved),
                                  magnitude)


class PagedKV:
    """Owns (or refers to) the tensors of a paged K/V cache and its C
    descriptor.  k and v are [n_pages][H][page_size][d]; order "token_major"
    stores them as [n_pages][page_size][H][d] instead (the views keep the
    first order).  residency "host_mapped" keeps the pages in pinned host
    memory, for fathom_append_kv and fathom_sparse_attention_paged."""

    def __init__(self, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int = 128,
                 dtype=None, order: str = "head_major", residency: str = "device",
                 device: Optional[int] = None):
        import torch
        dtype = torch.bfloat16 if dtype is None else dtype
        if order not in ("head_major", "token_major"):
            raise ValueError(f"unknown order {order!r}")
        if residency not in ("device", "host_mapped"):
            raise ValueError(f"unknown residency {residency!r}")
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
        shape = [n_pages, n_kv_heads, page_size, head_dim]
        if order == "token_major":
            shape[1], shape[2] = shape[2], shape[1]
        where = dict(device=dev) if residency == "device" else dict(pin_memory=True)
        k, v = (torch.zeros(shape, dtype=dtype, **where) for _ in range(2))
        if order == "token_major":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        self._set(k, v)

    @classmethod
    def from_tensors(cls, k, v):
        """A cache over existing tensors [n_pages][H][page_size][d] (views of
        any order of the first three axes, channels contiguous, equal strides)."""
        self = cls.__new__(cls)
        self._set(k, v)
        return self

    def _set(self, k, v):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype \
                or k.device != v.device or k.stride(3) != 1:
            raise ValueError("k and v: [n_pages][H][page_size][d] of one type, device and layout, "
                             "channels contiguous")
        if not (k.is_cuda or (k.is_pinned() and v.is_pinned())):
            raise ValueError("k and v: device or pinned host memory")
        self.k, self.v = k, v
        self.desc = fathom_kv_cache(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1),
                                    k.stride(2), k.shape[0], k.shape[2], k.shape[1], k.shape[3],
                                    _dtype_code(k.dtype))
