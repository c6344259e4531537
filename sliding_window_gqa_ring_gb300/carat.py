"""ctypes binding of libcarat.so: the same entry points, torch tensors in.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors must already live on the current CUDA device; the calls are
enqueued on torch's current stream (or the one passed) and return without
synchronising.  A missing library raises ``CaratError`` -- there is no CPU
fallback.

Layouts (see include/carat.h for the full contract):
  queries   bf16 [B][k][Hq][D]          out   fp32 [B][k][Hq][D]
  rings     bf16 [num_rings][window][Hkv][D]
  caches    bf16 [num_caches][capacity][Hkv][D]
  new rows  bf16 [B][k][Hkv][D]         displaced bf16 [B][k-1][2][Hkv][D]
  context_lengths int32 [B]; ring_ids / cache_ids int32 [B] or None
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_HERE, "libcarat.so")

CARAT_OK = 0
CARAT_ERR_INVALID_ARG = 1
CARAT_ERR_UNSUPPORTED = 2
CARAT_ERR_WORKSPACE = 3
CARAT_ERR_CUDA = 4
CARAT_DEV_BAD_CONTEXT = 0x1
CARAT_DEV_BAD_CACHE_ID = 0x2
CARAT_DEV_TIMEOUT = 0x4
CARAT_DEV_BAD_POSITION = 0x8
MAX_PROPOSALS = 16
MAX_TILE_ROWS = 128

EXPORTED = (
    "carat_ring_append", "carat_swa_attention", "carat_global_verify_attention",
    "carat_swa_workspace_bytes", "carat_global_workspace_bytes", "carat_get_device_status",
    "carat_status_string", "carat_abi_version", "carat_kernel_launches",
    "carat_swa_attention_noalloc", "carat_noalloc_scratch_bytes",
    "carat_swa_append_attention", "carat_global_append_verify_attention",
    "carat_ring_rollback", "carat_global_append_verify_attention_paged", "carat_paged_append",
    "carat_pool_create", "carat_pool_destroy", "carat_pool_alloc_ring", "carat_pool_free_ring",
    "carat_pool_alloc_pages", "carat_pool_free_pages", "carat_pool_stats",
    "carat_ring_append_fp8", "carat_ring_rollback_fp8", "carat_swa_attention_fp8",
    "carat_check_bounded_wait", "carat_launch_floor",
    "carat_paged_rope_append", "carat_paged_rope_append_fp8",
    "carat_global_verify_attention_paged", "carat_paged_verify_attention_fp8",
    "carat_paged_fp8_workspace_bytes",
    "carat_paged_chunk_attention", "carat_paged_chunk_workspace_bytes",
    "carat_pages_copy", "carat_paged_fork", "carat_pages_move",
    "carat_pool_share_pages", "carat_pool_plan_compaction",
)


class CaratError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


_lock = threading.Lock()
_lib = None


def _declare(lib):
    vp, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    lib.carat_ring_append.restype = i32
    lib.carat_ring_append.argtypes = [vp, vp, i32, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, vp]
    lib.carat_swa_attention.restype = i32
    lib.carat_swa_attention.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, i32, i32, i32, i32, i32,
                                        i32, f32, vp, sz, vp]
    lib.carat_global_verify_attention.restype = i32
    lib.carat_global_verify_attention.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32,
                                                  i32, i32, f32, vp, sz, vp]
    lib.carat_swa_workspace_bytes.restype = sz
    lib.carat_swa_workspace_bytes.argtypes = [i32] * 6
    lib.carat_global_workspace_bytes.restype = sz
    lib.carat_global_workspace_bytes.argtypes = [i32] * 6
    lib.carat_launch_floor.restype = i32
    lib.carat_launch_floor.argtypes = [i32, vp]
    lib.carat_check_bounded_wait.restype = i32
    lib.carat_check_bounded_wait.argtypes = [ctypes.c_uint64, vp]
    lib.carat_get_device_status.restype = i32
    lib.carat_get_device_status.argtypes = [ctypes.POINTER(ctypes.c_int32), i32, vp]
    lib.carat_status_string.restype = ctypes.c_char_p
    lib.carat_status_string.argtypes = [i32]
    lib.carat_abi_version.restype = i32
    lib.carat_abi_version.argtypes = []
    lib.carat_kernel_launches.restype = ctypes.c_uint64
    lib.carat_kernel_launches.argtypes = []
    lib.carat_swa_attention_noalloc.restype = i32
    lib.carat_swa_attention_noalloc.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, i32, i32, i32,
                                                i32, i32, i32, f32, vp]
    lib.carat_noalloc_scratch_bytes.restype = sz
    lib.carat_noalloc_scratch_bytes.argtypes = []
    lib.carat_swa_append_attention.restype = i32
    lib.carat_swa_append_attention.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, i32, i32,
                                               i32, i32, i32, i32, f32, vp, sz, vp]
    lib.carat_ring_rollback.restype = i32
    lib.carat_ring_rollback.argtypes = [vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
    lib.carat_global_append_verify_attention_paged.restype = i32
    lib.carat_global_append_verify_attention_paged.argtypes = [
        vp, vp, vp, vp, i32, vp, i32, i32, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, sz, vp]
    lib.carat_paged_append.restype = i32
    lib.carat_paged_append.argtypes = [vp, vp, i32, vp, i32, i32, vp, vp, vp, i32, i32, i32, i32,
                                       vp]
    lib.carat_pool_create.restype = vp
    lib.carat_pool_create.argtypes = [i32, i32]
    lib.carat_pool_destroy.restype = None
    lib.carat_pool_destroy.argtypes = [vp]
    lib.carat_pool_alloc_ring.restype = i32
    lib.carat_pool_alloc_ring.argtypes = [vp]
    lib.carat_pool_free_ring.restype = i32
    lib.carat_pool_free_ring.argtypes = [vp, i32]
    lib.carat_pool_alloc_pages.restype = i32
    lib.carat_pool_alloc_pages.argtypes = [vp, i32, ctypes.POINTER(ctypes.c_int32)]
    lib.carat_pool_free_pages.restype = i32
    lib.carat_pool_free_pages.argtypes = [vp, i32, ctypes.POINTER(ctypes.c_int32)]
    lib.carat_pool_stats.restype = i32
    lib.carat_pool_stats.argtypes = [vp, ctypes.POINTER(ctypes.c_int32)]
    lib.carat_ring_append_fp8.restype = i32
    lib.carat_ring_append_fp8.argtypes = [vp, vp, i32, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32,
                                          f32, f32, vp]
    lib.carat_ring_rollback_fp8.restype = i32
    lib.carat_ring_rollback_fp8.argtypes = [vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                            vp]
    lib.carat_swa_attention_fp8.restype = i32
    lib.carat_swa_attention_fp8.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, i32, i32, i32, i32,
                                            i32, i32, f32, f32, f32, vp, sz, vp]
    i64 = ctypes.c_int64
    lib.carat_paged_rope_append.restype = i32
    lib.carat_paged_rope_append.argtypes = [
        vp, vp, i32, vp, i32, i32, vp, vp, i64, vp, vp, i64, vp, i32, i32, i32, vp, vp, vp, i32, i32,
        i32, i32, i32, vp]
    lib.carat_paged_rope_append_fp8.restype = i32
    lib.carat_paged_rope_append_fp8.argtypes = [
        vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, vp, i64, vp, vp, i64, vp, i32, i32, i32, vp, vp,
        vp, i32, i32, i32, i32, i32, vp]
    lib.carat_global_verify_attention_paged.restype = i32
    lib.carat_global_verify_attention_paged.argtypes = [
        vp, vp, vp, vp, i32, vp, i32, i32, vp, i32, i32, i32, i32, i32, f32, vp, sz, vp]
    lib.carat_paged_verify_attention_fp8.restype = i32
    lib.carat_paged_verify_attention_fp8.argtypes = [
        vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp,
        sz, vp]
    lib.carat_paged_fp8_workspace_bytes.restype = sz
    lib.carat_paged_fp8_workspace_bytes.argtypes = [i32] * 6
    lib.carat_paged_chunk_attention.restype = i32
    lib.carat_paged_chunk_attention.argtypes = [
        vp, vp, vp, vp, i32, vp, i32, i32, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32, vp, sz, vp]
    lib.carat_paged_chunk_workspace_bytes.restype = sz
    lib.carat_paged_chunk_workspace_bytes.argtypes = [i32] * 5
    pages = [vp, vp, vp, vp, i32, i32, i64, i32, i32]
    lib.carat_pages_copy.restype = i32
    lib.carat_pages_copy.argtypes = pages + [vp, vp, vp, i32, vp]
    lib.carat_paged_fork.restype = i32
    lib.carat_paged_fork.argtypes = pages + [vp, i32, i32, vp, vp, vp, vp, vp, i32, vp]
    lib.carat_pages_move.restype = i32
    lib.carat_pages_move.argtypes = pages + [vp, vp, i32, vp, i64, vp]
    ids = ctypes.POINTER(ctypes.c_int32)
    lib.carat_pool_share_pages.restype = i32
    lib.carat_pool_share_pages.argtypes = [vp, i32, ids]
    lib.carat_pool_plan_compaction.restype = i32
    lib.carat_pool_plan_compaction.argtypes = [vp, i32, ids, ids]
    lib.carat_global_append_verify_attention.restype = i32
    lib.carat_global_append_verify_attention.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp, i32,
                                                         i32, i32, i32, i32, i32, f32, vp, sz, vp]
    return lib


def library():
    """The loaded libcarat.so (raises CaratError if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIBRARY):
                raise CaratError(CARAT_ERR_CUDA, f"libcarat.so not built ({LIBRARY}); run "
                                 "python -c 'import __graft_entry__ as g; g.build()'")
            _lib = _declare(ctypes.CDLL(LIBRARY))
    return _lib


_STATUS_TEXT = {
    CARAT_OK: "ok",
    CARAT_ERR_INVALID_ARG: "invalid argument",
    CARAT_ERR_UNSUPPORTED: "unsupported size",
    CARAT_ERR_WORKSPACE: "workspace missing or too small",
    CARAT_ERR_CUDA: "CUDA error",
}


def status_string(status: int) -> str:
    """Text for a status code (the same strings carat_status_string returns)."""
    return _STATUS_TEXT.get(status, "unknown status")


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor or None")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _expect(t, dtype, name):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _attention_args(out, queries, k_cache, v_cache, context_lengths, cache_dtype, what,
                    displaced=None, k_new=None, v_new=None):
    """Shape and dtype checks the C ABI cannot make (it sees only pointers and
    sizes): a cache of the wrong element type or head_dim would be read past
    its end on the GPU.  Returns (batch, k, q_heads, head_dim, num, rows,
    kv_heads) with num/rows the cache's first two dimensions."""
    _expect(queries, torch.bfloat16, f"{what}: queries")
    _expect(out, torch.float32, f"{what}: out")
    _expect(k_cache, cache_dtype, f"{what}: key cache")
    _expect(v_cache, cache_dtype, f"{what}: value cache")
    _expect(context_lengths, torch.int32, f"{what}: context_lengths")
    if queries.dim() != 4 or k_cache.dim() != 4:
        raise ValueError(f"{what}: queries and caches must be 4-D")
    batch, k, q_heads, head_dim = queries.shape
    num, rows, kv_heads, cache_dim = k_cache.shape
    if tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError(f"{what}: key and value caches differ in shape")
    if cache_dim != head_dim:
        raise ValueError(f"{what}: cache head_dim {cache_dim} != query head_dim {head_dim}")
    if tuple(out.shape) != tuple(queries.shape):
        raise ValueError(f"{what}: out must have the queries' shape")
    if tuple(context_lengths.shape) != (batch,):
        raise ValueError(f"{what}: context_lengths must be [batch]")
    if displaced is not None:
        _expect(displaced, cache_dtype, f"{what}: displaced")
        if displaced.dim() != 5 or displaced.shape[0] < batch or \
                tuple(displaced.shape[2:]) != (2, kv_heads, head_dim) or \
                (k > 1 and displaced.shape[1] < k - 1):
            raise ValueError(f"{what}: displaced must be [>=batch][>=k-1][2][kv_heads][head_dim]")
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if t is not None:
            _expect(t, torch.bfloat16, f"{what}: {name}")
            if tuple(t.shape) != (batch, k, kv_heads, head_dim):
                raise ValueError(f"{what}: {name} must be [batch][k][kv_heads][head_dim]")
    return batch, k, q_heads, head_dim, num, rows, kv_heads


def _check(status: int, what: str):
    if status != CARAT_OK:
        raise CaratError(status, what)


def carat_ring_append(k_ring, v_ring, k_new, v_new, context_lengths, *, ring_ids=None,
                      displaced=None, window=None, stream=None):
    """Write this step's K/V rows at slot = position mod window (lockstep K, V).

    k_new/v_new: bf16 [B][k][Hkv][D]; rings bf16 [num_rings][window][Hkv][D].
    """
    _expect(k_ring, torch.bfloat16, "k_ring")
    _expect(k_new, torch.bfloat16, "k_new")
    _expect(context_lengths, torch.int32, "context_lengths")
    num_rings, ring_window, kv_heads, head_dim = k_ring.shape
    batch, k = k_new.shape[0], k_new.shape[1]
    if window is None:
        window = ring_window
    _check(library().carat_ring_append(
        _ptr(k_ring), _ptr(v_ring), num_rings, _ptr(ring_ids), _ptr(k_new), _ptr(v_new),
        _ptr(context_lengths), k, _ptr(displaced), batch, kv_heads, head_dim, window,
        _stream(stream)), "carat_ring_append")


def swa_workspace_bytes(batch, proposal_count, q_heads, kv_heads, head_dim, window) -> int:
    return int(library().carat_swa_workspace_bytes(batch, proposal_count, q_heads, kv_heads,
                                                   head_dim, window))


def global_workspace_bytes(batch, proposal_count, q_heads, kv_heads, head_dim, capacity) -> int:
    return int(library().carat_global_workspace_bytes(batch, proposal_count, q_heads, kv_heads,
                                                      head_dim, capacity))


def carat_swa_attention(out, queries, k_ring, v_ring, context_lengths, *, scale, workspace,
                        ring_ids=None, displaced=None, stream=None):
    """Sliding-window attention read in place from the rotated rings.

    out fp32 [B][k][Hq][D]; queries bf16 [B][k][Hq][D]; workspace: a CUDA tensor
    of at least swa_workspace_bytes(...) bytes.
    """
    batch, k, q_heads, head_dim, num_rings, window, kv_heads = _attention_args(
        out, queries, k_ring, v_ring, context_lengths, torch.bfloat16, "carat_swa_attention",
        displaced=displaced)
    _check(library().carat_swa_attention(
        _ptr(out), _ptr(queries), _ptr(k_ring), _ptr(v_ring), num_rings, _ptr(ring_ids),
        _ptr(displaced), _ptr(context_lengths), k, batch, q_heads, kv_heads, head_dim, window,
        float(scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), "carat_swa_attention")


def carat_swa_attention_noalloc(out, queries, k_ring, v_ring, context_lengths, *, scale,
                                ring_ids=None, displaced=None, stream=None):
    """carat_swa_attention with the library's built-in scratch instead of a
    workspace, for callers that cannot allocate device memory.  Raises
    CaratError (CARAT_ERR_WORKSPACE) for sizes that need more scratch than
    noalloc_scratch_bytes().  Calls that overlap on the GPU share the scratch
    and race; order them on one stream."""
    batch, k, q_heads, head_dim, num_rings, window, kv_heads = _attention_args(
        out, queries, k_ring, v_ring, context_lengths, torch.bfloat16,
        "carat_swa_attention_noalloc", displaced=displaced)
    _check(library().carat_swa_attention_noalloc(
        _ptr(out), _ptr(queries), _ptr(k_ring), _ptr(v_ring), num_rings, _ptr(ring_ids),
        _ptr(displaced), _ptr(context_lengths), k, batch, q_heads, kv_heads, head_dim, window,
        float(scale), _stream(stream)), "carat_swa_attention_noalloc")


def noalloc_scratch_bytes() -> int:
    return int(library().carat_noalloc_scratch_bytes())


def carat_global_verify_attention(out, queries, key_cache, value_cache, context_lengths, *,
                                  scale, workspace, cache_ids=None, stream=None):
    """Grouped-head causal verify attention over a full cache (masked tail)."""
    batch, k, q_heads, head_dim, num_caches, capacity, kv_heads = _attention_args(
        out, queries, key_cache, value_cache, context_lengths, torch.bfloat16,
        "carat_global_verify_attention")
    _check(library().carat_global_verify_attention(
        _ptr(out), _ptr(queries), _ptr(key_cache), _ptr(value_cache), num_caches,
        _ptr(cache_ids), _ptr(context_lengths), k, batch, q_heads, kv_heads, head_dim, capacity,
        float(scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), "carat_global_verify_attention")


def carat_swa_append_attention(out, queries, k_ring, v_ring, k_new, v_new, context_lengths, *,
                                scale, workspace, ring_ids=None, displaced=None, stream=None):
    """Append this step's rows to the rings and attend, in one launch.  Rings
    are passed as before the step; afterwards they hold the new rows (and
    `displaced`, if given, the rows they overwrote, for carat_ring_rollback)."""
    batch, k, q_heads, head_dim, num_rings, window, kv_heads = _attention_args(
        out, queries, k_ring, v_ring, context_lengths, torch.bfloat16,
        "carat_swa_append_attention", displaced=displaced, k_new=k_new, v_new=v_new)
    _check(library().carat_swa_append_attention(
        _ptr(out), _ptr(queries), _ptr(k_ring), _ptr(v_ring), num_rings, _ptr(ring_ids),
        _ptr(displaced), _ptr(k_new), _ptr(v_new), _ptr(context_lengths), k, batch, q_heads,
        kv_heads, head_dim, window, float(scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "carat_swa_append_attention")


def carat_ring_rollback(k_ring, v_ring, displaced, context_lengths, accepted, proposal_count, *,
                        ring_ids=None, window=None, stream=None):
    """Keep only the first accepted[b] of the proposal_count rows the last
    append wrote; restore the slots of the rejected rows from `displaced`."""
    _expect(k_ring, torch.bfloat16, "k_ring")
    _expect(accepted, torch.int32, "accepted")
    num_rings, ring_window, kv_heads, head_dim = k_ring.shape
    batch = context_lengths.shape[0]
    _check(library().carat_ring_rollback(
        _ptr(k_ring), _ptr(v_ring), num_rings, _ptr(ring_ids), _ptr(displaced),
        _ptr(context_lengths), _ptr(accepted), int(proposal_count), batch, kv_heads, head_dim,
        ring_window if window is None else window, _stream(stream)), "carat_ring_rollback")


def carat_global_append_verify_attention(out, queries, key_cache, value_cache, k_new, v_new,
                                         context_lengths, *, scale, workspace, cache_ids=None,
                                         stream=None):
    """Append this step's rows to the global caches and run grouped verify
    attention, in one launch."""
    batch, k, q_heads, head_dim, num_caches, capacity, kv_heads = _attention_args(
        out, queries, key_cache, value_cache, context_lengths, torch.bfloat16,
        "carat_global_append_verify_attention", k_new=k_new, v_new=v_new)
    _check(library().carat_global_append_verify_attention(
        _ptr(out), _ptr(queries), _ptr(key_cache), _ptr(value_cache), num_caches,
        _ptr(cache_ids), _ptr(k_new), _ptr(v_new), _ptr(context_lengths), k, batch, q_heads,
        kv_heads, head_dim, capacity, float(scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "carat_global_append_verify_attention")


def carat_global_append_verify_attention_paged(out, queries, key_pages, value_pages, page_table,
                                               k_new, v_new, context_lengths, *, scale,
                                               workspace, stream=None):
    """Fused append + grouped verify attention over paged global caches.

    key_pages / value_pages bf16 [num_pages][page_rows][Hkv][D]; page_table
    int32 [B][max_pages] (device)."""
    _expect(page_table, torch.int32, "page_table")
    batch, k, q_heads, head_dim, num_pages, page_rows, kv_heads = _attention_args(
        out, queries, key_pages, value_pages, context_lengths, torch.bfloat16,
        "carat_global_append_verify_attention_paged", k_new=k_new, v_new=v_new)
    max_pages = page_table.shape[1]
    _check(library().carat_global_append_verify_attention_paged(
        _ptr(out), _ptr(queries), _ptr(key_pages), _ptr(value_pages), num_pages, _ptr(page_table),
        max_pages, page_rows, _ptr(k_new), _ptr(v_new), _ptr(context_lengths), k, batch,
        q_heads, kv_heads, head_dim, float(scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "carat_global_append_verify_attention_paged")


def carat_paged_append(key_pages, value_pages, page_table, k_new, v_new, context_lengths, *,
                       stream=None):
    """Write rows for positions context_lengths[b] + j through the page table: k_new and
    v_new bf16 [B][k][Hkv][D], a table line and a length for each request (or more)."""
    what = "carat_paged_append"
    for name, t in (("key_pages", key_pages), ("value_pages", value_pages), ("k_new", k_new),
                    ("v_new", v_new)):
        _expect(t, torch.bfloat16, f"{what}: {name}")
        if t.dim() != 4:
            raise ValueError(f"{what}: {name} must be 4-D")
    _expect(page_table, torch.int32, f"{what}: page_table")
    _expect(context_lengths, torch.int32, f"{what}: context_lengths")
    num_pages, page_rows, kv_heads, head_dim = key_pages.shape
    batch, k = k_new.shape[0], k_new.shape[1]
    if value_pages.shape != key_pages.shape:
        raise ValueError(f"{what}: key and value pages differ in shape")
    if tuple(k_new.shape) != (batch, k, kv_heads, head_dim) or v_new.shape != k_new.shape:
        raise ValueError(f"{what}: k_new and v_new must be [batch][k][{kv_heads}][{head_dim}]")
    if page_table.dim() != 2 or page_table.shape[0] < batch or context_lengths.dim() != 1 or \
            context_lengths.shape[0] < batch:
        raise ValueError(f"{what}: page_table and context_lengths must have a line for each of "
                         f"{batch} requests")
    _on_device(what, key_pages=key_pages, value_pages=value_pages, page_table=page_table,
               k_new=k_new, v_new=v_new, context_lengths=context_lengths)
    _check(library().carat_paged_append(
        _ptr(key_pages), _ptr(value_pages), num_pages, _ptr(page_table), page_table.shape[1],
        page_rows, _ptr(k_new), _ptr(v_new), _ptr(context_lengths), k, batch, kv_heads,
        head_dim, _stream(stream)), "carat_paged_append")


class Pool:
    """The library's host-side allocator of a shared pool's page ids."""

    def __init__(self, num_pages: int, pages_per_ring: int):
        self._lib = library()
        self._h = self._lib.carat_pool_create(int(num_pages), int(pages_per_ring))
        if not self._h:
            raise CaratError(CARAT_ERR_INVALID_ARG, "carat_pool_create")
        self.num_pages, self.pages_per_ring = int(num_pages), int(pages_per_ring)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            self._lib.carat_pool_destroy(h)
            self._h = None

    def alloc_ring(self) -> int:
        """Ring id (first page / pages_per_ring) of a whole free block, or -1."""
        return int(self._lib.carat_pool_alloc_ring(self._h))

    def free_ring(self, ring_id: int) -> bool:
        return self._lib.carat_pool_free_ring(self._h, int(ring_id)) == 0

    def alloc_pages(self, n: int):
        """n page ids, or None (nothing allocated) if fewer than n are free."""
        buf = (ctypes.c_int32 * max(int(n), 1))()
        got = self._lib.carat_pool_alloc_pages(self._h, int(n), buf)
        return None if got < 0 else [int(buf[i]) for i in range(got)]

    def free_pages(self, pages) -> bool:
        pages = list(pages)
        buf = (ctypes.c_int32 * max(len(pages), 1))(*pages)
        return self._lib.carat_pool_free_pages(self._h, len(pages), buf) == 0

    def share_pages(self, pages) -> bool:
        """One more owner for every listed page; free_pages takes one away."""
        pages = list(pages)
        buf = (ctypes.c_int32 * max(len(pages), 1))(*pages)
        return self._lib.carat_pool_share_pages(self._h, len(pages), buf) == 0

    def plan_compaction(self, max_moves: int):
        """(sources, destinations) of page moves that empty broken-up blocks.  The
        allocator counts them as done; carat_pages_move carries them out."""
        n = max(0, min(int(max_moves), self.num_pages))
        src, dst = (ctypes.c_int32 * max(n, 1))(), (ctypes.c_int32 * max(n, 1))()
        got = self._lib.carat_pool_plan_compaction(self._h, n, src, dst)
        if got < 0:
            raise CaratError(CARAT_ERR_INVALID_ARG, "carat_pool_plan_compaction")
        return list(src[:got]), list(dst[:got])

    def stats(self) -> dict:
        out = (ctypes.c_int32 * 4)()
        _check(0 if self._lib.carat_pool_stats(self._h, out) == 0 else CARAT_ERR_INVALID_ARG,
               "carat_pool_stats")
        return {"free_pages": out[0], "whole_free_blocks": out[1], "rings": out[2],
                "pages": out[3]}


def carat_get_device_status(clear: bool = True, stream=None) -> int:
    v = ctypes.c_int32(0)
    _check(library().carat_get_device_status(ctypes.byref(v), 1 if clear else 0, _stream(stream)),
           "carat_get_device_status")
    return int(v.value)


def carat_check_bounded_wait(limit_ns: int, stream=None) -> None:
    """Run the self-check of the library's bounded waits: a kernel waits on a
    barrier phase nothing completes, gives up after limit_ns and sets
    CARAT_DEV_TIMEOUT in the device status word (read it with
    carat_get_device_status)."""
    _check(library().carat_check_bounded_wait(ctypes.c_uint64(int(limit_ns)), _stream(stream)),
           "carat_check_bounded_wait")


def carat_launch_floor(dependent: bool = False, stream=None) -> None:
    """Launch one empty kernel (and, with dependent, an empty dependent launch
    after it): the floor under a call's measured time."""
    _check(library().carat_launch_floor(1 if dependent else 0, _stream(stream)),
           "carat_launch_floor")


def kernel_launches() -> int:
    """Kernels libcarat.so has launched in this process so far."""
    return int(library().carat_kernel_launches())


def workspace_tensor(nbytes: int, device=None) -> torch.Tensor:
    """A 256-byte aligned uint8 CUDA tensor of at least nbytes (torch owns it)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


# ---------------------------------------------------------------------------
# FP8 (e4m3) rings: uint8 tensors, one dequantisation scale per tensor
# ---------------------------------------------------------------------------

def carat_ring_append_fp8(k_ring, v_ring, k_new, v_new, context_lengths, *, k_scale, v_scale,
                          ring_ids=None, displaced=None, window=None, stream=None):
    """carat_ring_append into e4m3 rings (uint8 [num_rings][window][Hkv][D]);
    new rows stay bf16 and are quantised as e4m3(fp32(x * fp32(1/scale)))."""
    _expect(k_ring, torch.uint8, "k_ring")
    _expect(v_ring, torch.uint8, "v_ring")
    _expect(k_new, torch.bfloat16, "k_new")
    _expect(context_lengths, torch.int32, "context_lengths")
    if displaced is not None:
        _expect(displaced, torch.uint8, "displaced")
    num_rings, ring_window, kv_heads, head_dim = k_ring.shape
    batch, k = k_new.shape[0], k_new.shape[1]
    _check(library().carat_ring_append_fp8(
        _ptr(k_ring), _ptr(v_ring), num_rings, _ptr(ring_ids), _ptr(k_new), _ptr(v_new),
        _ptr(context_lengths), k, _ptr(displaced), batch, kv_heads, head_dim,
        ring_window if window is None else window, float(k_scale), float(v_scale),
        _stream(stream)), "carat_ring_append_fp8")


def carat_ring_rollback_fp8(k_ring, v_ring, displaced, context_lengths, accepted,
                            proposal_count, *, ring_ids=None, window=None, stream=None):
    """carat_ring_rollback for e4m3 rings and their uint8 displaced rows."""
    _expect(k_ring, torch.uint8, "k_ring")
    _expect(accepted, torch.int32, "accepted")
    num_rings, ring_window, kv_heads, head_dim = k_ring.shape
    batch = context_lengths.shape[0]
    _check(library().carat_ring_rollback_fp8(
        _ptr(k_ring), _ptr(v_ring), num_rings, _ptr(ring_ids), _ptr(displaced),
        _ptr(context_lengths), _ptr(accepted), int(proposal_count), batch, kv_heads, head_dim,
        ring_window if window is None else window, _stream(stream)), "carat_ring_rollback_fp8")


def carat_swa_attention_fp8(out, queries, k_ring, v_ring, context_lengths, *, scale, k_scale,
                            v_scale, workspace, ring_ids=None, displaced=None, stream=None):
    """Sliding-window attention over e4m3 rings (dequantised: byte value x scale)."""
    batch, k, q_heads, head_dim, num_rings, window, kv_heads = _attention_args(
        out, queries, k_ring, v_ring, context_lengths, torch.uint8, "carat_swa_attention_fp8",
        displaced=displaced)
    _check(library().carat_swa_attention_fp8(
        _ptr(out), _ptr(queries), _ptr(k_ring), _ptr(v_ring), num_rings, _ptr(ring_ids),
        _ptr(displaced), _ptr(context_lengths), k, batch, q_heads, kv_heads, head_dim, window,
        float(scale), float(k_scale), float(v_scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "carat_swa_attention_fp8")


# ---------------------------------------------------------------------------
# Rotary paged appends, and attention over e4m3 pages with a scale per block of
# tokens and KV head
# ---------------------------------------------------------------------------

def _on_device(what, **tensors):
    """Every tensor given is on the current CUDA device (a kernel would fault on
    a host pointer)."""
    device = torch.cuda.current_device()
    for name, t in tensors.items():
        if t is not None and not (t.is_cuda and t.get_device() == device):
            raise ValueError(f"{what}: {name} must be on the current CUDA device")


_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
# The current stream's handle and the current device without the objects torch
# makes for them (a call here is a few microseconds of host work in all).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_of(stream, device):
    return _raw_stream(device) if stream is None else _stream(stream)


def _plain(device, dtype, *tensors):
    """Every tensor is a contiguous one of this type on this device."""
    for t in tensors:
        if not (t.dtype is dtype and t.get_device() == device and t.is_contiguous()):
            return False
    return True


def _tokens(t, heads, head_dim, batch, k, name):
    """(pointer, token stride in elements) of a [B][k][heads][head_dim] tensor
    whose tokens are dense rows a fixed stride apart."""
    _expect(t, torch.bfloat16, name)
    if tuple(t.shape) != (batch, k, heads, head_dim):
        raise ValueError(f"{name} must be [batch][k][heads][head_dim] = "
                         f"{(batch, k, heads, head_dim)}, got {tuple(t.shape)}")
    s0, s1, s2, s3 = t.stride()
    if k == 1:
        s1 = s0 if batch > 1 else heads * head_dim
    if (head_dim > 1 and s3 != 1) or (heads > 1 and s2 != head_dim) or \
            (batch > 1 and s0 != k * s1):
        raise ValueError(f"{name}: a token's heads must be dense and its tokens equally spaced")
    return ctypes.c_void_p(t.data_ptr()), s1


def _paged_pool(key_pages, value_pages, page_table, context_lengths, dtype, batch, what):
    _expect(key_pages, dtype, f"{what}: key_pages")
    _expect(value_pages, dtype, f"{what}: value_pages")
    _expect(page_table, torch.int32, f"{what}: page_table")
    _expect(context_lengths, torch.int32, f"{what}: context_lengths")
    if key_pages.dim() != 4 or key_pages.shape != value_pages.shape:
        raise ValueError(f"{what}: key and value pages must be 4-D and alike")
    if page_table.dim() != 2 or page_table.shape[0] != batch:
        raise ValueError(f"{what}: page_table must be [batch][max_pages]")
    if tuple(context_lengths.shape) != (batch,):
        raise ValueError(f"{what}: context_lengths must be [batch]")
    return key_pages.shape


def _block_scales(k_scales, v_scales, num_pages, page_rows, kv_heads, what):
    """block_rows from the shape of the scales [num_pages][blocks][kv_heads]."""
    shape = k_scales.shape
    if len(shape) == 3 and shape[0] == num_pages and shape[2] == kv_heads and shape[1] > 0 and \
            page_rows % shape[1] == 0 and v_scales.shape == shape and \
            k_scales.dtype is _F32 and v_scales.dtype is _F32:
        return page_rows // shape[1]
    _expect(k_scales, torch.float32, f"{what}: k_scales")
    _expect(v_scales, torch.float32, f"{what}: v_scales")
    if k_scales.dim() != 3 or k_scales.shape != v_scales.shape or \
            k_scales.shape[0] != num_pages or k_scales.shape[2] != kv_heads or \
            k_scales.shape[1] < 1 or page_rows % k_scales.shape[1]:
        raise ValueError(f"{what}: scales must be [num_pages][page_rows / block_rows][kv_heads]")
    return page_rows // k_scales.shape[1]


def _rope_args(what, dtype, key_pages, value_pages, page_table, k_new, v_new, context_lengths,
               cos_sin, queries, queries_out, positions, new_counts, k_scales=None,
               v_scales=None):
    """The entry points' arguments.  The usual layout is recognised at once; any
    other goes through _rope_args_slow, which says what is wrong with it."""
    slow = (what, dtype, key_pages, value_pages, page_table, k_new, v_new, context_lengths,
            cos_sin, queries, queries_out, positions, new_counts, k_scales, v_scales)
    try:
        pool, new = key_pages.shape, k_new.shape
        num_pages, page_rows, kv_heads, head_dim = pool
        batch, k, h, d = new
        strides = k_new.stride()
        s0, s1, s2, s3 = strides
        rows, max_pages = page_table.shape
        table_rows, rotary_dim = cos_sin.shape
        device = key_pages.get_device()
        if not (h == kv_heads and d == head_dim and rows == batch and value_pages.shape == pool and
                v_new.shape == new and v_new.stride() == strides and s3 == 1 and s2 == d and
                s0 == k * s1 and k_new.dtype is _BF16 and v_new.dtype is _BF16 and
                k_new.get_device() == device and v_new.get_device() == device and
                device == _device() and context_lengths.shape == (batch,) and
                _plain(device, dtype, key_pages, value_pages) and
                _plain(device, _I32, page_table, context_lengths) and
                _plain(device, _F32, cos_sin)):
            return _rope_args_slow(*slow)
        q_heads, qp, qo, q_stride = 0, None, None, 0
        if queries is not None:
            qshape = queries.shape
            qb, qk, q_heads, qd = qshape
            t0, q_stride, t2, t3 = queries.stride()
            if not (qb == batch and qk == k and qd == d and t3 == 1 and t2 == d and
                    t0 == k * q_stride and queries.dtype is _BF16 and
                    queries.get_device() == device and queries_out.shape == qshape and
                    _plain(device, _BF16, queries_out)):
                return _rope_args_slow(*slow)
            qp, qo = queries.data_ptr(), queries_out.data_ptr()
        elif queries_out is not None:
            return _rope_args_slow(*slow)
        pp = cp = None
        if positions is not None:
            if positions.shape != (batch, k) or not _plain(device, _I32, positions):
                return _rope_args_slow(*slow)
            pp = positions.data_ptr()
        if new_counts is not None:
            if new_counts.shape != (batch,) or not _plain(device, _I32, new_counts):
                return _rope_args_slow(*slow)
            cp = new_counts.data_ptr()
        if k_scales is not None and not _plain(device, _F32, k_scales, v_scales):
            return _rope_args_slow(*slow)
    except (AttributeError, TypeError, ValueError):
        return _rope_args_slow(*slow)
    return ((num_pages, page_table.data_ptr(), max_pages, page_rows),
            (k_new.data_ptr(), v_new.data_ptr(), s1, qo, qp, q_stride, cos_sin.data_ptr(),
             table_rows, rotary_dim),
            (pp, cp, context_lengths.data_ptr(), k, batch, q_heads, kv_heads, head_dim), device)


def _rope_args_slow(what, dtype, key_pages, value_pages, page_table, k_new, v_new,
                    context_lengths, cos_sin, queries, queries_out, positions, new_counts,
                    k_scales, v_scales):
    if k_new.dim() != 4:
        raise ValueError(f"{what}: k_new must be [batch][k][kv_heads][head_dim]")
    batch, k = k_new.shape[0], k_new.shape[1]
    num_pages, page_rows, kv_heads, head_dim = _paged_pool(
        key_pages, value_pages, page_table, context_lengths, dtype, batch, what)
    _expect(cos_sin, torch.float32, f"{what}: cos_sin")
    if cos_sin.dim() != 2:
        raise ValueError(f"{what}: cos_sin must be [table_rows][rotary_dim]")
    kp, kv_stride = _tokens(k_new, kv_heads, head_dim, batch, k, f"{what}: k_new")
    vp, v_stride = _tokens(v_new, kv_heads, head_dim, batch, k, f"{what}: v_new")
    if kv_stride != v_stride:
        raise ValueError(f"{what}: k_new and v_new must have one token stride")
    q_heads, qp, q_stride = 0, None, 0
    if (queries is None) != (queries_out is None):
        raise ValueError(f"{what}: queries and queries_out go together")
    if queries is not None:
        if queries.dim() != 4:
            raise ValueError(f"{what}: queries must be [batch][k][q_heads][head_dim]")
        q_heads = queries.shape[2]
        qp, q_stride = _tokens(queries, q_heads, head_dim, batch, k, f"{what}: queries")
        _expect(queries_out, torch.bfloat16, f"{what}: queries_out")
        if queries_out.shape != queries.shape:
            raise ValueError(f"{what}: queries_out must have the queries' shape")
    if positions is not None:
        _expect(positions, torch.int32, f"{what}: positions")
        if tuple(positions.shape) != (batch, k):
            raise ValueError(f"{what}: positions must be [batch][k]")
    if new_counts is not None:
        _expect(new_counts, torch.int32, f"{what}: new_counts")
        if tuple(new_counts.shape) != (batch,):
            raise ValueError(f"{what}: new_counts must be [batch]")
    _on_device(what, key_pages=key_pages, value_pages=value_pages, page_table=page_table,
               k_new=k_new, v_new=v_new, context_lengths=context_lengths, cos_sin=cos_sin,
               queries=queries, queries_out=queries_out, positions=positions,
               new_counts=new_counts, k_scales=k_scales, v_scales=v_scales)
    head = (num_pages, _ptr(page_table), page_table.shape[1], page_rows)
    tail = (kp, vp, kv_stride, _ptr(queries_out), qp, q_stride, _ptr(cos_sin), cos_sin.shape[0],
            cos_sin.shape[1])
    rest = (_ptr(positions), _ptr(new_counts), _ptr(context_lengths), k, batch, q_heads, kv_heads,
            head_dim)
    for t in (key_pages, value_pages, k_scales, v_scales):
        _ptr(t)
    return head, tail, rest, key_pages.get_device()


def carat_paged_rope_append(key_pages, value_pages, page_table, k_new, v_new, context_lengths, *,
                            cos_sin, interleaved=False, queries=None, queries_out=None,
                            positions=None, new_counts=None, stream=None):
    """Rotate this step's keys (and queries, into queries_out) and write keys and
    values into bf16 pages [num_pages][page_rows][Hkv][D] at positions
    context_lengths[b] + j.

    k_new, v_new bf16 [B][k][Hkv][D] and queries bf16 [B][k][Hq][D] may be parts
    of a fused projection's output: a token's heads are dense, tokens a fixed
    stride apart.  cos_sin fp32 [table_rows][rotary_dim] (engine.rotary_table).
    positions int32 [B][k] (angles only; default context_lengths[b] + j);
    new_counts int32 [B]: rows request b really appends (default k)."""
    what = "carat_paged_rope_append"
    head, tail, rest, device = _rope_args(
        what, _BF16, key_pages, value_pages, page_table, k_new, v_new, context_lengths, cos_sin,
        queries, queries_out, positions, new_counts)
    _check((_lib or library()).carat_paged_rope_append(
        key_pages.data_ptr(), value_pages.data_ptr(), *head, *tail, 1 if interleaved else 0, *rest,
        _stream_of(stream, device)), what)


def carat_paged_rope_append_fp8(key_pages, value_pages, k_scales, v_scales, page_table, k_new,
                                v_new, context_lengths, *, cos_sin, interleaved=False,
                                queries=None, queries_out=None, positions=None, new_counts=None,
                                stream=None):
    """carat_paged_rope_append into e4m3 pages (uint8) with one power-of-two
    scale per block of tokens and KV head: k_scales, v_scales fp32
    [num_pages][page_rows / block_rows][Hkv], block_rows 16, 32, 64 or 128.  A
    block that starts in this call takes the least scale that holds its rows;
    one that already held rows keeps its scale or grows it, its older bytes
    then being rounded to the new one."""
    what = "carat_paged_rope_append_fp8"
    head, tail, rest, device = _rope_args(
        what, _U8, key_pages, value_pages, page_table, k_new, v_new, context_lengths, cos_sin,
        queries, queries_out, positions, new_counts, k_scales, v_scales)
    block_rows = _block_scales(k_scales, v_scales, head[0], head[3], rest[6], what)
    _check((_lib or library()).carat_paged_rope_append_fp8(
        key_pages.data_ptr(), value_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
        *head, block_rows, *tail, 1 if interleaved else 0, *rest, _stream_of(stream, device)), what)


def carat_global_verify_attention_paged(out, queries, key_pages, value_pages, page_table,
                                        context_lengths, *, scale, workspace, stream=None):
    """Grouped causal verify attention over bf16 pages that already hold this
    step's rows (e.g. after carat_paged_rope_append); out fp32 [B][k][Hq][D]."""
    what = "carat_global_verify_attention_paged"
    batch, k, q_heads, head_dim, num_pages, page_rows, kv_heads = _attention_args(
        out, queries, key_pages, value_pages, context_lengths, torch.bfloat16, what)
    _paged_pool(key_pages, value_pages, page_table, context_lengths, torch.bfloat16, batch, what)
    _on_device(what, out=out, queries=queries, key_pages=key_pages, value_pages=value_pages,
               page_table=page_table, context_lengths=context_lengths, workspace=workspace)
    _check(library().carat_global_verify_attention_paged(
        _ptr(out), _ptr(queries), _ptr(key_pages), _ptr(value_pages), num_pages, _ptr(page_table),
        page_table.shape[1], page_rows, _ptr(context_lengths), k, batch, q_heads, kv_heads,
        head_dim, float(scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), what)


def paged_fp8_workspace_bytes(batch, proposal_count, q_heads, kv_heads, head_dim, capacity) -> int:
    return int(library().carat_paged_fp8_workspace_bytes(batch, proposal_count, q_heads, kv_heads,
                                                         head_dim, capacity))


def carat_paged_verify_attention_fp8(out, queries, key_pages, value_pages, k_scales, v_scales,
                                     page_table, context_lengths, *, scale, workspace, window=0,
                                     new_counts=None, stream=None):
    """Decode / verify attention over e4m3 pages with block scales (as
    carat_paged_rope_append_fp8 writes them) that already hold this step's rows.

    out and queries bf16 [B][k][Hq][D]; window 0: every position up to the
    query's own, w > 0: the last w of them; new_counts int32 [B]: the queries
    request b really has (default k; rows of out behind them stay as they are);
    workspace: a CUDA tensor of at least paged_fp8_workspace_bytes(...) bytes."""
    what = "carat_paged_verify_attention_fp8"
    counts = None
    try:
        shape, pool = queries.shape, key_pages.shape
        batch, k, q_heads, head_dim = shape
        num_pages, page_rows, kv_heads, cache_dim = pool
        rows, max_pages = page_table.shape
        device = queries.get_device()
        usual = (cache_dim == head_dim and rows == batch and out.shape == shape and
                 value_pages.shape == pool and context_lengths.shape == (batch,) and
                 device == _device() and workspace.get_device() == device and
                 workspace.is_contiguous() and _plain(device, _BF16, out, queries) and
                 _plain(device, _U8, key_pages, value_pages) and
                 _plain(device, _I32, page_table, context_lengths) and
                 _plain(device, _F32, k_scales, v_scales))
        if new_counts is not None:
            usual = usual and new_counts.shape == (batch,) and _plain(device, _I32, new_counts)
            counts = new_counts.data_ptr()
    except (AttributeError, TypeError, ValueError):
        usual = False
    if not usual:
        _paged_fp8_explain(what, out, queries, key_pages, value_pages, k_scales, v_scales,
                           page_table, context_lengths, workspace, new_counts)
    block_rows = _block_scales(k_scales, v_scales, num_pages, page_rows, kv_heads, what)
    _check((_lib or library()).carat_paged_verify_attention_fp8(
        out.data_ptr(), queries.data_ptr(), key_pages.data_ptr(), value_pages.data_ptr(),
        k_scales.data_ptr(), v_scales.data_ptr(), num_pages, page_table.data_ptr(), max_pages,
        page_rows, block_rows, counts, context_lengths.data_ptr(), k, batch, q_heads, kv_heads,
        head_dim, max(-1, min(int(window), 0x7fffffff)), float(scale), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_of(stream, device)), what)


def _paged_fp8_explain(what, out, queries, key_pages, value_pages, k_scales, v_scales, page_table,
                       context_lengths, workspace, new_counts):
    """Raises what is wrong with the arguments."""
    _expect(out, torch.bfloat16, f"{what}: out")
    _expect(queries, torch.bfloat16, f"{what}: queries")
    if queries.dim() != 4 or out.shape != queries.shape:
        raise ValueError(f"{what}: queries must be [batch][k][q_heads][head_dim], out alike")
    batch, head_dim = queries.shape[0], queries.shape[3]
    num_pages, page_rows, kv_heads, cache_dim = _paged_pool(
        key_pages, value_pages, page_table, context_lengths, torch.uint8, batch, what)
    if cache_dim != head_dim:
        raise ValueError(f"{what}: cache head_dim {cache_dim} != query head_dim {head_dim}")
    _block_scales(k_scales, v_scales, num_pages, page_rows, kv_heads, what)
    if new_counts is not None:
        _expect(new_counts, torch.int32, f"{what}: new_counts")
        if tuple(new_counts.shape) != (batch,):
            raise ValueError(f"{what}: new_counts must be [batch]")
    _on_device(what, out=out, queries=queries, key_pages=key_pages, value_pages=value_pages,
               k_scales=k_scales, v_scales=v_scales, page_table=page_table,
               context_lengths=context_lengths, workspace=workspace, new_counts=new_counts)
    for t in (out, queries, key_pages, value_pages, k_scales, v_scales, page_table,
              context_lengths, workspace, new_counts):
        _ptr(t)
    raise ValueError(f"{what}: arguments do not fit together")


# ---------------------------------------------------------------------------
# Attention of a chunk of new tokens over bf16 pages
# ---------------------------------------------------------------------------

def paged_chunk_workspace_bytes(batch, proposal_count, q_heads, kv_heads, head_dim) -> int:
    return int(library().carat_paged_chunk_workspace_bytes(batch, proposal_count, q_heads,
                                                           kv_heads, head_dim))


def _int32(x):
    """An integer as a C int; one past its range keeps its sign."""
    return max(-1, min(int(x), 0x7fffffff))


def carat_paged_chunk_attention(out, queries, key_pages, value_pages, page_table, context_lengths,
                                *, scale, workspace=None, window=0, sinks=0, new_counts=None,
                                stream=None):
    """Attention of a chunk of new tokens (a prompt, a part of one, a decode or verify
    step) over bf16 pages [num_pages][page_rows][Hkv][D] that already hold their rows.

    out and queries bf16 [B][k][Hq][D], any k up to the capacity; window 0: every
    position up to the query's own, w > 0: the last w of them and the request's first
    `sinks` tokens; new_counts int32 [B]: the queries request b really has (default k;
    rows of out behind them stay as they are); workspace: a CUDA tensor of at least
    paged_chunk_workspace_bytes(...) bytes (None where that is 0)."""
    what = "carat_paged_chunk_attention"
    counts = None
    try:
        shape, pool = queries.shape, key_pages.shape
        batch, k, q_heads, head_dim = shape
        num_pages, page_rows, kv_heads, cache_dim = pool
        rows, max_pages = page_table.shape
        device = queries.get_device()
        usual = (cache_dim == head_dim and rows == batch and out.shape == shape and
                 value_pages.shape == pool and context_lengths.shape == (batch,) and
                 device == _device() and
                 _plain(device, _BF16, out, queries, key_pages, value_pages) and
                 _plain(device, _I32, page_table, context_lengths))
        if workspace is not None:
            usual = usual and workspace.get_device() == device and workspace.is_contiguous()
        if new_counts is not None:
            usual = usual and new_counts.shape == (batch,) and _plain(device, _I32, new_counts)
            counts = new_counts.data_ptr()
    except (AttributeError, TypeError, ValueError):
        usual = False
    if not usual:
        _paged_chunk_explain(what, out, queries, key_pages, value_pages, page_table,
                             context_lengths, workspace, new_counts)
    space, room = ((None, 0) if workspace is None else
                   (workspace.data_ptr(), workspace.numel() * workspace.element_size()))
    _check((_lib or library()).carat_paged_chunk_attention(
        out.data_ptr(), queries.data_ptr(), key_pages.data_ptr(), value_pages.data_ptr(),
        num_pages, page_table.data_ptr(), max_pages, page_rows, counts,
        context_lengths.data_ptr(), k, batch, q_heads, kv_heads, head_dim, _int32(window),
        _int32(sinks), float(scale), space, room, _stream_of(stream, device)), what)


def _paged_chunk_explain(what, out, queries, key_pages, value_pages, page_table, context_lengths,
                         workspace, new_counts):
    """Raises what is wrong with the arguments."""
    _expect(out, torch.bfloat16, f"{what}: out")
    _expect(queries, torch.bfloat16, f"{what}: queries")
    if queries.dim() != 4 or out.shape != queries.shape:
        raise ValueError(f"{what}: queries must be [batch][k][q_heads][head_dim], out alike")
    pool = _paged_pool(key_pages, value_pages, page_table, context_lengths, torch.bfloat16,
                       queries.shape[0], what)
    if pool[3] != queries.shape[3]:
        raise ValueError(f"{what}: cache head_dim {pool[3]} != query head_dim {queries.shape[3]}")
    if new_counts is not None:
        _expect(new_counts, torch.int32, f"{what}: new_counts")
        if tuple(new_counts.shape) != (queries.shape[0],):
            raise ValueError(f"{what}: new_counts must be [batch]")
    _on_device(what, out=out, queries=queries, key_pages=key_pages, value_pages=value_pages,
               page_table=page_table, context_lengths=context_lengths, workspace=workspace,
               new_counts=new_counts)
    for t in (out, queries, key_pages, value_pages, page_table, context_lengths, workspace,
              new_counts):
        _ptr(t)
    raise ValueError(f"{what}: arguments do not fit together")


# ---------------------------------------------------------------------------
# Operators on the pages of a pool
# ---------------------------------------------------------------------------

def hidden_pages(context_length: int, window: int, sinks: int, page_rows: int):
    """(first, end) of the entries of a request's page table whose pages no query at or
    behind position context_length sees any more under a sliding window with `sinks`
    first tokens: they can be freed (carat_pool_free_pages).  Empty without a window."""
    if window <= 0:
        return 0, 0
    first = -(-int(sinks) // page_rows)
    end = max(0, int(context_length) - int(window) + 1) // page_rows
    return (first, end) if end > first else (first, first)


def _page_args(what, key_pages, value_pages, k_scales, v_scales, lists, tables=None,
               num_pages=None):
    """The leading arguments of the operators on pages.  key_pages None (a move whose
    bytes have been moved already): the scales' shape, or num_pages, gives the pool."""
    if (k_scales is None) != (v_scales is None):
        raise ValueError(f"{what}: k_scales and v_scales go together")
    if (key_pages is None) != (value_pages is None):
        raise ValueError(f"{what}: key_pages and value_pages go together")
    first = next(iter(lists.values()))
    device = first.get_device()
    if key_pages is None:
        page_rows, row_bytes, block_rows, kv_heads = 1, 16, 0, 1
        if k_scales is not None:
            _expect(k_scales, torch.float32, f"{what}: k_scales")
            _expect(v_scales, torch.float32, f"{what}: v_scales")
            if k_scales.dim() != 3 or k_scales.shape != v_scales.shape:
                raise ValueError(f"{what}: scales must be 3-D and alike")
            num_pages, page_rows, kv_heads = k_scales.shape
            block_rows = 1
        if num_pages is None:
            raise ValueError(f"{what}: num_pages is needed without pages and scales")
    else:
        if key_pages.dtype not in (_BF16, _U8):
            raise TypeError(f"{what}: pages must be bf16 or uint8 (e4m3), got {key_pages.dtype}")
        _expect(value_pages, key_pages.dtype, f"{what}: value_pages")
        if key_pages.dim() != 4 or key_pages.shape != value_pages.shape:
            raise ValueError(f"{what}: key and value pages must be 4-D and alike")
        num_pages, page_rows, kv_heads, head_dim = key_pages.shape
        row_bytes = kv_heads * head_dim * key_pages.element_size()
        block_rows = 0
        if k_scales is not None:
            block_rows = _block_scales(k_scales, v_scales, num_pages, page_rows, kv_heads, what)
    for name, t in lists.items():
        if t is not None:
            _expect(t, torch.int32, f"{what}: {name}")
            _ptr(t)
            if t.dim() != 1 or t.shape != first.shape:
                raise ValueError(f"{what}: {name} must be one-dimensional, all lists alike")
    _on_device(what, key_pages=key_pages, value_pages=value_pages, k_scales=k_scales,
               v_scales=v_scales, **lists, **(tables or {}))
    return (_ptr(key_pages), _ptr(value_pages), _ptr(k_scales), _ptr(v_scales), int(num_pages),
            page_rows, row_bytes, block_rows, kv_heads), device


def _page_head(key_pages, value_pages, k_scales, v_scales):
    """(device, leading arguments) of the usual call, or None: _page_args says why."""
    try:
        pool = key_pages.shape
        num_pages, page_rows, kv_heads, head_dim = pool
        dtype, device = key_pages.dtype, key_pages.get_device()
        if device != _device() or value_pages.shape != pool or \
                not _plain(device, dtype, key_pages, value_pages):
            return None
        row_bytes = kv_heads * head_dim
        if dtype is _BF16:
            row_bytes *= 2
        elif dtype is not _U8:
            return None
        if k_scales is None:
            if v_scales is not None:
                return None
            return device, (key_pages.data_ptr(), value_pages.data_ptr(), None, None, num_pages,
                            page_rows, row_bytes, 0, kv_heads)
        shape = k_scales.shape
        pages, blocks, heads = shape
        if pages != num_pages or heads != kv_heads or blocks < 1 or page_rows % blocks or \
                v_scales.shape != shape or not _plain(device, _F32, k_scales, v_scales):
            return None
        return device, (key_pages.data_ptr(), value_pages.data_ptr(), k_scales.data_ptr(),
                        v_scales.data_ptr(), num_pages, page_rows, row_bytes, page_rows // blocks,
                        kv_heads)
    except (AttributeError, TypeError, ValueError):
        return None


def _lists(device, shape, *lists):
    """Every list is a contiguous int32 one of this shape on this device."""
    for t in lists:
        if not (t.shape == shape and t.dtype is _I32 and t.get_device() == device and
                t.is_contiguous()):
            return False
    return True


def carat_pages_copy(key_pages, value_pages, src, dst, *, rows=None, k_scales=None, v_scales=None,
                     stream=None):
    """Copy the first rows[i] rows (default: all) of page src[i] into page dst[i], keys,
    values and (e4m3 pages, uint8) the scales of their blocks.  src, dst, rows: int32
    lists on the device; a source below 0 is skipped."""
    what = "carat_pages_copy"
    usual = _page_head(key_pages, value_pages, k_scales, v_scales)
    if usual is not None and len(src.shape) == 1 and _lists(usual[0], src.shape, src, dst) and \
            (rows is None or _lists(usual[0], src.shape, rows)):
        device, head = usual
    else:
        head, device = _page_args(what, key_pages, value_pages, k_scales, v_scales,
                                  {"src": src, "dst": dst, "rows": rows})
    _check((_lib or library()).carat_pages_copy(
        *head, src.data_ptr(), dst.data_ptr(), None if rows is None else rows.data_ptr(),
        src.shape[0], _stream_of(stream, device)), what)


def carat_paged_fork(key_pages, value_pages, page_table, context_lengths, child_table, parents,
                     new_pages, *, child_lengths=None, k_scales=None, v_scales=None, stream=None):
    """Children of requests: child i's line of child_table takes over the whole pages of
    request parents[i], and the rows of its last, partly filled page are copied into page
    new_pages[i] (below 0: the child takes that page itself).  child_lengths[i] (optional)
    becomes the parent's context length."""
    what = "carat_paged_fork"
    usual = _page_head(key_pages, value_pages, k_scales, v_scales)
    lines = page_table.shape
    if usual is not None and len(lines) == 2 and len(parents.shape) == 1 and \
            _lists(usual[0], parents.shape, parents, new_pages) and \
            _lists(usual[0], lines, page_table) and \
            _lists(usual[0], lines[:1], context_lengths) and \
            _lists(usual[0], (parents.shape[0], lines[1]), child_table) and \
            (child_lengths is None or _lists(usual[0], parents.shape, child_lengths)):
        device, head = usual
    else:
        head, device = _fork_args(what, key_pages, value_pages, page_table, context_lengths,
                                  child_table, parents, new_pages, child_lengths, k_scales, v_scales)
    _check((_lib or library()).carat_paged_fork(
        *head, page_table.data_ptr(), lines[0], lines[1], context_lengths.data_ptr(),
        child_table.data_ptr(), None if child_lengths is None else child_lengths.data_ptr(),
        parents.data_ptr(), new_pages.data_ptr(), parents.shape[0], _stream_of(stream, device)),
        what)


def _fork_args(what, key_pages, value_pages, page_table, context_lengths, child_table, parents,
               new_pages, child_lengths, k_scales, v_scales):
    head, device = _page_args(
        what, key_pages, value_pages, k_scales, v_scales,
        {"parents": parents, "new_pages": new_pages, "child_lengths": child_lengths},
        {"page_table": page_table, "context_lengths": context_lengths, "child_table": child_table})
    for name, t in (("page_table", page_table), ("context_lengths", context_lengths),
                    ("child_table", child_table)):
        _expect(t, torch.int32, f"{what}: {name}")
        _ptr(t)
    if page_table.dim() != 2 or child_table.dim() != 2 or \
            child_table.shape[1] != page_table.shape[1] or \
            child_table.shape[0] != parents.shape[0]:
        raise ValueError(f"{what}: child_table must be [children][max_pages]")
    if tuple(context_lengths.shape) != (page_table.shape[0],):
        raise ValueError(f"{what}: context_lengths must be [parents' batch]")
    return head, device


def carat_pages_move(key_pages, value_pages, src, dst, *, page_table=None, k_scales=None,
                     v_scales=None, num_pages=None, stream=None):
    """Move whole pages src[i] to dst[i] (Pool.plan_compaction's list) and make every entry
    of page_table that names src[i] name dst[i].  key_pages and value_pages None: the bytes
    have been moved already, only scales and table follow (num_pages: the pool's, where
    there are no scales to tell)."""
    what = "carat_pages_move"
    usual = _page_head(key_pages, value_pages, k_scales, v_scales)
    if usual is not None and len(src.shape) == 1 and _lists(usual[0], src.shape, src, dst) and \
            (page_table is None or _lists(usual[0], page_table.shape, page_table)):
        device, head = usual
    else:
        if page_table is not None:
            _expect(page_table, torch.int32, f"{what}: page_table")
            _ptr(page_table)
        head, device = _page_args(what, key_pages, value_pages, k_scales, v_scales,
                                  {"src": src, "dst": dst}, {"page_table": page_table}, num_pages)
    table, entries = (None, 0) if page_table is None else (page_table.data_ptr(),
                                                           page_table.numel())
    _check((_lib or library()).carat_pages_move(
        *head, src.data_ptr(), dst.data_ptr(), src.shape[0], table, entries,
        _stream_of(stream, device)), what)
