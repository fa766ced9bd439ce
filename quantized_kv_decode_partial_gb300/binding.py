"""Thin Python binding of libpkvdecode.so (include/pkv_decode.h).

Argument marshalling only: shapes are read off the tensors, pointers and the
current CUDA stream are passed through, and PyTorch allocates the output and
the workspace (held between calls on the default stream, one per host thread
and device, up to 32 MB). Every step of the computation runs in the library's kernels;
there is no fallback, and a missing library raises ``LibraryNotBuilt``.
"""

from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple, Optional

import torch

from .build import LIB_PATH

EXPORTS = (
    "pkv_make_plan",
    "pkv_plan_for_current_device",
    "pkv_paged_decode_attention",
    "pkv_paged_decode_partial",
    "pkv_merge_partitions",
    "pkv_paged_decode_attention_no_alloc",
    "pkv_paged_decode_attention_host",
    "pkv_step_create",
    "pkv_step_run",
    "pkv_step_destroy",
    "pkv_paged_decode_append_attention",
    "pkv_paged_append",
    "pkv_make_sparse_plan",
    "pkv_sparse_plan_for_current_device",
    "pkv_update_block_bounds",
    "pkv_select_blocks",
    "pkv_selected_decode_attention",
    "pkv_sparse_decode_attention",
    "pkv_paged_gather",
    "pkv_strerror",
    "pkv_last_cuda_error",
    "pkv_set_wait_limit_ns",
    "pkv_version",
)

PKV_OK = 0
PKV_ERR_NULL_POINTER = -1
PKV_ERR_MISALIGNED = -2
PKV_ERR_BAD_LAYOUT = -3
PKV_ERR_BAD_PARAMS = -4
PKV_ERR_UNSUPPORTED_SHAPE = -5
PKV_ERR_WORKSPACE_TOO_SMALL = -6
PKV_ERR_CUDA = -7
PKV_ERR_SCRATCH_TOO_SMALL = -8
PKV_STATIC_SCRATCH_BYTES = 16 << 20

PKV_GROUP_BLOCK = -1  # PoolLayout.group_size of e4m3 pages (bits=8): one f32 scale per block and KV head

PKV_CONTRACTION_AUTO = 0
PKV_CONTRACTION_TENSOR = 1
PKV_CONTRACTION_CUDA_CORE = 2

PKV_SCHEDULE_AUTO = 0
PKV_SCHEDULE_PARTITIONS = 1
PKV_SCHEDULE_BALANCED = 2

PKV_DEVERR_BAD_BLOCK = 1
PKV_DEVERR_BAD_SEQ_LEN = 2
PKV_DEVERR_TIMEOUT = 4


class LibraryNotBuilt(RuntimeError):
    pass


class PkvError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"pkv error {code}: {message}")
        self.code = code


class PoolLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("num_blocks", "num_kv_heads", "block_size", "head_dim", "bits", "group_size", "v_head_dim")]


class DecodeParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("num_seqs", "num_q_heads", "n_query", "max_blocks_per_seq", "partition_tokens", "window",
                 "contraction", "schedule")]


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("partition_tokens", "max_partitions", "chunk_rows", "sm_count", "threads_per_cta",
                 "smem_bytes", "merge_in_cluster", "contraction")] + [("workspace_bytes", ctypes.c_size_t),
                                                                      ("balanced", ctypes.c_int32)]


class SparseParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("top_k", "first_blocks", "last_blocks")]


class SparsePlan(ctypes.Structure):
    _fields_ = [("attention", Plan), ("select_bytes", ctypes.c_size_t), ("workspace_bytes", ctypes.c_size_t)]


_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Loads (once) and returns the library with its prototypes declared."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise LibraryNotBuilt(f"{path} is missing: run __graft_entry__.build() or "
                              "python -m quantized_kv_decode_partial_gb300.build")
    lib = ctypes.CDLL(path)
    P, I32, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    lib.pkv_make_plan.argtypes = [ctypes.POINTER(PoolLayout), ctypes.POINTER(DecodeParams), I32, ctypes.POINTER(Plan)]
    lib.pkv_make_plan.restype = ctypes.c_int
    lib.pkv_plan_for_current_device.argtypes = [ctypes.POINTER(PoolLayout), ctypes.POINTER(DecodeParams),
                                                ctypes.POINTER(Plan)]
    lib.pkv_plan_for_current_device.restype = ctypes.c_int
    lib.pkv_paged_decode_attention.argtypes = [ctypes.POINTER(PoolLayout), ctypes.POINTER(DecodeParams),
                                               P, P, P, P, P, P, P, P, P, F, P, P, SZ, P, P]
    lib.pkv_paged_decode_attention.restype = ctypes.c_int
    lib.pkv_paged_decode_partial.argtypes = lib.pkv_paged_decode_attention.argtypes
    lib.pkv_paged_decode_partial.restype = ctypes.c_int
    lib.pkv_merge_partitions.argtypes = [ctypes.POINTER(PoolLayout), ctypes.POINTER(DecodeParams), P, P, SZ, P,
                                         P, P]
    lib.pkv_merge_partitions.restype = ctypes.c_int
    lib.pkv_paged_decode_attention_no_alloc.argtypes = [ctypes.POINTER(PoolLayout), ctypes.POINTER(DecodeParams),
                                                        P, P, P, P, P, P, P, P, P, F, P, P, P]
    lib.pkv_paged_decode_attention_no_alloc.restype = ctypes.c_int
    lib.pkv_paged_decode_attention_host.argtypes = [ctypes.POINTER(PoolLayout), ctypes.POINTER(DecodeParams),
                                                    P, P, SZ, P, P, P, P, P, P, P, P, P, P, P, P, F, P, P, SZ, P, P]
    lib.pkv_paged_decode_attention_host.restype = ctypes.c_int
    lib.pkv_step_create.argtypes = [ctypes.POINTER(PoolLayout), ctypes.POINTER(DecodeParams),
                                    P, P, SZ, P, P, P, P, P, P, P, P, P, P, P, P, F, P, P, SZ, P, P,
                                    ctypes.POINTER(ctypes.c_void_p)]
    lib.pkv_step_create.restype = ctypes.c_int
    lib.pkv_step_run.argtypes = [P]
    lib.pkv_step_run.restype = ctypes.c_int
    lib.pkv_step_destroy.argtypes = [P]
    lib.pkv_step_destroy.restype = None
    lib.pkv_paged_decode_append_attention.argtypes = [ctypes.POINTER(PoolLayout), ctypes.POINTER(DecodeParams),
                                                      P, P, P, P, P, P, P, P, P, P, P, F, P, P, SZ, P, P]
    lib.pkv_paged_decode_append_attention.restype = ctypes.c_int
    lib.pkv_paged_append.argtypes = [ctypes.POINTER(PoolLayout), I32, I32, I32, P, P, P, P, P, P, P, P, P, P, P, P]
    lib.pkv_paged_append.restype = ctypes.c_int
    lib.pkv_paged_gather.argtypes = [P, I32, I32, I32, I32, P, P, I32, I32, I32, P, P, P]
    lib.pkv_paged_gather.restype = ctypes.c_int
    LPS = [ctypes.POINTER(PoolLayout), ctypes.POINTER(DecodeParams), ctypes.POINTER(SparseParams)]
    lib.pkv_make_sparse_plan.argtypes = LPS + [I32, ctypes.POINTER(SparsePlan)]
    lib.pkv_make_sparse_plan.restype = ctypes.c_int
    lib.pkv_sparse_plan_for_current_device.argtypes = LPS + [ctypes.POINTER(SparsePlan)]
    lib.pkv_sparse_plan_for_current_device.restype = ctypes.c_int
    lib.pkv_update_block_bounds.argtypes = [ctypes.POINTER(PoolLayout), I32, I32, I32, P, P, P, P, P, P, P, P]
    lib.pkv_update_block_bounds.restype = ctypes.c_int
    lib.pkv_select_blocks.argtypes = LPS + [P, P, P, P, P, P, P, P, SZ, P, P]
    lib.pkv_select_blocks.restype = ctypes.c_int
    lib.pkv_selected_decode_attention.argtypes = LPS + [P, P, P, P, P, P, P, P, P, F, P, P, SZ, P, P]
    lib.pkv_selected_decode_attention.restype = ctypes.c_int
    lib.pkv_sparse_decode_attention.argtypes = LPS + [P, P, P, P, P, P, P, P, P, P, F, P, P, P, SZ, P, P]
    lib.pkv_sparse_decode_attention.restype = ctypes.c_int
    lib.pkv_strerror.argtypes = [ctypes.c_int]
    lib.pkv_strerror.restype = ctypes.c_char_p
    lib.pkv_last_cuda_error.argtypes = []
    lib.pkv_last_cuda_error.restype = ctypes.c_char_p
    lib.pkv_version.argtypes = []
    lib.pkv_version.restype = ctypes.c_int
    lib.pkv_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.pkv_set_wait_limit_ns.restype = ctypes.c_uint64
    if path == LIB_PATH:
        _lib = lib
    return lib


def _check(rc: int, lib) -> None:
    if rc != PKV_OK:
        msg = lib.pkv_strerror(rc).decode()
        if rc == PKV_ERR_CUDA:
            msg += ": " + lib.pkv_last_cuda_error().decode()
        raise PkvError(rc, msg)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def v_head_dim_of(v_pool: torch.Tensor, bits: int) -> int:
    """Value head dim of a V pool: its row's bits (bf16 values, affine words, e4m3 codes) over the stored bits."""
    return v_pool.shape[-1] * v_pool.element_size() * 8 // bits


def layout_for(k_pool: torch.Tensor, head_dim: int, bits: int, group_size: int = 64,
               v_pool: Optional[torch.Tensor] = None) -> PoolLayout:
    nb, hk, bs, width = k_pool.shape
    if width * k_pool.element_size() * 8 != head_dim * bits:
        raise ValueError(f"k_pool rows of {width} {k_pool.dtype} are not {head_dim} values of {bits} bits")
    dv = 0 if v_pool is None else v_head_dim_of(v_pool, bits)
    return PoolLayout(nb, hk, bs, head_dim, bits, group_size, 0 if dv == head_dim else dv)


def _out_like(q: torch.Tensor, layout: PoolLayout) -> torch.Tensor:
    dv = layout.v_head_dim or layout.head_dim
    return torch.empty(q.shape[:-1] + (dv,), dtype=q.dtype, device=q.device)


_plan_cache = {}


def _plan_key(layout: PoolLayout, params: DecodeParams):
    return (torch.cuda.current_device(),) + tuple(getattr(layout, f) for f, _ in PoolLayout._fields_) + \
        tuple(getattr(params, f) for f, _ in DecodeParams._fields_)


def _cached_plan(layout: PoolLayout, params: DecodeParams) -> Plan:
    key = _plan_key(layout, params)
    plan = _plan_cache.get(key)
    if plan is None:
        plan = make_plan(layout, params)
        if len(_plan_cache) > 1024:
            _plan_cache.clear()
        _plan_cache[key] = plan
    return plan


def set_wait_limit_ns(ns: int) -> int:
    """Bound of one main-loop pipeline wait for decode calls made from now on
    (pkv_set_wait_limit_ns; 0 restores the default of one second). Returns the
    previous bound."""
    return int(load_library().pkv_set_wait_limit_ns(int(ns)))


def make_plan(layout: PoolLayout, params: DecodeParams, sm_count: Optional[int] = None) -> Plan:
    """The library's plan (partition size, workspace bytes) for these shapes."""
    lib = load_library()
    plan = Plan()
    if sm_count is None:
        rc = lib.pkv_plan_for_current_device(ctypes.byref(layout), ctypes.byref(params), ctypes.byref(plan))
    else:
        rc = lib.pkv_make_plan(ctypes.byref(layout), ctypes.byref(params), sm_count, ctypes.byref(plan))
    _check(rc, lib)
    return plan


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the current stream's handle without building a Stream object, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


class _Workspaces(threading.local):
    """The default stream's workspaces of one host thread, a growing one per device. Calls on
    that stream run one after the other, and the launches of one thread's call are not mixed
    with another call's, so they may share it; a call on any other stream (a captured one
    among them) gets a workspace of its own. So does one that needs more than MOST_HELD: a step
    that large hides what the allocator takes, and its memory goes back when it returns."""

    MOST_HELD = 32 << 20

    def __init__(self):
        self.held = {}

    def get(self, device: torch.device, index: int, stream: int, nbytes: int) -> torch.Tensor:
        if stream != 0 or nbytes > self.MOST_HELD:
            return torch.empty(nbytes, dtype=torch.uint8, device=device)
        ws = self.held.get(index)
        if ws is None or ws.numel() < nbytes:
            ws = self.held[index] = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return ws


_workspaces = _Workspaces()


class _Call:
    """What a call's shapes settle: the argument structures and the plan."""

    __slots__ = ("layout", "params", "layout_ref", "params_ref", "sparse", "sparse_ref", "workspace_bytes", "out_shape",
                 "like_q")

    def __init__(self, layout, params, q, sparse=None):
        if q.get_device() < 0:
            raise ValueError("expected CUDA tensors")
        self.layout, self.params, self.sparse = layout, params, sparse
        self.layout_ref, self.params_ref = ctypes.byref(layout), ctypes.byref(params)
        self.sparse_ref = None if sparse is None else ctypes.byref(sparse)
        dv = layout.v_head_dim or layout.head_dim
        self.out_shape = tuple(q.shape[:-1]) + (dv,)
        self.like_q = self.out_shape == tuple(q.shape)

    def new_out(self, q):
        if self.like_q:
            return torch.empty_like(q, memory_format=torch.contiguous_format)
        return torch.empty(self.out_shape, dtype=q.dtype, device=q.device)


_calls = {}


def _remember(key, call):
    if len(_calls) > 1024:
        _calls.clear()
    _calls[key] = call
    return call


def _require(dtype: torch.dtype, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, not {t.dtype}")


def _check_tensors(index: int, *tensors) -> None:
    """All contiguous and on device `index`."""
    for t in tensors:
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous and on one device")


def _require_shape(name: str, t: Optional[torch.Tensor], *shape: int) -> None:
    if t is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must be of shape {list(shape)}, not {list(t.shape)}")


def _types(tensors) -> tuple:
    """Shapes and types, for a key."""
    return tuple([None if t is None else (t.shape, t.dtype) for t in tensors])


_E4M3_DTYPES = (torch.float8_e4m3fn, torch.uint8)


def _check_block_scales(k_pool, v_pool, bits: int, group_size: int, *scales) -> None:
    if bits == 8 and group_size == PKV_GROUP_BLOCK:
        for pool in (k_pool, v_pool):
            if pool is not None and pool.dtype not in _E4M3_DTYPES:
                raise TypeError(f"e4m3 pages are float8_e4m3fn (or uint8) codes, not {pool.dtype}")
        cells = k_pool.shape[:2]
        for s in scales:
            if s is None:
                continue
            if s.dtype is not torch.float32:
                raise TypeError(f"scales of e4m3 pages are float32 [num_blocks, num_kv_heads], not {s.dtype}")
            if s.shape != cells or not s.is_contiguous():
                raise ValueError("scales of e4m3 pages are contiguous [num_blocks, num_kv_heads] planes")


def _check_planes(k_pool, v_pool, bits: int, group_size: int, k_dim: int, **planes) -> None:
    """The scale and bias planes of pages of codes; affine ones are bf16 [NB, HK, BS, D / 64]."""
    if bits == 8 and group_size == PKV_GROUP_BLOCK:
        _check_block_scales(k_pool, v_pool, bits, group_size, planes.get("k_scales"), planes.get("v_scales"))
    elif bits != 16:
        _require(torch.bfloat16, **planes)
        for name, t in planes.items():
            d = k_dim if name[0] == "k" else v_head_dim_of(v_pool, bits)
            _require_shape(name, t, *k_pool.shape[:3], d // 64)


def _require_decode_shapes(q, k_pool, v_pool, block_tables, seq_lens) -> None:
    """Types and shapes of a decode call over e4m3 pages (k_pool's rows are checked by layout_for)."""
    _require(torch.bfloat16, q=q)
    _require(torch.int32, block_tables=block_tables, seq_lens=seq_lens)
    _require_shape("v_pool", v_pool, *k_pool.shape[:3], v_pool.shape[-1])
    _require_shape("block_tables", block_tables, q.shape[0], block_tables.shape[-1])
    _require_shape("seq_lens", seq_lens, q.shape[0])


def _decode_call(q, k_pool, v_pool, block_tables, bits, group_size, partition_tokens, window, contraction, schedule,
                 e4m3=None) -> _Call:
    """Cached by what settles the call; runs with q's device current. e4m3: of such pages, what
    else is checked (seq_lens, k_scales, v_scales)."""
    key = (q.get_device(), q.shape, k_pool.shape, k_pool.dtype, v_pool.shape, v_pool.dtype, block_tables.shape, bits, group_size,
           partition_tokens, window, contraction, schedule)
    if e4m3 is not None:
        key += (q.dtype, block_tables.dtype) + _types(e4m3)
    call = _calls.get(key)
    if call is None:
        if e4m3 is not None:
            _check_block_scales(k_pool, v_pool, bits, group_size, *e4m3[1:])
            _require_decode_shapes(q, k_pool, v_pool, block_tables, e4m3[0])
        B, HQ, N, D = q.shape
        call = _Call(layout_for(k_pool, D, bits, group_size, v_pool),
                     DecodeParams(B, HQ, N, block_tables.shape[1], partition_tokens, window, contraction, schedule), q)
        call.workspace_bytes = _cached_plan(call.layout, call.params).workspace_bytes
        _remember(key, call)
    return call


def paged_decode_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                           block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float, *,
                           bits: int = 16, group_size: int = 64,
                           k_scales: Optional[torch.Tensor] = None, k_biases: Optional[torch.Tensor] = None,
                           v_scales: Optional[torch.Tensor] = None, v_biases: Optional[torch.Tensor] = None,
                           partition_tokens: int = 0, window: int = 0, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None,
                           error_flag: Optional[torch.Tensor] = None, contraction: int = 0,
                           schedule: int = 0) -> torch.Tensor:
    """Decode attention over a paged cache (see include/pkv_decode.h).

    q bf16 [B, HQ, N, D]; pools bf16 [NB, HK, BS, D] (bits=16) or int32 code
    words [NB, HK, BS, D*bits/32] with bf16 scale/bias planes [NB, HK, BS, D/64],
    or float8_e4m3fn (or uint8) codes [NB, HK, BS, D] with f32 scale planes [NB, HK]
    (bits=8, group_size=PKV_GROUP_BLOCK, no biases);
    block_tables int32 [B, max_blocks]; seq_lens int32 [B]. Runs on the current
    CUDA stream of q's device and returns bf16 [B, HQ, N, D].
    """
    lib = load_library()
    e4m3 = (seq_lens, k_scales, v_scales) if group_size == PKV_GROUP_BLOCK and bits == 8 else None
    with _on_device(q.device):
        call = _decode_call(q, k_pool, v_pool, block_tables, bits, group_size, partition_tokens, window, contraction,
                            schedule, e4m3)
        index = q.get_device()
        if e4m3 is not None:
            _check_tensors(index, q, k_pool, v_pool, block_tables, seq_lens, k_scales, v_scales, out, workspace,
                           error_flag)
            if out is not None:
                _require(torch.bfloat16, out=out)
                _require_shape("out", out, *call.out_shape)
        stream = _raw_stream(index)
        if out is None:
            out = call.new_out(q)
        if workspace is None and call.workspace_bytes:
            workspace = _workspaces.get(q.device, index, stream, call.workspace_bytes)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        rc = lib.pkv_paged_decode_attention(
            call.layout_ref, call.params_ref, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
            _ptr(k_scales), _ptr(k_biases), _ptr(v_scales), _ptr(v_biases), block_tables.data_ptr(),
            seq_lens.data_ptr(), float(scale), out.data_ptr(), _ptr(workspace), ws_bytes, _ptr(error_flag),
            stream)
    if rc != PKV_OK:
        _check(rc, lib)
    return out


def paged_decode_append_attention(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                                  k_pool: torch.Tensor, v_pool: torch.Tensor, block_tables: torch.Tensor,
                                  seq_lens: torch.Tensor, scale: float, *, bits: int = 16, group_size: int = 64,
                                  k_scales: Optional[torch.Tensor] = None, k_biases: Optional[torch.Tensor] = None,
                                  v_scales: Optional[torch.Tensor] = None, v_biases: Optional[torch.Tensor] = None,
                                  partition_tokens: int = 0, window: int = 0, out: Optional[torch.Tensor] = None,
                                  workspace: Optional[torch.Tensor] = None,
                                  error_flag: Optional[torch.Tensor] = None, contraction: int = 0,
                                  schedule: int = 0) -> torch.Tensor:
    """One decode step with its write (pkv_paged_decode_append_attention): writes
    k_new/v_new bf16 [B, HK, N, D] at cache positions seq_lens[b]-N .. seq_lens[b]-1
    (seq_lens counts the new rows), then attends as ``paged_decode_attention``."""
    lib = load_library()
    with _on_device(q.device):
        stream = _raw_stream(q.get_device())
        call = _decode_call(q, k_pool, v_pool, block_tables, bits, group_size, partition_tokens, window, contraction,
                            schedule)
        if out is None:
            out = call.new_out(q)
        if workspace is None and call.workspace_bytes:
            workspace = _workspaces.get(q.device, q.get_device(), stream, call.workspace_bytes)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        rc = lib.pkv_paged_decode_append_attention(
            call.layout_ref, call.params_ref, q.data_ptr(), _ptr(k_new), _ptr(v_new), k_pool.data_ptr(),
            v_pool.data_ptr(), _ptr(k_scales), _ptr(k_biases), _ptr(v_scales), _ptr(v_biases), block_tables.data_ptr(),
            seq_lens.data_ptr(), float(scale), out.data_ptr(), _ptr(workspace), ws_bytes, _ptr(error_flag),
            stream)
    if rc != PKV_OK:
        _check(rc, lib)
    return out


class HostDecodeStep:
    """One decode step driven from host memory (a pkv_step: pkv_paged_decode_attention_host
    prepared once).

    The step's host inputs (q, lengths, the new K/V rows for the fused step, block
    tables) live in one pinned block with a device twin. Each call enqueues the decode
    (fused with the append when ``k_new``/``v_new`` are given); the kernels read the
    inputs from the pinned block and write the output into pinned ``out_host`` over
    NVLink-C2C (the library falls back to copies where the memory is not mapped).
    Write the next step's values into ``host[name]`` (views of the pinned block)
    before calling again; ``copy_tables=False`` keeps the block tables out of the
    per-step data (the device copy made at construction is used, until
    ``refresh_tables()``). Pools, scale/bias planes and the workspace are device
    tensors, as for ``paged_decode_attention``.
    """

    def __init__(self, q: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, k_pool: torch.Tensor,
                 v_pool: torch.Tensor, scale: float, *, k_new: Optional[torch.Tensor] = None,
                 v_new: Optional[torch.Tensor] = None, bits: int = 16, group_size: int = 64, k_scales=None,
                 k_biases=None, v_scales=None, v_biases=None, partition_tokens: int = 0, window: int = 0,
                 workspace: Optional[torch.Tensor] = None, error_flag: Optional[torch.Tensor] = None, stream=None,
                 copy_tables: bool = True, contraction: int = 0, schedule: int = 0):
        self.lib = lib = load_library()
        _check_block_scales(k_pool, v_pool, bits, group_size, k_scales, v_scales)
        dev = k_pool.device
        if group_size == PKV_GROUP_BLOCK and bits == 8:
            _require_decode_shapes(q, k_pool, v_pool, block_tables, seq_lens)
            _check_tensors(k_pool.get_device(), k_pool, v_pool, k_scales, v_scales, workspace, error_flag)
        B, HQ, N, D = q.shape
        self.layout = layout_for(k_pool, D, bits, group_size, v_pool)
        self.params = DecodeParams(B, HQ, N, block_tables.shape[1], partition_tokens, window, contraction,
                                   schedule)
        named = [("q", q), ("seq_lens", seq_lens)]
        if k_new is not None:
            named += [("k_new", k_new), ("v_new", v_new)]
        named.append(("block_tables", block_tables))  # last: a per-step copy can stop before it
        offs, total = {}, 0
        for name, t in named:  # 256-byte aligned slots
            offs[name] = total
            total += -(-(t.numel() * t.element_size()) // 256) * 256
        self.block_host = torch.empty(total, dtype=torch.uint8, pin_memory=True)
        self.block_dev = torch.empty(total, dtype=torch.uint8, device=dev)
        self.host, self.dev = {}, {}
        for name, t in named:
            n = t.numel() * t.element_size()
            self.host[name] = self.block_host[offs[name]:offs[name] + n].view(t.dtype).view(t.shape)
            self.dev[name] = self.block_dev[offs[name]:offs[name] + n].view(t.dtype).view(t.shape)
            self.host[name].copy_(t.cpu())
        self.dev["block_tables"].copy_(self.host["block_tables"])
        # bytes copied per step: everything up to the tables' slot, or the whole block
        self.in_bytes = total if copy_tables else offs["block_tables"]
        with _on_device(dev):
            plan = _cached_plan(self.layout, self.params)
            self.out = _out_like(self.dev["q"], self.layout)
            if workspace is None and plan.workspace_bytes:
                workspace = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=dev)
            st = (stream or torch.cuda.current_stream(dev)).cuda_stream
        self.out_host = torch.empty(self.out.shape, dtype=self.out.dtype, pin_memory=True)
        self.h2d_bytes, self.d2h_bytes = self.in_bytes, self.out_host.numel() * self.out_host.element_size()
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        self._keep = (k_pool, v_pool, k_scales, k_biases, v_scales, v_biases, workspace, error_flag)
        d = self.dev
        handle = ctypes.c_void_p()
        with _on_device(dev):
            rc = lib.pkv_step_create(
                ctypes.byref(self.layout), ctypes.byref(self.params), _ptr(self.block_host), _ptr(self.block_dev),
                self.in_bytes, _ptr(self.out_host), _ptr(d["q"]), _ptr(d.get("k_new")), _ptr(d.get("v_new")),
                _ptr(k_pool), _ptr(v_pool), _ptr(k_scales), _ptr(k_biases), _ptr(v_scales), _ptr(v_biases),
                _ptr(d["block_tables"]), _ptr(d["seq_lens"]), float(scale), _ptr(self.out), _ptr(workspace),
                ws_bytes, _ptr(error_flag), st, ctypes.byref(handle))
        _check(rc, lib)
        self._handle = handle
        self._run = lib.pkv_step_run
        self._destroy = lib.pkv_step_destroy
        self._device = dev

    def refresh_tables(self):
        """Copies the host block tables to the device now (synchronously)."""
        self.dev["block_tables"].copy_(self.host["block_tables"])

    def __call__(self) -> torch.Tensor:
        """Enqueues the step (pkv_step_run) and returns the pinned output tensor,
        which holds the result once the stream reaches this point."""
        rc = self._run(self._handle)
        if rc != PKV_OK:
            _check(rc, self.lib)
        return self.out_host

    def __del__(self):
        # the handle is host memory only; work in flight keeps using the tensors, which
        # the caller keeps alive as long as it needs the results
        handle = getattr(self, "_handle", None)
        if handle is not None and handle.value:
            self._destroy(handle)
            self._handle = None


class _Stay:
    """The call's device is current already."""

    __slots__ = ()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


class _Switch:
    """Makes another device current for the call."""

    __slots__ = ("index", "prev")

    def __init__(self, index: int, prev: int):
        self.index, self.prev = index, prev

    def __enter__(self):
        torch.cuda.set_device(self.index)
        return self

    def __exit__(self, *exc):
        torch.cuda.set_device(self.prev)
        return False


_stay = _Stay()
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on_index(index: int):
    cur = _current_device()
    return _stay if cur == index else _Switch(index, cur)


def _on_device(device: torch.device):
    return _stay if device.index is None else _on_index(device.index)


def paged_decode_passes(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                        block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float, *, passes: str,
                        bits: int = 16, group_size: int = 64, k_scales=None, k_biases=None, v_scales=None,
                        v_biases=None, partition_tokens: int = 0, window: int = 0,
                        out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        error_flag: Optional[torch.Tensor] = None, contraction: int = 0,
                        schedule: int = 0) -> torch.Tensor:
    """One pass of the decode: ``passes="partial"`` (pkv_paged_decode_partial) or
    ``"merge"`` (pkv_merge_partitions). ``out`` and, with more than one
    partition, ``workspace`` must be given so the two calls share them."""
    lib = load_library()
    _check_block_scales(k_pool, v_pool, bits, group_size, k_scales, v_scales)
    if group_size == PKV_GROUP_BLOCK and bits == 8:
        _require_decode_shapes(q, k_pool, v_pool, block_tables, seq_lens)
        _check_tensors(q.get_device(), q, k_pool, v_pool, block_tables, seq_lens, k_scales, v_scales, out, workspace,
                       error_flag)
        if out is not None:
            _require(torch.bfloat16, out=out)
            _require_shape("out", out, *q.shape[:-1], v_head_dim_of(v_pool, bits))
    B, HQ, N, D = q.shape
    layout = layout_for(k_pool, D, bits, group_size, v_pool)
    params = DecodeParams(B, HQ, N, block_tables.shape[1], partition_tokens, window, contraction, schedule)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _on_device(q.device):
        stream = torch.cuda.current_stream(q.device).cuda_stream
        if passes == "partial":
            rc = lib.pkv_paged_decode_partial(
                ctypes.byref(layout), ctypes.byref(params), _ptr(q), _ptr(k_pool), _ptr(v_pool),
                _ptr(k_scales), _ptr(k_biases), _ptr(v_scales), _ptr(v_biases), _ptr(block_tables),
                _ptr(seq_lens), float(scale), _ptr(out), _ptr(workspace), ws_bytes, _ptr(error_flag), stream)
        elif passes == "merge":
            rc = lib.pkv_merge_partitions(ctypes.byref(layout), ctypes.byref(params), _ptr(seq_lens),
                                          _ptr(workspace), ws_bytes, _ptr(out), _ptr(error_flag), stream)
        else:
            raise ValueError(passes)
    _check(rc, lib)
    return out


def paged_append(k_new: torch.Tensor, v_new: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                 k_pool: torch.Tensor, v_pool: torch.Tensor, *, bits: int = 16, group_size: int = 64,
                 k_scales=None, k_biases=None, v_scales=None, v_biases=None,
                 error_flag: Optional[torch.Tensor] = None) -> None:
    """Writes k_new/v_new bf16 [B, HK, n_new, D] at positions seq_lens[b].. of each
    sequence (quantising affine and e4m3 pages); see include/pkv_decode.h."""
    lib = load_library()
    index, tables = k_new.get_device(), block_tables.shape
    B, HK, n_new, D = k_new.shape
    key = ("append", index, k_pool.shape, k_pool.dtype, v_pool.shape, v_pool.dtype, D, bits, group_size)
    e4m3 = group_size == PKV_GROUP_BLOCK and bits == 8
    if e4m3:
        key += _types((k_new, v_new, block_tables, seq_lens, k_scales, v_scales))
    call = _calls.get(key)
    if call is None:
        if e4m3:
            _check_block_scales(k_pool, v_pool, bits, group_size, k_scales, v_scales)
            _require(torch.bfloat16, k_new=k_new, v_new=v_new)
            _require(torch.int32, block_tables=block_tables, seq_lens=seq_lens)
            _require_shape("v_pool", v_pool, *k_pool.shape[:3], v_pool.shape[-1])
            _require_shape("k_new", k_new, B, k_pool.shape[1], n_new, D)
            _require_shape("v_new", v_new, B, k_pool.shape[1], n_new, v_head_dim_of(v_pool, bits))
            _require_shape("block_tables", block_tables, B, tables[-1])
            _require_shape("seq_lens", seq_lens, B)
            _check_tensors(index, k_new, v_new, block_tables, seq_lens, k_pool, v_pool)
        call = _remember(key, _Call(layout_for(k_pool, D, bits, group_size, v_pool), DecodeParams(), k_new))
    if e4m3:
        _check_tensors(index, k_new, v_new, block_tables, seq_lens, k_pool, v_pool, k_scales, v_scales, error_flag)
    with _on_index(index):
        rc = lib.pkv_paged_append(call.layout_ref, B, tables[1], n_new, k_new.data_ptr(), v_new.data_ptr(),
                                  block_tables.data_ptr(), seq_lens.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
                                  _ptr(k_scales), _ptr(k_biases), _ptr(v_scales), _ptr(v_biases), _ptr(error_flag),
                                  _raw_stream(index))
    if rc != PKV_OK:
        _check(rc, lib)


def paged_gather(pool: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, max_len: int,
                 out: Optional[torch.Tensor] = None, error_flag: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Bit-exact gather of one pool plane [NB, HK, BS, W] into [B, HK, max_len, W]."""
    lib = load_library()
    nb, hk, bs = pool.shape[:3]
    row_bytes = pool[0, 0, 0].numel() * pool.element_size()
    B = block_tables.shape[0]
    if out is None:
        out = torch.zeros((B, hk, max_len) + tuple(pool.shape[3:]), dtype=pool.dtype, device=pool.device)
    with _on_device(pool.device):
        stream = torch.cuda.current_stream(pool.device).cuda_stream
        rc = lib.pkv_paged_gather(_ptr(pool), nb, hk, bs, row_bytes, _ptr(block_tables), _ptr(seq_lens), B,
                                  block_tables.shape[1], max_len, _ptr(out), _ptr(error_flag), stream)
    _check(rc, lib)
    return out


def make_sparse_plan(layout: PoolLayout, params: DecodeParams, sparse: SparseParams,
                     sm_count: Optional[int] = None) -> SparsePlan:
    """The library's plan of a sparse step (workspace bytes, the attention's own plan)."""
    lib = load_library()
    plan = SparsePlan()
    args = (ctypes.byref(layout), ctypes.byref(params), ctypes.byref(sparse))
    if sm_count is None:
        rc = lib.pkv_sparse_plan_for_current_device(*args, ctypes.byref(plan))
    else:
        rc = lib.pkv_make_sparse_plan(*args, sm_count, ctypes.byref(plan))
    _check(rc, lib)
    return plan


def update_block_bounds(k_pool: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                        k_bounds: torch.Tensor, *, n_new: int, bits: int = 16, group_size: int = 64,
                        k_scales: Optional[torch.Tensor] = None, k_biases: Optional[torch.Tensor] = None,
                        error_flag: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Brings k_bounds bf16 [NB, HK, 2, D] (each block's smallest and largest key, elementwise)
    up to date after the last n_new rows of every sequence were appended (seq_lens counts
    them); see include/pkv_decode.h. Returns k_bounds."""
    lib = load_library()
    key = ("bounds", k_bounds.get_device(), k_pool.shape, k_pool.dtype, k_bounds.shape, k_bounds.dtype, block_tables.shape,
           block_tables.dtype, seq_lens.shape, seq_lens.dtype, bits, group_size)
    if bits != 16:
        key += _types((k_scales, k_biases))
    call = _calls.get(key)
    if call is None:
        D = k_pool.shape[-1] * k_pool.element_size() * 8 // bits
        _check_planes(k_pool, None, bits, group_size, D, k_scales=k_scales, k_biases=k_biases)
        _require(torch.bfloat16, k_bounds=k_bounds)
        _require(torch.int32, block_tables=block_tables, seq_lens=seq_lens)
        _require_shape("k_bounds", k_bounds, k_pool.shape[0], k_pool.shape[1], 2, D)
        _require_shape("seq_lens", seq_lens, block_tables.shape[0])
        layout = layout_for(k_pool, D, bits, group_size)
        if D == 192:  # the values are not looked at; no pages have 192-dim ones
            layout.v_head_dim = 128
        call = _remember(key, _Call(layout, DecodeParams(), k_bounds))
    _check_tensors(k_bounds.get_device(), k_pool, block_tables, seq_lens, k_bounds, k_scales, k_biases, error_flag)
    B, max_blocks = block_tables.shape
    with _on_device(k_pool.device):
        rc = lib.pkv_update_block_bounds(call.layout_ref, B, max_blocks, n_new, k_pool.data_ptr(), _ptr(k_scales),
                                         _ptr(k_biases), block_tables.data_ptr(), seq_lens.data_ptr(),
                                         k_bounds.data_ptr(), _ptr(error_flag), _raw_stream(k_pool.get_device()))
    if rc != PKV_OK:
        _check(rc, lib)
    return k_bounds


class BlockSelection(NamedTuple):
    """Blocks chosen for a step (pkv_select_blocks): ``blocks`` int32 [B, HK, top_k], their places
    in the sequence; ``tables`` [B, HK, top_k] and ``lens`` [B, HK], the form the attention over
    them reads."""

    blocks: torch.Tensor
    tables: torch.Tensor
    lens: torch.Tensor


def select_blocks(q: torch.Tensor, k_bounds: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, *,
                  block_size: int, top_k: int, first_blocks: int = 1, last_blocks: int = 1,
                  out: Optional[BlockSelection] = None, workspace: Optional[torch.Tensor] = None,
                  error_flag: Optional[torch.Tensor] = None) -> BlockSelection:
    """Chooses top_k blocks for each (sequence, KV head) of queries q bf16 [B, HQ, N, D] by their
    bounds (pkv_select_blocks). Depends on the bounds alone, whatever the pages' format."""
    lib = load_library()
    with _on_device(q.device):
        stream = _raw_stream(q.get_device())
        key = ("select", q.get_device(), q.shape, q.dtype, k_bounds.shape, k_bounds.dtype, block_tables.shape,
               block_tables.dtype, seq_lens.shape, seq_lens.dtype, block_size, top_k, first_blocks, last_blocks)
        call = _calls.get(key)
        if call is None:
            B, HQ, N, D = q.shape
            _require(torch.bfloat16, q=q, k_bounds=k_bounds)
            _require(torch.int32, block_tables=block_tables, seq_lens=seq_lens)
            nb, hk = k_bounds.shape[:2]
            _require_shape("k_bounds", k_bounds, nb, hk, 2, D)
            _require_shape("block_tables", block_tables, B, block_tables.shape[1])
            _require_shape("seq_lens", seq_lens, B)
            call = _Call(PoolLayout(nb, hk, block_size, D, 16, 64, 64 if D == 64 else 128),
                         DecodeParams(B, HQ, N, block_tables.shape[1]), q,
                         SparseParams(top_k, first_blocks, last_blocks))
            call.workspace_bytes = make_sparse_plan(call.layout, call.params, call.sparse).select_bytes
            _remember(key, call)
        B, hk = q.shape[0], k_bounds.shape[1]
        if out is None:
            new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=q.device)
            out = BlockSelection(new(B, hk, top_k), new(B, hk, top_k), new(B, hk))
        else:
            _require(torch.int32, blocks=out.blocks, tables=out.tables, lens=out.lens)
            _require_shape("out.blocks", out.blocks, B, hk, top_k)
            _require_shape("out.tables", out.tables, B, hk, top_k)
            _require_shape("out.lens", out.lens, B, hk)
        _check_tensors(q.get_device(), q, k_bounds, block_tables, seq_lens, *out, workspace, error_flag)
        if workspace is None and call.workspace_bytes:
            workspace = _workspaces.get(q.device, q.get_device(), stream, call.workspace_bytes)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        rc = lib.pkv_select_blocks(call.layout_ref, call.params_ref, call.sparse_ref, q.data_ptr(),
                                   k_bounds.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(),
                                   _ptr(out.blocks), out.tables.data_ptr(), out.lens.data_ptr(), _ptr(workspace),
                                   ws_bytes, _ptr(error_flag), stream)
    if rc != PKV_OK:
        _check(rc, lib)
    return out


def selected_decode_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, selection: BlockSelection,
                              scale: float, *, bits: int = 16, group_size: int = 64,
                              k_scales: Optional[torch.Tensor] = None, k_biases: Optional[torch.Tensor] = None,
                              v_scales: Optional[torch.Tensor] = None, v_biases: Optional[torch.Tensor] = None,
                              partition_tokens: int = 0, out: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None, error_flag: Optional[torch.Tensor] = None,
                              contraction: int = 0, schedule: int = 0) -> torch.Tensor:
    """Decode attention over chosen blocks (pkv_selected_decode_attention); otherwise as
    ``paged_decode_attention``."""
    lib = load_library()
    tables, lens = selection.tables, selection.lens
    with _on_device(q.device):
        key = ("selected", q.get_device(), q.shape, q.dtype, k_pool.shape, k_pool.dtype, v_pool.shape, v_pool.dtype, tables.shape,
               tables.dtype, lens.shape, lens.dtype, bits, group_size, partition_tokens, contraction, schedule)
        if bits != 16:
            key += _types((k_scales, k_biases, v_scales, v_biases))
        call = _calls.get(key)
        if call is None:
            B, HQ, N, D = q.shape
            _check_planes(k_pool, v_pool, bits, group_size, D, k_scales=k_scales, k_biases=k_biases, v_scales=v_scales,
                          v_biases=v_biases)
            layout = layout_for(k_pool, D, bits, group_size, v_pool)
            top_k = tables.shape[-1]
            _require(torch.bfloat16, q=q)
            _require(torch.int32, tables=tables, lens=lens)
            _require_shape("v_pool", v_pool, *k_pool.shape[:3], v_pool.shape[-1])
            _require_shape("selection.tables", tables, B, layout.num_kv_heads, top_k)
            _require_shape("selection.lens", lens, B, layout.num_kv_heads)
            # which blocks were taken is settled: any numbers that hold the new rows
            sparse = SparseParams(top_k, 0, 1 + -(-(N - 1) // layout.block_size))
            call = _Call(layout, DecodeParams(B, HQ, N, top_k, partition_tokens, 0, contraction, schedule), q, sparse)
            call.workspace_bytes = make_sparse_plan(layout, call.params, sparse).attention.workspace_bytes
            _remember(key, call)
        _check_tensors(q.get_device(), q, k_pool, v_pool, tables, lens, k_scales, k_biases, v_scales, v_biases, out,
                       workspace, error_flag)
        stream = _raw_stream(q.get_device())
        if out is None:
            out = call.new_out(q)
        else:
            _require(torch.bfloat16, out=out)
            _require_shape("out", out, *call.out_shape)
        if workspace is None and call.workspace_bytes:
            workspace = _workspaces.get(q.device, q.get_device(), stream, call.workspace_bytes)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        rc = lib.pkv_selected_decode_attention(
            call.layout_ref, call.params_ref, call.sparse_ref, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
            _ptr(k_scales), _ptr(k_biases), _ptr(v_scales), _ptr(v_biases), tables.data_ptr(), lens.data_ptr(), float(scale),
            out.data_ptr(), _ptr(workspace), ws_bytes, _ptr(error_flag), stream)
    if rc != PKV_OK:
        _check(rc, lib)
    return out


def sparse_decode_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, k_bounds: torch.Tensor,
                            block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float, *, top_k: int,
                            first_blocks: int = 1, last_blocks: int = 1, bits: int = 16, group_size: int = 64,
                            k_scales: Optional[torch.Tensor] = None, k_biases: Optional[torch.Tensor] = None,
                            v_scales: Optional[torch.Tensor] = None, v_biases: Optional[torch.Tensor] = None,
                            blocks: Optional[torch.Tensor] = None, partition_tokens: int = 0,
                            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                            error_flag: Optional[torch.Tensor] = None, contraction: int = 0,
                            schedule: int = 0) -> torch.Tensor:
    """Decode attention over the top_k blocks of each (sequence, KV head) that the bounds k_bounds
    bf16 [NB, HK, 2, D] score highest for the queries, the first_blocks first and last_blocks
    last always among them (pkv_sparse_decode_attention). ``blocks`` int32 [B, HK, top_k]
    receives the choice. Otherwise as ``paged_decode_attention``."""
    lib = load_library()
    with _on_device(q.device):
        key = ("sparse", q.get_device(), q.shape, q.dtype, k_pool.shape, k_pool.dtype, v_pool.shape, v_pool.dtype, k_bounds.shape,
               k_bounds.dtype, block_tables.shape, block_tables.dtype, seq_lens.shape, seq_lens.dtype,
               None if blocks is None else (blocks.shape, blocks.dtype), bits, group_size, partition_tokens,
               contraction, schedule, top_k, first_blocks, last_blocks)
        if bits != 16:
            key += _types((k_scales, k_biases, v_scales, v_biases))
        call = _calls.get(key)
        if call is None:
            B, HQ, N, D = q.shape
            _check_planes(k_pool, v_pool, bits, group_size, D, k_scales=k_scales, k_biases=k_biases, v_scales=v_scales,
                          v_biases=v_biases)
            layout = layout_for(k_pool, D, bits, group_size, v_pool)
            _require(torch.bfloat16, q=q, k_bounds=k_bounds)
            _require(torch.int32, block_tables=block_tables, seq_lens=seq_lens, blocks=blocks)
            _require_shape("k_bounds", k_bounds, layout.num_blocks, layout.num_kv_heads, 2, D)
            _require_shape("v_pool", v_pool, *k_pool.shape[:3], v_pool.shape[-1])
            _require_shape("block_tables", block_tables, B, block_tables.shape[1])
            _require_shape("seq_lens", seq_lens, B)
            _require_shape("blocks", blocks, B, layout.num_kv_heads, top_k)
            call = _Call(layout, DecodeParams(B, HQ, N, block_tables.shape[1], partition_tokens, 0, contraction, schedule),
                         q, SparseParams(top_k, first_blocks, last_blocks))
            call.workspace_bytes = make_sparse_plan(layout, call.params, call.sparse).workspace_bytes
            _remember(key, call)
        _check_tensors(q.get_device(), q, k_pool, v_pool, k_bounds, block_tables, seq_lens, blocks, out, k_scales, k_biases,
                       v_scales, v_biases, workspace, error_flag)
        stream = _raw_stream(q.get_device())
        if out is None:
            out = call.new_out(q)
        else:
            _require(torch.bfloat16, out=out)
            _require_shape("out", out, *call.out_shape)
        if workspace is None:
            workspace = _workspaces.get(q.device, q.get_device(), stream, call.workspace_bytes)
        ws_bytes = workspace.numel() * workspace.element_size()
        rc = lib.pkv_sparse_decode_attention(
            call.layout_ref, call.params_ref, call.sparse_ref, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
            _ptr(k_scales), _ptr(k_biases), _ptr(v_scales), _ptr(v_biases), k_bounds.data_ptr(),
            block_tables.data_ptr(), seq_lens.data_ptr(), float(scale), _ptr(blocks), out.data_ptr(), workspace.data_ptr(),
            ws_bytes, _ptr(error_flag), stream)
    if rc != PKV_OK:
        _check(rc, lib)
    return out
