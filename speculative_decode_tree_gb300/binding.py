"""Thin Python binding of the C ABI in include/ddtree_verify.h.

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the cudaStream_t, return codes become exceptions.  Every step
of the verify path runs in the library's CUDA kernels; there is no CPU
fallback, and loading fails loudly when the library has not been built.
"""
from __future__ import annotations

import copy
import ctypes
import os
from typing import Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "libddtree_verify.so")

DDTREE_OK = 0
DDTREE_EINVAL = 1
DDTREE_EWORKSPACE = 2
DDTREE_EUNSUPPORTED = 3
DDTREE_ELAUNCH = 4
DDTREE_EDEVICE_DATA = 5
DDTREE_ECUDA = 6

DDTREE_ST_BAD_INDEX = 0x1
DDTREE_ST_BAD_PARENT = 0x2
DDTREE_ST_BAD_LENGTH = 0x4
DDTREE_ST_TIMEOUT = 0x8
DDTREE_ST_OVERLAP = 0x10
DDTREE_ST_BAD_MASK = 0x20
DDTREE_ST_NO_PAGES = 0x40
DDTREE_ST_BAD_SCALE = 0x80

DDTREE_ROPE_PLAIN = 0
DDTREE_ROPE_LINEAR = 1
DDTREE_ROPE_YARN = 2

DDTREE_BF16 = 0
DDTREE_FP16 = 1

DDTREE_KERNEL_AUTO = 0
DDTREE_KERNEL_SIMT = 1
DDTREE_KERNEL_TC = 2
DDTREE_KERNEL_TC2 = 3

EXPORTS = (
    "ddtree_verify_mla_plan", "ddtree_verify_mla_plan_ex", "ddtree_verify_mla_workspace_size",
    "ddtree_verify_mla", "ddtree_verify_mla_batched", "ddtree_build_ancestor_mask",
    "ddtree_verify_mla_check", "ddtree_status_str", "ddtree_verify_mla_batched_timed",
    "ddtree_verify_mla_noalloc", "ddtree_accept_greedy_workspace_size", "ddtree_accept_greedy",
    "ddtree_relocate_kv_workspace_size", "ddtree_relocate_kv",
    "ddtree_tree_from_mask_workspace_size", "ddtree_tree_from_mask", "ddtree_step_maps",
    "ddtree_rope_init", "ddtree_mla_append", "ddtree_draft_append",
    "ddtree_draft_attention_plan", "ddtree_draft_attention_workspace_size", "ddtree_draft_attention",
    "ddtree_draft8_append", "ddtree_draft8_read",
    "ddtree_draft8_attention_plan", "ddtree_draft8_attention_workspace_size", "ddtree_draft8_attention",
    "ddtree_prompt_attention_plan", "ddtree_prompt_attention_workspace_size", "ddtree_prompt_attention",
)


class Plan(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("n_nodes", ctypes.c_int32), ("n_heads", ctypes.c_int32),
        ("rows_per_req", ctypes.c_int32), ("pool_rows", ctypes.c_int64),
        ("max_keys", ctypes.c_int32), ("kernel", ctypes.c_int32), ("tile_keys", ctypes.c_int32),
        ("chunk_keys", ctypes.c_int32), ("total_splits", ctypes.c_int32),
        ("row_tile", ctypes.c_int32), ("row_tiles", ctypes.c_int32), ("num_sms", ctypes.c_int32),
        ("q_latent_row_stride", ctypes.c_int32), ("q_rope_row_stride", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_int64), ("off_partial_lse", ctypes.c_int64),
        ("off_partial_o", ctypes.c_int64), ("fused_combine", ctypes.c_int32),
        ("wait_limit_us", ctypes.c_int32), ("reserved", ctypes.c_int32 * 6),
    ]

    def as_dict(self) -> dict:
        return {k: getattr(self, k) for k, _ in self._fields_ if k != "reserved"}


class Rope(ctypes.Structure):
    """A rotation (ddtree_rope_t), made by ddtree_rope_init."""
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("mscale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turns", ctypes.c_uint64 * 128)]


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class _Cache8Struct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + \
               [(n, ctypes.c_int64) for n in ("n_pages", "page_stride", "token_stride", "head_stride")] + \
               [(n, ctypes.c_int32) for n in ("page_size", "n_kv_heads", "head_dim", "block_tokens")]


class DraftPlan(ctypes.Structure):
    """ddtree_draft_plan_t (include/ddtree_draft.h)."""
    _fields_ = [(n, ctypes.c_int32) for n in ("n_tokens", "n_heads", "n_kv_heads", "head_dim", "dtype", "page_size",
                                              "window", "n_sinks", "row_tile", "tile_keys", "n_shares", "wait_limit_us")] + \
               [(n, ctypes.c_int64) for n in ("q_stride", "out_stride", "workspace_bytes")]


class Draft8Plan(ctypes.Structure):
    """ddtree_draft8_plan_t (include/ddtree_draft8.h)."""
    _fields_ = [(n, ctypes.c_int32) for n in ("n_tokens", "n_heads", "n_kv_heads", "head_dim", "dtype", "page_size", "block_tokens",
                                              "window", "n_sinks", "row_tiles", "tile_keys", "n_shares")] + \
               [(n, ctypes.c_int64) for n in ("q_stride", "out_stride", "workspace_bytes")]


class PromptPlan(ctypes.Structure):
    """ddtree_prompt_plan_t (include/ddtree_prompt.h)."""
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "n_heads", "n_kv_heads", "head_dim", "dtype", "window", "n_sinks", "q_rows", "k_rows",
                                              "wait_limit_us", "tile_tokens", "max_items")] + \
               [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride", "out_stride", "workspace_bytes")]


class DDTreeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {code} ({ddtree_status_str(code)})")


_lib = None


def library() -> ctypes.CDLL:
    """Load the in-tree library once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                           "(run speculative_decode_tree_gb300.build.build())")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    P = ctypes.POINTER(Plan)
    L.ddtree_verify_mla_plan.argtypes = [i32, i32, i32, vp, i64, P]
    L.ddtree_verify_mla_plan_ex.argtypes = [i32, i32, i32, vp, i64, i32, i32, P]
    L.ddtree_verify_mla_workspace_size.argtypes = [P]
    L.ddtree_verify_mla_workspace_size.restype = sz
    L.ddtree_verify_mla.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, f32, vp, vp, vp, vp]
    L.ddtree_verify_mla_batched.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, f32, vp, vp, vp, sz, vp]
    L.ddtree_verify_mla_batched_timed.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, f32, vp, vp, vp, sz,
                                                  vp, vp]
    L.ddtree_build_ancestor_mask.argtypes = [vp, i32, i32, vp, vp, vp]
    L.ddtree_verify_mla_noalloc.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, f32, vp, vp, vp]
    L.ddtree_verify_mla_check.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
    L.ddtree_status_str.argtypes = [i32]
    L.ddtree_status_str.restype = ctypes.c_char_p
    L.ddtree_accept_greedy_workspace_size.argtypes = [i32, i32]
    L.ddtree_accept_greedy_workspace_size.restype = sz
    L.ddtree_accept_greedy.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.ddtree_accept_greedy.restype = i32
    L.ddtree_relocate_kv_workspace_size.argtypes = [i64]
    L.ddtree_relocate_kv_workspace_size.restype = sz
    L.ddtree_relocate_kv.argtypes = [i32, i64, vp, i64, vp, vp, vp, vp, vp, sz, vp]
    L.ddtree_relocate_kv.restype = i32
    L.ddtree_tree_from_mask_workspace_size.argtypes = [i32, i32]
    L.ddtree_tree_from_mask_workspace_size.restype = sz
    L.ddtree_tree_from_mask.argtypes = [i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.ddtree_tree_from_mask.restype = i32
    L.ddtree_step_maps.argtypes = [i32, i32, i32, i64, vp, i32, i32, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp,
                                   vp, vp, i64, vp, vp, vp, vp, vp, vp]
    L.ddtree_step_maps.restype = i32
    f64 = ctypes.c_double
    L.ddtree_rope_init.argtypes = [i32, i32, f64, i32, f64, i32, f64, f64, f64, vp]
    L.ddtree_rope_init.restype = i32
    L.ddtree_mla_append.argtypes = [i64, i32, vp, vp, i64, vp, f32, vp, i64, i64, vp, vp, vp, i64, vp, i64, i64, vp, vp]
    L.ddtree_mla_append.restype = i32
    L.ddtree_draft_append.argtypes = [i64, i32, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp, f32, vp, vp, vp, i64, vp, vp]
    L.ddtree_draft_append.restype = i32
    L.ddtree_draft_attention_plan.argtypes = [i32, i32, vp, i32, i32, i32, vp]
    L.ddtree_draft_attention_plan.restype = i32
    L.ddtree_draft_attention_workspace_size.argtypes = [vp]
    L.ddtree_draft_attention_workspace_size.restype = sz
    L.ddtree_draft_attention.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, f32, vp, vp, vp, sz, vp]
    L.ddtree_draft_attention.restype = i32
    L.ddtree_draft8_append.argtypes = [i64, i32, i32, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp, f32, vp, vp, vp, i64, vp, vp]
    L.ddtree_draft8_append.restype = i32
    L.ddtree_draft8_read.argtypes = [i64, i32, vp, vp, vp, i64, vp, i64, vp, vp]
    L.ddtree_draft8_read.restype = i32
    L.ddtree_draft8_attention_plan.argtypes = [i32, i32, vp, i32, i32, i32, i32, vp]
    L.ddtree_draft8_attention_plan.restype = i32
    L.ddtree_draft8_attention_workspace_size.argtypes = [vp]
    L.ddtree_draft8_attention_workspace_size.restype = sz
    L.ddtree_draft8_attention.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, f32, vp, vp, vp, sz, vp]
    L.ddtree_draft8_attention.restype = i32
    L.ddtree_prompt_attention_plan.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, vp]
    L.ddtree_prompt_attention_plan.restype = i32
    L.ddtree_prompt_attention_workspace_size.argtypes = [vp]
    L.ddtree_prompt_attention_workspace_size.restype = sz
    L.ddtree_prompt_attention.argtypes = [vp, vp, vp, vp, vp, vp, f32, vp, vp, vp, sz, vp]
    L.ddtree_prompt_attention.restype = i32
    for name in ("ddtree_verify_mla_plan", "ddtree_verify_mla_plan_ex", "ddtree_verify_mla",
                 "ddtree_verify_mla_batched", "ddtree_build_ancestor_mask", "ddtree_verify_mla_check",
                 "ddtree_verify_mla_batched_timed", "ddtree_verify_mla_noalloc"):
        getattr(L, name).restype = i32
    _lib = L
    return L


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dev(t: torch.Tensor, dtype: torch.dtype, name: str, numel: Optional[int] = None,
         contiguous: bool = True, device: Optional[int] = None) -> int:
    """Device pointer of `t` after checking what the kernels rely on: a CUDA
    tensor of `dtype` on the current device (`device`, when the caller looked
    it up once for several tensors), contiguous (unless the caller checks its
    layout), holding at least `numel` elements.  The C ABI trusts the sizes it
    derives itself, so an undersized or foreign buffer is rejected here,
    before any launch."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    cur = torch.cuda.current_device() if device is None else device
    if t.get_device() != cur:
        raise ValueError(f"{name} is on {t.device}, not the current device cuda:{cur}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs at least {numel}")
    return t.data_ptr()


def _q(t: torch.Tensor, name: str, rows: int, width: int, row_stride: int, device: Optional[int] = None) -> int:
    """Pointer of a query operand: `rows` rows of `width` bf16 values whose
    starts are `row_stride` elements apart (width when 0), e.g. views
    q[..., :512] and q[..., 512:] of one [tokens, heads, 576] tensor."""
    stride = row_stride or width
    _dev(t, torch.bfloat16, name, contiguous=False, device=device)
    shape, strides = t.shape, t.stride()
    if len(shape) < 2 or shape[-1] != width or strides[-1] != 1 or t.numel() != rows * width:
        raise ValueError(f"{name} must be [..., {width}] with {rows} rows of unit-stride elements")
    expect = stride
    for d in range(len(shape) - 2, -1, -1):  # every leading dimension steps whole rows
        if shape[d] > 1 and strides[d] != expect:
            raise ValueError(f"{name}: row stride must be {stride} elements (plan q_*_row_stride)")
        expect *= shape[d]
    return t.data_ptr()


# The current stream's handle without a Stream object around it (0.2 us instead
# of 3 us of host time); the public call where torch has no such function.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(rc: int, where: str) -> None:
    if rc != DDTREE_OK:
        raise DDTreeError(rc, where)


def ddtree_status_str(code: int) -> str:
    return library().ddtree_status_str(int(code)).decode()


def ddtree_verify_mla_plan(batch: int, n_nodes: int, n_heads: int, prefix_lens: Sequence[int],
                           pool_rows: int) -> Plan:
    arr = (ctypes.c_int32 * max(len(prefix_lens), 1))(*[int(p) for p in prefix_lens])
    plan = Plan()
    _check(library().ddtree_verify_mla_plan(batch, n_nodes, n_heads, ctypes.cast(arr, ctypes.c_void_p),
                                            int(pool_rows), ctypes.byref(plan)), "plan")
    return plan


def ddtree_verify_mla_plan_ex(batch: int, n_nodes: int, n_heads: int, prefix_lens: Sequence[int],
                              pool_rows: int, num_sms: int, kernel: int = DDTREE_KERNEL_AUTO) -> Plan:
    arr = (ctypes.c_int32 * max(len(prefix_lens), 1))(*[int(p) for p in prefix_lens])
    plan = Plan()
    _check(library().ddtree_verify_mla_plan_ex(batch, n_nodes, n_heads, ctypes.cast(arr, ctypes.c_void_p),
                                               int(pool_rows), int(num_sms), int(kernel),
                                               ctypes.byref(plan)), "plan_ex")
    return plan


def ddtree_verify_mla_workspace_size(plan: Plan) -> int:
    return int(library().ddtree_verify_mla_workspace_size(ctypes.byref(plan)))


def ddtree_verify_mla(q_latent, q_rope, kv_pool, kv_indices, prefix_len: int, tree_parent,
                      n_nodes: int, n_heads: int, sm_scale: float, out, lse, workspace,
                      stream=None) -> None:
    bf, i32 = torch.bfloat16, torch.int32
    lib = library()
    rows = int(n_nodes) * int(n_heads)
    args = (_dev(q_latent, bf, "q_latent", rows * 512), _dev(q_rope, bf, "q_rope", rows * 64),
            _dev(kv_pool, bf, "kv_pool"), _dev(kv_indices, i32, "kv_indices", int(prefix_len) + int(n_nodes)),
            int(prefix_len), _dev(tree_parent, i32, "tree_parent", int(n_nodes)),
            int(n_nodes), int(n_heads), float(sm_scale), _dev(out, bf, "out", rows * 512),
            _dev(lse, torch.float32, "lse", rows))
    # The workspace must hold what the library's own plan for this shape needs.
    plan = ddtree_verify_mla_plan(1, n_nodes, n_heads, [prefix_len], 0)
    rc = lib.ddtree_verify_mla(*args, _dev(workspace, torch.uint8, "workspace", plan.workspace_bytes),
                               _stream(stream))
    _check(rc, "ddtree_verify_mla")


def ddtree_verify_mla_noalloc(q_latent, q_rope, kv_pool, kv_indices, prefix_len: int, tree_parent,
                              n_nodes: int, n_heads: int, sm_scale: float, out, lse,
                              stream=None) -> None:
    """ddtree_verify_mla without a workspace: for callers that cannot allocate
    device memory; the partials use the library's built-in scratch array."""
    bf, i32 = torch.bfloat16, torch.int32
    rows = int(n_nodes) * int(n_heads)
    rc = library().ddtree_verify_mla_noalloc(
        _dev(q_latent, bf, "q_latent", rows * 512), _dev(q_rope, bf, "q_rope", rows * 64),
        _dev(kv_pool, bf, "kv_pool"), _dev(kv_indices, i32, "kv_indices", int(prefix_len) + int(n_nodes)),
        int(prefix_len), _dev(tree_parent, i32, "tree_parent", int(n_nodes)),
        int(n_nodes), int(n_heads), float(sm_scale), _dev(out, bf, "out", rows * 512),
        _dev(lse, torch.float32, "lse", rows), _stream(stream))
    _check(rc, "ddtree_verify_mla_noalloc")


def _batched_args(plan: Plan, q_latent, q_rope, kv_pool, kv_indices, kv_indptr, prefix_lens, tree_parent,
                  sm_scale, out, lse, workspace):
    bf, i32 = torch.bfloat16, torch.int32
    b, t, rows = plan.batch, plan.n_nodes, plan.batch * plan.rows_per_req
    pool_numel = plan.pool_rows * 576 if plan.pool_rows > 0 else None
    ql = _q(q_latent, "q_latent", rows, 512, plan.q_latent_row_stride)  # a CUDA tensor on the current device
    d = q_latent.get_device()  # so the current device, for the call's other tensors
    return (ctypes.byref(plan), ql,
            _q(q_rope, "q_rope", rows, 64, plan.q_rope_row_stride, d),
            _dev(kv_pool, bf, "kv_pool", pool_numel, device=d),
            _dev(kv_indices, i32, "kv_indices", device=d), _dev(kv_indptr, i32, "kv_indptr", b + 1, device=d),
            _dev(prefix_lens, i32, "prefix_lens", b, device=d), _dev(tree_parent, i32, "tree_parent", b * t, device=d),
            float(sm_scale), _dev(out, bf, "out", rows * 512, device=d), _dev(lse, torch.float32, "lse", rows, device=d),
            _dev(workspace, torch.uint8, "workspace", plan.workspace_bytes, device=d), workspace.numel())


def ddtree_verify_mla_batched(plan: Plan, q_latent, q_rope, kv_pool, kv_indices, kv_indptr,
                              prefix_lens, tree_parent, sm_scale: float, out, lse, workspace,
                              stream=None) -> None:
    rc = library().ddtree_verify_mla_batched(
        *_batched_args(plan, q_latent, q_rope, kv_pool, kv_indices, kv_indptr, prefix_lens, tree_parent,
                       sm_scale, out, lse, workspace), _stream(stream))
    _check(rc, "ddtree_verify_mla_batched")


class BoundVerify:
    """ddtree_verify_mla_batched with its arguments checked and marshalled
    once, for callers whose buffers stay the same from call to call (a decode
    loop with static buffers).  Calling the object launches the verify on
    `stream`.  It keeps references to the plan and tensors; they must not be
    resized or moved in place (`resize_`, `set_`) while the object is used."""

    def __init__(self, plan: Plan, q_latent, q_rope, kv_pool, kv_indices, kv_indptr, prefix_lens,
                 tree_parent, sm_scale: float, out, lse, workspace):
        self._keep = (plan, q_latent, q_rope, kv_pool, kv_indices, kv_indptr, prefix_lens, tree_parent,
                      out, lse, workspace)
        self._args = _batched_args(plan, q_latent, q_rope, kv_pool, kv_indices, kv_indptr, prefix_lens,
                                   tree_parent, sm_scale, out, lse, workspace)
        self._fn = library().ddtree_verify_mla_batched

    def __call__(self, stream=None) -> None:
        _check(self._fn(*self._args, _stream(stream)), "ddtree_verify_mla_batched")


def ddtree_verify_mla_batched_timed(plan: Plan, q_latent, q_rope, kv_pool, kv_indices, kv_indptr,
                                    prefix_lens, tree_parent, sm_scale: float, out, lse, workspace,
                                    stage_events, stream=None) -> None:
    """As ddtree_verify_mla_batched, recording three torch.cuda.Event objects
    (before the partial kernel, between partial and combine, after combine)."""
    evs = (ctypes.c_void_p * 3)(*[None if e is None else e.cuda_event for e in stage_events])
    rc = library().ddtree_verify_mla_batched_timed(
        *_batched_args(plan, q_latent, q_rope, kv_pool, kv_indices, kv_indptr, prefix_lens, tree_parent,
                       sm_scale, out, lse, workspace), _stream(stream), ctypes.cast(evs, ctypes.c_void_p))
    _check(rc, "ddtree_verify_mla_batched_timed")


def ddtree_build_ancestor_mask(tree_parent, batch: int, n_nodes: int, anc_out, status=None,
                               stream=None) -> None:
    rc = library().ddtree_build_ancestor_mask(
        _dev(tree_parent, torch.int32, "tree_parent"), int(batch), int(n_nodes),
        _dev(anc_out, torch.int64, "anc_out"),
        None if status is None else _dev(status, torch.int32, "status"), _stream(stream))
    _check(rc, "ddtree_build_ancestor_mask")


def ddtree_verify_mla_check(workspace, stream=None) -> int:
    """Synchronising read of the device status word; returns its DDTREE_ST_* bits."""
    v = ctypes.c_uint32(0)
    rc = library().ddtree_verify_mla_check(_dev(workspace, torch.uint8, "workspace"), _stream(stream),
                                           ctypes.byref(v))
    if rc not in (DDTREE_OK, DDTREE_EDEVICE_DATA):
        raise DDTreeError(rc, "ddtree_verify_mla_check")
    return int(v.value)


def ddtree_accept_greedy_workspace_size(batch: int, n_nodes: int) -> int:
    return int(library().ddtree_accept_greedy_workspace_size(int(batch), int(n_nodes)))


def ddtree_accept_greedy(logits: torch.Tensor, draft_tokens: torch.Tensor, tree_parent: torch.Tensor,
                         kv_indices: torch.Tensor, kv_indptr: torch.Tensor, prefix_lens: torch.Tensor,
                         accept_len: torch.Tensor, next_token: torch.Tensor, accepted_nodes: torch.Tensor,
                         commit_indices: torch.Tensor, freed_indices: torch.Tensor, workspace: torch.Tensor,
                         stream=None) -> None:
    """Greedy acceptance + commit (include/ddtree_accept.h).  logits [B, T+1, V]
    bf16; the int32 outputs are [B] and [B, T]."""
    B, T1, V = logits.shape
    T = T1 - 1
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    i32 = torch.int32
    _check(library().ddtree_accept_greedy(
        B, T, V, _dev(logits, torch.bfloat16, "logits"), _dev(draft_tokens, i32, "draft_tokens"),
        _dev(tree_parent, i32, "tree_parent"), _dev(kv_indices, i32, "kv_indices"),
        _dev(kv_indptr, i32, "kv_indptr"), _dev(prefix_lens, i32, "prefix_lens"),
        _dev(accept_len, i32, "accept_len"), _dev(next_token, i32, "next_token"),
        _dev(accepted_nodes, i32, "accepted_nodes"), _dev(commit_indices, i32, "commit_indices"),
        _dev(freed_indices, i32, "freed_indices"), _dev(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream)), "accept_greedy")


def ddtree_relocate_kv_workspace_size(pool_rows: int) -> int:
    return int(library().ddtree_relocate_kv_workspace_size(int(pool_rows)))


def ddtree_relocate_kv(kv_pool: torch.Tensor, kv_indices: torch.Tensor, kv_indptr: torch.Tensor,
                       dest_base: torch.Tensor, total_rows: int, workspace: torch.Tensor,
                       old_indices: Optional[torch.Tensor] = None, stream=None) -> None:
    """Tier-1 relocation (include/ddtree_relocate.h): moves each request's rows
    to [dest_base[b], dest_base[b] + n_b) and rewrites kv_indices in place."""
    i32 = torch.int32
    _check(library().ddtree_relocate_kv(
        int(dest_base.numel()), int(total_rows), _dev(kv_pool, torch.bfloat16, "kv_pool"), int(kv_pool.shape[0]),
        _dev(kv_indices, i32, "kv_indices"), _dev(kv_indptr, i32, "kv_indptr"), _dev(dest_base, i32, "dest_base"),
        None if old_indices is None else _dev(old_indices, i32, "old_indices"),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)), "relocate_kv")


def ddtree_tree_from_mask_workspace_size(batch: int, n_nodes: int) -> int:
    return int(library().ddtree_tree_from_mask_workspace_size(int(batch), int(n_nodes)))


def ddtree_tree_from_mask(custom_mask: torch.Tensor, mask_indptr: torch.Tensor, prefix_lens: torch.Tensor,
                          tree_parent: torch.Tensor, workspace: torch.Tensor,
                          anc_bits: Optional[torch.Tensor] = None, stream=None) -> None:
    """Flattened custom tree mask -> parent array (include/ddtree_mask.h).
    custom_mask uint8 (or bool) flat; tree_parent int32 [B, T] output."""
    m = custom_mask.view(torch.uint8) if custom_mask.dtype == torch.bool else custom_mask
    B_, T = tree_parent.shape
    _check(library().ddtree_tree_from_mask(
        int(B_), int(T), _dev(m, torch.uint8, "custom_mask"), _dev(mask_indptr, torch.int64, "mask_indptr"),
        _dev(prefix_lens, torch.int32, "prefix_lens"), _dev(tree_parent, torch.int32, "tree_parent"),
        None if anc_bits is None else _dev(anc_bits, torch.int64, "anc_bits"),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)), "tree_from_mask")


class _Bound:
    """A call whose arguments are checked and marshalled once, for callers
    whose buffers stay the same (see BoundVerify).  Calling the object launches
    on `stream`, with the device of the buffers current.  It keeps references
    to the tensors; they must not be resized or moved in place while the object
    is used.  Plans, rotations and a cache's layout are kept as they were when
    they were checked: later changes of the caller's do not reach the call."""
    _entry = ""

    def _bind(self, args, keep) -> None:
        lib = library()
        # Arguments are converted here, not at every call: a function object of
        # its own without argument types takes the converted ones as they are
        # (1.2 us instead of 2.8 us for 26 arguments).
        types = getattr(lib, self._entry).argtypes
        self._args, self._keep = tuple(t.from_param(v) for t, v in zip(types, args, strict=False)), keep
        self._fn = lib[self._entry]
        self._fn.restype = ctypes.c_int
        self._device = torch.cuda.current_device()

    def __call__(self, stream=None) -> None:
        device = torch.cuda.current_device()
        if device != self._device:
            raise ValueError(f"{self._entry}: bound on cuda:{self._device}, which is not the current device")
        handle = _raw_stream(device) if stream is None and _raw_stream is not None else _stream(stream)
        rc = self._fn(*self._args, ctypes.c_void_p(handle))
        if rc != DDTREE_OK:
            raise DDTreeError(rc, self._entry)


def _kept(x):
    """A copy of a plan, a rotation or a cache (whose tensors stay the same)."""
    if isinstance(x, (DraftCache, Draft8Cache)):
        own = copy.copy(x)
        own.struct = _kept(x.struct)
        return own
    return type(x).from_buffer_copy(x)


def _opt(t: Optional[torch.Tensor], dtype: torch.dtype, name: str, numel: Optional[int] = None,
         device: Optional[int] = None) -> Optional[int]:
    return None if t is None else _dev(t, dtype, name, numel, device=device)


def _maps_args(page_table, prefix_lens, max_new, page_size, n_pages, kv_indptr, kv_indices, new_slots, positions,
               table_row, new_lens, tree_parent, pages_held, free_pages, free_head, pages_held_out, free_head_out,
               new_indptr, token_rows, status):
    i32 = torch.int32
    table = _dev(page_table, i32, "page_table")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [rows, pages of a row]")
    d = page_table.get_device()
    b, t = int(prefix_lens.numel()), int(max_new)
    n_free = 0 if free_pages is None else int(free_pages.numel())
    indptr = _dev(kv_indptr, i32, "kv_indptr", b + 1, device=d)
    indices = _opt(kv_indices, i32, "kv_indices", device=d)
    if kv_indices is not None and kv_indices.numel() == 0:
        indices = indptr  # an empty list has no address, and a null one asks for none; nothing is written there
    return (b, t, int(page_size), int(n_pages), table, int(page_table.shape[0]), int(page_table.shape[1]),
            _opt(table_row, i32, "table_row", b, d), _dev(prefix_lens, i32, "prefix_lens", device=d),
            _opt(new_lens, i32, "new_lens", b, d), _opt(tree_parent, i32, "tree_parent", b * t, d),
            _opt(pages_held, i32, "pages_held", b, d), _opt(free_pages, i32, "free_pages", device=d), n_free,
            _opt(free_head, i32, "free_head", 1, d), _opt(pages_held_out, i32, "pages_held_out", b, d),
            _opt(free_head_out, i32, "free_head_out", 1, d), indptr,
            indices, 0 if kv_indices is None else int(kv_indices.numel()),
            _opt(new_indptr, i32, "new_indptr", b + 1, d), _dev(new_slots, i32, "new_slots", b * t, device=d),
            _dev(positions, i32, "positions", b * t, device=d), _opt(token_rows, i32, "token_rows", b * t, d),
            _opt(status, i32, "status", 1, d))


def ddtree_step_maps(page_table: torch.Tensor, prefix_lens: torch.Tensor, max_new: int, page_size: int, n_pages: int,
                     kv_indptr: torch.Tensor, kv_indices: Optional[torch.Tensor], new_slots: torch.Tensor,
                     positions: torch.Tensor, *, table_row: Optional[torch.Tensor] = None,
                     new_lens: Optional[torch.Tensor] = None, tree_parent: Optional[torch.Tensor] = None,
                     pages_held: Optional[torch.Tensor] = None, free_pages: Optional[torch.Tensor] = None,
                     free_head: Optional[torch.Tensor] = None, pages_held_out: Optional[torch.Tensor] = None,
                     free_head_out: Optional[torch.Tensor] = None, new_indptr: Optional[torch.Tensor] = None,
                     token_rows: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """Page-table growth, verify index layout, slots and positions of a step
    from the requests' lengths (include/ddtree_maps.h).  page_table int32
    [rows, pages of a row], grown in place; the batch is prefix_lens.numel()."""
    _check(library().ddtree_step_maps(
        *_maps_args(page_table, prefix_lens, max_new, page_size, n_pages, kv_indptr, kv_indices, new_slots, positions,
                    table_row, new_lens, tree_parent, pages_held, free_pages, free_head, pages_held_out,
                    free_head_out, new_indptr, token_rows, status), _stream(stream)), "ddtree_step_maps")


class BoundStepMaps(_Bound):
    """ddtree_step_maps with its arguments checked and marshalled once."""
    _entry = "ddtree_step_maps"

    def __init__(self, page_table, prefix_lens, max_new: int, page_size: int, n_pages: int, kv_indptr, kv_indices,
                 new_slots, positions, *, table_row=None, new_lens=None, tree_parent=None, pages_held=None,
                 free_pages=None, free_head=None, pages_held_out=None, free_head_out=None, new_indptr=None,
                 token_rows=None, status=None):
        a = (page_table, prefix_lens, max_new, page_size, n_pages, kv_indptr, kv_indices, new_slots, positions,
             table_row, new_lens, tree_parent, pages_held, free_pages, free_head, pages_held_out, free_head_out,
             new_indptr, token_rows, status)
        self._bind(_maps_args(*a), a)


def ddtree_rope_init(rot_dim: int, *, theta: float, interleaved: bool = False, scaling: int = DDTREE_ROPE_PLAIN,
                     factor: float = 1.0, original_positions: int = 1, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     mscale: float = 0.0) -> Rope:
    """A rotation for the append calls (include/ddtree_append.h); host only.
    DDTREE_ROPE_YARN needs `factor` and `original_positions`."""
    rope = Rope()
    _check(library().ddtree_rope_init(int(rot_dim), int(bool(interleaved)), float(theta), int(scaling), float(factor),
                                      int(original_positions), float(beta_fast), float(beta_slow), float(mscale),
                                      ctypes.addressof(rope)), "ddtree_rope_init")
    return rope


def _rows(t: torch.Tensor, dtype: torch.dtype, name: str, shape: tuple, device: int) -> int:
    """Pointer of a strided tensor of `shape` whose last dimension is dense."""
    p = _dev(t, dtype, name, contiguous=False, device=device)
    if tuple(t.shape) != shape or t.stride(-1) != 1:
        raise ValueError(f"{name} must be {list(shape)} with unit-stride columns, got {list(t.shape)}")
    return p


def _step(t: torch.Tensor, d: int, least: int) -> int:
    """Stride of dimension d; a dimension of one element has none of its own."""
    return int(t.stride(d)) if t.shape[d] > 1 else least


def _mla_append_args(rope, kv_new, positions, slots, kv_pool, latent_weight, eps, q_rope, q_out, status):
    bf, i32 = torch.bfloat16, torch.int32
    if kv_new.dim() != 2 or kv_pool.dim() != 2 or kv_pool.shape[1] != 576:
        raise ValueError("kv_new must be [tokens, 576] and kv_pool [rows, 576]")
    pool = _dev(kv_pool, bf, "kv_pool")
    d, n = kv_pool.get_device(), int(kv_new.shape[0])
    kv = _rows(kv_new, bf, "kv_new", (n, 576), d)
    heads, q, o = 0, (None, 64, 64), (None, 64, 64)
    if (q_rope is None) != (q_out is None):
        raise ValueError("q_rope and q_out come together")
    if q_rope is not None and q_rope.numel() > 0:
        heads = int(q_rope.shape[1])
        q = (_rows(q_rope, bf, "q_rope", (n, heads, 64), d), _step(q_rope, 0, 64), _step(q_rope, 1, 64))
        o = (_rows(q_out, bf, "q_out", (n, heads, 64), d), _step(q_out, 0, 64), _step(q_out, 1, 64))
    return (n, heads, ctypes.addressof(rope), kv, _step(kv_new, 0, 576),
            _opt(latent_weight, bf, "latent_weight", 512, d), float(eps), *q,
            _dev(positions, i32, "positions", n, device=d), _dev(slots, i32, "slots", n, device=d), pool,
            int(kv_pool.shape[0]), *o, _opt(status, i32, "status", 1, d))


def ddtree_mla_append(rope: Rope, kv_new: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
                      kv_pool: torch.Tensor, *, latent_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      q_rope: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                      status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Norm, rotation and pool rows of new tokens, and their queries' rope part
    (include/ddtree_append.h).  kv_new [N, 576] (rows may be strided), q_rope
    and q_out [N, H, 64] (tokens and heads may be strided; q_out may be q_rope)."""
    _check(library().ddtree_mla_append(
        *_mla_append_args(rope, kv_new, positions, slots, kv_pool, latent_weight, eps, q_rope, q_out, status),
        _stream(stream)), "ddtree_mla_append")


class BoundMlaAppend(_Bound):
    """ddtree_mla_append with its arguments checked and marshalled once."""
    _entry = "ddtree_mla_append"

    def __init__(self, rope: Rope, kv_new, positions, slots, kv_pool, *, latent_weight=None, eps: float = 1e-6,
                 q_rope=None, q_out=None, status=None):
        a = (_kept(rope), kv_new, positions, slots, kv_pool, latent_weight, eps, q_rope, q_out, status)
        self._bind(_mla_append_args(*a), a)


class DraftCache:
    """The drafter's paged cache (ddtree_draft_cache_t): k and v are
    [pages, page_size, kv_heads, head_dim] tensors of one dtype (bf16 or fp16)
    and equal strides; a view with the heads outside the tokens serves too."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        dtype = {torch.bfloat16: DDTREE_BF16, torch.float16: DDTREE_FP16}.get(k.dtype)
        if dtype is None:
            raise TypeError(f"a draft cache is bfloat16 or float16, got {k.dtype}")
        if k.dim() != 4:
            raise ValueError("a draft cache is [pages, page_size, kv_heads, head_dim]")
        kp = _rows(k, k.dtype, "k cache", tuple(k.shape), torch.cuda.current_device())
        vp = _rows(v, k.dtype, "v cache", tuple(k.shape), k.get_device())
        step = [_step(k, d, int(k.shape[3])) for d in range(3)]
        if step != [_step(v, d, int(k.shape[3])) for d in range(3)]:
            raise ValueError("the key and value caches must have equal strides")
        self.k, self.v = k, v
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = (int(x) for x in k.shape)
        self.struct = _CacheStruct(kp, vp, self.n_pages, *step, self.page_size, self.n_kv_heads, self.head_dim, dtype)


def _cache_device(cache: DraftCache) -> int:
    """The cache's device, which must be the current one: the call launches there."""
    d = cache.k.get_device()
    if d != torch.cuda.current_device():
        raise ValueError(f"the cache is on {cache.k.device}, not the current device")
    return d


def _draft_append_args(cache, rope, q, k, v, positions, slots, q_out, q_weight, k_weight, eps, status):
    dt, i32, d = cache.k.dtype, torch.int32, _cache_device(cache)
    n, dim, kvh = int(k.shape[0]), cache.head_dim, cache.n_kv_heads

    def heads(t, name, h):
        p = _rows(t, dt, name, (n, h, dim), d)
        if h > 1 and n and t.stride(1) != dim:
            raise ValueError(f"{name}: heads must be {dim} elements apart")
        return p, _step(t, 0, h * dim)
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    h = int(q.shape[1]) if q is not None else 0
    qa, oa = (heads(q, "q", h), heads(q_out, "q_out", h)) if h else ((None, 0), (None, 0))
    return (n, h, ctypes.addressof(cache.struct), ctypes.addressof(rope), *qa, *heads(k, "k", kvh), *heads(v, "v", kvh),
            _opt(q_weight, dt, "q_weight", dim, d), _opt(k_weight, dt, "k_weight", dim, d), float(eps),
            _dev(positions, i32, "positions", n, device=d), _dev(slots, i32, "slots", n, device=d), *oa,
            _opt(status, i32, "status", 1, d))


def ddtree_draft_append(cache: DraftCache, rope: Rope, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                        positions: torch.Tensor, slots: torch.Tensor, q_out: Optional[torch.Tensor], *,
                        q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                        eps: float = 1e-6, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Head norms, rotation and cache rows of the drafter's new tokens
    (include/ddtree_append.h).  q [N, H, D], k and v [N, Hkv, D] (tokens may be
    strided, as parts of one projection); q_out [N, H, D], which may be q."""
    _check(library().ddtree_draft_append(
        *_draft_append_args(cache, rope, q, k, v, positions, slots, q_out, q_weight, k_weight, eps, status),
        _stream(stream)), "ddtree_draft_append")


class BoundDraftAppend(_Bound):
    """ddtree_draft_append with its arguments checked and marshalled once."""
    _entry = "ddtree_draft_append"

    def __init__(self, cache: DraftCache, rope: Rope, q, k, v, positions, slots, q_out, *, q_weight=None, k_weight=None,
                 eps: float = 1e-6, status=None):
        a = (_kept(cache), _kept(rope), q, k, v, positions, slots, q_out, q_weight, k_weight, eps, status)
        self._bind(_draft_append_args(*a), a)


def ddtree_draft_attention_plan(n_tokens: int, n_heads: int, cache: DraftCache, window: int = 0, n_sinks: int = 0,
                                num_sms: int = 0) -> DraftPlan:
    """Plan of the drafter's attention (include/ddtree_draft.h): one for all lengths."""
    plan = DraftPlan()
    _check(library().ddtree_draft_attention_plan(int(n_tokens), int(n_heads), ctypes.addressof(cache.struct), int(window),
                                                 int(n_sinks), int(num_sms), ctypes.addressof(plan)), "draft_attention_plan")
    return plan


def ddtree_draft_attention_workspace_size(plan: DraftPlan) -> int:
    return int(library().ddtree_draft_attention_workspace_size(ctypes.addressof(plan)))


def _draft_attention_args(plan, q, cache, page_table, positions, sm_scale, out, workspace, token_rows, lse):
    dt, i32, d = cache.k.dtype, torch.int32, _cache_device(cache)
    n, h, dim = plan.n_tokens, plan.n_heads, plan.head_dim
    if cache.head_dim != dim:
        raise ValueError("the plan was made for another cache")

    def heads(t, name, stride):
        p = _rows(t, dt, name, (n, h, dim), d)
        if (h > 1 and t.stride(1) != dim) or (n > 1 and t.stride(0) != (stride or h * dim)):
            raise ValueError(f"{name}: heads must be {dim} and tokens {stride or h * dim} elements apart (plan q_stride, out_stride)")
        return p
    table = _dev(page_table, i32, "page_table", device=d)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [rows, pages of a row]")
    return (ctypes.addressof(plan), heads(q, "q", plan.q_stride), ctypes.addressof(cache.struct), table,
            int(page_table.shape[0]), int(page_table.shape[1]), _opt(token_rows, i32, "token_rows", n, d),
            _dev(positions, i32, "positions", n, device=d), float(sm_scale), heads(out, "out", plan.out_stride),
            _opt(lse, torch.float32, "lse", n * h, d),
            _dev(workspace, torch.uint8, "workspace", plan.workspace_bytes, device=d), int(workspace.numel()))


def ddtree_draft_attention(plan: DraftPlan, q: torch.Tensor, cache: DraftCache, page_table: torch.Tensor,
                           positions: torch.Tensor, sm_scale: float, out: torch.Tensor, workspace: torch.Tensor, *,
                           token_rows: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                           stream=None) -> None:
    """The drafter's attention of one new token per request over its paged
    cache (include/ddtree_draft.h).  q and out [N, H, D], lse [N, H].
    Probabilities meet V in the cache's type; everything else is in 32 bits."""
    _check(library().ddtree_draft_attention(
        *_draft_attention_args(plan, q, cache, page_table, positions, sm_scale, out, workspace, token_rows, lse),
        _stream(stream)), "ddtree_draft_attention")


class BoundDraftAttention(_Bound):
    """ddtree_draft_attention with its arguments checked and marshalled once."""
    _entry = "ddtree_draft_attention"

    def __init__(self, plan: DraftPlan, q, cache: DraftCache, page_table, positions, sm_scale: float, out, workspace, *,
                 token_rows=None, lse=None):
        a = (_kept(plan), q, _kept(cache), page_table, positions, sm_scale, out, workspace, token_rows, lse)
        self._bind(_draft_attention_args(*a), a)


_DTYPES = {torch.bfloat16: DDTREE_BF16, torch.float16: DDTREE_FP16}


def _dtype_code(dtype: torch.dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"the type must be bfloat16 or float16, got {dtype}")
    return code


class Draft8Cache:
    """The drafter's paged cache in 8 bits (ddtree_draft8_cache_t): k and v are
    [pages, page_size, kv_heads, head_dim] tensors of float8_e4m3fn (or their
    bytes, uint8) with equal strides, as in DraftCache; k_scale and v_scale
    are contiguous [pages, ceil(page_size / block_tokens), kv_heads] float32
    tensors.  Scales of zero are blocks that nothing was written to."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, block_tokens: int):
        if k.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise TypeError(f"an 8-bit draft cache is float8_e4m3fn or uint8, got {k.dtype}")
        if k.dim() != 4:
            raise ValueError("a draft cache is [pages, page_size, kv_heads, head_dim]")
        kp = _rows(k, k.dtype, "k cache", tuple(k.shape), torch.cuda.current_device())
        d = k.get_device()
        vp = _rows(v, k.dtype, "v cache", tuple(k.shape), d)
        step = [_step(k, i, -(-int(k.shape[3]) // 16) * 16) for i in range(3)]
        if step != [_step(v, i, -(-int(k.shape[3]) // 16) * 16) for i in range(3)]:
            raise ValueError("the key and value caches must have equal strides")
        self.k, self.v, self.k_scale, self.v_scale, self.block_tokens = k, v, k_scale, v_scale, int(block_tokens)
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = (int(x) for x in k.shape)
        if self.block_tokens < 1:
            raise ValueError("block_tokens must be at least 1")
        shape = (self.n_pages, -(-self.page_size // self.block_tokens), self.n_kv_heads)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _dev(t, torch.float32, name, device=d)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        self.struct = _Cache8Struct(kp, vp, k_scale.data_ptr(), v_scale.data_ptr(), self.n_pages, *step, self.page_size,
                                    self.n_kv_heads, self.head_dim, self.block_tokens)


def _head_rows(t, dtype, name, n, h, dim, device):
    """Pointer and row stride of a [n, h, dim] tensor whose heads lie next to each other."""
    p = _rows(t, dtype, name, (n, h, dim), device)
    if h > 1 and n and t.stride(1) != dim:
        raise ValueError(f"{name}: heads must be {dim} elements apart")
    return p, _step(t, 0, h * dim)


def _draft8_append_args(cache, rope, q, k, v, positions, slots, q_out, q_weight, k_weight, eps, status):
    dt, i32, d = k.dtype, torch.int32, _cache_device(cache)
    n, dim, kvh = int(k.shape[0]), cache.head_dim, cache.n_kv_heads
    code = _dtype_code(dt)
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    h = int(q.shape[1]) if q is not None else 0
    qa, oa = (None, 0), (None, 0)
    if h:
        qa, oa = _head_rows(q, dt, "q", n, h, dim, d), _head_rows(q_out, dt, "q_out", n, h, dim, d)
    return (n, h, code, ctypes.addressof(cache.struct), ctypes.addressof(rope), *qa, *_head_rows(k, dt, "k", n, kvh, dim, d),
            *_head_rows(v, dt, "v", n, kvh, dim, d), _opt(q_weight, dt, "q_weight", dim, d), _opt(k_weight, dt, "k_weight", dim, d),
            float(eps), _dev(positions, i32, "positions", n, device=d), _dev(slots, i32, "slots", n, device=d), *oa,
            _opt(status, i32, "status", 1, d))


def ddtree_draft8_append(cache: Draft8Cache, rope: Rope, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                         positions: torch.Tensor, slots: torch.Tensor, q_out: Optional[torch.Tensor], *,
                         q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                         eps: float = 1e-6, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Head norms and rotation of the drafter's new tokens, keys and values
    quantised into their blocks (include/ddtree_draft8.h).  Tensors as in
    ddtree_draft_append; tokens of one block follow one another."""
    _check(library().ddtree_draft8_append(
        *_draft8_append_args(cache, rope, q, k, v, positions, slots, q_out, q_weight, k_weight, eps, status),
        _stream(stream)), "ddtree_draft8_append")


class BoundDraft8Append(_Bound):
    """ddtree_draft8_append with its arguments checked and marshalled once."""
    _entry = "ddtree_draft8_append"

    def __init__(self, cache: Draft8Cache, rope: Rope, q, k, v, positions, slots, q_out, *, q_weight=None, k_weight=None,
                 eps: float = 1e-6, status=None):
        a = (_kept(cache), _kept(rope), q, k, v, positions, slots, q_out, q_weight, k_weight, eps, status)
        self._bind(_draft8_append_args(*a), a)


def _draft8_read_args(cache, slots, k_out, v_out, status):
    d = _cache_device(cache)
    one = k_out if k_out is not None else v_out
    if one is None:
        raise ValueError("one of k_out and v_out at least")
    n, code = int(one.shape[0]), _dtype_code(one.dtype)
    outs = [(None, 0) if t is None else _head_rows(t, one.dtype, name, n, cache.n_kv_heads, cache.head_dim, d)
            for t, name in ((k_out, "k_out"), (v_out, "v_out"))]
    return (n, code, ctypes.addressof(cache.struct), _dev(slots, torch.int32, "slots", n, device=d), *outs[0], *outs[1],
            _opt(status, torch.int32, "status", 1, d))


def ddtree_draft8_read(cache: Draft8Cache, slots: torch.Tensor, k_out: Optional[torch.Tensor], v_out: Optional[torch.Tensor], *,
                       status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Rows of the 8-bit cache in 16 bits (include/ddtree_draft8.h): k_out and
    v_out [N, Hkv, D], bf16 or fp16 (rows may be strided), either may be None."""
    _check(library().ddtree_draft8_read(*_draft8_read_args(cache, slots, k_out, v_out, status), _stream(stream)),
           "ddtree_draft8_read")


class BoundDraft8Read(_Bound):
    """ddtree_draft8_read with its arguments checked and marshalled once."""
    _entry = "ddtree_draft8_read"

    def __init__(self, cache: Draft8Cache, slots, k_out, v_out, *, status=None):
        a = (_kept(cache), slots, k_out, v_out, status)
        self._bind(_draft8_read_args(*a), a)


def ddtree_draft8_attention_plan(n_tokens: int, n_heads: int, cache: Draft8Cache, dtype: torch.dtype, window: int = 0,
                                 n_sinks: int = 0, num_sms: int = 0) -> Draft8Plan:
    """Plan of the drafter's attention over its 8-bit cache (include/ddtree_draft8.h):
    one for all lengths.  dtype: of q and out, bf16 or fp16."""
    plan = Draft8Plan()
    _check(library().ddtree_draft8_attention_plan(int(n_tokens), int(n_heads), ctypes.addressof(cache.struct), _dtype_code(dtype),
                                                  int(window), int(n_sinks), int(num_sms), ctypes.addressof(plan)),
           "draft8_attention_plan")
    return plan


def ddtree_draft8_attention_workspace_size(plan: Draft8Plan) -> int:
    return int(library().ddtree_draft8_attention_workspace_size(ctypes.addressof(plan)))


def _plan_rows(t, dtype, name, n, h, dim, stride, device, fields):
    """Pointer of a [n, h, dim] tensor laid out as a plan says (stride 0: contiguous rows)."""
    p = _rows(t, dtype, name, (n, h, dim), device)
    if (h > 1 and t.stride(1) != dim) or (n > 1 and t.stride(0) != (stride or h * dim)):
        raise ValueError(f"{name}: heads must be {dim} and rows {stride or h * dim} elements apart (plan {fields})")
    return p


def _draft8_attention_args(plan, q, cache, page_table, positions, sm_scale, out, workspace, token_rows, lse):
    dt, i32, d = q.dtype, torch.int32, _cache_device(cache)
    n, h, dim = plan.n_tokens, plan.n_heads, plan.head_dim
    if cache.head_dim != dim:
        raise ValueError("the plan was made for another cache")
    if _dtype_code(dt) != plan.dtype:
        raise TypeError(f"the plan was made for another type than {dt}")
    table = _dev(page_table, i32, "page_table", device=d)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [rows, pages of a row]")
    return (ctypes.addressof(plan), _plan_rows(q, dt, "q", n, h, dim, plan.q_stride, d, "q_stride"),
            ctypes.addressof(cache.struct), table, int(page_table.shape[0]), int(page_table.shape[1]),
            _opt(token_rows, i32, "token_rows", n, d), _dev(positions, i32, "positions", n, device=d), float(sm_scale),
            _plan_rows(out, dt, "out", n, h, dim, plan.out_stride, d, "out_stride"), _opt(lse, torch.float32, "lse", n * h, d),
            _dev(workspace, torch.uint8, "workspace", plan.workspace_bytes, device=d), int(workspace.numel()))


def ddtree_draft8_attention(plan: Draft8Plan, q: torch.Tensor, cache: Draft8Cache, page_table: torch.Tensor,
                            positions: torch.Tensor, sm_scale: float, out: torch.Tensor, workspace: torch.Tensor, *,
                            token_rows: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """ddtree_draft_attention over the 8-bit cache (include/ddtree_draft8.h).
    q and out [N, H, D], lse [N, H]."""
    _check(library().ddtree_draft8_attention(
        *_draft8_attention_args(plan, q, cache, page_table, positions, sm_scale, out, workspace, token_rows, lse),
        _stream(stream)), "ddtree_draft8_attention")


class BoundDraft8Attention(_Bound):
    """ddtree_draft8_attention with its arguments checked and marshalled once."""
    _entry = "ddtree_draft8_attention"

    def __init__(self, plan: Draft8Plan, q, cache: Draft8Cache, page_table, positions, sm_scale: float, out, workspace, *,
                 token_rows=None, lse=None):
        a = (_kept(plan), q, _kept(cache), page_table, positions, sm_scale, out, workspace, token_rows, lse)
        self._bind(_draft8_attention_args(*a), a)


def ddtree_prompt_attention_plan(batch: int, q_rows: int, k_rows: int, n_heads: int, n_kv_heads: int, head_dim: int, dtype: torch.dtype,
                                 window: int = 0, n_sinks: int = 0) -> PromptPlan:
    """Plan of the attention over whole prompts (include/ddtree_prompt.h), for
    packed buffers of q_rows and k_rows rows and up to `batch` sequences of
    any lengths; host only."""
    plan = PromptPlan()
    _check(library().ddtree_prompt_attention_plan(int(batch), int(q_rows), int(k_rows), int(n_heads), int(n_kv_heads), int(head_dim),
                                                  _dtype_code(dtype), int(window), int(n_sinks), ctypes.addressof(plan)),
           "prompt_attention_plan")
    return plan


def ddtree_prompt_attention_workspace_size(plan: PromptPlan) -> int:
    return int(library().ddtree_prompt_attention_workspace_size(ctypes.addressof(plan)))


def _prompt_attention_args(plan, q, k, v, q_indptr, k_indptr, sm_scale, out, workspace, lse):
    dt, i32, f = q.dtype, torch.int32, torch.cuda.current_device()
    if _dtype_code(dt) != plan.dtype:
        raise TypeError(f"the plan was made for another type than {dt}")
    h, kvh, dim = plan.n_heads, plan.n_kv_heads, plan.head_dim
    plan = type(plan).from_buffer_copy(plan)  # the call's own: strides are the tensors' where the plan leaves them out
    pointers = []
    for t, name, rows, heads in ((q, "q", plan.q_rows, h), (k, "k", plan.k_rows, kvh), (v, "v", plan.k_rows, kvh), (out, "out", plan.q_rows, h)):
        p = _rows(t, dt, name, (rows, heads, dim), f)
        if heads > 1 and t.stride(1) != dim:
            raise ValueError(f"{name}: heads must be {dim} elements apart")
        field = f"{name}_stride"
        if getattr(plan, field) == 0:
            setattr(plan, field, _step(t, 0, heads * dim))
        elif rows > 1 and t.stride(0) != getattr(plan, field):
            raise ValueError(f"{name}: rows must be {getattr(plan, field)} elements apart (plan {field})")
        pointers.append(p)
    args = (ctypes.addressof(plan), *pointers[:3], _dev(q_indptr, i32, "q_indptr", plan.batch + 1, device=f),
            _opt(k_indptr, i32, "k_indptr", plan.batch + 1, f), float(sm_scale), pointers[3],
            _opt(lse, torch.float32, "lse", plan.q_rows * h, f),
            _dev(workspace, torch.uint8, "workspace", plan.workspace_bytes, device=f), int(workspace.numel()))
    return args, plan


def ddtree_prompt_attention(plan: PromptPlan, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_indptr: torch.Tensor,
                            k_indptr: Optional[torch.Tensor], sm_scale: float, out: torch.Tensor, workspace: torch.Tensor, *,
                            lse: Optional[torch.Tensor] = None, stream=None) -> None:
    """Causal attention over packed prompts (include/ddtree_prompt.h).  q and
    out [q_rows, H, D], k and v [k_rows, Hkv, D] (rows may be strided, as parts
    of one projection), q_indptr and k_indptr [batch + 1] (None: the same),
    lse [q_rows, H]."""
    args, plan = _prompt_attention_args(plan, q, k, v, q_indptr, k_indptr, sm_scale, out, workspace, lse)
    _check(library().ddtree_prompt_attention(*args, _stream(stream)), "ddtree_prompt_attention")


class BoundPromptAttention(_Bound):
    """ddtree_prompt_attention with its arguments checked and marshalled once."""
    _entry = "ddtree_prompt_attention"

    def __init__(self, plan: PromptPlan, q, k, v, q_indptr, k_indptr, sm_scale: float, out, workspace, *, lse=None):
        args, kept = _prompt_attention_args(plan, q, k, v, q_indptr, k_indptr, sm_scale, out, workspace, lse)
        self._bind(args, (kept, q, k, v, q_indptr, k_indptr, out, workspace, lse))
