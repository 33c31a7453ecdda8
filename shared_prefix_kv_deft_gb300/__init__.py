"""Python binding of the GB300 DeFT tree-attention decode library.

A thin ctypes layer over the C ABI in include/deft.h (libdeft.so, built by
`shared_prefix_kv_deft_gb300.build.build()`): the functions below have the
C names and only marshal arguments.  PyTorch provides device memory and the
current CUDA stream; every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if libdeft.so is missing or a call
fails, an exception is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from dataclasses import dataclass
from typing import Tuple, Optional

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libdeft.so")

DEFT_OUT_BF16 = 0
DEFT_OUT_F32 = 1

# deft_plan_array values (include/deft.h)
ARRAYS = {
    "chunk_seg_off": (0, np.int32), "chunk_q_off": (1, np.int32), "chunk_q": (2, np.int32),
    "seg_node": (3, np.int32), "seg_tok_begin": (4, np.int32), "seg_tok_len": (5, np.int32),
    "seg_mask": (6, np.uint64), "chunk_mask": (7, np.uint64), "q_slot_off": (8, np.int32),
    "q_slot": (9, np.int32), "node_cover": (10, np.uint64), "node_order": (11, np.int32),
    "fma_items": (12, np.int32), "mma_items": (13, np.int32), "fallback_items": (14, np.int32),
    "naive_chunk_seg_off": (15, np.int32), "naive_chunk_q": (16, np.int32),
    "naive_seg_node": (17, np.int32), "naive_seg_tok_begin": (18, np.int32),
    "naive_seg_tok_len": (19, np.int32), "naive_q_slot_off": (20, np.int32),
    "naive_q_slot": (21, np.int32), "fma_direct": (22, np.uint32),
    "fallback_direct": (23, np.uint32), "merge_q": (24, np.int32),
}

# Symbols the header declares (checked by the tests).
EXPORTS = ["deft_plan", "deft_plan_at", "deft_plan_ex", "deft_plan_rebuild", "deft_plan_stats_get",
           "deft_plan_get", "deft_plan_upload", "deft_workspace_bytes", "deft_tree_attn",
           "deft_naive_attn", "deft_tree_attn_ex", "deft_step_status", "deft_check_pages",
           "deft_plan_update", "deft_pages_create", "deft_pages_free", "deft_pages_alloc",
           "deft_pages_retain", "deft_pages_release", "deft_pages_free_count", "deft_pages_refcount",
           "deft_plan_free", "deft_status_str", "deft_version", "deft_trace_enable",
           "deft_trace_read", "deft_tree_attn_noalloc", "deft_tree_attn_host",
           "deft_page_table_workspace_bytes", "deft_page_table", "deft_kv_write", "deft_prompt_plan",
           "deft_prompt_plan_rebuild", "deft_prompt_plan_upload", "deft_prompt_plan_stats_get",
           "deft_prompt_plan_get", "deft_prompt_plan_free", "deft_prompt_workspace_bytes",
           "deft_prompt_attn", "deft_prompt_status", "deft_qkv_write", "deft_qkv_write4", "deft_kv4_page_bytes",
           "deft_kv_unpack4", "deft_tree_attn4"]

KERNEL_NAMES = {0: "phase1_fma", 1: "phase1_mma", 2: "phase2_merge", 3: "phase1_kv4"}
PLAN_TREE_ONLY = 1   # deft_plan_ex flags
PLAN_TENSOR_PACK = 2
# deft_page_table's counts[3]
TABLE_BAD_LENGTH = 1
TABLE_BAD_PREV = 2
TABLE_NO_FREE_PAGE = 4
TABLE_PAGE_CAP = 8
TABLE_TOKEN_CAP = 16
# deft_tree_attn_ex flags
STEP_NAIVE = 1
STEP_CUDA_CORES = 2
STEP_SEPARATE_MERGE = 4


class DeftError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status} ({status_str(status)})")
        self.status = status


class TraceRecord(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("family", ctypes.c_int32),
                ("bucket", ctypes.c_int32), ("fallback", ctypes.c_int32),
                ("items", ctypes.c_int32), ("ms", ctypes.c_float)]


class PlanStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_nodes", "num_queries", "gqa_group", "chunk_target", "mask_words", "num_chunks",
        "num_segments", "num_slots", "num_fma_items", "num_mma_items", "num_fallback_items",
        "max_chunk_tokens", "max_slots_per_query", "naive_num_chunks", "naive_num_slots",
        "naive_num_segments", "num_merge_queries", "reserved0")] + [(n, ctypes.c_int64) for n in (
        "unique_tokens", "naive_tokens", "planned_tokens", "pair_tokens", "device_bytes")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class PromptStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_nodes", "num_prompts", "num_rows", "num_items", "num_units", "num_split_items", "ctas",
        "reserved0")] + [(n, ctypes.c_int64) for n in ("pair_tokens", "partial_slots", "device_bytes")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class QkTurn(ctypes.Structure):
    _fields_ = [("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("num_positions", ctypes.c_int32),
                ("cos_sin", ctypes.c_void_p), ("position", ctypes.c_void_p)]


_lib = None


def load(path: str = LIB_PATH):
    """Load libdeft.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "shared_prefix_kv_deft_gb300.build.build() (no fallback exists)")
    lib = ctypes.CDLL(path)
    P, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    lib.deft_plan.argtypes = [P, P, i32, P, i32, i32, i32, ctypes.POINTER(P)]
    lib.deft_plan_at.argtypes = [P, P, i32, P, P, i32, i32, i32, ctypes.POINTER(P)]
    lib.deft_plan_ex.argtypes = [P, P, i32, P, P, i32, i32, i32, i32, ctypes.POINTER(P)]
    lib.deft_plan_rebuild.argtypes = [P, P, P, i32, P, P, i32, i32, i32, i32]
    lib.deft_plan_stats_get.argtypes = [P, ctypes.POINTER(PlanStats)]
    lib.deft_plan_get.argtypes = [P, i32, P, sz]
    lib.deft_plan_upload.argtypes = [P, P]
    lib.deft_workspace_bytes.argtypes = [P, i32, i32]
    lib.deft_workspace_bytes.restype = sz
    attn = [P, P, P, P, P, i32, i32, i32, i32, i32, f32, P, P, i32, P, P, sz, P]
    lib.deft_tree_attn.argtypes = attn
    lib.deft_naive_attn.argtypes = attn
    lib.deft_tree_attn_ex.argtypes = attn[:-1] + [i32, P]
    lib.deft_tree_attn_host.argtypes = [P] + attn[:-1] + [P, P, P]
    lib.deft_step_status.argtypes = [P, P, ctypes.POINTER(i32)]
    lib.deft_check_pages.argtypes = [P, i32, P, P, ctypes.c_int64, i32, i32]
    lib.deft_plan_update.argtypes = [P, P, i32]
    lib.deft_pages_create.argtypes = [i32, ctypes.POINTER(P)]
    lib.deft_pages_free.argtypes = [P]
    lib.deft_pages_free.restype = None
    for fn in ("deft_pages_alloc", "deft_pages_retain", "deft_pages_release"):
        getattr(lib, fn).argtypes = [P, i32, P]
    lib.deft_pages_free_count.argtypes = [P]
    lib.deft_pages_refcount.argtypes = [P, i32]
    lib.deft_tree_attn_noalloc.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, f32, P, P,
                                           i32, P, P]
    lib.deft_plan_free.argtypes = [P]
    lib.deft_plan_free.restype = None
    lib.deft_status_str.argtypes = [ctypes.c_int]
    lib.deft_status_str.restype = ctypes.c_char_p
    lib.deft_version.argtypes = []
    lib.deft_trace_enable.argtypes = [i32]
    lib.deft_trace_read.argtypes = [ctypes.POINTER(TraceRecord), i32, ctypes.POINTER(i32)]
    i64 = ctypes.c_int64
    lib.deft_page_table_workspace_bytes.argtypes = [i32]
    lib.deft_page_table_workspace_bytes.restype = sz
    lib.deft_page_table.argtypes = [P, i32, P, P, P, i32, i64, P, i32, i32, P, P, i32, P, P, i32, P, P, sz, P]
    lib.deft_kv_write.argtypes = [P, P, i32, i64, i64, P, i32, P, P, i32, i32, i32, i32, P]
    prompt = [P, P, i32, P, P, i32, i32, i32]
    lib.deft_prompt_plan.argtypes = prompt + [ctypes.POINTER(P)]
    lib.deft_prompt_plan_rebuild.argtypes = [P] + prompt
    lib.deft_prompt_plan_upload.argtypes = [P, P]
    lib.deft_prompt_plan_stats_get.argtypes = [P, ctypes.POINTER(PromptStats)]
    lib.deft_prompt_plan_get.argtypes = [P, i32, P, sz]
    lib.deft_prompt_plan_free.argtypes = [P]
    lib.deft_prompt_plan_free.restype = None
    lib.deft_prompt_workspace_bytes.argtypes = [P, i32, i32]
    lib.deft_prompt_workspace_bytes.restype = sz
    lib.deft_prompt_attn.argtypes = [P, i64, i32, P, P, P, P, i32, i32, i32, i32, i32, f32, P, P, i32, P, P, sz, P]
    lib.deft_prompt_status.argtypes = [P, P, ctypes.POINTER(i32)]
    qkv = [P, P, P, i32, i64, i64, i64, P, i32, ctypes.POINTER(QkTurn), P, P, P]
    lib.deft_qkv_write.argtypes = qkv + [i32, i32, i32, i32, i32, P]
    lib.deft_qkv_write4.argtypes = qkv + [f32, f32, i32, i32, i32, i32, i32, P]
    lib.deft_tree_attn4.argtypes = [P, P, P, f32, f32] + attn[3:]
    lib.deft_kv4_page_bytes.argtypes = [i32]
    lib.deft_kv4_page_bytes.restype = sz
    lib.deft_kv_unpack4.argtypes = [P, P, f32, f32, i32, P, i32, P, P, i32, i32, i32, P]
    for fn in ("deft_plan", "deft_plan_at", "deft_plan_ex", "deft_plan_rebuild", "deft_plan_stats_get",
               "deft_plan_get", "deft_plan_upload", "deft_tree_attn", "deft_naive_attn", "deft_version",
               "deft_trace_enable", "deft_trace_read", "deft_tree_attn_noalloc", "deft_tree_attn_ex",
               "deft_step_status", "deft_check_pages", "deft_plan_update", "deft_pages_create",
               "deft_pages_alloc", "deft_pages_retain", "deft_pages_release", "deft_pages_free_count",
               "deft_pages_refcount", "deft_page_table", "deft_kv_write", "deft_prompt_plan",
               "deft_prompt_plan_rebuild", "deft_prompt_plan_upload", "deft_prompt_plan_stats_get",
               "deft_prompt_plan_get", "deft_prompt_attn", "deft_prompt_status", "deft_qkv_write", "deft_qkv_write4",
               "deft_kv_unpack4", "deft_tree_attn4"):
        getattr(lib, fn).restype = ctypes.c_int
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load().deft_status_str(int(status)).decode()


def _check(fn: str, rc: int):
    if rc != 0:
        raise DeftError(fn, rc)


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _plan_flags(naive: bool, tensor_pack: bool) -> int:
    return (0 if naive else PLAN_TREE_ONLY) | (PLAN_TENSOR_PACK if tensor_pack else 0)


def _ptr(a: np.ndarray) -> int:
    # The address as an int (ctypes converts it for c_void_p parameters);
    # cheaper than building a ctypes pointer object.
    return a.ctypes.data


class Plan:
    """Owner of a deft_plan_t handle (deft_plan_ex ... deft_plan_free).
    query_pos: per query, the token of its node it sits at (-1: the last);
    None: every query at its node's last token.  naive=False: tree-only plan
    (DEFT_PLAN_TREE_ONLY; deft_naive_attn refuses it)."""

    def __init__(self, parent, node_len, query_node, chunk_target: int = 256, gqa_group: int = 1,
                 query_pos=None, naive: bool = True, tensor_pack: bool = False):
        lib = load()
        par, ln, qn = _i32(parent), _i32(node_len), _i32(query_node)
        pos = None if query_pos is None else _i32(query_pos)
        h = ctypes.c_void_p()
        _check("deft_plan_ex", lib.deft_plan_ex(_ptr(par), _ptr(ln), int(par.shape[0]), _ptr(qn),
                                                None if pos is None else _ptr(pos), int(qn.shape[0]),
                                                int(chunk_target), int(gqa_group),
                                                _plan_flags(naive, tensor_pack), ctypes.byref(h)))
        self.handle = h
        self._stats = None
        self._staged = {}

    def _stage(self, slot: int, a) -> Tuple[int, int]:
        """a copied into this plan's int32 staging buffer `slot` (kept across
        rebuilds, its address taken once): (length, address).  The library
        copies the inputs it keeps, so the buffers are only read during the
        call."""
        a = np.asarray(a)
        n = int(a.shape[0])
        buf, addr = self._staged.get(slot, (None, 0))
        if buf is None or buf.shape[0] < n:
            buf = np.empty(max(2 * n, 64), dtype=np.int32)
            addr = buf.ctypes.data
            self._staged[slot] = (buf, addr)
        buf[:n] = a
        return n, addr

    @property
    def stats(self) -> dict:
        """deft_plan_stats_get, read once per build."""
        if self._stats is None:
            st = PlanStats()
            _check("deft_plan_stats_get", load().deft_plan_stats_get(self.handle, ctypes.byref(st)))
            self._stats = st.as_dict()
        return self._stats

    def rebuild(self, parent, node_len, query_node, chunk_target: int = 256, gqa_group: int = 1,
                query_pos=None, naive: bool = True, tensor_pack: bool = False):
        """deft_plan_rebuild: plan a new tree into this plan, keeping its device
        allocation and staging buffer; upload() again before the next step.
        On error (DeftError) the plan is unchanged."""
        n, par = self._stage(0, parent)
        n_len, ln = self._stage(1, node_len)
        nq, qn = self._stage(2, query_node)
        pos = None if query_pos is None else self._stage(3, query_pos)[1]
        if n_len != n:
            raise ValueError("parent and node_len differ in length")
        _check("deft_plan_rebuild", load().deft_plan_rebuild(
            self.handle, par, ln, n, qn, pos, nq, int(chunk_target), int(gqa_group),
            _plan_flags(naive, tensor_pack)))
        self._stats = None

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _lib is not None:
            _lib.deft_plan_free(h)
            self.handle = None

    def _count(self, name: str) -> int:
        s = self.stats
        W, C, S = s["mask_words"], s["num_chunks"], s["num_segments"]
        counts = {
            "chunk_seg_off": C + 1, "chunk_q_off": C + 1, "chunk_q": s["num_slots"],
            "seg_node": S, "seg_tok_begin": S, "seg_tok_len": S, "seg_mask": S * W,
            "chunk_mask": C * W, "q_slot_off": s["num_queries"] + 1, "q_slot": s["num_slots"],
            "node_cover": s["num_nodes"] * W, "node_order": s["num_nodes"],
            "fma_items": 3 * s["num_fma_items"], "mma_items": 3 * s["num_mma_items"],
            "fallback_items": 3 * s["num_fallback_items"],
            "naive_chunk_seg_off": s["naive_num_chunks"] + 1,
            "naive_chunk_q": s["naive_num_slots"], "naive_seg_node": s["naive_num_segments"],
            "naive_seg_tok_begin": s["naive_num_segments"],
            "naive_seg_tok_len": s["naive_num_segments"],
            "naive_q_slot_off": s["num_queries"] + 1, "naive_q_slot": s["naive_num_slots"],
            "fma_direct": s["num_fma_items"], "fallback_direct": s["num_fallback_items"],
            "merge_q": s["num_merge_queries"],
        }
        return counts[name]

    def get(self, name: str) -> np.ndarray:
        """Host copy of one plan array (deft_plan_get)."""
        which, dt = ARRAYS[name]
        out = np.zeros(max(self._count(name), 1), dtype=dt)
        _check("deft_plan_get", load().deft_plan_get(self.handle, which, _ptr(out), out.nbytes))
        return out[: self._count(name)]

    def upload(self, stream=None):
        _check("deft_plan_upload", load().deft_plan_upload(self.handle, _stream(stream)))

    def workspace_bytes(self, num_q_heads: int, head_dim: int) -> int:
        return int(load().deft_workspace_bytes(self.handle, int(num_q_heads), int(head_dim)))

    def update(self, node_len):
        """deft_plan_update: the same tree with new node lengths (tokens
        appended, pruned subtrees at 0); upload() again before the next step."""
        n, ln = self._stage(1, node_len)
        _check("deft_plan_update", load().deft_plan_update(self.handle, ln, n))
        self._stats = None

    def step_status(self, stream=None) -> int:
        """deft_step_status: 0, or the code of a kernel wait that ran out in an
        earlier step (the codes are cleared by the call)."""
        code = ctypes.c_int32()
        rc = load().deft_step_status(self.handle, _stream(stream), ctypes.byref(code))
        if rc not in (0, -9):
            _check("deft_step_status", rc)
        return int(code.value)


def _stream(stream):
    """The raw cudaStream_t (an int) of `stream`, or of torch's current
    stream when it is None."""
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            # The current stream's handle without building a Stream object
            # (~0.3 us against ~3 us for torch.cuda.current_stream()).
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


@dataclass
class StepBuffers:
    out: "object"
    lse: "object"
    workspace: "object"


def alloc_buffers(plan: Plan, num_queries: int, num_q_heads: int, head_dim: int, device="cuda",
                  out_dtype: int = DEFT_OUT_BF16) -> StepBuffers:
    """Device output, lse and workspace tensors for one step (torch memory)."""
    import torch
    odt = torch.bfloat16 if out_dtype == DEFT_OUT_BF16 else torch.float32
    ws = plan.workspace_bytes(num_q_heads, head_dim)
    return StepBuffers(torch.empty((num_queries, num_q_heads, head_dim), dtype=odt, device=device),
                       torch.empty((num_queries, num_q_heads), dtype=torch.float32, device=device),
                       torch.empty(ws, dtype=torch.uint8, device=device))


def _attn(fn_name: str, q, k_pages, v_pages, node_page_off, page_id, plan: Plan,
          bufs: Optional[StepBuffers] = None, scale: Optional[float] = None,
          out_dtype: int = DEFT_OUT_BF16, stream=None, flags: int = 0):
    torch = _need_torch()
    lib = load()
    Q, Hq, d = q.shape
    Hkv, P = k_pages.shape[1], k_pages.shape[2]
    if bufs is None:
        with _allocating_for(stream):
            bufs = alloc_buffers(plan, Q, Hq, d, q.device, out_dtype)
    for t in (q, k_pages, v_pages):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("q, k_pages and v_pages must be contiguous bf16 CUDA tensors")
    for t in (node_page_off, page_id):
        if t.dtype != torch.int32 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("node_page_off and page_id must be contiguous int32 CUDA tensors")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    odt = DEFT_OUT_BF16 if bufs.out.dtype == torch.bfloat16 else DEFT_OUT_F32
    args = [q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), node_page_off.data_ptr(),
            page_id.data_ptr(), int(k_pages.shape[0]), int(Hq), int(Hkv), int(d),
            int(P), float(scale), plan.handle, bufs.out.data_ptr(), odt,
            bufs.lse.data_ptr(), bufs.workspace.data_ptr(), int(bufs.workspace.numel())]
    if fn_name == "deft_tree_attn_ex":
        args.append(int(flags))
    rc = getattr(lib, fn_name)(*args, _stream(stream))
    _check(fn_name, rc)
    return bufs.out, bufs.lse


def deft_tree_attn(q, k_pages, v_pages, node_page_off, page_id, plan: Plan, bufs=None,
                   scale=None, out_dtype=DEFT_OUT_BF16, stream=None, flags: int = 0):
    """One DeFT tree-attention step; returns (out, lse) device tensors.
    bufs None: allocated from the memory of the stream the call runs on.
    flags (STEP_*): deft_tree_attn_ex's options; 0 calls deft_tree_attn."""
    return _attn("deft_tree_attn_ex" if flags else "deft_tree_attn", q, k_pages, v_pages,
                 node_page_off, page_id, plan, bufs, scale, out_dtype, stream, flags)


def _host_step_args(q_host, q, k_pages, v_pages, node_page_off, page_id, plan: Plan, bufs: StepBuffers,
                    out_host, lse_host, scale):
    """The checked arguments of deft_tree_attn_host, the stream left out."""
    import torch
    Q, Hq, d = q.shape
    Hkv, P = k_pages.shape[1], k_pages.shape[2]
    for t in (q, k_pages, v_pages):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("q, k_pages and v_pages must be contiguous bf16 CUDA tensors")
    if q_host.dtype != torch.bfloat16 or not q_host.is_contiguous() or q_host.is_cuda or q_host.shape != q.shape:
        raise ValueError("q_host must be a contiguous bf16 host tensor shaped like q")
    for h, dv in ((out_host, bufs.out), (lse_host, bufs.lse)):
        if h.is_cuda or not h.is_contiguous() or h.dtype != dv.dtype or h.shape != dv.shape:
            raise ValueError("out_host / lse_host must be contiguous host tensors shaped like the outputs")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    odt = DEFT_OUT_BF16 if bufs.out.dtype == torch.bfloat16 else DEFT_OUT_F32
    return (q_host.data_ptr(), q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), node_page_off.data_ptr(),
            page_id.data_ptr(), int(k_pages.shape[0]), int(Hq), int(Hkv), int(d), int(P), float(scale), plan.handle,
            bufs.out.data_ptr(), odt, bufs.lse.data_ptr(), bufs.workspace.data_ptr(), int(bufs.workspace.numel()),
            out_host.data_ptr(), lse_host.data_ptr())


def deft_tree_attn_host(q_host, q, k_pages, v_pages, node_page_off, page_id, plan: Plan, bufs: StepBuffers,
                        out_host, lse_host, scale=None, stream=None):
    """deft_tree_attn_host: q_host (host, pinned for an asynchronous copy) is
    copied into the device buffer q, the step runs, and out / lse are copied
    into out_host / lse_host, all on the stream; synchronise it before
    reading the host outputs."""
    args = _host_step_args(q_host, q, k_pages, v_pages, node_page_off, page_id, plan, bufs, out_host, lse_host,
                           scale)
    _check("deft_tree_attn_host", load().deft_tree_attn_host(*args, _stream(stream)))
    return out_host, lse_host


class HostStep:
    """deft_tree_attn_host bound to one set of buffers, for a decode loop
    that runs the same shapes every step: the arguments are checked and
    marshalled once, each call is one library call on the stream.  The
    object holds the tensors and the plan, so their addresses stay valid;
    refill q_host (and rebuild or update the plan, then upload it) between
    calls, and synchronise the stream before reading out_host / lse_host."""

    def __init__(self, q_host, q, k_pages, v_pages, node_page_off, page_id, plan: Plan, bufs: StepBuffers,
                 out_host, lse_host, scale=None):
        self._args = _host_step_args(q_host, q, k_pages, v_pages, node_page_off, page_id, plan, bufs, out_host,
                                     lse_host, scale)
        self._held = (q_host, q, k_pages, v_pages, node_page_off, page_id, plan, bufs, out_host, lse_host)
        self._fn = load().deft_tree_attn_host
        self.out_host, self.lse_host = out_host, lse_host

    def __call__(self, stream=None):
        rc = self._fn(*self._args, _stream(stream))
        if rc:
            _check("deft_tree_attn_host", rc)
        return self.out_host, self.lse_host


def deft_naive_attn(q, k_pages, v_pages, node_page_off, page_id, plan: Plan, bufs=None,
                    scale=None, out_dtype=DEFT_OUT_BF16, stream=None):
    """The per-query flash-decoding form of the same step (IO comparison)."""
    return _attn("deft_naive_attn", q, k_pages, v_pages, node_page_off, page_id, plan, bufs,
                 scale, out_dtype, stream)


def deft_plan(parent, node_len, query_node, chunk_target: int = 256, gqa_group: int = 1,
              query_pos=None, naive: bool = True, tensor_pack: bool = False) -> Plan:
    return Plan(parent, node_len, query_node, chunk_target, gqa_group, query_pos, naive, tensor_pack)


class PagePool:
    """deft_pages_*: a host pool of KV page numbers with reference counts."""

    def __init__(self, num_pages: int):
        h = ctypes.c_void_p()
        _check("deft_pages_create", load().deft_pages_create(int(num_pages), ctypes.byref(h)))
        self.handle = h

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _lib is not None:
            _lib.deft_pages_free(h)
            self.handle = None

    def alloc(self, n: int) -> np.ndarray:
        out = np.zeros(max(int(n), 1), dtype=np.int32)
        _check("deft_pages_alloc", load().deft_pages_alloc(self.handle, int(n), _ptr(out)))
        return out[: int(n)]

    def retain(self, ids):
        ids = _i32(ids)
        _check("deft_pages_retain", load().deft_pages_retain(self.handle, int(ids.size),
                                                             _ptr(ids) if ids.size else None))

    def release(self, ids):
        ids = _i32(ids)
        _check("deft_pages_release", load().deft_pages_release(self.handle, int(ids.size),
                                                               _ptr(ids) if ids.size else None))

    @property
    def free_count(self) -> int:
        return int(load().deft_pages_free_count(self.handle))

    def refcount(self, page: int) -> int:
        return int(load().deft_pages_refcount(self.handle, int(page)))


def _allocating_for(stream):
    """Context in which tensors come from the memory of the stream that the
    call runs on: a tensor of another stream's could still be in use there,
    and one that the call drops would be handed out again while it runs."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        # ExternalStream(0) is a stream of torch's pool, not the default one.
        stream = _torch.cuda.ExternalStream(stream) if stream else _torch.cuda.default_stream()
    return _torch.cuda.stream(stream)


def _launch_stream(stream, *tensors) -> int:
    """The raw stream to launch on.  Raises unless every tensor is on the
    current CUDA device (the library launches there)."""
    dev = _torch.cuda.current_device()
    for t in tensors:
        if t.get_device() != dev:      # -1: not on a GPU
            raise ValueError("tensors must be on the current CUDA device")
    if stream is None:
        raw = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(dev)
    return _stream(stream)


_torch = None


def _need_torch():
    """torch, imported at the first call that takes tensors."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _heads_packed(shape, stride) -> bool:
    """Whether [tokens, heads, head_dim] holds each token's heads
    contiguously (the stride of a dimension of one element says nothing)."""
    return shape[0] == 0 or (stride[2] == 1 and (shape[1] == 1 or stride[1] == shape[2]))


def _index_tensor(t, name: str) -> int:
    """The length of a contiguous one-dimensional int32 tensor."""
    n, = t.shape if t.dim() == 1 else (-1,)
    if n < 0 or t.dtype != _torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous one-dimensional int32 tensor")
    return n


@dataclass
class PageTable:
    """Outputs of deft_page_table (int32 CUDA tensors): node_page_off and
    page_id as the steps take them, tok_off / slot of the new tokens, counts =
    (pages, pages taken from the free list, new tokens, 0 or TABLE_*).
    workspace: page_table_workspace(num_nodes)."""
    page_off: "object"
    page_id: "object"
    tok_off: "object"
    slot: "object"
    counts: "object"
    workspace: "object" = None


def page_table_workspace(num_nodes: int, device="cuda"):
    """Device workspace deft_page_table needs for so many nodes (None: none)."""
    import torch
    n = int(load().deft_page_table_workspace_bytes(int(num_nodes)))
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def alloc_page_table(num_nodes: int, max_pages: int, max_tokens: int, device="cuda") -> PageTable:
    """Tensors for a table of at most max_pages pages and max_tokens new tokens."""
    import torch

    def new(n):
        return torch.empty(int(n), dtype=torch.int32, device=device)
    return PageTable(new(num_nodes + 1), new(max_pages), new(num_nodes + 1), new(max_tokens), new(4),
                     page_table_workspace(num_nodes, device))


def deft_page_table(node_len, free_pages, prev=None, table: Optional[PageTable] = None, max_pages: Optional[int] = None,
                    max_tokens: Optional[int] = None, page_size: int = 16, stream=None) -> PageTable:
    """deft_page_table: page table and slot map of the nodes' new tokens.
    prev: (prev_len, prev_page_off, prev_page_id) of the earlier table, None:
    every node starts empty.  table: the tensors to write (reused between
    steps); None: allocated for max_pages and max_tokens, from the memory of
    the stream the call runs on."""
    _need_torch()
    n, n_free = _index_tensor(node_len, "node_len"), _index_tensor(free_pages, "free_pages")
    if table is None:
        if max_pages is None or max_tokens is None:
            raise ValueError("max_pages and max_tokens are needed to allocate a table")
        with _allocating_for(stream):
            table = alloc_page_table(n, max_pages, max_tokens, node_len.device)
    off, ids, tok, slot, counts, ws = (table.page_off, table.page_id, table.tok_off, table.slot, table.counts,
                                       table.workspace)
    n_ids, n_slots = _index_tensor(ids, "page_id"), _index_tensor(slot, "slot")
    if _index_tensor(off, "page_off") <= n or _index_tensor(tok, "tok_off") <= n or _index_tensor(counts, "counts") < 4:
        raise ValueError("page_off and tok_off need num_nodes + 1 entries, counts 4")
    used = [node_len, free_pages, off, ids, tok, slot, counts]
    pl = po = pi = None
    n_prev = n_prev_ids = 0
    if prev is not None:
        t_len, t_off, t_id = prev
        n_prev, n_prev_ids = _index_tensor(t_len, "prev_len"), _index_tensor(t_id, "prev_page_id")
        if _index_tensor(t_off, "prev_page_off") < n_prev:
            raise ValueError("prev_page_off is shorter than prev_len")
        used += prev
        if n_prev:
            pl, po, pi = t_len.data_ptr(), t_off.data_ptr(), t_id.data_ptr()
    ws_ptr, ws_bytes = None, 0
    if ws is not None:
        used.append(ws)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    st = _launch_stream(stream, *used)
    rc = load().deft_page_table(node_len.data_ptr(), n, pl, po, pi, n_prev, n_prev_ids, free_pages.data_ptr(), n_free,
                                int(page_size), off.data_ptr(), ids.data_ptr(), n_ids, tok.data_ptr(), slot.data_ptr(),
                                n_slots, counts.data_ptr(), ws_ptr, ws_bytes, st)
    if rc:
        _check("deft_page_table", rc)
    return table


def deft_kv_write(k, v, slot, k_pages, v_pages, stream=None):
    """deft_kv_write: rows of k and v ([tokens, num_kv_heads, head_dim], bf16
    or fp32, views with any token stride) into the pages at their slots; rows
    with a slot outside the pool (-1) are skipped."""
    torch = _need_torch()
    shape, ks, vs, dt = k.shape, k.stride(), v.stride(), k.dtype
    if len(shape) != 3 or v.shape != shape or v.dtype != dt or dt not in (torch.bfloat16, torch.float32):
        raise ValueError("k and v must be alike: [tokens, heads, head_dim], bf16 or fp32")
    T, Hkv, d = shape
    if not _heads_packed(shape, ks) or not _heads_packed(shape, vs):
        raise ValueError("the heads of a token must be contiguous")
    pool = _check_pools(k_pages, v_pages, d)
    if pool[1] != Hkv:
        raise ValueError("k_pages and v_pages have another number of heads")
    if _index_tensor(slot, "slot") != T:
        raise ValueError("slot must have one entry per token")
    st = _launch_stream(stream, k, v, slot, k_pages, v_pages)
    rc = load().deft_kv_write(k.data_ptr(), v.data_ptr(), DEFT_OUT_BF16 if dt == torch.bfloat16 else DEFT_OUT_F32, ks[0],
                              vs[0], slot.data_ptr(), T, k_pages.data_ptr(), v_pages.data_ptr(), pool[0], Hkv, d,
                              pool[2], st)
    if rc:
        _check("deft_kv_write", rc)


def _check_pools(k_pages, v_pages, head_dim):
    """The shape of the page pools, after their checks."""
    shape, bf16 = k_pages.shape, _torch.bfloat16
    if len(shape) != 4 or v_pages.shape != shape or shape[3] != head_dim or k_pages.dtype != bf16 or \
            v_pages.dtype != bf16 or not k_pages.is_contiguous() or not v_pages.is_contiguous():
        raise ValueError("k_pages and v_pages must be contiguous bf16 [pages, heads, page_size, head_dim], alike")
    return shape


def kv4_page_bytes(head_dim: int) -> int:
    """Bytes of one head's page of a 4-bit cache (0: not a head_dim it has)."""
    return int(load().deft_kv4_page_bytes(int(head_dim)))


def alloc_kv4_pages(num_pages: int, num_kv_heads: int, head_dim: int, device="cuda"):
    """(k4_pages, v4_pages) of a 4-bit cache, uint8 [pages, heads, kv4_page_bytes(head_dim)]."""
    import torch
    shape = (int(num_pages), int(num_kv_heads), kv4_page_bytes(head_dim))
    if shape[2] == 0:
        raise ValueError("a 4-bit cache has a head_dim of 64 or 128")
    return tuple(torch.empty(shape, dtype=torch.uint8, device=device) for _ in "kv")


def _check_pools4(k4_pages, v4_pages, head_dim):
    """(pages, heads) of the 4-bit pools, after their checks."""
    shape = k4_pages.shape
    if len(shape) != 3 or v4_pages.shape != shape or shape[2] != 9 * head_dim or k4_pages.dtype != _torch.uint8 or \
            v4_pages.dtype != _torch.uint8 or not k4_pages.is_contiguous() or not v4_pages.is_contiguous():
        raise ValueError("k4_pages and v4_pages must be contiguous uint8 [pages, heads, 9 * head_dim], alike")
    return shape


def _qkv_args(q, k, v, slot, position, cos_sin, interleaved, q_norm, k_norm, eps, q_out, stream):
    """The checked arguments of the append calls up to q_out, the tensors they
    name, the heads and q_out itself."""
    shape, dt = k.shape, k.dtype
    bf16 = dt is _torch.bfloat16
    if len(shape) != 3 or v.shape != shape or v.dtype is not dt or not (bf16 or dt is _torch.float32):
        raise ValueError("k and v must be alike: [tokens, heads, head_dim], bf16 or fp32")
    T, Hkv, d = shape
    ks, vs = k.stride(), v.stride()
    if not _heads_packed(shape, ks) or not _heads_packed(shape, vs):
        raise ValueError("the heads of a token must be contiguous")
    if _index_tensor(slot, "slot") != T:
        raise ValueError("slot must have one entry per token")
    used = [k, v, slot]
    Hq = qs = 0
    q_ptr = out_ptr = None
    if q is not None:
        q_shape, q_st = q.shape, q.stride()
        if len(q_shape) != 3 or q_shape[0] != T or q_shape[2] != d or q.dtype is not dt or not _heads_packed(q_shape, q_st):
            raise ValueError("q must be [tokens, heads, head_dim] of k's dtype with the heads of a token contiguous")
        Hq, qs = q_shape[1], q_st[0]
        if q_out is None:
            with _allocating_for(stream):
                q_out = _torch.empty((T, Hq, d), dtype=_torch.bfloat16, device=q.device)
        elif q_out.shape != q_shape or q_out.dtype is not _torch.bfloat16 or not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous bf16, shaped like q")
        used += (q, q_out)
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None or q_norm is not None:
        raise ValueError("q_out and q_norm go with q")
    turn = None
    if cos_sin is not None or q_norm is not None or k_norm is not None:
        qn = kn = table = pos = None
        rows = rot = 0
        if q_norm is not None:
            qn = _norm_pointer(q_norm, d, dt, "q_norm")
            used.append(q_norm)
        if k_norm is not None:
            kn = _norm_pointer(k_norm, d, dt, "k_norm")
            used.append(k_norm)
        if cos_sin is not None:
            if cos_sin.dim() != 2 or cos_sin.dtype is not _torch.float32 or not cos_sin.is_contiguous():
                raise ValueError("cos_sin must be contiguous fp32 [positions, rot_dim]")
            if position is None or _index_tensor(position, "position") != T:
                raise ValueError("position must have one entry per token")
            rows, rot = cos_sin.shape
            table, pos = cos_sin.data_ptr(), position.data_ptr()
            used += (cos_sin, position)
        turn = ctypes.byref(QkTurn(qn, kn, eps, rot, 1 if interleaved else 0, rows, table, pos))
    args = (q_ptr, k.data_ptr(), v.data_ptr(), DEFT_OUT_BF16 if bf16 else DEFT_OUT_F32, qs, ks[0], vs[0], slot.data_ptr(), T,
            turn, out_ptr)
    return args, used, (Hq, Hkv, d), q_out


def _norm_pointer(w, head_dim, dtype, name):
    if w.shape != (head_dim,) or w.dtype is not dtype or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [head_dim] tensor of k's dtype")
    return w.data_ptr()


def deft_qkv_write(q, k, v, slot, k_pages, v_pages, position=None, cos_sin=None, interleaved: bool = False, q_norm=None,
                   k_norm=None, eps: float = 1e-6, q_out=None, stream=None):
    """deft_qkv_write: rows of a projection ([tokens, heads, head_dim], bf16 or
    fp32, views with any token stride) to the cache: q and k normed for each
    head (q_norm, k_norm: weights, None: no norm) and rotated (cos_sin
    [positions, rot_dim]: cosines, then sines; None: no rotation) by position,
    k and v into the pages at their slots; returns q_out, bf16 (allocated from
    the memory of the stream the call runs on when None).  q None: k and v
    alone."""
    _need_torch()
    args, used, (Hq, Hkv, d), q_out = _qkv_args(q, k, v, slot, position, cos_sin, interleaved, q_norm, k_norm, eps, q_out, stream)
    pool = _check_pools(k_pages, v_pages, d)
    if pool[1] != Hkv:
        raise ValueError("k_pages and v_pages have another number of heads")
    st = _launch_stream(stream, k_pages, v_pages, *used)
    rc = load().deft_qkv_write(*args, k_pages.data_ptr(), v_pages.data_ptr(), pool[0], Hq, Hkv, d, pool[2], st)
    if rc:
        _check("deft_qkv_write", rc)
    return q_out


def deft_qkv_write4(q, k, v, slot, k4_pages, v4_pages, position=None, cos_sin=None, interleaved: bool = False,
                    q_norm=None, k_norm=None, eps: float = 1e-6, q_out=None, k_scale: float = 1.0, v_scale: float = 1.0,
                    stream=None):
    """deft_qkv_write4: deft_qkv_write into the 4-bit pools of
    alloc_kv4_pages, quantised with k_scale and v_scale."""
    _need_torch()
    args, used, (Hq, Hkv, d), q_out = _qkv_args(q, k, v, slot, position, cos_sin, interleaved, q_norm, k_norm, eps, q_out, stream)
    pool = _check_pools4(k4_pages, v4_pages, d)
    if pool[1] != Hkv:
        raise ValueError("k4_pages and v4_pages have another number of heads")
    st = _launch_stream(stream, k4_pages, v4_pages, *used)
    rc = load().deft_qkv_write4(*args, k4_pages.data_ptr(), v4_pages.data_ptr(), k_scale, v_scale, pool[0], Hq, Hkv, d, 16, st)
    if rc:
        _check("deft_qkv_write4", rc)
    return q_out


def deft_kv_unpack4(k4_pages, v4_pages, page_id, k_pages=None, v_pages=None, k_scale: float = 1.0, v_scale: float = 1.0,
                    stream=None):
    """deft_kv_unpack4: the listed pages of a 4-bit cache as bf16 pages
    [listed, heads, 16, head_dim], in the list's order; returns (k_pages,
    v_pages), allocated from the memory of the stream the call runs on when
    None."""
    torch = _need_torch()
    if k4_pages.dim() != 3 or k4_pages.shape[2] % 9:
        raise ValueError("k4_pages must be [pages, heads, 9 * head_dim]")
    pages, Hkv, d = k4_pages.shape[0], k4_pages.shape[1], k4_pages.shape[2] // 9
    _check_pools4(k4_pages, v4_pages, d)
    n = _index_tensor(page_id, "page_id")
    if (k_pages is None) != (v_pages is None):
        raise ValueError("k_pages and v_pages go together")
    if k_pages is None:
        with _allocating_for(stream):
            k_pages, v_pages = (torch.empty((n, Hkv, 16, d), dtype=torch.bfloat16, device=k4_pages.device) for _ in "kv")
    shape = _check_pools(k_pages, v_pages, d)
    if shape[0] < n or shape[1] != Hkv or shape[2] != 16:
        raise ValueError("k_pages and v_pages must hold the listed pages, [listed, heads, 16, head_dim]")
    st = _launch_stream(stream, k4_pages, v4_pages, page_id, k_pages, v_pages)
    rc = load().deft_kv_unpack4(k4_pages.data_ptr(), v4_pages.data_ptr(), k_scale, v_scale, pages, page_id.data_ptr(), n,
                                k_pages.data_ptr(), v_pages.data_ptr(), Hkv, d, 16, st)
    if rc:
        _check("deft_kv_unpack4", rc)
    return k_pages, v_pages


def deft_tree_attn4(q, k4_pages, v4_pages, node_page_off, page_id, plan: Plan, bufs: Optional[StepBuffers] = None,
                    scale: Optional[float] = None, out_dtype: int = DEFT_OUT_BF16, k_scale: float = 1.0,
                    v_scale: float = 1.0, stream=None):
    """deft_tree_attn4: one tree-attention step over the 4-bit pools of
    alloc_kv4_pages, written with k_scale and v_scale; returns (out, lse).
    bufs: alloc_buffers(plan, queries, num_q_heads, head_dim); None: allocated
    from the memory of the stream the call runs on."""
    torch = _need_torch()
    shape = q.shape
    if len(shape) != 3 or q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [queries, num_q_heads, head_dim]")
    Q, Hq, d = shape
    pool = _check_pools4(k4_pages, v4_pages, d)
    stats = plan.stats
    if Q != stats["num_queries"]:
        raise ValueError("q must have one row per query of the plan")
    if _index_tensor(node_page_off, "node_page_off") < stats["num_nodes"]:
        raise ValueError("node_page_off is shorter than the plan's nodes")
    _index_tensor(page_id, "page_id")
    if bufs is None:
        with _allocating_for(stream):
            bufs = alloc_buffers(plan, Q, Hq, d, q.device, out_dtype)
    out, lse, ws = bufs.out, bufs.lse, bufs.workspace
    odt = out.dtype
    if out.shape != shape or odt not in (torch.bfloat16, torch.float32) or not out.is_contiguous():
        raise ValueError("out must be contiguous bf16 or fp32, shaped like q")
    if lse.shape != (Q, Hq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [queries, num_q_heads]")
    st = _launch_stream(stream, q, k4_pages, v4_pages, node_page_off, page_id, out, lse, ws)
    if Q == 0:
        return out, lse
    rc = load().deft_tree_attn4(
        q.data_ptr(), k4_pages.data_ptr(), v4_pages.data_ptr(), k_scale, v_scale, node_page_off.data_ptr(),
        page_id.data_ptr(), pool[0], Hq, pool[1], d, 16, 1.0 / math.sqrt(d) if scale is None else float(scale), plan.handle,
        out.data_ptr(), DEFT_OUT_BF16 if odt == torch.bfloat16 else DEFT_OUT_F32, lse.data_ptr(), ws.data_ptr(),
        ws.numel() * ws.element_size(), st)
    if rc:
        _check("deft_tree_attn4", rc)
    return out, lse


PROMPT_ARRAYS = {"nodes": (0, 2), "items": (1, 12), "cta_off": (2, 1), "cta_unit": (3, 1), "merges": (4, 4)}


class PromptPlan:
    """Owner of a deft_prompt_plan_t handle.  parent None: every node a root;
    prompt_len None: every prompt its whole node (an entry -1: the same)."""

    def __init__(self, parent, node_len, prompt_node, num_kv_heads: int, gqa_group: int = 1, prompt_len=None):
        h = ctypes.c_void_p()
        args = self._args(parent, node_len, prompt_node, num_kv_heads, gqa_group, prompt_len)
        _check("deft_prompt_plan", load().deft_prompt_plan(*args[0], ctypes.byref(h)))
        self.handle = h
        self._stats = None

    @staticmethod
    def _args(parent, node_len, prompt_node, num_kv_heads, gqa_group, prompt_len):
        ln, pn = _i32(node_len), _i32(prompt_node)
        par = None if parent is None else _i32(parent)
        pl = None if prompt_len is None else _i32(prompt_len)
        if par is not None and par.shape != ln.shape:
            raise ValueError("parent and node_len differ in length")
        if pl is not None and pl.shape != pn.shape:
            raise ValueError("prompt_node and prompt_len differ in length")
        # The arrays are held until the call has returned.
        return (None if par is None else _ptr(par), _ptr(ln), int(ln.shape[0]), _ptr(pn),
                None if pl is None else _ptr(pl), int(pn.shape[0]), int(num_kv_heads), int(gqa_group)), (par, ln, pn, pl)

    def rebuild(self, parent, node_len, prompt_node, num_kv_heads: int, gqa_group: int = 1, prompt_len=None):
        """deft_prompt_plan_rebuild; upload() again before the next step."""
        args = self._args(parent, node_len, prompt_node, num_kv_heads, gqa_group, prompt_len)
        _check("deft_prompt_plan_rebuild", load().deft_prompt_plan_rebuild(self.handle, *args[0]))
        self._stats = None

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _lib is not None:
            _lib.deft_prompt_plan_free(h)
            self.handle = None

    @property
    def stats(self) -> dict:
        """deft_prompt_plan_stats_get, read once per build."""
        if self._stats is None:
            st = PromptStats()
            _check("deft_prompt_plan_stats_get", load().deft_prompt_plan_stats_get(self.handle, ctypes.byref(st)))
            self._stats = st.as_dict()
        return self._stats

    def get(self, name: str) -> np.ndarray:
        """Host copy of one plan array (deft_prompt_plan_get), a row per record."""
        which, width = PROMPT_ARRAYS[name]
        s = self.stats
        n = {"nodes": s["num_nodes"], "items": s["num_items"], "cta_off": 153, "cta_unit": s["num_units"],
             "merges": s["num_split_items"]}[name]
        out = np.zeros(max(n * width, 1), dtype=np.int32)
        _check("deft_prompt_plan_get", load().deft_prompt_plan_get(self.handle, which, _ptr(out), out.nbytes))
        return out[: n * width].reshape(n, width) if width > 1 else out[:n]

    def upload(self, stream=None):
        _check("deft_prompt_plan_upload", load().deft_prompt_plan_upload(self.handle, _stream(stream)))

    def workspace_bytes(self, num_q_heads: int, head_dim: int) -> int:
        return int(load().deft_prompt_workspace_bytes(self.handle, int(num_q_heads), int(head_dim)))

    def step_status(self, stream=None) -> int:
        """deft_prompt_status: 0, or the code of a kernel wait that ran out."""
        code = ctypes.c_int32()
        rc = load().deft_prompt_status(self.handle, _stream(stream), ctypes.byref(code))
        if rc not in (0, -9):
            _check("deft_prompt_status", rc)
        return int(code.value)


def deft_prompt_attn(q, k_pages, v_pages, node_page_off, page_id, plan: PromptPlan, bufs: Optional[StepBuffers] = None,
                     scale: Optional[float] = None, out_dtype: int = DEFT_OUT_BF16, stream=None):
    """Causal attention of the plan's prompts: q [rows, num_q_heads,
    head_dim] bf16 (any token stride), rows packed prompt by prompt; returns
    (out, lse).  bufs: alloc_buffers(plan, rows, num_q_heads, head_dim); None:
    allocated from the memory of the stream the call runs on."""
    torch = _need_torch()
    shape, qs = q.shape, q.stride()
    if len(shape) != 3 or q.dtype != torch.bfloat16 or not _heads_packed(shape, qs):
        raise ValueError("q must be bf16 [rows, num_q_heads, head_dim] with the heads of a token contiguous")
    T, Hq, d = shape
    if bufs is None:
        with _allocating_for(stream):
            bufs = alloc_buffers(plan, T, Hq, d, q.device, out_dtype)
    out, lse, ws = bufs.out, bufs.lse, bufs.workspace
    pool = _check_pools(k_pages, v_pages, d)
    stats = plan.stats
    rows = stats["num_rows"]
    if _index_tensor(node_page_off, "node_page_off") < stats["num_nodes"]:
        raise ValueError("node_page_off is shorter than the plan's nodes")
    _index_tensor(page_id, "page_id")
    os, ls, odt = out.shape, lse.shape, out.dtype
    if len(os) != 3 or os[1] != Hq or os[2] != d or os[0] < rows or odt not in (torch.bfloat16, torch.float32) or \
            not out.is_contiguous():
        raise ValueError("out must be contiguous bf16 or fp32 [rows, num_q_heads, head_dim]")
    if len(ls) != 2 or ls[1] != Hq or ls[0] < rows or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [rows, num_q_heads]")
    st = _launch_stream(stream, q, k_pages, v_pages, node_page_off, page_id, out, lse, ws)
    if T == 0 and rows == 0:
        return out, lse
    rc = load().deft_prompt_attn(
        q.data_ptr(), qs[0] if T > 1 else Hq * d, T, k_pages.data_ptr(), v_pages.data_ptr(), node_page_off.data_ptr(),
        page_id.data_ptr(), pool[0], Hq, pool[1], d, pool[2], 1.0 / math.sqrt(d) if scale is None else float(scale),
        plan.handle, out.data_ptr(), DEFT_OUT_BF16 if odt == torch.bfloat16 else DEFT_OUT_F32, lse.data_ptr(),
        ws.data_ptr(), ws.numel() * ws.element_size(), st)
    if rc:
        _check("deft_prompt_attn", rc)
    return out, lse


def deft_check_pages(node_len, node_page_off, page_id, num_pages: int, page_size: int = 16) -> int:
    """deft_check_pages on host arrays: 0 (DEFT_OK) or the status code."""
    ln, npo, pid = _i32(node_len), _i32(node_page_off), _i32(page_id)
    return int(load().deft_check_pages(_ptr(ln), int(ln.shape[0]), _ptr(npo),
                                       _ptr(pid) if pid.size else None, int(pid.size),
                                       int(num_pages), int(page_size)))


def trace_enable(on: bool = True):
    _check("deft_trace_enable", load().deft_trace_enable(1 if on else 0))


def trace_read(cap: int = 1 << 16):
    """Per-launch records since the last read: list of dicts (waits for the events)."""
    recs = (TraceRecord * cap)()
    n = ctypes.c_int32()
    _check("deft_trace_read", load().deft_trace_read(recs, cap, ctypes.byref(n)))
    return [{"kernel": KERNEL_NAMES.get(r.kernel, str(r.kernel)), "family": r.family,
             "bucket": r.bucket, "fallback": r.fallback, "items": r.items, "ms": r.ms}
            for r in recs[: n.value]]


def version() -> int:
    return int(load().deft_version())
