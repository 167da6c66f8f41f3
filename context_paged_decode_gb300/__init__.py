"""Python binding of libdcp.so, the GB300 hot path of Decode Context Parallelism.

Argument marshalling only: every step runs in the library's CUDA kernels.
PyTorch supplies device memory and the current stream.  The functions carry
the C names without the ``dcp_`` prefix; see ``include/dcp.h`` for the
meaning, layout and error behaviour of every argument.

If the shared library is missing or fails to load, every call raises: there
is no fallback implementation.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdcp.so")
MAX_RANKS = 16

F32, BF16 = 0, 1
KIND_GQA, KIND_MLA, KIND_SFA = 0, 1, 2
_DT = {torch.float32: F32, torch.bfloat16: BF16}


class DcpError(RuntimeError):
    pass


class Layout(C.Structure):
    _fields_ = [("dcp_size", C.c_int32), ("block_size", C.c_int32), ("interleave", C.c_int32)]

    def __init__(self, dcp_size, block_size, interleave=1):
        super().__init__(int(dcp_size), int(block_size), int(interleave))

    def __repr__(self):
        return f"Layout(dcp={self.dcp_size}, bs={self.block_size}, I={self.interleave})"


class RankPtrs(C.Structure):
    _fields_ = [("ptr", C.c_void_p * MAX_RANKS)]


class PagedKVStruct(C.Structure):
    _fields_ = [("k", RankPtrs), ("v", RankPtrs), ("num_blocks", C.c_int64),
                ("block_table", C.c_void_p), ("max_vblocks", C.c_int32),
                ("bt_rank_stride", C.c_int64)]


class PagedKV8Struct(C.Structure):
    _fields_ = [("k", RankPtrs), ("v", RankPtrs), ("scale", RankPtrs), ("num_blocks", C.c_int64),
                ("block_table", C.c_void_p), ("max_vblocks", C.c_int32),
                ("bt_rank_stride", C.c_int64)]


class ScoresStruct(C.Structure):
    _fields_ = [("cap", C.c_float), ("window", C.c_int32), ("prefix", C.c_int32),
                ("slopes", C.c_void_p), ("first", C.c_void_p)]


class PagesStruct(C.Structure):
    _fields_ = [("block_table", C.c_void_p), ("seq_lens", C.c_void_p), ("ref_count", C.c_void_p),
                ("free_bits", C.c_void_p), ("num_reqs", C.c_int32), ("max_vblocks", C.c_int32),
                ("bt_rank_stride", C.c_int64), ("num_blocks", C.c_int64)]


class PoolSetStruct(C.Structure):
    _fields_ = [("ptr", C.c_void_p), ("num_pools", C.c_int32), ("num_heads", C.c_int32),
                ("row_bytes", C.c_int32), ("num_blocks", C.c_int64)]


_lib = None
_bind = None     # the native extension, once it knows the library
_loaded_from = LIB_PATH


def _load_binding():
    """Load the library and the extension that hands tensors to it (once)."""
    global _bind
    load()
    try:
        from . import _binding
    except ImportError as e:
        raise DcpError(f"the native binding is not built ({e}): build it with "
                       "__graft_entry__.build()") from None
    _binding.init(_loaded_from, DcpError)
    _bind = _binding
    return _bind


def load(path: str = LIB_PATH):
    """Load libdcp.so (once).  Raises if it is missing: there is no fallback."""
    global _lib, _bind, _loaded_from
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise DcpError(f"{path} not found: build it with __graft_entry__.build()")
    lib = C.CDLL(path)
    i32, i64, vp, f32 = C.c_int32, C.c_int64, C.c_void_p, C.c_float
    L, RP, PK, PG, PS = Layout, RankPtrs, PagedKVStruct, PagesStruct, PoolSetStruct
    P8, SF = PagedKV8Struct, ScoresStruct
    sig = {
        "dcp_strerror": (C.c_char_p, [C.c_int]),
        "dcp_version": (C.c_int, []),
        "dcp_local_seq_lens": (C.c_int, [L, vp, i32, vp, vp, vp]),
        "dcp_slot_mapping": (C.c_int, [L, vp, vp, i64, vp, i32, i32, i64, i64, vp, vp, vp, vp]),
        "dcp_cache_write_gqa": (C.c_int, [L, vp, vp, i64, i32, i32, C.c_int, vp, i64, RP, RP, vp,
                                          vp]),
        "dcp_cache_write_mla": (C.c_int, [L, vp, i64, i32, C.c_int, vp, i64, RP, vp, vp]),
        "dcp_gather_context_mla": (C.c_int, [L, PK, i32, i32, C.c_int, vp, vp, i64, vp, vp, vp]),
        "dcp_decode_workspace_size": (C.c_int, [L, C.c_int, i32, i32, i32, i32,
                                                C.POINTER(C.c_size_t)]),
        "dcp_decode_partial_gqa": (C.c_int, [L, vp, i32, i32, i32, i32, f32, C.c_int, PK, vp, vp,
                                             vp, vp, C.c_size_t, vp, vp]),
        "dcp_lse_merge": (C.c_int, [i32, vp, vp, i32, i32, i32, vp, vp, C.c_int, vp, vp]),
        "dcp_lse_merge_swa": (C.c_int, [i32, vp, vp, vp, vp, i32, i32, i32, vp, vp, C.c_int, vp,
                                        vp]),
        "dcp_decode_gqa": (C.c_int, [L, vp, i32, i32, i32, i32, f32, C.c_int, PK, vp, vp, vp,
                                     C.c_int, vp, vp, C.c_size_t, vp, vp]),
        "dcp_decode_gqa_noalloc": (C.c_int, [L, vp, i32, i32, i32, i32, f32, C.c_int, PK, vp, vp,
                                             vp, C.c_int, vp, vp, vp]),
        "dcp_decode_partial_mla": (C.c_int, [L, vp, i32, i32, i32, i32, f32, C.c_int, PK, vp, vp,
                                             vp, vp, C.c_size_t, vp, vp]),
        "dcp_decode_mla": (C.c_int, [L, vp, i32, i32, i32, i32, f32, C.c_int, PK, vp, vp, vp,
                                     C.c_int, vp, vp, C.c_size_t, vp, vp]),
        "dcp_sfa_remap": (C.c_int, [L, vp, i32, i32, vp, vp, i32, i64, i64, vp, vp, vp, vp]),
        "dcp_topk_workspace_size": (C.c_int, [L, i32, i32, C.POINTER(C.c_size_t)]),
        "dcp_topk_local": (C.c_int, [L, vp, i32, i32, vp, i32, vp, vp]),
        "dcp_topk_merge": (C.c_int, [i32, vp, i32, i32, vp, C.c_size_t, vp, vp, vp]),
        "dcp_topk": (C.c_int, [L, vp, i32, i32, vp, i32, vp, vp, vp, C.c_size_t, vp]),
        "dcp_sfa_compact_workspace_size": (C.c_int, [L, i64, C.POINTER(C.c_size_t)]),
        "dcp_sfa_compact_blocks": (C.c_int, [L, vp, vp, i32, i32, vp, i32, PK, i32, C.c_int, i64,
                                             vp, vp, vp, vp, vp, C.c_size_t, vp, vp]),
        "dcp_sfa_decode_partial": (C.c_int, [L, vp, i32, i32, i32, i32, f32, C.c_int, PK, vp, vp,
                                             i32, vp, vp, vp, vp]),
        "dcp_sfa_decode": (C.c_int, [L, vp, i32, i32, i32, i32, f32, C.c_int, PK, vp, i32, vp, vp,
                                     vp, C.c_int, vp, vp, C.c_size_t, vp, vp]),
        "dcp_tree_workspace_size": (C.c_int, [L, i32, i32, i32, i32, i32, C.c_int,
                                              C.POINTER(C.c_size_t)]),
        "dcp_tree_partial_gqa": (C.c_int, [L, vp, vp, i32, i32, i32, i32, i32, i32, f32, C.c_int,
                                           PK, vp, vp, vp, vp, vp, C.c_size_t, vp, vp]),
        "dcp_tree_decode_gqa": (C.c_int, [L, vp, vp, i32, i32, i32, i32, i32, i32, f32, C.c_int,
                                          PK, vp, vp, vp, vp, C.c_int, vp, vp, C.c_size_t, vp,
                                          vp]),
        "dcp_rope_write_gqa": (C.c_int, [L, vp, i64, vp, i64, vp, i64, i64, i32, i32, i32, C.c_int,
                                         vp, i32, vp, vp, i32, i32, f32, vp, i64, RP, RP, vp, vp,
                                         vp, vp]),
        "dcp_rope_write_mla": (C.c_int, [L, vp, i64, vp, i64, i64, i32, i32, C.c_int, vp, i32, vp,
                                         vp, i32, i32, f32, vp, i64, RP, vp, vp, vp]),
        "dcp_pages_init": (C.c_int, [L, PG, vp]),
        "dcp_pages_workspace_size": (C.c_int, [L, PG, i32, C.POINTER(C.c_size_t)]),
        "dcp_pages_resize": (C.c_int, [L, PG, vp, vp, i32, vp, vp, vp, C.c_size_t, vp, vp]),
        "dcp_pages_fork": (C.c_int, [L, PG, vp, vp, i32, vp, vp, vp, C.c_size_t, vp, vp]),
        "dcp_pages_copy": (C.c_int, [L, PS, vp, vp, i32, i32, vp, vp]),
        "dcp_cache_compact": (C.c_int, [L, PS, vp, i32, i32, i64, vp, vp, vp, i32, vp, vp, vp]),
        "dcp_q8_append_gqa": (C.c_int, [L, vp, i64, vp, i64, i32, vp, vp, i32, i32, i32, C.c_int,
                                        P8, vp, vp]),
        "dcp_q8_gather_gqa": (C.c_int, [L, P8, i32, i32, i32, vp, vp, i64, vp, vp, C.c_int, vp,
                                        vp]),
        "dcp_q8_decode_gqa": (C.c_int, [L, vp, i32, i32, i32, i32, f32, C.c_int, P8, vp, SF, vp,
                                        vp, C.c_int, vp, vp, C.c_size_t, vp, vp]),
        "dcp_q8_partial_gqa": (C.c_int, [L, vp, i32, i32, i32, i32, f32, C.c_int, P8, vp, SF, vp,
                                         vp, vp, C.c_size_t, vp, vp]),
        "dcp_scored_decode_gqa": (C.c_int, [L, vp, i32, i32, i32, i32, f32, C.c_int, PK, vp, SF,
                                            vp, vp, C.c_int, vp, vp, C.c_size_t, vp, vp]),
        "dcp_scored_partial_gqa": (C.c_int, [L, vp, i32, i32, i32, i32, f32, C.c_int, PK, vp, SF,
                                             vp, vp, vp, C.c_size_t, vp, vp]),
        "dcp_scored_workspace_size": (C.c_int, [L, i32, i32, i32, i32, i32,
                                                C.POINTER(C.c_size_t)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib, _bind, _loaded_from = lib, None, os.path.abspath(path)
    return lib


def exported_symbols():
    """Names of the C entry points this binding expects the library to export."""
    return ["dcp_strerror", "dcp_version", "dcp_local_seq_lens", "dcp_slot_mapping",
            "dcp_cache_write_gqa", "dcp_cache_write_mla", "dcp_gather_context_mla",
            "dcp_decode_workspace_size",
            "dcp_decode_partial_gqa", "dcp_lse_merge", "dcp_lse_merge_swa", "dcp_decode_gqa",
            "dcp_decode_gqa_noalloc",
            "dcp_decode_partial_mla",
            "dcp_decode_mla", "dcp_sfa_remap", "dcp_topk_workspace_size", "dcp_topk_local", "dcp_topk_merge",
            "dcp_topk", "dcp_sfa_compact_workspace_size", "dcp_sfa_compact_blocks",
            "dcp_sfa_decode_partial", "dcp_sfa_decode",
            "dcp_tree_workspace_size", "dcp_tree_partial_gqa", "dcp_tree_decode_gqa",
            "dcp_rope_write_gqa", "dcp_rope_write_mla", "dcp_pages_init",
            "dcp_pages_workspace_size", "dcp_pages_resize", "dcp_pages_fork", "dcp_pages_copy",
            "dcp_cache_compact", "dcp_q8_append_gqa", "dcp_q8_gather_gqa", "dcp_q8_decode_gqa",
            "dcp_q8_partial_gqa", "dcp_scored_decode_gqa", "dcp_scored_partial_gqa",
            "dcp_scored_workspace_size"]


def _check(rc):
    if rc != 0:
        msg = load().dcp_strerror(rc).decode()
        raise DcpError(f"libdcp error {rc}: {msg}")


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _dtype(t):
    try:
        return _DT[t.dtype]
    except KeyError:
        raise DcpError(f"unsupported dtype {t.dtype}") from None


def _cuda_contig(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise DcpError("tensors must be contiguous CUDA tensors")


def rank_ptrs(tensors) -> RankPtrs:
    rp = RankPtrs()
    for i, t in enumerate(tensors or []):
        rp.ptr[i] = t.data_ptr()
    return rp


def _rank_stride(block_table, ranks=1) -> int:
    """Entries between two ranks' tables; 0 for a table that all ranks share."""
    if block_table.dim() == 2 or block_table.shape[0] == 1:
        return 0
    if block_table.shape[0] < ranks:
        raise DcpError(f"{block_table.shape[0]} block tables for {ranks} ranks")
    return block_table.shape[1] * block_table.shape[2]


class PagedKV:
    """Per-rank paged pools plus the block table, as the decode calls read them.

    k_pools / v_pools: one tensor per rank (GQA: [num_blocks, Hkv, bs, d];
    latent: [num_blocks, bs, kv_dim], v_pools None).  block_table:
    [dcp, B, max_vb] int32 (one table per rank), or a table that all ranks
    share: [B, max_vb] or [1, B, max_vb].
    """

    def __init__(self, k_pools, v_pools, block_table, num_blocks):
        self.k_pools = list(k_pools)
        self.v_pools = list(v_pools) if v_pools is not None else None
        self.block_table = block_table
        self.num_blocks = int(num_blocks)
        _cuda_contig(block_table, *self.k_pools, *(self.v_pools or []))
        if block_table.dtype != torch.int32:
            raise DcpError("block_table must be int32")
        self.max_vb = block_table.shape[-1]
        self.bt_rank_stride = _rank_stride(block_table)

    def struct(self, layout=None) -> PagedKVStruct:
        """The C struct, for a call of this layout (which needs a table for each rank, or one)."""
        if layout is not None:
            _rank_stride(self.block_table, layout.dcp_size)
        s = PagedKVStruct()
        s.k = rank_ptrs(self.k_pools)
        s.v = rank_ptrs(self.v_pools)
        s.num_blocks = self.num_blocks
        s.block_table = self.block_table.data_ptr()
        s.max_vblocks = self.max_vb
        s.bt_rank_stride = self.bt_rank_stride
        return s


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def local_seq_lens(layout, seq_lens, out=None, err=None, stream=None):
    lib = load()
    _cuda_contig(seq_lens)
    B = seq_lens.shape[0]
    if out is None:
        out = torch.empty((B, layout.dcp_size), dtype=torch.int32, device=seq_lens.device)
    _check(lib.dcp_local_seq_lens(layout, _p(seq_lens), B, _p(out), _p(err), _stream(stream)))
    return out


def slot_mapping(layout, req_idx, positions, block_table, num_blocks, out_rank=None,
                 out_slot=None, err=None, stream=None):
    lib = load()
    _cuda_contig(req_idx, positions, block_table)
    T = req_idx.shape[0]
    B, max_vb = block_table.shape[-2:]
    stride = _rank_stride(block_table, layout.dcp_size)
    dev = req_idx.device
    if out_rank is None:
        out_rank = torch.empty(T, dtype=torch.int32, device=dev)
    if out_slot is None:
        out_slot = torch.empty((layout.dcp_size, T), dtype=torch.int64, device=dev)
    _check(lib.dcp_slot_mapping(layout, _p(req_idx), _p(positions), T, _p(block_table), B, max_vb,
                                stride, int(num_blocks), _p(out_rank), _p(out_slot), _p(err),
                                _stream(stream)))
    return out_rank, out_slot


def cache_write_gqa(layout, k, v, slot, k_pools, v_pools, num_blocks, err=None, stream=None):
    lib = load()
    _cuda_contig(k, v, slot)
    T, Hkv, d = k.shape
    _check(lib.dcp_cache_write_gqa(layout, _p(k), _p(v), T, Hkv, d, _dtype(k), _p(slot),
                                   int(num_blocks), rank_ptrs(k_pools), rank_ptrs(v_pools),
                                   _p(err), _stream(stream)))


def cache_write_mla(layout, kv, slot, pools, num_blocks, err=None, stream=None):
    lib = load()
    _cuda_contig(kv, slot)
    T, dk = kv.shape
    _check(lib.dcp_cache_write_mla(layout, _p(kv), T, dk, _dtype(kv), _p(slot), int(num_blocks),
                                   rank_ptrs(pools), _p(err), _stream(stream)))


def gather_context_mla(layout, kv: PagedKV, req_idx, positions, out=None, err=None,
                       stream=None):
    """Rows of tokens (req_idx[t], positions[t]) from the sharded latent cache."""
    lib = load()
    _cuda_contig(req_idx, positions)
    T = req_idx.shape[0]
    pool = kv.k_pools[0]
    kv_dim = pool.shape[-1]
    B = kv.block_table.shape[-2]
    if out is None:
        out = torch.empty((T, kv_dim), dtype=pool.dtype, device=pool.device)
    _check(lib.dcp_gather_context_mla(layout, kv.struct(layout), B, kv_dim, _dtype(pool),
                                      _p(req_idx), _p(positions), T, _p(out), _p(err),
                                      _stream(stream)))
    return out


def decode_workspace_size(layout, kind, num_reqs, num_q_heads, num_kv_heads, head_dim_v):
    lib = load()
    n = C.c_size_t(0)
    _check(lib.dcp_decode_workspace_size(layout, kind, num_reqs, num_q_heads, num_kv_heads,
                                         head_dim_v, C.byref(n)))
    return n.value


def _workspace(layout, kind, B, Hq, Hkv, dv, device, workspace):
    need = decode_workspace_size(layout, kind, B, Hq, Hkv, dv)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    return workspace


def decode_partial_gqa(layout, q, kv: PagedKV, local_lens, scale, part_o=None, part_lse=None,
                       workspace=None, err=None, stream=None):
    lib = load()
    _cuda_contig(q, local_lens)
    B, Hq, d = q.shape
    Hkv = kv.k_pools[0].shape[1]
    dev = q.device
    if part_o is None:
        part_o = torch.empty((layout.dcp_size, B, Hq, d), dtype=torch.float32, device=dev)
    if part_lse is None:
        part_lse = torch.empty((layout.dcp_size, B, Hq), dtype=torch.float32, device=dev)
    ws = _workspace(layout, KIND_GQA, B, Hq, Hkv, d, dev, workspace)
    _check(lib.dcp_decode_partial_gqa(layout, _p(q), B, Hq, Hkv, d, float(scale), _dtype(q),
                                      kv.struct(layout), _p(local_lens), _p(part_o), _p(part_lse),
                                      _p(ws), ws.numel(), _p(err), _stream(stream)))
    return part_o, part_lse


def decode_gqa(layout, q, kv: PagedKV, local_lens, scale, sink=None, out_dtype=None, out=None,
               out_lse=None, workspace=None, err=None, stream=None):
    lib = load()
    _cuda_contig(q, local_lens, sink)
    B, Hq, d = q.shape
    Hkv = kv.k_pools[0].shape[1]
    dev = q.device
    odt = out_dtype or q.dtype
    if out is None:
        out = torch.empty((B, Hq, d), dtype=odt, device=dev)
    if out_lse is None:
        out_lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    ws = _workspace(layout, KIND_GQA, B, Hq, Hkv, d, dev, workspace)
    _check(lib.dcp_decode_gqa(layout, _p(q), B, Hq, Hkv, d, float(scale), _dtype(q),
                              kv.struct(layout), _p(local_lens), _p(sink), _p(out), _dtype(out),
                              _p(out_lse), _p(ws), ws.numel(), _p(err), _stream(stream)))
    return out, out_lse


def decode_gqa_noalloc(layout, q, kv: PagedKV, local_lens, scale, sink=None, out_dtype=None,
                       out=None, out_lse=None, err=None, stream=None):
    """dcp_decode_gqa without a caller workspace: the library's fixed 16 MiB
    device array holds the split-KV scratch (for callers that cannot allocate;
    calls that overlap on the GPU race on that array)."""
    lib = load()
    _cuda_contig(q, local_lens, sink)
    B, Hq, d = q.shape
    Hkv = kv.k_pools[0].shape[1]
    dev = q.device
    odt = out_dtype or q.dtype
    if out is None:
        out = torch.empty((B, Hq, d), dtype=odt, device=dev)
    if out_lse is None:
        out_lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    _check(lib.dcp_decode_gqa_noalloc(layout, _p(q), B, Hq, Hkv, d, float(scale), _dtype(q),
                                      kv.struct(layout), _p(local_lens), _p(sink), _p(out),
                                      _dtype(out), _p(out_lse), _p(err), _stream(stream)))
    return out, out_lse


def lse_merge(part_o, part_lse, sink=None, out_dtype=torch.float32, out=None, out_lse=None,
              stream=None):
    lib = load()
    _cuda_contig(part_o, part_lse, sink)
    n, B, H, dv = part_o.shape
    dev = part_o.device
    if out is None:
        out = torch.empty((B, H, dv), dtype=out_dtype, device=dev)
    if out_lse is None:
        out_lse = torch.empty((B, H), dtype=torch.float32, device=dev)
    _check(lib.dcp_lse_merge(n, _p(part_o), _p(part_lse), B, H, dv, _p(sink), _p(out),
                             _dtype(out), _p(out_lse), _stream(stream)))
    return out, out_lse


def lse_merge_swa(part_o, part_lse, swa_o, swa_lse, sink=None, out_dtype=torch.float32, out=None,
                  out_lse=None, stream=None):
    """Merge the per-rank partials with ONE replicated-window partial (+ sink)."""
    lib = load()
    _cuda_contig(part_o, part_lse, swa_o, swa_lse, sink)
    n, B, H, dv = part_o.shape
    dev = part_o.device
    if out is None:
        out = torch.empty((B, H, dv), dtype=out_dtype, device=dev)
    if out_lse is None:
        out_lse = torch.empty((B, H), dtype=torch.float32, device=dev)
    _check(lib.dcp_lse_merge_swa(n, _p(part_o), _p(part_lse), _p(swa_o), _p(swa_lse), B, H, dv,
                                 _p(sink), _p(out), _dtype(out), _p(out_lse), _stream(stream)))
    return out, out_lse


def decode_partial_mla(layout, q, kv: PagedKV, local_lens, scale, v_dim=512, part_o=None,
                       part_lse=None, workspace=None, err=None, stream=None):
    lib = load()
    _cuda_contig(q, local_lens)
    B, Hq, dk = q.shape
    dev = q.device
    if part_o is None:
        part_o = torch.empty((layout.dcp_size, B, Hq, v_dim), dtype=torch.float32, device=dev)
    if part_lse is None:
        part_lse = torch.empty((layout.dcp_size, B, Hq), dtype=torch.float32, device=dev)
    ws = _workspace(layout, KIND_MLA, B, Hq, 1, v_dim, dev, workspace)
    _check(lib.dcp_decode_partial_mla(layout, _p(q), B, Hq, dk, v_dim, float(scale), _dtype(q),
                                      kv.struct(layout), _p(local_lens), _p(part_o), _p(part_lse),
                                      _p(ws), ws.numel(), _p(err), _stream(stream)))
    return part_o, part_lse


def decode_mla(layout, q, kv: PagedKV, local_lens, scale, v_dim=512, sink=None, out_dtype=None,
               out=None, out_lse=None, workspace=None, err=None, stream=None):
    lib = load()
    _cuda_contig(q, local_lens, sink)
    B, Hq, dk = q.shape
    dev = q.device
    odt = out_dtype or q.dtype
    if out is None:
        out = torch.empty((B, Hq, v_dim), dtype=odt, device=dev)
    if out_lse is None:
        out_lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    ws = _workspace(layout, KIND_MLA, B, Hq, 1, v_dim, dev, workspace)
    _check(lib.dcp_decode_mla(layout, _p(q), B, Hq, dk, v_dim, float(scale), _dtype(q),
                              kv.struct(layout), _p(local_lens), _p(sink), _p(out), _dtype(out),
                              _p(out_lse), _p(ws), ws.numel(), _p(err), _stream(stream)))
    return out, out_lse


def sfa_remap(layout, topk, seq_lens, block_table, num_blocks, out_rank=None, out_slot=None,
              err=None, stream=None):
    lib = load()
    _cuda_contig(topk, seq_lens, block_table)
    B, K = topk.shape
    max_vb, stride = block_table.shape[-1], _rank_stride(block_table, layout.dcp_size)
    if out_rank is None:
        out_rank = torch.empty((B, K), dtype=torch.int32, device=topk.device)
    if out_slot is None:
        out_slot = torch.empty((B, K), dtype=torch.int32, device=topk.device)
    _check(lib.dcp_sfa_remap(layout, _p(topk), B, K, _p(seq_lens), _p(block_table), max_vb,
                             stride, int(num_blocks), _p(out_rank), _p(out_slot), _p(err),
                             _stream(stream)))
    return out_rank, out_slot


def topk_local(layout, local_scores, local_lens, k, cand=None, stream=None):
    """Per-rank top-k candidate keys [dcp, B, k] (uint64 stored as int64)."""
    lib = load()
    _cuda_contig(local_scores, local_lens)
    dcp_, B, max_local = local_scores.shape
    if cand is None:
        cand = torch.empty((dcp_, B, k), dtype=torch.int64, device=local_scores.device)
    _check(lib.dcp_topk_local(layout, _p(local_scores), B, max_local, _p(local_lens), k, _p(cand),
                              _stream(stream)))
    return cand


def topk_merge(cand, stream=None):
    lib = load()
    _cuda_contig(cand)
    dcp_, B, k = cand.shape
    dev = cand.device
    ws = torch.empty(B * k * 8, dtype=torch.uint8, device=dev)
    ids = torch.empty((B, k), dtype=torch.int32, device=dev)
    scores = torch.empty((B, k), dtype=torch.float32, device=dev)
    _check(lib.dcp_topk_merge(dcp_, _p(cand), B, k, _p(ws), ws.numel(), _p(ids), _p(scores),
                              _stream(stream)))
    return ids, scores


def topk(layout, local_scores, local_lens, k, stream=None):
    """Exact global top-k ids and scores [B, k] from per-rank local scores."""
    lib = load()
    _cuda_contig(local_scores, local_lens)
    dcp_, B, max_local = local_scores.shape
    dev = local_scores.device
    n = C.c_size_t(0)
    _check(lib.dcp_topk_workspace_size(layout, B, k, C.byref(n)))
    ws = torch.empty(max(n.value, 1), dtype=torch.uint8, device=dev)
    ids = torch.empty((B, k), dtype=torch.int32, device=dev)
    scores = torch.empty((B, k), dtype=torch.float32, device=dev)
    _check(lib.dcp_topk(layout, _p(local_scores), B, max_local, _p(local_lens), k, _p(ids),
                        _p(scores), _p(ws), ws.numel(), _stream(stream)))
    return ids, scores


def sfa_compact_blocks(layout, kv: PagedKV, topk, q_req, seq_lens, max_blocks, err=None,
                       stream=None):
    """Compact the referenced latent blocks; returns (blocks, ids, counts, index)."""
    lib = load()
    _cuda_contig(topk, q_req, seq_lens)
    Q, K = topk.shape
    pool = kv.k_pools[0]
    kv_dim, bs = pool.shape[-1], pool.shape[-2]
    dev = pool.device
    n = C.c_size_t(0)
    _check(lib.dcp_sfa_compact_workspace_size(layout, kv.num_blocks, C.byref(n)))
    ws = torch.empty(max(n.value, 1), dtype=torch.uint8, device=dev)
    blocks = torch.empty((max(max_blocks, 1), bs, kv_dim), dtype=pool.dtype, device=dev)
    ids = torch.empty(max(max_blocks, 1), dtype=torch.int32, device=dev)
    counts = torch.empty(layout.dcp_size, dtype=torch.int32, device=dev)
    index = torch.empty((Q, K), dtype=torch.int64, device=dev)
    _check(lib.dcp_sfa_compact_blocks(layout, _p(topk), _p(q_req), Q, K, _p(seq_lens),
                                      kv.block_table.shape[-2], kv.struct(layout), kv_dim,
                                      _dtype(pool), int(max_blocks), _p(blocks), _p(ids), _p(counts),
                                      _p(index), _p(ws), ws.numel(), _p(err), _stream(stream)))
    return blocks, ids, counts, index


def sfa_decode_partial(layout, q, kv: PagedKV, sel_rank, sel_slot, scale, v_dim=512,
                       part_o=None, part_lse=None, err=None, stream=None):
    lib = load()
    _cuda_contig(q, sel_rank, sel_slot)
    B, Hq, dk = q.shape
    K = sel_rank.shape[1]
    dev = q.device
    if part_o is None:
        part_o = torch.empty((layout.dcp_size, B, Hq, v_dim), dtype=torch.float32, device=dev)
    if part_lse is None:
        part_lse = torch.empty((layout.dcp_size, B, Hq), dtype=torch.float32, device=dev)
    _check(lib.dcp_sfa_decode_partial(layout, _p(q), B, Hq, dk, v_dim, float(scale), _dtype(q),
                                      kv.struct(layout), _p(sel_rank), _p(sel_slot), K, _p(part_o),
                                      _p(part_lse), _p(err), _stream(stream)))
    return part_o, part_lse


def sfa_decode(layout, q, kv: PagedKV, topk, seq_lens, scale, v_dim=512, sink=None,
               out_dtype=None, out=None, out_lse=None, workspace=None, err=None, stream=None):
    lib = load()
    _cuda_contig(q, topk, seq_lens, sink)
    B, Hq, dk = q.shape
    K = topk.shape[1]
    dev = q.device
    odt = out_dtype or q.dtype
    if out is None:
        out = torch.empty((B, Hq, v_dim), dtype=odt, device=dev)
    if out_lse is None:
        out_lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    ws = _workspace(layout, KIND_SFA, B, Hq, 1, v_dim, dev, workspace)
    _check(lib.dcp_sfa_decode(layout, _p(q), B, Hq, dk, v_dim, float(scale), _dtype(q),
                              kv.struct(layout), _p(topk), K, _p(seq_lens), _p(sink), _p(out),
                              _dtype(out), _p(out_lse), _p(ws), ws.numel(), _p(err),
                              _stream(stream)))
    return out, out_lse


# ---------------------------------------------------------------------------
# around the decode step: drafted token trees, rotary positions, pages
# ---------------------------------------------------------------------------
# These calls are short (a few microseconds on the GPU), so their arguments are
# checked and handed to the C ABI by a native extension (binding/dcp_binding.cpp).
# Whatever it refuses, and every error of the library, is a DcpError.

def tree_workspace_size(layout, num_reqs, max_tree, num_q_heads, num_kv_heads, head_dim, dtype):
    """Bytes of workspace of tree_decode_gqa and tree_partial_gqa for this shape."""
    if dtype not in _DT:
        raise DcpError(f"unsupported dtype {dtype}")
    n = C.c_size_t(0)
    _check(load().dcp_tree_workspace_size(layout, num_reqs, max_tree, num_q_heads, num_kv_heads,
                                          head_dim, _DT[dtype], C.byref(n)))
    return n.value


def tree_decode_gqa(layout, q, kv: PagedKV, q_start, ctx_lens, tree_mask, scale, max_tree,
                    sink=None, out_dtype=None, out=None, out_lse=None, workspace=None, err=None,
                    stream=None):
    """Attention of drafted token trees: q [N, Hq, d] holds the nodes of all
    requests, packed; node j of request b is stored at position ctx_lens[b] + j.
    tree_mask [N] int64: bit j = sees node j of its request."""
    return (_bind or _load_binding()).tree(
        False, layout, q, kv, q_start, ctx_lens, tree_mask, scale, max_tree, sink, out_dtype, out,
        out_lse, workspace, err, stream)


def tree_partial_gqa(layout, q, kv: PagedKV, q_start, ctx_lens, tree_mask, scale, max_tree,
                     part_o=None, part_lse=None, workspace=None, err=None, stream=None):
    """tree_decode_gqa's per-rank partials, for lse_merge."""
    return (_bind or _load_binding()).tree(
        True, layout, q, kv, q_start, ctx_lens, tree_mask, scale, max_tree, None, None, part_o,
        part_lse, workspace, err, stream)


def rope_write_gqa(layout, q, k, v, positions, inv_freq, slot, k_pools, v_pools, num_blocks,
                   axis=None, interleaved=False, scaling=1.0, q_out=None, k_out=None, err=None,
                   stream=None):
    """Rotate q and k by their positions and write k, v into the cache at
    `slot`; returns the rotated q.  q, k, v may be slices of one projection."""
    return (_bind or _load_binding()).rope(
        False, layout, q, k, v, positions, inv_freq, slot, k_pools, v_pools, num_blocks, axis,
        interleaved, scaling, q_out, k_out, err, stream)


def rope_write_mla(layout, q, kv, positions, inv_freq, slot, pools, num_blocks, axis=None,
                   interleaved=True, scaling=1.0, q_out=None, err=None, stream=None):
    """Rotate the last entries of q's heads and of the latent rows, and write
    the rows into the cache at `slot`; returns the rotated q."""
    return (_bind or _load_binding()).rope(
        True, layout, q, kv, None, positions, inv_freq, slot, pools, None, num_blocks, axis,
        interleaved, scaling, q_out, None, err, stream)


class Pages:
    """Who holds which page of the cache (see dcp_pages_t).

    block_table [T, B, max_vb] int32 with T = dcp tables (one per rank) or 1 (a
    table that all ranks share), seq_lens [B] int32, ref_count [T, num_blocks]
    int32, free_bits [T, ceil(num_blocks / 32)] int32.  ``Pages.new`` makes them.
    The other calls take the table as it is, a shared one too.
    """

    def __init__(self, block_table, seq_lens, ref_count, free_bits, num_blocks):
        self.block_table, self.seq_lens = block_table, seq_lens
        self.ref_count, self.free_bits = ref_count, free_bits
        self.num_blocks = int(num_blocks)
        T, B, _ = block_table.shape
        for t, shape in ((block_table, block_table.shape), (seq_lens, (B,)),
                         (ref_count, (T, self.num_blocks)),
                         (free_bits, (T, (self.num_blocks + 31) // 32))):
            if t.dtype != torch.int32 or t.shape != shape or not t.is_cuda or \
                    not t.is_contiguous():
                raise DcpError(f"the pages' state: a contiguous int32 CUDA tensor of shape "
                               f"{tuple(shape)} is needed, got {t.dtype} {tuple(t.shape)} on "
                               f"{t.device}")

    @classmethod
    def new(cls, layout, num_reqs, max_vblocks, num_blocks, shared=False, device="cuda",
            stream=None):
        T = 1 if shared else layout.dcp_size
        mk = lambda *shape: torch.empty(shape, dtype=torch.int32, device=device)  # noqa: E731
        # memory of another stream may still be in use by work queued there
        with torch.cuda.stream(stream):
            p = cls(mk(T, num_reqs, max_vblocks), mk(num_reqs), mk(T, num_blocks),
                    mk(T, (num_blocks + 31) // 32), num_blocks)
        pages_init(layout, p, stream=stream)
        return p


def pages_init(layout, pages: Pages, stream=None):
    """Every request unused, every page free."""
    (_bind or _load_binding()).pages_init(layout, pages, stream)


def pages_resize(layout, pages: Pages, req, new_lens, copy_src=None, copy_dst=None, workspace=None,
                 err=None, stream=None):
    """Requests req [n] to lengths new_lens [n]: admit, grow, trim or free.
    Returns (copy_src, copy_dst) [tables, n] for pages_copy."""
    return (_bind or _load_binding()).pages(False, layout, pages, req, new_lens, copy_src, copy_dst,
                                            workspace, err, stream)


def pages_fork(layout, pages: Pages, parent, child, copy_src=None, copy_dst=None, workspace=None,
               err=None, stream=None):
    """child [n] become copies of parent [n]: full pages shared, open ones to
    be copied.  Returns (copy_src, copy_dst) [tables, n] for pages_copy."""
    return (_bind or _load_binding()).pages(True, layout, pages, parent, child, copy_src, copy_dst,
                                            workspace, err, stream)


class PoolSet:
    """Pools of one shape (keys and values of all layers), each a list of one
    tensor per rank: [num_blocks, heads, block_size, d], or [num_blocks,
    block_size, d] for latent rows.  Keeps the tensors and their addresses.  A
    pool named more than once (layers that share a cache) counts once."""

    def __init__(self, pools):
        # twice the same moves would read what the first had written
        self.pools = tuple({tuple((t.data_ptr(), t.shape) for t in p): p
                            for p in map(tuple, pools)}.values())
        flat = [t for p in self.pools for t in p]
        if not flat or len({len(p) for p in self.pools}) != 1:
            raise DcpError("a pool set needs pools with one tensor per rank each")
        first = flat[0]
        if first.dim() not in (3, 4):
            raise DcpError("pools must be [blocks, heads, block_size, d] or [blocks, block_size, d]")
        for t in flat:
            if t.dtype != first.dtype or t.shape != first.shape or t.device != first.device or \
                    not t.is_cuda or not t.is_contiguous() or t.data_ptr() % 16:
                raise DcpError("the pools of a set must be contiguous, 16-byte aligned CUDA "
                               "tensors of one type, shape and device")
        if sum(len({t.data_ptr() for t in p}) for p in self.pools) != \
                len({t.data_ptr() for t in flat}):
            raise DcpError("two pools of a set are alike on one rank and not on another")
        self.ranks = len(self.pools[0])
        self.num_blocks, self.block_size = first.shape[0], first.shape[-2]
        self.num_heads = first.shape[1] if first.dim() == 4 else 1
        self.row_bytes = first.shape[-1] * first.element_size()
        self.ptr = torch.tensor([[t.data_ptr() for t in p] for p in self.pools],
                                dtype=torch.int64).to(first.device)


def pages_copy(layout, pools: PoolSet, copy_src, copy_dst, err=None, stream=None):
    """Copy pages copy_src -> copy_dst [tables, n] inside every pool (-1: nothing)."""
    (_bind or _load_binding()).pages_copy(layout, pools, copy_src, copy_dst, err, stream)


def cache_compact(layout, pools: PoolSet, block_table, num_blocks, ctx_lens, path, path_len,
                  new_lens=None, err=None, stream=None):
    """Move the accepted drafted tokens path [B, max_path] (nodes behind
    ctx_lens [B], path_len [B] of them) together behind the context, in every
    pool; returns the new lengths [B].  block_table [dcp, B, max_vb], or one
    that all ranks share: [B, max_vb] or [1, B, max_vb]."""
    return (_bind or _load_binding()).cache_compact(layout, pools, block_table, num_blocks,
                                                    ctx_lens, path, path_len, new_lens, err, stream)


# ---------------------------------------------------------------------------
# the cache in 8 bits, and scored decode attention
# ---------------------------------------------------------------------------

class PagedKV8:
    """A paged cache in 8 bits (see dcp_paged_kv8_t): per-rank pools k_pools and
    v_pools [num_blocks, Hkv, bs, d] of torch.float8_e4m3fn, per-rank scales
    [num_blocks, Hkv, 4] float32 (of a page and head that of its keys, that of
    its values, and two unused), and the block table as for PagedKV."""

    def __init__(self, k_pools, v_pools, scales, block_table, num_blocks):
        self.k_pools, self.v_pools, self.scales = list(k_pools), list(v_pools), list(scales)
        self.block_table = block_table
        self.num_blocks = int(num_blocks)
        _cuda_contig(block_table, *self.k_pools, *self.v_pools, *self.scales)
        if block_table.dtype != torch.int32:
            raise DcpError("block_table must be int32")
        if any(t.dtype != torch.float8_e4m3fn for t in self.k_pools + self.v_pools):
            raise DcpError("the pools of an 8-bit cache must be float8_e4m3fn")
        if any(t.dtype != torch.float32 or t.dim() != 3 or t.shape[-1] != 4 for t in self.scales):
            raise DcpError("scales must be float32 [blocks, heads, 4]")

    @classmethod
    def new(cls, layout, num_blocks, num_kv_heads, head_dim, block_table):
        """An empty cache on the table's device: what its pages hold is written
        before it is read, but for the scales' unused numbers, which are zeros."""
        mk = lambda: [torch.empty((num_blocks, num_kv_heads, layout.block_size, head_dim),  # noqa: E731
                                  dtype=torch.float8_e4m3fn, device=block_table.device)
                      for _ in range(layout.dcp_size)]
        return cls(mk(), mk(), [torch.zeros((num_blocks, num_kv_heads, 4), device=block_table.device)
                                for _ in range(layout.dcp_size)], block_table, num_blocks)

    def struct(self, layout=None):
        raise DcpError("a cache in 8 bits: the q8_ calls read it")


class Scores:
    """How scores are formed and which tokens are seen (see dcp_scores_t): a cap
    (0: none), a window of the last tokens (0: all) with the document's first
    `prefix` tokens beside it, slopes [Hq] float32 of a bias by distance, and
    the first token [B] int32 of each request's document."""

    def __init__(self, cap=0.0, window=0, prefix=0, slopes=None, first=None):
        self.cap, self.window, self.prefix = float(cap), int(window), int(prefix)
        self.slopes, self.first = slopes, first


def scored_workspace_size(layout, num_reqs, num_q_heads, num_kv_heads, head_dim, per_rank=False):
    """Bytes of workspace of the scored_ and q8_ attention calls for this shape."""
    n = C.c_size_t(0)
    _check(load().dcp_scored_workspace_size(layout, num_reqs, num_q_heads, num_kv_heads, head_dim,
                                            int(per_rank), C.byref(n)))
    return n.value


def q8_append_gqa(layout, k, v, kv: PagedKV8, q_start, ctx_lens, err=None, stream=None):
    """Quantise k, v [N, Hkv, d] into the cache: rows q_start[b] .. q_start[b+1]
    go to positions ctx_lens[b] .. of request b.  k, v may be slices of one
    projection."""
    (_bind or _load_binding()).q8_append(layout, k, v, kv, q_start, ctx_lens, err, stream)


def q8_gather_gqa(layout, kv: PagedKV8, req_idx, positions, dtype=torch.bfloat16, k_out=None,
                  v_out=None, err=None, stream=None):
    """Keys and values [N, Hkv, d] of tokens (req_idx[t], positions[t])."""
    return (_bind or _load_binding()).q8_gather(layout, kv, req_idx, positions, dtype, k_out, v_out,
                                                err, stream)


def q8_decode_gqa(layout, q, kv: PagedKV8, seq_lens, scale, scores=None, sink=None, out_dtype=None,
                  out=None, out_lse=None, workspace=None, err=None, stream=None):
    """decode_gqa over a cache in 8 bits, from the lengths [B] themselves."""
    return (_bind or _load_binding()).scored(True, False, layout, q, kv, seq_lens, scale, scores,
                                             sink, out_dtype, out, out_lse, workspace, err, stream)


def q8_partial_gqa(layout, q, kv: PagedKV8, seq_lens, scale, scores=None, part_o=None,
                   part_lse=None, workspace=None, err=None, stream=None):
    """q8_decode_gqa's per-rank partials, for lse_merge."""
    return (_bind or _load_binding()).scored(True, True, layout, q, kv, seq_lens, scale, scores,
                                             None, None, part_o, part_lse, workspace, err, stream)


def scored_decode_gqa(layout, q, kv: PagedKV, seq_lens, scale, scores, sink=None, out_dtype=None,
                      out=None, out_lse=None, workspace=None, err=None, stream=None):
    """decode_gqa with scores formed as `scores` says, from the lengths [B]."""
    return (_bind or _load_binding()).scored(False, False, layout, q, kv, seq_lens, scale, scores,
                                             sink, out_dtype, out, out_lse, workspace, err, stream)


def scored_partial_gqa(layout, q, kv: PagedKV, seq_lens, scale, scores, part_o=None, part_lse=None,
                       workspace=None, err=None, stream=None):
    """scored_decode_gqa's per-rank partials, for lse_merge."""
    return (_bind or _load_binding()).scored(False, True, layout, q, kv, seq_lens, scale, scores,
                                             None, None, part_o, part_lse, workspace, err, stream)


def q8_pages_copy(layout, caches, copy_src, copy_dst, err=None, stream=None):
    """pages_copy for the caches (of all layers) in 8 bits: their pages and their
    scales.  `caches` is a Q8Pools."""
    pages_copy(layout, caches.pages, copy_src, copy_dst, err=err, stream=stream)
    pages_copy(Layout(layout.dcp_size, 1, 1), caches.scales, copy_src, copy_dst, stream=stream)


class Q8Pools:
    """The pools and scales of several PagedKV8 of one shape, for q8_pages_copy."""

    def __init__(self, caches):
        caches = list(caches)
        # as bytes: the copies move them unchanged
        self.pages = PoolSet([[t.view(torch.uint8) for t in p]
                              for c in caches for p in (c.k_pools, c.v_pools)])
        # a head's scales are 16 bytes, its page's one row
        self.scales = PoolSet([[t.unsqueeze(2) for t in c.scales] for c in caches])
