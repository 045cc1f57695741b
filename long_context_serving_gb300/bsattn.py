"""Thin ctypes binding of libbsattn.so (include/bsattn.h).

Argument marshalling only: every step of the decode path runs in the library's
CUDA kernels. Tensors are passed as raw device pointers; the stream is the
caller's current torch stream unless one is given. A missing library raises.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbsattn.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "bsattn.h")

# bs_status
BS_OK = 0
BS_ERR_INVALID_ARG = 1
BS_ERR_SHAPE = 2
BS_ERR_ALIGN = 3
BS_ERR_CAPACITY = 4
BS_ERR_CUDA = 5
BS_ERR_DEVICE_BOUNDS = 6
BS_ERR_TIMEOUT = 7
# bs_dtype, bs_head_class, bs_group_reduce
BS_BF16, BS_FP32, BS_E4M3, BS_INT8 = 0, 1, 2, 3
BS_STREAMING, BS_RETRIEVAL, BS_DUAL = 0, 1, 2
BS_GROUP_MAX, BS_GROUP_MEAN = 0, 1
BS_MAX_DRAFT = 64


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages_per_unit", ctypes.c_int32), ("max_blocks_per_unit", ctypes.c_int32),
                ("max_sel_per_unit", ctypes.c_int32), ("max_subs_per_unit", ctypes.c_int32),
                ("max_gather_pages_per_unit", ctypes.c_int32), ("n_pages", ctypes.c_int64),
                ("kv_dtype", ctypes.c_int), ("q_dtype", ctypes.c_int)]


class KV(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class HeadCfg(ctypes.Structure):
    _fields_ = [("cls", ctypes.c_void_p), ("block_tokens", ctypes.c_void_p), ("sub_tokens", ctypes.c_void_p),
                ("k_total", ctypes.c_void_p), ("k_evict", ctypes.c_void_p), ("sink_tokens", ctypes.c_void_p),
                ("local_tokens", ctypes.c_void_p), ("sum_off", ctypes.c_void_p), ("sum_rows", ctypes.c_void_p)]


class StepIO(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("summaries", ctypes.c_void_p), ("scores", ctypes.c_void_p),
                ("evict_logits", ctypes.c_void_p), ("alive", ctypes.c_void_p), ("evict_bias", ctypes.c_void_p),
                ("prev_idx", ctypes.c_void_p),
                ("prev_cnt", ctypes.c_void_p), ("cur_idx", ctypes.c_void_p), ("cur_cnt", ctypes.c_void_p),
                ("added", ctypes.c_void_p), ("added_cnt", ctypes.c_void_p), ("removed", ctypes.c_void_p),
                ("removed_cnt", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("dev_status", ctypes.c_void_p)]


class HostKV(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64)]


class BlockCache(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("slot_block", ctypes.c_void_p), ("block_slot", ctypes.c_void_p),
                ("slots_per_unit", ctypes.c_int32), ("pages_per_slot", ctypes.c_int32)]


class HostTables(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("block_tokens", ctypes.c_void_p),
                ("evict_bias", ctypes.c_void_p), ("max_blocks_per_unit", ctypes.c_int32)]


class Pools(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class PageMap(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("ref_count", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p)]


class PageCopies(ctypes.Structure):
    _fields_ = [("pairs", ctypes.c_void_p), ("count", ctypes.c_void_p), ("capacity", ctypes.c_int32)]


class Rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("magnitude", ctypes.c_float), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class Drafts(ctypes.Structure):
    _fields_ = [("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("n_rows", ctypes.c_int64), ("row_begin", ctypes.c_void_p), ("n_draft", ctypes.c_void_p),
                ("visible", ctypes.c_void_p), ("max_draft", ctypes.c_int32)]


class BsError(RuntimeError):
    def __init__(self, call: str, status: int, text: str):
        super().__init__(f"{call} returned {status} ({text})")
        self.status = status


_P = ctypes.POINTER
_SIGS = {
    "bs_check_head_cfg": (ctypes.c_int, [_P(Dims), _P(HeadCfg), ctypes.c_void_p]),
    "bs_build_block_summaries": (ctypes.c_int, [_P(Dims), _P(KV), _P(HeadCfg), ctypes.c_void_p, ctypes.c_int32,
                                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "bs_score_blocks": (ctypes.c_int, [_P(Dims), ctypes.c_void_p, _P(HeadCfg), ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "bs_select_topk": (ctypes.c_int, [_P(Dims), _P(HeadCfg), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p]),
    "bs_sparse_decode_attn": (ctypes.c_int, [_P(Dims), ctypes.c_void_p, _P(KV), _P(HeadCfg), ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "bs_block_setdiff": (ctypes.c_int, [_P(Dims), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "bs_sparse_decode_attn_noalloc": (ctypes.c_int, [_P(Dims), ctypes.c_void_p, _P(KV), _P(HeadCfg),
                                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                     ctypes.c_void_p]),
    "bs_decode_step": (ctypes.c_int, [_P(Dims), _P(KV), _P(HeadCfg), _P(StepIO), ctypes.c_int, ctypes.c_void_p]),
    "bs_block_swap": (ctypes.c_int, [_P(Dims), _P(HeadCfg), ctypes.c_void_p, _P(HostKV), _P(BlockCache),
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p]),
    "bs_cpu_sparse_attn": (ctypes.c_int, [_P(Dims), ctypes.c_void_p, _P(HostKV), _P(HostTables), ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int]),
    "bs_lse_merge": (ctypes.c_int, [_P(Dims), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "bs_quant_append": (ctypes.c_int, [_P(Dims), _P(Pools), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                       ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]),
    "bs_pages_workspace_size": (ctypes.c_size_t, [_P(Dims)]),
    "bs_pages_reserve": (ctypes.c_int, [_P(Dims), _P(PageMap), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p, ctypes.c_void_p]),
    "bs_pages_fork": (ctypes.c_int, [_P(Dims), _P(PageMap), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                     _P(PageCopies), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                     ctypes.c_void_p]),
    "bs_pages_free": (ctypes.c_int, [_P(Dims), _P(PageMap), ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.c_void_p]),
    "bs_pages_compact": (ctypes.c_int, [_P(Dims), _P(PageMap), _P(PageCopies), ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "bs_pages_copy": (ctypes.c_int, [_P(Dims), _P(Pools), _P(PageCopies), ctypes.c_void_p, ctypes.c_void_p]),
    "bs_rope_append": (ctypes.c_int, [_P(Dims), _P(Rope), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, _P(Pools),
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p]),
    "bs_prefill_attn": (ctypes.c_int, [_P(Dims), ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, _P(KV), _P(HeadCfg),
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                       ctypes.c_void_p]),
    "bs_prefill_workspace_size": (ctypes.c_size_t, [_P(Dims), ctypes.c_int64, ctypes.c_int32]),
    "bs_tree_decode_attn": (ctypes.c_int, [_P(Dims), ctypes.c_void_p, ctypes.c_int64, _P(KV), _P(HeadCfg),
                                           ctypes.c_void_p, ctypes.c_void_p, _P(Drafts), ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                           ctypes.c_void_p]),
    "bs_tree_workspace_size": (ctypes.c_size_t, [_P(Dims), ctypes.c_int32]),
    "bs_tree_commit": (ctypes.c_int, [_P(Dims), _P(Pools), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                      ctypes.c_void_p]),
    "bs_workspace_size": (ctypes.c_size_t, [_P(Dims)]),
    "bs_decode_step_launches": (ctypes.c_int, [_P(Dims)]),
    "bs_set_wait_limit_ns": (ctypes.c_int, [ctypes.c_uint64]),
    "bs_wait_limit_ns": (ctypes.c_uint64, []),
    "bs_status_string": (ctypes.c_char_p, [ctypes.c_int]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library. Raises when it has not been built: there is no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with long_context_serving_gb300.build.build()")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/bsattn.h declares."""
    text = open(HEADER, encoding="utf-8").read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(bs_[a-z_]+)\s*\(", text)))


def status_string(status: int) -> str:
    return lib().bs_status_string(status).decode()


def _check(call: str, status: int) -> None:
    if status != BS_OK:
        raise BsError(call, status, status_string(status))


def _ptr(t) -> int | None:
    if type(t) is torch.Tensor:
        return t.data_ptr()
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return t.ctypes.data          # a numpy array (host memory)


def _current_stream():
    """A function for the raw handle of the current stream. The handle alone, through torch's own
    internals where it has them: a Stream object takes longer than a call's launches."""
    raw, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
    if raw is None or device is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw(device())


_current = _current_stream()


def _stream(stream) -> int | None:
    if stream is None:
        return _current()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def check_head_cfg(dims: Dims, cfg_host: HeadCfg, seq_lens_host) -> int:
    """Host-side check of a head configuration held in host memory; returns the status."""
    return lib().bs_check_head_cfg(ctypes.byref(dims), ctypes.byref(cfg_host), _ptr(seq_lens_host))


def build_block_summaries(dims, kv, cfg, tok_begin, max_new_tokens, summaries, dev_status, stream=None):
    _check("bs_build_block_summaries",
           lib().bs_build_block_summaries(ctypes.byref(dims), ctypes.byref(kv), ctypes.byref(cfg), _ptr(tok_begin),
                                          int(max_new_tokens), _ptr(summaries), _ptr(dev_status), _stream(stream)))


def score_blocks(dims, q, cfg, seq_lens, summaries, group_reduce, scores, dev_status, stream=None):
    _check("bs_score_blocks",
           lib().bs_score_blocks(ctypes.byref(dims), _ptr(q), ctypes.byref(cfg), _ptr(seq_lens), _ptr(summaries),
                                 int(group_reduce), _ptr(scores), _ptr(dev_status), _stream(stream)))


def select_topk(dims, cfg, seq_lens, scores, evict_logits, alive, sel_idx, sel_cnt, dev_status, stream=None):
    _check("bs_select_topk",
           lib().bs_select_topk(ctypes.byref(dims), ctypes.byref(cfg), _ptr(seq_lens), _ptr(scores),
                                _ptr(evict_logits), _ptr(alive), _ptr(sel_idx), _ptr(sel_cnt), _ptr(dev_status),
                                _stream(stream)))


def sparse_decode_attn(dims, q, kv, cfg, sel_idx, sel_cnt, out, lse, workspace, dev_status, stream=None,
                       evict_bias=None):
    """a4. evict_bias (None: plain softmax) is the ED-DMA logit bias of every block,
    fp32 [units][max_blocks_per_unit] on the device."""
    _check("bs_sparse_decode_attn",
           lib().bs_sparse_decode_attn(ctypes.byref(dims), _ptr(q), ctypes.byref(kv), ctypes.byref(cfg),
                                       _ptr(sel_idx), _ptr(sel_cnt), _ptr(evict_bias), _ptr(out), _ptr(lse),
                                       _ptr(workspace), _nbytes(workspace), _ptr(dev_status), _stream(stream)))


def block_setdiff(dims, prev_idx, prev_cnt, cur_idx, cur_cnt, added, added_cnt, removed, removed_cnt, dev_status,
                  stream=None):
    _check("bs_block_setdiff",
           lib().bs_block_setdiff(ctypes.byref(dims), _ptr(prev_idx), _ptr(prev_cnt), _ptr(cur_idx), _ptr(cur_cnt),
                                  _ptr(added), _ptr(added_cnt), _ptr(removed), _ptr(removed_cnt), _ptr(dev_status),
                                  _stream(stream)))


def sparse_decode_attn_noalloc(dims, q, kv, cfg, sel_idx, sel_cnt, out, lse, dev_status, stream=None,
                               evict_bias=None):
    """bs_sparse_decode_attn for callers that cannot allocate a workspace: the library's
    fixed per-device scratch array stands in for it (see include/bsattn.h)."""
    _check("bs_sparse_decode_attn_noalloc",
           lib().bs_sparse_decode_attn_noalloc(ctypes.byref(dims), _ptr(q), ctypes.byref(kv), ctypes.byref(cfg),
                                               _ptr(sel_idx), _ptr(sel_cnt), _ptr(evict_bias), _ptr(out),
                                               _ptr(lse), _ptr(dev_status), _stream(stream)))


def decode_step(dims, kv, cfg, io: StepIO, group_reduce=BS_GROUP_MAX, stream=None):
    """All five steps of one layer's decode step (two launches)."""
    _check("bs_decode_step", lib().bs_decode_step(ctypes.byref(dims), ctypes.byref(kv), ctypes.byref(cfg),
                                                  ctypes.byref(io), int(group_reduce), _stream(stream)))


def block_swap(dims, cfg, seq_lens, host: HostKV, cache: BlockCache, added, added_cnt, removed, removed_cnt,
               dev_status, stream=None):
    """Move the blocks the set-difference adds from host memory into the GPU block cache."""
    _check("bs_block_swap",
           lib().bs_block_swap(ctypes.byref(dims), ctypes.byref(cfg), _ptr(seq_lens), ctypes.byref(host),
                               ctypes.byref(cache), _ptr(added), _ptr(added_cnt), _ptr(removed), _ptr(removed_cnt),
                               _ptr(dev_status), _stream(stream)))


def cpu_sparse_attn(dims, q, kv: HostKV, tables: HostTables, sel_idx, sel_cnt, out, lse, n_threads: int):
    """Attention of the listed blocks on the host cores (every buffer in host memory)."""
    _check("bs_cpu_sparse_attn",
           lib().bs_cpu_sparse_attn(ctypes.byref(dims), _ptr(q), ctypes.byref(kv), ctypes.byref(tables),
                                    _ptr(sel_idx), _ptr(sel_cnt), _ptr(out), _ptr(lse), int(n_threads)))


def lse_merge(dims, out_a, lse_a, out_b, lse_b, out, lse, stream=None):
    """Merge two partial attention results over disjoint token sets (device memory)."""
    _check("bs_lse_merge", lib().bs_lse_merge(ctypes.byref(dims), _ptr(out_a), _ptr(lse_a), _ptr(out_b),
                                              _ptr(lse_b), _ptr(out), _ptr(lse), _stream(stream)))


def quant_append(dims, pools: Pools, page_table, seq_lens, tok_begin, row_begin, k_new, v_new, row_stride: int,
                 n_rows: int, max_new_tokens: int, dev_status, stream=None):
    """Quantise new tokens' K and V into the pages of an 8-bit cache."""
    _check("bs_quant_append",
           lib().bs_quant_append(ctypes.byref(dims), ctypes.byref(pools), _ptr(page_table), _ptr(seq_lens),
                                 _ptr(tok_begin), _ptr(row_begin), _ptr(k_new), _ptr(v_new), int(row_stride),
                                 int(n_rows), int(max_new_tokens), _ptr(dev_status), _stream(stream)))


def pages_reserve(dims, page_map: PageMap, new_lens, workspace, dev_status, stream=None):
    """Free pages for every entry below ceil(new_lens / 16) that holds none."""
    _check("bs_pages_reserve",
           lib().bs_pages_reserve(ctypes.byref(dims), ctypes.byref(page_map), _ptr(new_lens), _ptr(workspace),
                                  _nbytes(workspace), _ptr(dev_status), _stream(stream)))


def pages_fork(dims, page_map: PageMap, src, dst, copies: PageCopies, workspace, dev_status, stream=None):
    """Slots dst become copies of sequences src: full pages shared, partial last pages listed in copies."""
    if src.numel() != dst.numel():
        raise ValueError(f"src and dst differ in length: {src.numel()} and {dst.numel()}")
    _check("bs_pages_fork",
           lib().bs_pages_fork(ctypes.byref(dims), ctypes.byref(page_map), _ptr(src), _ptr(dst), src.numel(),
                               ctypes.byref(copies), _ptr(workspace), _nbytes(workspace), _ptr(dev_status),
                               _stream(stream)))


def pages_free(dims, page_map: PageMap, seqs, dev_status, stream=None):
    """The sequences give up their pages; their lengths become 0."""
    _check("bs_pages_free",
           lib().bs_pages_free(ctypes.byref(dims), ctypes.byref(page_map), _ptr(seqs), seqs.numel(),
                               _ptr(dev_status), _stream(stream)))


def pages_compact(dims, page_map: PageMap, copies: PageCopies, n_live, workspace, dev_status, stream=None):
    """Moves the pages in use below their number, n_live; the moves are listed in copies."""
    _check("bs_pages_compact",
           lib().bs_pages_compact(ctypes.byref(dims), ctypes.byref(page_map), ctypes.byref(copies), _ptr(n_live),
                                  _ptr(workspace), _nbytes(workspace), _ptr(dev_status), _stream(stream)))


def pages_copy(dims, pools: Pools, copies: PageCopies, dev_status, stream=None):
    """Copies the listed pages (and their scales) of one layer's pools."""
    _check("bs_pages_copy",
           lib().bs_pages_copy(ctypes.byref(dims), ctypes.byref(pools), ctypes.byref(copies), _ptr(dev_status),
                               _stream(stream)))


def rope_append(dims, rope: Rope, q, k, v, row_stride: int, n_rows: int, positions, row_seq, pools, page_table, q_out,
                k_out, dev_status, stream=None):
    """Queries and keys normalised per head and rotated; with pools, K and V written into their pages."""
    _check("bs_rope_append",
           lib().bs_rope_append(ctypes.byref(dims), ctypes.byref(rope), _ptr(q), _ptr(k), _ptr(v), int(row_stride),
                                int(n_rows), _ptr(positions), _ptr(row_seq),
                                None if pools is None else ctypes.byref(pools), _ptr(page_table), _ptr(q_out),
                                _ptr(k_out), _ptr(dev_status), _stream(stream)))


def prefill_attn(dims, q, q_stride: int, n_rows: int, kv, cfg, tok_begin, row_begin, max_new_tokens: int, out, lse,
                 workspace, dev_status, stream=None):
    """New tokens attend the cache that holds them: everything before them, or sinks and a window."""
    _check("bs_prefill_attn",
           lib().bs_prefill_attn(ctypes.byref(dims), _ptr(q), int(q_stride), int(n_rows), ctypes.byref(kv),
                                 ctypes.byref(cfg), _ptr(tok_begin), _ptr(row_begin), int(max_new_tokens), _ptr(out),
                                 _ptr(lse), _ptr(workspace), 0 if workspace is None else _nbytes(workspace),
                                 _ptr(dev_status), _stream(stream)))


def tree_decode_attn(dims, q, q_stride: int, kv, cfg, sel_idx, sel_cnt, drafts: Drafts, out, lse, workspace, dev_status,
                     stream=None):
    """A tree of drafted tokens attends the selected blocks and its own ancestors."""
    _check("bs_tree_decode_attn",
           lib().bs_tree_decode_attn(ctypes.byref(dims), _ptr(q), int(q_stride), ctypes.byref(kv), ctypes.byref(cfg),
                                     _ptr(sel_idx), _ptr(sel_cnt), ctypes.byref(drafts), _ptr(out), _ptr(lse),
                                     _ptr(workspace), 0 if workspace is None else _nbytes(workspace),
                                     _ptr(dev_status), _stream(stream)))


def tree_commit(dims, pools: Pools, page_table, seq_lens, tok_begin, row_begin, path, path_stride: int, k_new, v_new,
                row_stride: int, n_rows: int, dev_status, stream=None):
    """The accepted drafts' K and V, along a path through each tree, appended to the cache."""
    _check("bs_tree_commit",
           lib().bs_tree_commit(ctypes.byref(dims), ctypes.byref(pools), _ptr(page_table), _ptr(seq_lens),
                                _ptr(tok_begin), _ptr(row_begin), _ptr(path), int(path_stride), _ptr(k_new),
                                _ptr(v_new), int(row_stride), int(n_rows), _ptr(dev_status), _stream(stream)))


def prefill_workspace_size(dims, n_rows: int, max_new_tokens: int) -> int:
    return int(lib().bs_prefill_workspace_size(ctypes.byref(dims), int(n_rows), int(max_new_tokens)))


def tree_workspace_size(dims, max_draft: int) -> int:
    return int(lib().bs_tree_workspace_size(ctypes.byref(dims), int(max_draft)))


def pages_workspace_size(dims) -> int:
    return int(lib().bs_pages_workspace_size(ctypes.byref(dims)))


def workspace_size(dims) -> int:
    return int(lib().bs_workspace_size(ctypes.byref(dims)))


def decode_step_launches(dims) -> int:
    """Kernels one decode_step call launches for these dims (0 on bad dims)."""
    return int(lib().bs_decode_step_launches(ctypes.byref(dims)))


def set_wait_limit_ns(limit_ns: int) -> None:
    """Limit of every device-side wait of the calls launched from now on (default 1 s)."""
    _check("bs_set_wait_limit_ns", lib().bs_set_wait_limit_ns(int(limit_ns)))


def wait_limit_ns() -> int:
    return int(lib().bs_wait_limit_ns())
