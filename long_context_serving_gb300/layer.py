"""Device buffers of one attention layer's decode state, laid out for libbsattn.

PyTorch here only allocates device memory, copies inputs in and scatters logical
tokens into the paged pool; every step of the decode path is a libbsattn call.
"""
from __future__ import annotations

import contextlib
import ctypes

import numpy as np
import torch

from . import bsattn as B


def _cdiv(a: int, b: int) -> int:
    return -(-a // b)


def _kv_tensor(arr: np.ndarray, dtype: str, device) -> torch.Tensor:
    if dtype == "bf16":
        return torch.from_numpy(np.ascontiguousarray(arr).view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(arr, dtype=np.float32)).to(device)


def _on(stream):
    """torch's own work on `stream` too (a Stream, a raw handle, or None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream))))


class PagedLayer:
    """One layer of a workload: paged K/V pools, head configuration, summaries and the
    per-step buffers of the five calls.

    ``workload`` is any object with the fields of ``workloads.Workload`` (shapes, head
    properties, logical K/V/q arrays, eviction logits, page table).
    ``fill``: value written into pool slots that hold no token yet, so that a kernel
    reading past T would show up (NaN by default).
    ``preload_all``: put every token of every step in the pool now (otherwise tokens
    enter the pool when their step appends them).
    ``q_fp32``: pass the queries as fp32 (the same values, widened) over a bf16 cache.
    ``kv8``: "e4m3" or "int8" keeps the cache in 8 bits with a scale per page; tokens enter
    it through bs_quant_append (slots without a token hold NaN, or 85 in INT8).
    """

    def __init__(self, wl, device="cuda", fill=float("nan"), preload_all=False, q_fp32=False, ed_dma=False,
                 kv8=None):
        self.wl = wl
        if kv8 not in (None, "e4m3", "int8"):
            raise ValueError(f"kv8 is None, 'e4m3' or 'int8', not {kv8!r}")
        self.kv8 = kv8
        # ED-DMA attention: the eviction logits also enter the attention as block logits.
        self.ed_dma = bool(ed_dma)
        self.device = torch.device(device)
        U, d, G = wl.U, wl.d, wl.G
        T_cap = wl.T_cap
        g = wl.g.astype(np.int64)
        s = wl.s.astype(np.int64)
        max_pages = int(wl.page_table.shape[1])
        n_sink = np.array([_cdiv(int(wl.sink[u]), int(g[u])) for u in range(U)])
        n_local = np.array([_cdiv(int(wl.local[u]), int(g[u])) + 1 for u in range(U)])
        n_blk_cap = np.array([_cdiv(T_cap, int(g[u])) for u in range(U)])
        sel_u = np.minimum(n_sink + n_local + wl.k.astype(np.int64), n_blk_cap)
        self.max_sel = int(sel_u.max())
        self.max_blocks = int(n_blk_cap.max())
        sub_rows = np.array([_cdiv(T_cap, int(s[u])) for u in range(U)], dtype=np.int64)
        self.dims = B.Dims(batch=wl.B, n_q_heads=wl.Hq, n_kv_heads=wl.Hkv, head_dim=d, page_size=16,
                           max_pages_per_unit=max_pages, max_blocks_per_unit=self.max_blocks,
                           max_sel_per_unit=self.max_sel, max_subs_per_unit=int(sub_rows.max()),
                           max_gather_pages_per_unit=int((sel_u * g // 16).max()), n_pages=int(wl.n_pages),
                           kv_dtype={"e4m3": B.BS_E4M3, "int8": B.BS_INT8}[kv8] if kv8
                           else B.BS_BF16 if wl.dtype == "bf16" else B.BS_FP32,
                           q_dtype=B.BS_BF16 if wl.dtype == "bf16" and not q_fp32 else B.BS_FP32)

        dev = self.device
        i32 = lambda a: torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device=dev)  # noqa: E731
        # Head configuration (struct of arrays) and summary offsets.
        sum_off = np.zeros(U, dtype=np.int64)
        sum_off[1:] = np.cumsum(sub_rows * d)[:-1]
        self.cfg_arrays = dict(cls=i32(wl.cls), block_tokens=i32(wl.g), sub_tokens=i32(wl.s), k_total=i32(wl.k),
                               k_evict=i32(wl.k_e), sink_tokens=i32(wl.sink), local_tokens=i32(wl.local),
                               sum_off=torch.as_tensor(sum_off, device=dev), sum_rows=i32(sub_rows))
        self.cfg = B.HeadCfg(**{k: v.data_ptr() for k, v in self.cfg_arrays.items()})
        host = dict(cls=wl.cls, block_tokens=wl.g, sub_tokens=wl.s, k_total=wl.k, k_evict=wl.k_e,
                    sink_tokens=wl.sink, local_tokens=wl.local, sum_off=sum_off, sum_rows=sub_rows)
        self._cfg_host = {k: np.ascontiguousarray(v, dtype=np.int64 if k == "sum_off" else np.int32)
                          for k, v in host.items()}
        cfg_host = B.HeadCfg(**{k: v.ctypes.data for k, v in self._cfg_host.items()})
        T_last = (wl.T_prefill + wl.steps).astype(np.int32)
        st = B.check_head_cfg(self.dims, cfg_host, T_last)
        if st != B.BS_OK:
            raise B.BsError("bs_check_head_cfg", st, B.status_string(st))

        # Paged pools.
        kv_dt = torch.bfloat16 if wl.dtype == "bf16" else torch.float32
        self.page_table = i32(wl.page_table)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.k_scale = self.v_scale = None
        if kv8:
            code = torch.float8_e4m3fn if kv8 == "e4m3" else torch.int8
            self.k_pool = torch.full((wl.n_pages, 16, d), 0x7F if kv8 == "e4m3" else 85, dtype=torch.uint8,
                                     device=dev).view(code)
            self.v_pool = self.k_pool.clone()
            self.k_scale = torch.full((wl.n_pages,), float("nan"), dtype=torch.float32, device=dev)
            self.v_scale = self.k_scale.clone()
            self.pools = B.Pools(k_pool=self.k_pool.data_ptr(), v_pool=self.v_pool.data_ptr(),
                                 k_scale=self.k_scale.data_ptr(), v_scale=self.v_scale.data_ptr())
        else:
            self.k_pool = torch.full((wl.n_pages, 16, d), fill, dtype=kv_dt, device=dev)
            self.v_pool = torch.full((wl.n_pages, 16, d), fill, dtype=kv_dt, device=dev)
        self._pt_long = self.page_table.long()
        self._K = _kv_tensor(wl.K, wl.dtype, dev)          # logical [U][T_cap][d], source of appends
        self._V = _kv_tensor(wl.V, wl.dtype, dev)
        upto = np.full(wl.B, T_cap, np.int64) if preload_all else wl.T_prefill.astype(np.int64)
        if preload_all and kv8:       # (a shorter sequence has no pages past its last step)
            upto = np.minimum(upto, T_last.astype(np.int64))
        self._write_tokens(np.zeros(wl.B, np.int64), upto)

        self.q = _kv_tensor(wl.q, wl.dtype, dev)           # [steps][B][Hq][d]
        if q_fp32:
            self.q = self.q.float().contiguous()
        self.seq_lens = i32(np.stack([wl.T_prefill + i + 1 for i in range(wl.steps)]))  # [steps][B]
        self.tok_begin = self.seq_lens - 1
        self.prefill_lens = i32(wl.T_prefill)
        self.zeros_b = torch.zeros(wl.B, dtype=torch.int32, device=dev)
        self.kv = B.KV(k_pool=self.k_pool.data_ptr(), v_pool=self.v_pool.data_ptr(),
                       page_table=self.page_table.data_ptr(), seq_lens=0,
                       k_scale=self.k_scale.data_ptr() if kv8 else 0, v_scale=self.v_scale.data_ptr() if kv8 else 0)

        # Per-step state and outputs.
        MB, MS = self.max_blocks, self.max_sel
        self.summaries = torch.full((int(sub_rows.sum()) * d,), float("nan"), dtype=torch.float32, device=dev)
        self.scores = torch.zeros((U, MB), dtype=torch.float32, device=dev)
        self.evict = None
        self.alive = None
        if wl.evict is not None:
            ev = np.full((U, MB), -np.inf, np.float32)
            ev[:, :wl.evict.shape[1]] = wl.evict[:, :MB]
            self.evict = torch.as_tensor(ev, device=dev)
            self.alive = torch.ones((U, MB), dtype=torch.uint8, device=dev)
        if self.ed_dma and self.evict is None:
            raise ValueError("ED-DMA attention needs a workload with eviction logits")
        self.sel = [torch.full((U, MS), -1, dtype=torch.int32, device=dev) for _ in range(2)]
        self.cnt = [torch.zeros(U, dtype=torch.int32, device=dev) for _ in range(2)]
        self.cur = 0                                         # index of the buffer the next select writes
        self.added = torch.full((U, MS), -1, dtype=torch.int32, device=dev)
        self.added_cnt = torch.zeros(U, dtype=torch.int32, device=dev)
        self.removed = torch.full((U, MS), -1, dtype=torch.int32, device=dev)
        self.removed_cnt = torch.zeros(U, dtype=torch.int32, device=dev)
        self.out = torch.zeros((wl.B, wl.Hq, d), dtype=torch.float32, device=dev)
        self.lse = torch.zeros((wl.B, wl.Hq), dtype=torch.float32, device=dev)
        self.workspace = torch.zeros(max(B.workspace_size(self.dims) // 4, 4), dtype=torch.float32, device=dev)

    # -- caller-side KV writes (not a step of the method) --------------------------
    def _write_tokens(self, lo: np.ndarray, hi: np.ndarray) -> None:
        """Copy logical tokens [lo[b], hi[b]) of every unit into their pool pages."""
        wl = self.wl
        if self.kv8:
            self._quant_append(lo, hi)
            return
        for b in range(wl.B):
            if hi[b] <= lo[b]:
                continue
            t = torch.arange(int(lo[b]), int(hi[b]), device=self.device)
            for u in range(b * wl.Hkv, (b + 1) * wl.Hkv):
                phys = self._pt_long[u, t // 16]
                self.k_pool[phys, t % 16] = self._K[u, t]
                self.v_pool[phys, t % 16] = self._V[u, t]

    def _quant_append(self, lo: np.ndarray, hi: np.ndarray) -> None:
        """The same into an 8-bit cache: the sequences' new tokens as packed rows of all KV
        heads, quantised into their pages."""
        wl = self.wl
        n = np.maximum(hi - lo, 0)
        if n.sum() == 0:
            return
        dt = torch.float32 if self.dims.q_dtype == B.BS_FP32 else torch.bfloat16

        def rows(x):
            parts = [x[b * wl.Hkv:(b + 1) * wl.Hkv, int(lo[b]):int(lo[b] + n[b])].transpose(0, 1) for b in range(wl.B)]
            return torch.cat(parts).reshape(int(n.sum()), wl.Hkv * wl.d).to(dt).contiguous()

        i32 = lambda a: torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device=self.device)  # noqa: E731
        B.quant_append(self.dims, self.pools, self.page_table, i32(lo + n), i32(lo), i32(np.cumsum(n) - n),
                       rows(self._K), rows(self._V), wl.Hkv * wl.d, int(n.sum()), int(n.max()), self.status)

    def append(self, step: int) -> None:
        """Write the token appended at ``step`` (position T_prefill + step) into the pools."""
        lo = self.wl.T_prefill.astype(np.int64) + step
        self._write_tokens(lo, lo + 1)

    # -- the five calls ------------------------------------------------------------
    def kv_at(self, seq_lens: torch.Tensor) -> B.KV:
        return B.KV(k_pool=self.kv.k_pool, v_pool=self.kv.v_pool, page_table=self.kv.page_table,
                    seq_lens=seq_lens.data_ptr(), k_scale=self.kv.k_scale, v_scale=self.kv.v_scale)

    def prefill(self, stream=None) -> None:
        """Summaries of every prefilled token."""
        max_new = int(self.wl.T_prefill.max())
        if max_new == 0:       # an empty cache: the first decode step's update covers token 0
            return
        B.build_block_summaries(self.dims, self.kv_at(self.prefill_lens), self.cfg, self.zeros_b, max(max_new, 1),
                                self.summaries, self.status, stream)

    def update_summaries(self, step: int, stream=None) -> None:
        """Recompute the sub-block holding the token appended at ``step``."""
        B.build_block_summaries(self.dims, self.kv_at(self.seq_lens[step]), self.cfg, self.tok_begin[step], 1,
                                self.summaries, self.status, stream)

    def score(self, step: int, group_reduce=B.BS_GROUP_MAX, stream=None) -> None:
        B.score_blocks(self.dims, self.q[step], self.cfg, self.seq_lens[step], self.summaries, group_reduce,
                       self.scores, self.status, stream)

    def select(self, step: int, stream=None) -> None:
        B.select_topk(self.dims, self.cfg, self.seq_lens[step], self.scores, self.evict, self.alive,
                      self.sel[self.cur], self.cnt[self.cur], self.status, stream)

    def attend(self, step: int, stream=None) -> None:
        B.sparse_decode_attn(self.dims, self.q[step], self.kv_at(self.seq_lens[step]), self.cfg, self.sel[self.cur],
                             self.cnt[self.cur], self.out, self.lse, self.workspace, self.status, stream,
                             evict_bias=self.evict if self.ed_dma else None)

    def setdiff(self, stream=None) -> None:
        prev = 1 - self.cur
        B.block_setdiff(self.dims, self.sel[prev], self.cnt[prev], self.sel[self.cur], self.cnt[self.cur],
                        self.added, self.added_cnt, self.removed, self.removed_cnt, self.status, stream)

    def step_io(self, step: int) -> B.StepIO:
        """Buffers of bs_decode_step for ``step`` (current selection buffer ``self.cur``)."""
        prev = 1 - self.cur
        ptr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        return B.StepIO(q=self.q[step].data_ptr(), summaries=self.summaries.data_ptr(),
                        scores=self.scores.data_ptr(), evict_logits=ptr(self.evict), alive=ptr(self.alive),
                        evict_bias=ptr(self.evict) if self.ed_dma else 0,
                        prev_idx=self.sel[prev].data_ptr(), prev_cnt=self.cnt[prev].data_ptr(),
                        cur_idx=self.sel[self.cur].data_ptr(), cur_cnt=self.cnt[self.cur].data_ptr(),
                        added=self.added.data_ptr(), added_cnt=self.added_cnt.data_ptr(),
                        removed=self.removed.data_ptr(), removed_cnt=self.removed_cnt.data_ptr(),
                        out=self.out.data_ptr(), lse=self.lse.data_ptr(), workspace=self.workspace.data_ptr(),
                        workspace_bytes=self.workspace.numel() * 4, dev_status=self.status.data_ptr())

    def fused_step(self, step: int, group_reduce=B.BS_GROUP_MAX, stream=None) -> None:
        """The same decode step through bs_decode_step (two launches), then advance."""
        B.decode_step(self.dims, self.kv_at(self.seq_lens[step]), self.cfg, self.step_io(step), group_reduce,
                      stream)
        self.advance()

    # -- prompts and drafts --------------------------------------------------------
    # What these calls allocate and upload belongs to the stream they run on, workspaces too: calls on
    # two streams share nothing, and memory given back is reused behind the kernels that read it.
    def prefill_attend(self, q: torch.Tensor, lo, hi, stream=None):
        """Tokens [lo[b], hi[b]) of every sequence, already in the cache, attend it: q bf16
        [rows][Hq][d], the sequences' rows one behind another. Streaming heads look at their
        sink and window, the others at everything. Returns out (packed) and lse."""
        self._check_q(q)
        lo, hi = self._per_sequence("lo", lo), self._per_sequence("hi", hi)
        n = hi - lo
        most = max(1, int(n.max()))
        with _on(stream):
            out, lse = self._rows_out(q)
            lens, begin, first = self._i32(hi), self._i32(lo), self._i32(np.cumsum(n) - n)
            ws = self._rows_workspace(B.prefill_workspace_size(self.dims, q.shape[0], most))
            B.prefill_attn(self.dims, q, q.stride(0), q.shape[0], self.kv_at(lens), self.cfg, begin, first, most, out, lse,
                           ws, self.status, stream)
        return out, lse

    def draft_attend(self, q: torch.Tensor, k_new, v_new, n_draft, visible, lens, stream=None):
        """Trees of drafts, n_draft[b] of them for sequence b, attend the blocks of the last selection
        (the one that became the previous) and the drafts that `visible` (int64, a row's mask) names;
        lens[b] tokens are in the cache. k_new, v_new: rows of all KV heads, bf16. Returns out (packed)
        and lse."""
        self._check_q(q)
        rows = q.shape[0]
        self._check_new(k_new, v_new, rows, torch.bfloat16)
        if visible.dtype != torch.int64 or not visible.is_contiguous() or visible.numel() < rows or visible.device.type != self.device.type:
            raise ValueError("visible is int64, contiguous, a mask for every row, on the layer's device")
        n, lens = self._per_sequence("n_draft", n_draft), self._per_sequence("lens", lens)
        most = max(1, int(n.max()))
        last = 1 - self.cur
        with _on(stream):
            out, lse = self._rows_out(q)
            at, first, count = self._i32(lens), self._i32(np.cumsum(n) - n), self._i32(n)
            drafts = B.Drafts(k_new=k_new.data_ptr(), v_new=v_new.data_ptr(), row_stride=k_new.stride(0), n_rows=rows,
                              row_begin=first.data_ptr(), n_draft=count.data_ptr(), visible=visible.data_ptr(), max_draft=most)
            ws = self._rows_workspace(B.tree_workspace_size(self.dims, most))
            B.tree_decode_attn(self.dims, q, q.stride(0), self.kv_at(at), self.cfg, self.sel[last], self.cnt[last], drafts,
                               out, lse, ws, self.status, stream)
        return out, lse

    def commit_drafts(self, k_new, v_new, n_draft, path, lens, stream=None) -> None:
        """The accepted drafts of each sequence, path[b] (node numbers, -1 behind the last), enter the
        cache behind its lens[b] tokens, and the means that the next step scores with follow."""
        n, lens = self._per_sequence("n_draft", n_draft), self._per_sequence("lens", lens)
        path = np.asarray(path, np.int64)
        if path.ndim != 2 or path.shape[0] != self.wl.B:
            raise ValueError("path is [batch][nodes]")
        live = path >= 0
        if (live[:, 1:] & ~live[:, :-1]).any() or (path >= np.maximum(n, 0)[:, None]).any():
            raise ValueError("a path names its own sequence's drafts, and -1 only behind the last")
        rows = int(n.sum())
        if not live.any():
            return
        self._check_new(k_new, v_new, rows, torch.float32 if self.dims.q_dtype == B.BS_FP32 else torch.bfloat16)
        pools = self.pools if self.kv8 else B.Pools(k_pool=self.k_pool.data_ptr(), v_pool=self.v_pool.data_ptr())
        with _on(stream):
            to, begin, first, nodes = self._i32(lens + live.sum(1)), self._i32(lens), self._i32(np.cumsum(n) - n), self._i32(path)
            B.tree_commit(self.dims, pools, self.page_table, to, begin, first, nodes, path.shape[1], k_new, v_new,
                          k_new.stride(0), rows, self.status, stream)
            # (a step renews the sub-block of its own token only)
            B.build_block_summaries(self.dims, self.kv_at(to), self.cfg, begin, path.shape[1], self.summaries, self.status, stream)

    def _i32(self, a) -> torch.Tensor:
        return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device=self.device)

    def _per_sequence(self, name: str, a) -> np.ndarray:
        a = np.asarray(a, np.int64)
        if a.shape != (self.wl.B,):
            raise ValueError(f"{name} has one number a sequence ({self.wl.B}), not shape {a.shape}")
        return a

    def _check_q(self, q: torch.Tensor) -> None:
        wl = self.wl
        if q.dtype != torch.bfloat16 or q.ndim != 3 or tuple(q.shape[1:]) != (wl.Hq, wl.d) or q.stride(2) != 1 or \
                (wl.Hq > 1 and q.stride(1) != wl.d) or q.device.type != self.device.type:
            raise ValueError(f"q is bf16 [rows][{wl.Hq}][{wl.d}] on the layer's device, a row's heads one behind another")

    def _check_new(self, k_new: torch.Tensor, v_new: torch.Tensor, rows: int, dtype) -> None:
        width = self.wl.Hkv * self.wl.d
        for x in (k_new, v_new):
            flat = x.ndim == 2 and x.shape[1] == width and x.stride(1) == 1
            heads = x.ndim == 3 and tuple(x.shape[1:]) == (self.wl.Hkv, self.wl.d) and x.stride(2) == 1 and \
                (self.wl.Hkv == 1 or x.stride(1) == self.wl.d)
            if not (flat or heads) or x.dtype != dtype or x.shape[0] < rows or x.stride(0) != k_new.stride(0) or \
                    x.device.type != self.device.type:
                raise ValueError(f"k_new and v_new are {dtype} rows of {width} elements, {rows} of them at least, of one "
                                 "stride, on the layer's device")

    def _rows_out(self, q: torch.Tensor):
        return (torch.zeros(tuple(q.shape), dtype=q.dtype, device=self.device),
                torch.zeros(tuple(q.shape[:2]), dtype=torch.float32, device=self.device))

    def _rows_workspace(self, size: int) -> torch.Tensor:
        return torch.empty(max(size, 16), dtype=torch.uint8, device=self.device)

    def advance(self) -> None:
        """The current selection becomes the previous one."""
        self.cur = 1 - self.cur

    def step(self, step: int, group_reduce=B.BS_GROUP_MAX, stream=None) -> None:
        """One decode step of this layer (after the caller appended its KV): a1 update,
        a2 scores, a3 selection, a4 attention, a5 set-difference."""
        self.update_summaries(step, stream)
        self.score(step, group_reduce, stream)
        self.select(step, stream)
        self.attend(step, stream)
        self.setdiff(stream)
        self.advance()

    # -- host views ----------------------------------------------------------------
    def set_selection(self, lists: dict, which: int | None = None) -> None:
        """Overwrite selections of some units (unit -> ascending block list)."""
        which = self.cur if which is None else which
        sel = self.sel[which].cpu()
        cnt = self.cnt[which].cpu()
        for u, lst in lists.items():
            sel[u] = -1
            sel[u, :len(lst)] = torch.as_tensor(list(lst), dtype=torch.int32)
            cnt[u] = len(lst)
        self.sel[which].copy_(sel)
        self.cnt[which].copy_(cnt)

    def selection(self, which: int) -> list:
        sel = self.sel[which].cpu().numpy()
        cnt = self.cnt[which].cpu().numpy()
        return [sel[u, :cnt[u]].tolist() for u in range(self.wl.U)]

    def unit_summaries(self, u: int, rows: int) -> np.ndarray:
        off = int(self._cfg_host["sum_off"][u])
        d = self.wl.d
        return self.summaries[off:off + rows * d].view(rows, d).cpu().numpy()

    def read_status(self) -> int:
        return int(self.status.item())
