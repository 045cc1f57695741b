"""Plain float64 forms of the calls on rows of new tokens, and small caches to try them on."""
from __future__ import annotations

import numpy as np
import torch

import _quant as Q
from long_context_serving_gb300 import bsattn as B

HALF_BF16 = 2.0 ** -8          # half a step of bf16, relative
CODE = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
KIND = {"bf16": B.BS_BF16, "fp32": B.BS_FP32, "e4m3": B.BS_E4M3, "int8": B.BS_INT8}


def i32(a, device="cuda"):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device=device)


def bf16(x):
    """x rounded to bf16 as float32."""
    return torch.as_tensor(np.asarray(x, np.float32)).bfloat16().float().numpy()


class Cache:
    """Units of lens[b] tokens over a permuted pool; slots without a token hold NaN (85 in INT8).
    K, V: float64 [unit][T][d], the values the pool stands for."""

    def __init__(self, B_, Hkv, G, d, lens, kind, seed=0, spare=4, max_pages=None, k_std=1.0, **dims):
        rng = np.random.default_rng(seed)
        self.B, self.Hkv, self.G, self.d, self.kind = B_, Hkv, G, d, kind
        self.lens = np.asarray(lens, np.int64)
        U = B_ * Hkv
        pages = np.repeat(-(-self.lens // 16), Hkv)
        P = max_pages or max(1, int(pages.max()))
        n_pages = int(pages.sum()) + spare
        perm = rng.permutation(n_pages)
        table = np.full((U, P), -1, np.int32)
        raw = {}
        at = 0
        for u in range(U):
            table[u, :pages[u]] = perm[at:at + pages[u]]
            at += pages[u]
        self.K, self.V = [], []
        for name, std in (("k", k_std), ("v", 1.0)):
            vals = []
            if kind in ("bf16", "fp32"):
                pool = np.full((n_pages, 16, d), np.nan, np.float32)
                scale = None
            else:
                pool = np.full((n_pages, 16, d), 0x7F if kind == "e4m3" else 85, np.uint8)
                scale = np.full(n_pages, np.nan, np.float32)
            for u in range(U):
                T = int(self.lens[u // Hkv])
                x = (std * rng.standard_normal((T, d))).astype(np.float32)
                if kind == "bf16":
                    x = bf16(x)
                val = x.astype(np.float64)
                for lp in range(pages[u]):
                    rows = x[lp * 16:(lp + 1) * 16]
                    ph = table[u, lp]
                    if scale is None:
                        pool[ph, :len(rows)] = rows
                    else:
                        # (any scale may stand in a cache, not only those an append writes)
                        s = np.float32(np.abs(rows).max() / (400 if kind == "e4m3" else 120))
                        c = Q.round_half_even(rows / s, kind)
                        pool[ph, :len(rows)], scale[ph] = c, s
                        val[lp * 16:(lp + 1) * 16] = Q.decode(c, kind) * np.float64(s)
                vals.append(val)
            raw[name] = (pool, scale)
            setattr(self, name.upper(), vals)
        self.table_np = table
        self.table = i32(table)
        dev = {}
        for name, (pool, scale) in raw.items():
            t = torch.as_tensor(pool).to("cuda")
            dev[name] = t.to(CODE[kind]) if kind in ("bf16", "fp32") else t.view(CODE[kind])
            dev[name + "s"] = None if scale is None else torch.as_tensor(scale).to("cuda")
        self.k, self.v, self.ks, self.vs = dev["k"], dev["v"], dev["ks"], dev["vs"]
        self.seq_lens = i32(self.lens)
        base = dict(batch=B_, n_q_heads=Hkv * G, n_kv_heads=Hkv, head_dim=d, page_size=16, max_pages_per_unit=P,
                    max_blocks_per_unit=max(1, P), max_sel_per_unit=max(1, P), max_subs_per_unit=max(1, 16 * P),
                    max_gather_pages_per_unit=max(1, P), n_pages=n_pages, kv_dtype=KIND[kind], q_dtype=B.BS_BF16)
        base.update(dims)
        self.dims = B.Dims(**base)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def kv(self):
        p = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        return B.KV(k_pool=p(self.k), v_pool=p(self.v), page_table=p(self.table), seq_lens=p(self.seq_lens),
                    k_scale=p(self.ks), v_scale=p(self.vs))

    def pools(self):
        p = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        return B.Pools(k_pool=p(self.k), v_pool=p(self.v), k_scale=p(self.ks), v_scale=p(self.vs))


def attend_row(q, K, V):
    """One row's attention over the keys that it sees, float64: out, lse, and what bounds the error:
    the weighted |V| and the largest sum of |q K| / sqrt(d)."""
    d = q.shape[0]
    if len(K) == 0:
        return np.zeros(d), -np.inf, np.zeros(d), 0.0
    x = K @ q / np.sqrt(d)
    top = x.max()
    w = np.exp(x - top)
    l = w.sum()
    return w @ V / l, top + np.log(l), w @ np.abs(V) / l, float((np.abs(K) @ np.abs(q)).max() / np.sqrt(d))


def check_row(out, lse, want, where):
    """out (bf16) and lse (fp32) of a row against float64. A weight enters as bf16, half a step of
    itself off, so a sum of them by as much of the weighted |V|; the result is rounded once more. A
    logit's fp32 sum of d products, in any order, is off by at most (d + 2) half steps of fp32 of the
    sum of its terms' magnitudes (d <= 128: under 2^-16), a weight by as much relative, lse by as much."""
    o, z, a, x = want
    logit = 2.0 ** -16 * (1 + x)
    tol = HALF_BF16 * (np.abs(o) + a * (1 + HALF_BF16)) + 2 * logit * a + 1e-38
    bad = ~(np.abs(out - o) <= tol)
    assert not bad.any(), (where, out[bad][:4], o[bad][:4], tol[bad][:4])
    if lse is not None:
        assert (np.isneginf(lse) and np.isneginf(z)) or abs(lse - z) <= logit + 2.0 ** -22 * abs(z), (where, lse, z)


def prefill_seen(p, T, streaming, sink, local):
    t = np.arange(T)
    seen = t <= p
    return seen & ((t < sink) | (t > p - local)) if streaming else seen
