"""The operators of prompts and of drafted tokens over the paged cache, as a serving loop
calls them: their cases, their plain forms and their definition in 64 bits.

    rope     queries and keys of new tokens normalised per head (or not) and rotated to their
             positions; K and V of tokens that enter a bf16 or fp32 cache written to their pages
    prefill  attention of new prompt tokens over the cache that holds them: all earlier tokens,
             or (streaming heads) a few first tokens and a window
    tree     attention of a tree of drafted tokens over the selected blocks and their ancestors
    commit   the accepted drafts' K and V, along a path through the tree, appended to the cache

With `own` false, run() computes them with elementary torch operations; with `own` true
it calls the framework.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
E4M3_MAX = 448.0
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "bf16": torch.bfloat16, "fp32": torch.float32}


def _cdiv(a, b):
    return -(-a // b)


# ----------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------
def listed():
    return [
        # One decode token for each of 64 sequences of up to 128K tokens, with norms.
        dict(name="rope_decode", op="rope", B=64, Hq=32, Hkv=8, d=128, old_lo=1000, old_hi=131071, new_lo=1, new_hi=1,
             rot=128, inter=False, norm=True, act="bf16", code="bf16"),
        # Prompts of many lengths behind cached prefixes, rotation alone.
        dict(name="rope_prompt", op="rope", B=6, Hq=28, Hkv=4, d=128, old_lo=0, old_hi=4001, new_lo=1501, new_hi=8192,
             rot=128, inter=False, norm=False, act="bf16", code="bf16"),
        # Three small trees of drafts, which enter no cache yet; half of each head rotated, in pairs of neighbours.
        dict(name="rope_drafts", op="rope", B=3, Hq=8, Hkv=2, d=64, old_lo=90, old_hi=70000, new_lo=5, new_hi=13,
             rot=32, inter=True, norm=True, act="fp32", code="none"),
        # A first prompt of a few words on one small unit: latency alone.
        dict(name="prefill_first", op="prefill", B=1, Hkv=1, G=4, d=64, old_lo=0, old_hi=0, new_lo=17, new_hi=17,
             streaming=0, sink=128, local=2048, code="int8"),
        # The second half of a 16K prompt, half streaming and half retrieval heads.
        dict(name="prefill_chunk", op="prefill", B=1, Hkv=8, G=4, d=128, old_lo=8192, old_hi=8192, new_lo=8192,
             new_hi=8192, streaming=4, sink=128, local=2048, code="bf16"),
        # Ragged chunks over ragged prefixes, groups of seven, windows everywhere, an 8-bit cache.
        dict(name="prefill_ragged_window", op="prefill", B=4, Hkv=4, G=7, d=128, old_lo=0, old_hi=14001, new_lo=333,
             new_hi=2048, streaming=4, sink=128, local=2048, code="e4m3"),
        # One token a sequence that looks at all it has: the batch's dense decode step.
        dict(name="prefill_single", op="prefill", B=32, Hkv=8, G=4, d=128, old_lo=2001, old_hi=16383, new_lo=1, new_hi=1,
             streaming=2, sink=128, local=2048, code="bf16"),
        # Eight drafts of one 32K session.
        dict(name="tree_session", op="tree", B=1, Hkv=8, G=4, d=128, T_lo=32768, T_hi=32768, g="32", frac=0.05,
             streaming=4, n_lo=8, n_hi=8, code="bf16"),
        # Ragged trees over a ragged batch with groups of seven, an 8-bit cache.
        dict(name="tree_ragged", op="tree", B=8, Hkv=4, G=7, d=128, T_lo=32769, T_hi=65533, g="64", frac=0.05,
             streaming=0, n_lo=5, n_hi=31, code="e4m3"),
        # The widest trees over four 128K sequences, a granularity of its own for each head.
        dict(name="tree_wide", op="tree", B=4, Hkv=8, G=4, d=128, T_lo=131069, T_hi=131069, g="16,32,64,128", frac=0.08,
             streaming=2, n_lo=64, n_hi=64, code="bf16"),
        # A batch's accepted drafts enter an 8-bit cache.
        dict(name="commit_batch", op="commit", B=64, Hkv=8, d=128, T_lo=5, T_hi=127, n=24, acc_lo=0, acc_hi=6,
             code="e4m3", act="bf16"),
        # One short answer's two accepted drafts.
        dict(name="commit_one", op="commit", B=1, Hkv=2, d=64, T_lo=31, T_hi=31, n=8, acc_lo=2, acc_hi=2, code="bf16",
             act="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "prefill", "prefill", "tree", "tree", "commit"])
    B, Hkv, d = _log_int(rng, 1, 64), rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128])
    if op == "rope":
        act = rng.choice(["bf16", "bf16", "fp32"])
        code = rng.choice(["bf16", "fp32", "none"])
        G = rng.randint(1, 8)
        new_hi = _log_int(rng, 1, max(1, min(8192, 28000 * 36 * 128 // ((G + 2) * Hkv * d * B))))
        if code == "none":
            new_hi = min(new_hi, 64)
        old_hi = _log_int(rng, 1, 131000)
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, old_lo=rng.randint(0, old_hi), old_hi=old_hi,
                    new_lo=rng.randint(0, new_hi), new_hi=new_hi, rot=rng.choice([d, d, d // 2, 16]),
                    inter=rng.random() < 0.4, norm=rng.random() < 0.5, act=act, code=code)
    if op == "prefill":
        G = rng.randint(1, 8)
        # (rows x keys of the plain form's logits, at most those of the largest listed case)
        most = 8 * 32768 * 16384
        T_hi = _log_int(rng, 1, max(1, min(16384, most // (B * Hkv * G))))
        new_hi = _log_int(rng, 1, max(1, min(T_hi, most // (B * Hkv * G * T_hi))))
        old_hi = T_hi - new_hi
        window = rng.random() < 0.5
        return dict(op=op, B=B, Hkv=Hkv, G=G, d=d, old_lo=rng.randint(0, old_hi), old_hi=old_hi,
                    new_lo=rng.randint(0, new_hi), new_hi=new_hi, streaming=rng.randint(0, Hkv) if window else 0,
                    sink=rng.choice([0, 1, 4, 37, 128]), local=_log_int(rng, 1, 4096),
                    code=rng.choice(["bf16", "bf16", "e4m3", "int8"]))
    if op == "tree":
        most = min(131072, 4 * 8 * 131069 // (B * Hkv))
        T_hi = _log_int(rng, 1, most)
        n_hi = _log_int(rng, 1, 64)
        return dict(op=op, B=B, Hkv=Hkv, G=rng.randint(1, 8), d=d, T_lo=rng.randint(max(1, T_hi // 2), T_hi), T_hi=T_hi,
                    g=rng.choice(["16", "32", "64", "128", "48", "16,32,64,128"]), frac=rng.uniform(0.02, 0.08),
                    streaming=rng.randint(0, 1), n_lo=rng.randint(0, n_hi), n_hi=n_hi,
                    code=rng.choice(["bf16", "bf16", "e4m3", "int8"]))
    n = rng.randint(1, 64)
    hi = rng.randint(1, min(n, 12))
    return dict(op=op, B=B, Hkv=Hkv, d=d, T_lo=rng.randint(0, 40), T_hi=rng.randint(40, 200), n=n,
                acc_lo=rng.randint(0, hi), acc_hi=hi, code=rng.choice(["e4m3", "int8", "bf16", "fp32"]),
                act=rng.choice(["bf16", "fp32"]))


# ----------------------------------------------------------------------------------
# Sizes that a case fixes (the same for every seed)
# ----------------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n numbers spread over [lo, hi], both ends among them where n allows."""
    if n == 1:
        return np.array([hi], np.int64)
    return np.array([lo + (hi - lo) * i // (n - 1) for i in range(n)], np.int64)


def _old_new(case):
    """Tokens of each sequence already there, and new ones."""
    old = _spread(case["old_lo"], case["old_hi"], case["B"])
    return old, _spread(case["new_lo"], case["new_hi"], case["B"])[::-1].copy()


def _streams(case, U):
    return np.array([(u % case["Hkv"]) < case["streaming"] for u in range(U)])


def _tree_sizes(case):
    """Per unit: T, g and selected blocks; per sequence: drafts."""
    B, Hkv = case["B"], case["Hkv"]
    gs = [int(x) for x in case["g"].split(",")]
    T = np.repeat(_spread(case["T_lo"], case["T_hi"], B), Hkv)
    U = B * Hkv
    g = np.array([gs[(u * 5 + u // Hkv) % len(gs)] for u in range(U)], np.int64)
    n_blk = -(-T // g)
    streams = _streams(case, U)
    n_loc = np.where(streams, -(-2048 // g), 1)
    k = np.where(streams, 0, np.maximum(1, (case["frac"] * n_blk).astype(np.int64)))
    cnt = np.minimum(n_blk, 1 + n_loc + k)
    return T, g, cnt, streams, _spread(case["n_lo"], case["n_hi"], B)[::-1].copy()


def _accepted(case):
    return np.roll(_spread(case["acc_lo"], case["acc_hi"], case["B"]), case["B"] // 3)


def _elem(name):
    return 4 if name == "fp32" else 2 if name == "bf16" else 1


def work(case):
    op, d = case["op"], case["d"]
    if op == "rope":
        old, new = _old_new(case)
        rows, a = int(new.sum()), _elem(case["act"])
        heads = case["Hq"] + case["Hkv"]
        nbytes = rows * heads * d * a + rows * case["Hq"] * d * a + rows * 4
        if case["code"] == "none":
            nbytes += rows * case["Hkv"] * d * a
        else:
            nbytes += rows * case["Hkv"] * d * (a + 2 * _elem(case["code"])) + rows * 4
        return {"bytes": nbytes, "flops": rows * heads * (4 * d if case["norm"] else 0) + rows * heads * case["rot"] * 3}
    if op == "prefill":
        old, new = _old_new(case)
        nbytes = flops = 0
        page = 8 if case["code"] in ("e4m3", "int8") else 0
        for h in range(case["Hkv"]):
            for o, n in zip(old.tolist(), new.tolist()):
                if n == 0:
                    continue
                T = o + n
                if h < case["streaming"]:
                    p = np.arange(o, T)
                    first = np.maximum(p + 1 - case["local"], 0)
                    pairs = int((p + 1 - first + np.minimum(first, case["sink"])).sum())
                    keys = T - int(first[0]) + min(int(first[0]), case["sink"])
                else:
                    pairs, keys = n * o + n * (n + 1) // 2, T
                flops += 4 * d * case["G"] * pairs
                nbytes += keys * d * 2 * _elem(case["code"]) + _cdiv(keys, PAGE) * (4 + page)
                nbytes += n * case["G"] * (d * 4 + 4)
        return {"bytes": nbytes, "flops": flops}
    if op == "tree":
        T, g, cnt, _, n = _tree_sizes(case)
        G, Hkv = case["G"], case["Hkv"]
        tok = (cnt - 1) * g + (T - (-(-T // g) - 1) * g)
        nu = np.repeat(n, Hkv)
        has = nu > 0
        page = 8 if case["code"] in ("e4m3", "int8") else 0
        nbytes = int((tok * has).sum()) * d * 2 * _elem(case["code"]) + int((-(-tok // PAGE) * has).sum()) * (4 + page)
        nbytes += int((cnt * has).sum()) * 4 + int(nu.sum()) * d * 2 * 2 + int(nu.sum()) * G * (d * 4 + 4)
        pairs = int((tok * nu).sum()) + int((nu * (nu + 1) // 2).sum())
        return {"bytes": nbytes, "flops": 4 * d * G * pairs}
    acc = _accepted(case)
    T = _spread(case["T_lo"], case["T_hi"], case["B"])
    tok = int(acc.sum()) * case["Hkv"]
    nbytes = 2 * d * tok * (_elem(case["act"]) + _elem(case["code"])) + tok * 4
    if case["code"] in ("e4m3", "int8"):
        nbytes += 4 * d * int((T % PAGE)[acc > 0].sum()) * case["Hkv"]
    return {"bytes": nbytes, "flops": 4 * tok * d}


# ----------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------
def _dev():
    return torch.device("cuda")


def _gen(seed):
    return torch.Generator(device=_dev()).manual_seed(int(seed) * 7919 + 29)


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device=_dev())


def _page_scale(amax, code):
    """The scale of a page whose largest magnitude is amax (fp32): for E4M3 the smallest
    power of two that brings it to 448 or less, for INT8 amax / 127; at least 2^-126, and 0
    for a page of zeros."""
    tiny = torch.tensor(2.0 ** -126, device=amax.device)
    if code == "int8":
        s = torch.maximum(amax / torch.full_like(amax, 127.0), tiny)
    else:
        bits = amax.view(torch.int32)
        e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
        s = ((e.clamp(min=-126) + 127) << 23).view(torch.float32)
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _encode(x, s, code):
    """Codes of the values x (fp32) at scale s."""
    y = torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x))
    if code == "int8":
        return torch.nan_to_num(torch.round(y).clamp(-127, 127), nan=0.0).to(torch.int8)
    return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _random_pool(n_pages, d, code, gen, spread=0.5):
    """A pool of pages of normal values, a spread of its own for each page; its codes and scales."""
    pool = torch.empty((n_pages, PAGE, d), dtype=CODES[code], device=_dev())
    scale = torch.zeros(n_pages, dtype=torch.float32, device=_dev())
    for a in range(0, n_pages, 65536):
        b = min(n_pages, a + 65536)
        x = torch.randn((b - a, PAGE, d), generator=gen, device=_dev())
        x *= torch.exp(spread * torch.randn((b - a, 1, 1), generator=gen, device=_dev()))
        if code in ("bf16", "fp32"):
            pool[a:b] = x.to(CODES[code])
        else:
            s = _page_scale(x.abs().amax((1, 2)), code)
            pool[a:b] = _encode(x, s.view(-1, 1, 1), code)
            scale[a:b] = s
    return pool, scale


def _tables(pages, rng, spare=3, first=None):
    """A page table of `pages` logical pages a unit (from logical page `first` on), scattered over
    a pool; its number of pages."""
    pages = np.asarray(pages, np.int64)
    first = np.zeros_like(pages) if first is None else np.asarray(first, np.int64)
    n = np.maximum(pages - first, 0)
    table = np.full((len(pages), max(1, int(pages.max()))), -1, np.int32)
    perm = rng.permutation(int(n.sum()) + spare)
    at = 0
    for u in range(len(pages)):
        table[u, first[u]:first[u] + n[u]] = perm[at:at + n[u]]
        at += n[u]
    return table, int(n.sum()) + spare


def _tree(n, rng):
    """A random tree of n nodes, root first: depth of each node, ancestors of each (bit j: node j, itself
    among them), parents. Half the time a node extends the newest branch."""
    depth, seen, parent = np.zeros(n, np.int64), [0] * n, np.full(n, -1, np.int64)
    for i in range(n):
        if i > 0:
            parent[i] = i - 1 if rng.random() < 0.5 else int(rng.integers(i))
            depth[i], seen[i] = depth[parent[i]] + 1, seen[parent[i]]
        seen[i] |= 1 << i
    return depth, seen, parent


def prepare(case, seed):
    return {"rope": _prep_rope, "prefill": _prep_prefill, "tree": _prep_tree, "commit": _prep_commit}[case["op"]](
        dict(case), int(seed))


def _prep_rope(case, seed):
    gen, rng = _gen(seed), np.random.default_rng(seed)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    act = CODES[case["act"]]
    old, new = _old_new(case)
    rows = int(new.sum())
    b = np.repeat(np.arange(case["B"]), new)
    i = np.arange(rows) - np.repeat(np.cumsum(new) - new, new)
    pos = old[b] + i
    if case["code"] == "none":       # drafts: as deep in their tree as behind the context
        pos = old[b] + np.concatenate([_tree(int(n), rng)[0] for n in new]) if rows else pos
    # the model's fused projection leaves one row a token: Q heads, K heads, V heads
    qkv = torch.randn((max(rows, 1), (Hq + 2 * Hkv) * d), generator=gen, device=_dev())
    qkv *= torch.exp(0.5 * torch.randn((max(rows, 1), 1), generator=gen, device=_dev()))
    s = dict(case=case, qkv=qkv.to(act), rows=rows, pos=_i32(pos), seq=_i32(b),
             freq=torch.as_tensor(500000.0 ** (-2.0 * np.arange(case["rot"] // 2) / case["rot"]), device=_dev()),
             wq=1 + 0.1 * torch.randn(d, generator=gen, device=_dev()) if case["norm"] else None,
             wk=1 + 0.1 * torch.randn(d, generator=gen, device=_dev()) if case["norm"] else None, eps=1e-6,
             q_out=torch.zeros((rows, Hq, d), dtype=act, device=_dev()), k_out=None,
             status=torch.zeros(1, dtype=torch.int32, device=_dev()))
    if case["code"] == "none":
        s["k_out"] = torch.zeros((rows, Hkv, d), dtype=act, device=_dev())
    else:
        total = np.where(new > 0, old + new, 0)
        table, n_pages = _tables(np.repeat(-(-total // PAGE), Hkv), rng, first=np.repeat(old // PAGE, Hkv))
        s["table"], s["n_pages"] = _i32(table), n_pages
        s["k"] = torch.zeros((n_pages, PAGE, d), dtype=CODES[case["code"]], device=_dev())
        s["v"] = torch.zeros_like(s["k"])
    return s


def _prep_prefill(case, seed):
    gen, rng = _gen(seed), np.random.default_rng(seed)
    B, Hkv, G, d = case["B"], case["Hkv"], case["G"], case["d"]
    old, new = _old_new(case)
    U, rows = B * Hkv, int(new.sum())
    table, n_pages = _tables(np.repeat(-(-(old + new) // PAGE), Hkv), rng)
    k, ks = _random_pool(n_pages, d, case["code"], gen, 0.2)
    v, vs = _random_pool(n_pages, d, case["code"], gen)
    streams = _streams(case, U)
    return dict(case=case, k=k, v=v, ks=ks, vs=vs, table=_i32(table), old=_i32(old), lens=_i32(old + new),
                row0=_i32(np.cumsum(new) - new), rows=rows, max_new=int(new.max()), max_len=int((old + new).max()),
                cls=_i32(np.where(streams, 0, 1)), sink=_i32(np.full(U, case["sink"])),
                local=_i32(np.full(U, case["local"])),
                q=(1.5 * torch.randn((max(rows, 1), Hkv * G * d), generator=gen, device=_dev())).bfloat16(),
                out=torch.zeros((rows, Hkv * G, d), dtype=torch.bfloat16, device=_dev()),
                lse=torch.zeros((rows, Hkv * G), dtype=torch.float32, device=_dev()),
                status=torch.zeros(1, dtype=torch.int32, device=_dev()))


def _prep_tree(case, seed):
    gen, rng = _gen(seed), np.random.default_rng(seed)
    B, Hkv, G, d = case["B"], case["Hkv"], case["G"], case["d"]
    T, g, cnt, streams, n = _tree_sizes(case)
    U, rows = B * Hkv, int(n.sum())
    table, n_pages = _tables(-(-T // PAGE), rng)
    n_blk = -(-T // g)
    sel = np.full((U, int(cnt.max())), -1, np.int32)
    for u in range(U):
        c, nb = int(cnt[u]), int(n_blk[u])
        loc = min(nb, int(-(-2048 // g[u]))) if streams[u] else 1
        forced = np.union1d([0], np.arange(nb - loc, nb))
        rest = np.setdiff1d(np.arange(nb), forced)
        pick = rng.choice(rest, size=max(0, c - len(forced)), replace=False)
        mine = np.sort(np.concatenate([forced, pick]))
        sel[u, :c] = np.concatenate([mine[:c - 1], mine[-1:]])
    k, ks = _random_pool(n_pages, d, case["code"], gen, 0.2)
    v, vs = _random_pool(n_pages, d, case["code"], gen)
    seen = [_tree(int(x), rng)[1] for x in n]
    flat = np.array([m for s in seen for m in s] or [0], np.uint64)
    return dict(case=case, k=k, v=v, ks=ks, vs=vs, table=_i32(table), lens=_i32(T.reshape(B, Hkv)[:, 0]), g=_i32(g),
                sel=_i32(sel), cnt=_i32(cnt), max_blocks=int(n_blk.max()), max_gather=int((cnt * g // PAGE).max()),
                n=_i32(n), row0=_i32(np.cumsum(n) - n), rows=rows, max_draft=max(1, int(n.max())),
                seen=torch.as_tensor(flat.view(np.int64), device=_dev()),
                q=(1.5 * torch.randn((max(rows, 1), Hkv * G * d), generator=gen, device=_dev())).bfloat16(),
                kv_new=torch.randn((max(rows, 1), 2 * Hkv * d), generator=gen, device=_dev()).bfloat16(),
                out=torch.zeros((rows, Hkv * G, d), dtype=torch.bfloat16, device=_dev()),
                lse=torch.zeros((rows, Hkv * G), dtype=torch.float32, device=_dev()),
                status=torch.zeros(1, dtype=torch.int32, device=_dev()))


def _prep_commit(case, seed):
    gen, rng = _gen(seed), np.random.default_rng(seed)
    B, Hkv, d, n = case["B"], case["Hkv"], case["d"], case["n"]
    T, acc = _spread(case["T_lo"], case["T_hi"], B), _accepted(case)
    table, n_pages = _tables(np.repeat(-(-(T + acc) // PAGE), Hkv), rng)
    k, ks = _random_pool(n_pages, d, case["code"], gen)
    v, vs = _random_pool(n_pages, d, case["code"], gen)
    kv_new = torch.randn((B * n, 2 * Hkv * d), generator=gen, device=_dev())
    kv_new *= torch.exp(torch.randn((B * n, 1), generator=gen, device=_dev()))
    # the accepted path: nodes of rising index, as a walk down the tree visits them
    path = np.full((B, max(1, case["acc_hi"])), -1, np.int32)
    for b in range(B):
        path[b, :acc[b]] = np.sort(rng.choice(n, size=int(acc[b]), replace=False))
    return dict(case=case, k=k, v=v, ks=ks, vs=vs, table=_i32(table), old=_i32(T), lens=_i32(T + acc),
                row0=_i32(np.arange(B) * n), path=_i32(path), total=int(acc.sum()), kv_new=kv_new.to(CODES[case["act"]]),
                status=torch.zeros(1, dtype=torch.int32, device=_dev()))


# ----------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "prefill": _own_prefill, "tree": _own_tree, "commit": _own_commit}[op](state)
    return {"rope": _plain_rope, "prefill": _plain_prefill, "tree": _plain_tree, "commit": _plain_commit}[op](state)


def _rope_out(s):
    return {"q": s["q_out"], "k": s["k_out"]} if s["case"]["code"] == "none" else {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _pools_out(s):
    out = {"k": s["k"], "v": s["v"]}
    if s["case"]["code"] in ("e4m3", "int8"):
        out.update(k_scale=s["ks"], v_scale=s["vs"])
    return out


# -- plain forms -------------------------------------------------------------------
def _plain_rotate(x, w, s):
    """x [rows][heads][d] normalised with the weights w (None: not) and rotated, in fp32."""
    c = s["case"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
    angle = s["pos"].double().view(-1, 1, 1) * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    r = c["rot"]
    if c["inter"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_rope(s):
    c = s["case"]
    Hq, Hkv, d, R = c["Hq"], c["Hkv"], c["d"], s["rows"]
    x = s["qkv"][:R].view(R, Hq + 2 * Hkv, d)
    s["q_out"].copy_(_plain_rotate(x[:, :Hq], s["wq"], s))
    k = _plain_rotate(x[:, Hq:Hq + Hkv], s["wk"], s)
    if c["code"] == "none":
        s["k_out"].copy_(k)
    else:
        unit = s["seq"].long().view(-1, 1) * Hkv + torch.arange(Hkv, device=_dev())
        at = s["pos"].long().view(-1, 1)
        page = s["table"].long()[unit, at // PAGE]
        s["k"][page, at % PAGE] = k.to(s["k"].dtype)
        s["v"][page, at % PAGE] = x[:, Hq + Hkv:].to(s["v"].dtype)
    return _rope_out(s)


def _rows_of(n, R):
    """Sequence and index there of each of R packed rows (n: rows of each sequence)."""
    b = torch.repeat_interleave(torch.arange(n.numel(), device=_dev()), n, output_size=R)
    return b, torch.arange(R, device=_dev()) - (torch.cumsum(n, 0) - n)[b]


def _plain_softmax(x, V, s, b, i):
    """out, lse of the logits x [units][new][G][keys] over the values V; rows (b, i) kept."""
    c = s["case"]
    B, Hkv, G, d = c["B"], c["Hkv"], c["G"], c["d"]
    U, n = x.shape[0], x.shape[1]
    m = x.amax(3, keepdim=True)
    base = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(base).exp_()
    l = p.sum(3, keepdim=True)
    o = torch.matmul(p.view(U, n * G, -1), V).view(U, n, G, d) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (base + torch.log(l)).view(B, Hkv, n, G)
    s["out"].copy_(o.view(B, Hkv, n, G, d)[b, :, i].reshape(-1, Hkv * G, d))
    s["lse"].copy_(lse[b, :, i].reshape(-1, Hkv * G))
    return {"out": s["out"], "lse": s["lse"]}


def _padded(x, s, n):
    """Rows of the packed x [rows][...] as [B][longest][...] (rows past a sequence's own: any)."""
    at = s["row0"].long().view(-1, 1) + torch.arange(n, device=_dev())
    return x[at.clamp(max=x.shape[0] - 1)]


def _values(pool, scale, phys, code):
    x = pool[phys].float()
    return x * scale[phys].view(*phys.shape, 1, 1) if code in ("e4m3", "int8") else x


def _plain_prefill(s):
    c = s["case"]
    B, Hkv, G, d = c["B"], c["Hkv"], c["G"], c["d"]
    U, n, P = B * Hkv, s["max_new"], _cdiv(s["max_len"], PAGE)
    if s["rows"] == 0:
        return {"out": s["out"], "lse": s["lse"]}
    phys = s["table"][:, :P].long().clamp(min=0)
    K = _values(s["k"], s["ks"], phys, c["code"]).view(U, P * PAGE, d)
    V = _values(s["v"], s["vs"], phys, c["code"]).view(U, P * PAGE, d)
    q = _padded(s["q"], s, n).float().view(B, n, Hkv, G, d).transpose(1, 2).reshape(U, n * G, d)
    x = torch.matmul(q, K.transpose(1, 2)).mul_(1.0 / math.sqrt(d)).view(U, n, G, -1)
    t = torch.arange(P * PAGE, device=_dev()).view(1, 1, -1)
    p = (s["old"].long().view(B, 1, 1) + torch.arange(n, device=_dev()).view(1, -1, 1)).repeat_interleave(Hkv, 0)
    near = (t < s["sink"].long().view(U, 1, 1)) | (t > p - s["local"].long().view(U, 1, 1))
    seen = (t <= p) & (near | (s["cls"].view(U, 1, 1) != 0))
    x.masked_fill_(~seen.unsqueeze(2), -math.inf)
    b, i = _rows_of(s["lens"].long() - s["old"].long(), s["rows"])
    return _plain_softmax(x, V, s, b, i)


def _plain_tree(s):
    c = s["case"]
    B, Hkv, G, d = c["B"], c["Hkv"], c["G"], c["d"]
    U, P, n = s["table"].shape[0], s["table"].shape[1], s["max_draft"]
    if s["rows"] == 0:
        return {"out": s["out"], "lse": s["lse"]}
    ppb = (s["g"].long() // PAGE).view(U, 1)
    T = s["lens"].long().repeat_interleave(Hkv).view(U, 1)
    at = torch.arange(s["max_gather"], device=_dev()).view(1, -1)
    blk = torch.gather(s["sel"].long(), 1, (at // ppb).clamp(max=s["sel"].shape[1] - 1))
    page = blk * ppb + at % ppb
    used = (at // ppb < s["cnt"].long().view(U, 1)) & (page * PAGE < T)
    phys = torch.gather(s["table"].long(), 1, page.clamp(0, P - 1))
    phys = torch.where(used, phys, torch.zeros_like(phys))
    tok = page.unsqueeze(2) * PAGE + torch.arange(PAGE, device=_dev())
    seen = (used.unsqueeze(2) & (tok < T.unsqueeze(2))).view(U, 1, 1, -1).expand(U, n, 1, -1)
    K = _values(s["k"], s["ks"], phys, c["code"]).view(U, -1, d)
    V = _values(s["v"], s["vs"], phys, c["code"]).view(U, -1, d)
    # the drafts behind the cache, each seen by the rows whose mask has its bit
    new = _padded(s["kv_new"], s, n).float().view(B, n, 2, Hkv, d).permute(2, 0, 3, 1, 4).reshape(2, U, n, d)
    j = torch.arange(n, device=_dev())
    bits = (_padded(s["seen"], s, n).view(B, n, 1) >> j) & 1
    bits = ((bits == 1) & (j < s["n"].long().view(B, 1, 1))).repeat_interleave(Hkv, 0).unsqueeze(2)
    seen = torch.cat([seen, bits], 3)
    q = _padded(s["q"], s, n).float().view(B, n, Hkv, G, d).transpose(1, 2).reshape(U, n * G, d)
    x = torch.matmul(q, torch.cat([K, new[0]], 1).transpose(1, 2)).mul_(1.0 / math.sqrt(d)).view(U, n, G, -1)
    x.masked_fill_(~seen, -math.inf)
    b, i = _rows_of(s["n"].long(), s["rows"])
    return _plain_softmax(x, torch.cat([V, new[1]], 1), s, b, i)


def _plain_commit(s):
    c = s["case"]
    B, Hkv, d, code, R = c["B"], c["Hkv"], c["d"], c["code"], s["total"]
    if R == 0:
        return _pools_out(s)
    old = s["old"].long()
    acc = s["lens"].long() - old
    b, i = _rows_of(acc, R)
    row = s["row0"].long()[b] + s["path"].long()[b, i]
    t = old[b] + i
    u = b.view(-1, 1) * Hkv + torch.arange(Hkv, device=_dev())
    phys = s["table"].long()[u, (t // PAGE).view(-1, 1)]                       # [rows, Hkv]
    slot = (t % PAGE).view(-1, 1).expand(-1, Hkv)
    new = s["kv_new"][row].float().view(R, 2, Hkv, d)
    if code in ("bf16", "fp32"):
        s["k"][phys, slot] = new[:, 0].to(s["k"].dtype)
        s["v"][phys, slot] = new[:, 1].to(s["v"].dtype)
        return _pools_out(s)
    # pages that held tokens before: the page of position old, where it ends inside a page
    first = (old // PAGE).clamp(max=s["table"].shape[1] - 1)
    keeps = ((old % PAGE > 0) & (acc > 0)).repeat_interleave(Hkv)
    head_page = s["table"].long()[torch.arange(B * Hkv, device=_dev()), first.repeat_interleave(Hkv)][keeps]
    n_old = (old % PAGE).repeat_interleave(Hkv)[keeps]
    for pool, scale, x in ((s["k"], s["ks"], new[:, 0]), (s["v"], s["vs"], new[:, 1])):
        amax = torch.zeros(scale.shape[0], device=_dev())
        amax.scatter_reduce_(0, phys.reshape(-1), x.abs().amax(2).reshape(-1), "amax")
        had = torch.zeros_like(scale)
        had[head_page] = scale[head_page]
        to = torch.maximum(had, _page_scale(amax, code))
        # codes already there, at the page's new scale
        at, was = to[head_page], scale[head_page]
        again = _encode(pool[head_page].float() * was.view(-1, 1, 1), at.view(-1, 1, 1), code)
        keep = (torch.arange(PAGE, device=_dev()).view(1, -1) < n_old.view(-1, 1)) & (at > was).view(-1, 1)
        raw = pool.view(torch.uint8)
        raw[head_page] = torch.where(keep.unsqueeze(2), again.view(torch.uint8), raw[head_page])
        raw[phys, slot] = _encode(x, to[phys].unsqueeze(2), code).view(torch.uint8)
        scale[phys.reshape(-1)] = to[phys.reshape(-1)]
    return _pools_out(s)


# -- the framework's calls -----------------------------------------------------------
def _handle(s):
    """What a program keeps between calls: the dims, the pointer structs, the workspaces."""
    h = s.get("handle")
    if h is not None:
        return h
    from long_context_serving_gb300 import bsattn as A

    c = s["case"]
    types = {"e4m3": A.BS_E4M3, "int8": A.BS_INT8, "bf16": A.BS_BF16, "fp32": A.BS_FP32}
    Hkv, d = c["Hkv"], c["d"]
    Hq = c.get("Hq", Hkv * c.get("G", 1))
    dims = A.Dims(batch=c["B"], n_q_heads=Hq, n_kv_heads=Hkv, head_dim=d, page_size=PAGE,
                  max_pages_per_unit=s["table"].shape[1] if "table" in s else 1, max_blocks_per_unit=s.get("max_blocks", 1),
                  max_sel_per_unit=s["sel"].shape[1] if "sel" in s else 1, max_subs_per_unit=1,
                  max_gather_pages_per_unit=s.get("max_gather", 1), n_pages=s["k"].shape[0] if "k" in s else 1,
                  kv_dtype=types.get(c["code"], A.BS_BF16), q_dtype=types[c.get("act", "bf16")])
    h = dict(A=A, dims=dims)
    p = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    eight = c["code"] in ("e4m3", "int8")
    scales = dict(k_scale=p(s["ks"]) if eight else 0, v_scale=p(s["vs"]) if eight else 0)
    if c["op"] == "rope":
        h["rope"] = A.Rope(inv_freq=p(s["freq"]), rot_dim=c["rot"], interleaved=int(c["inter"]), magnitude=1.0,
                           q_weight=p(s["wq"]), k_weight=p(s["wk"]), eps=s["eps"])
        x = s["qkv"]
        h["qkv"] = x[:, :Hq * d], x[:, Hq * d:(Hq + Hkv) * d], x[:, (Hq + Hkv) * d:]
        h["pools"] = A.Pools(k_pool=p(s["k"]), v_pool=p(s["v"])) if "k" in s else None
    elif c["op"] == "commit":
        h["pools"] = A.Pools(k_pool=p(s["k"]), v_pool=p(s["v"]), **scales)
        h["new"] = s["kv_new"][:, :Hkv * d], s["kv_new"][:, Hkv * d:]
    else:
        h["kv"] = A.KV(k_pool=p(s["k"]), v_pool=p(s["v"]), page_table=p(s["table"]), seq_lens=p(s["lens"]), **scales)
        if c["op"] == "prefill":
            h["cfg"] = A.HeadCfg(cls=p(s["cls"]), sink_tokens=p(s["sink"]), local_tokens=p(s["local"]))
            size = A.prefill_workspace_size(dims, s["rows"], s["max_new"])
        else:
            h["cfg"] = A.HeadCfg(block_tokens=p(s["g"]))
            h["drafts"] = A.Drafts(k_new=p(s["kv_new"]), v_new=p(s["kv_new"][:, Hkv * d:]),
                                   row_stride=s["kv_new"].stride(0), n_rows=s["rows"], row_begin=p(s["row0"]),
                                   n_draft=p(s["n"]), visible=p(s["seen"]), max_draft=s["max_draft"])
            size = A.tree_workspace_size(dims, s["max_draft"])
        h["ws"] = torch.zeros(max(size, 16) // 4, dtype=torch.int32, device=_dev())
    s["handle"] = h
    return h


def _own_rope(s):
    h = _handle(s)
    q, k, v = h["qkv"]
    if s["rows"] > 0:
        h["A"].rope_append(h["dims"], h["rope"], q, k, v, s["qkv"].stride(0), s["rows"], s["pos"], s["seq"], h["pools"],
                           s.get("table"), s["q_out"], s["k_out"], s["status"])
    return _rope_out(s)


def _own_prefill(s):
    h = _handle(s)
    if s["rows"] > 0:
        h["A"].prefill_attn(h["dims"], s["q"], s["q"].stride(0), s["rows"], h["kv"], h["cfg"], s["old"], s["row0"],
                            s["max_new"], s["out"], s["lse"], h["ws"], s["status"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_tree(s):
    h = _handle(s)
    if s["rows"] > 0:
        h["A"].tree_decode_attn(h["dims"], s["q"], s["q"].stride(0), h["kv"], h["cfg"], s["sel"], s["cnt"], h["drafts"],
                                s["out"], s["lse"], h["ws"], s["status"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_commit(s):
    h = _handle(s)
    k, v = h["new"]
    if s["total"] > 0:
        h["A"].tree_commit(h["dims"], h["pools"], s["table"], s["lens"], s["old"], s["row0"], s["path"],
                           s["path"].shape[1], k, v, s["kv_new"].stride(0), s["kv_new"].shape[0], s["status"])
    return _pools_out(s)


# ----------------------------------------------------------------------------------
# The definition in 64 bits
# ----------------------------------------------------------------------------------
def exact(case, seed):
    """Rotation and attention in float64, unit by unit; commits value by value, but for INT8 codes,
    which are of quotients rounded to fp32 (E4M3 scales are powers of two): no such value."""
    if case["op"] == "rope":
        return _exact_rope(prepare(case, seed))
    if case["op"] == "prefill":
        return _exact_prefill(prepare(case, seed))
    if case["op"] == "tree":
        return _exact_tree(prepare(case, seed))
    return _exact_commit(prepare(case, seed)) if case["code"] != "int8" else None


def _exact_rope(s):
    c = s["case"]
    Hq, Hkv, d, R, r = c["Hq"], c["Hkv"], c["d"], s["rows"], c["rot"]
    x = s["qkv"][:R].double().view(R, Hq + 2 * Hkv, d).clone()
    for lo, hi, w in ((0, Hq, s["wq"]), (Hq, Hq + Hkv, s["wk"])):
        if w is not None:
            x[:, lo:hi] /= torch.sqrt(x[:, lo:hi].square().sum(-1, keepdim=True) / d + s["eps"])
            x[:, lo:hi] *= w.double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=_dev()), s["pos"].double().view(-1, 1) * s["freq"])
    first = torch.arange(0, r, 2, device=_dev()) if c["inter"] else torch.arange(r // 2, device=_dev())
    second = first + (1 if c["inter"] else r // 2)
    z = torch.complex(x[:, :Hq + Hkv, first], x[:, :Hq + Hkv, second]) * turn.unsqueeze(1)
    x[:, :Hq + Hkv, first], x[:, :Hq + Hkv, second] = z.real, z.imag
    if c["code"] == "none":
        return {"q": x[:, :Hq], "k": x[:, Hq:Hq + Hkv]}
    k, v = s["k"].double(), s["v"].double()
    table = s["table"].long()
    for h in range(Hkv):
        page = table[s["seq"].long() * Hkv + h, s["pos"].long() // PAGE]
        k[page, s["pos"].long() % PAGE] = x[:, Hq + h]
        v[page, s["pos"].long() % PAGE] = x[:, Hq + Hkv + h]
    return {"q": x[:, :Hq], "k": k, "v": v}


def _unit_kv(s, u, tokens):
    """K and V of these tokens of a unit in float64."""
    page, at = s["table"].long()[u, tokens // PAGE], tokens % PAGE
    got = []
    for pool, scale in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        x = (pool.view(torch.uint8)[page, at].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[page, at]).double()
        got.append(x * scale.double()[page, None] if s["case"]["code"] in ("e4m3", "int8") else x)
    return got


def _exact_rows(q, K, V, seen):
    """out, lse of queries q [rows][G][d] over keys of which row i sees seen[i]."""
    x = torch.einsum("igd,td->igt", q, K) / math.sqrt(K.shape[1])
    x = torch.where(seen[:, None, :], x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, 2)
    return torch.einsum("igt,td->igd", torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None]), V), lse


def _exact_prefill(s):
    c = s["case"]
    Hkv, G, d = c["Hkv"], c["G"], c["d"]
    out, lse = torch.zeros_like(s["out"], dtype=torch.float64), torch.zeros_like(s["lse"], dtype=torch.float64)
    old, new = _old_new(c)
    at = 0
    for b in range(c["B"]):
        o, n = int(old[b]), int(new[b])
        q = s["q"][at:at + n].double().view(n, Hkv, G, d)
        t = torch.arange(o + n, device=_dev())
        for h in range(Hkv):
            K, V = _unit_kv(s, b * Hkv + h, t)
            for a in range(0, n, 1024):
                p = torch.arange(o + a, o + min(n, a + 1024), device=_dev()).view(-1, 1)
                seen = t <= p
                if h < c["streaming"]:
                    seen &= (t < c["sink"]) | (p - t < c["local"])
                end = int(p[-1, 0]) + 1
                y, z = _exact_rows(q[a:a + 1024, h], K[:end], V[:end], seen[:, :end])
                out[at + a:at + a + len(p), h * G:(h + 1) * G], lse[at + a:at + a + len(p), h * G:(h + 1) * G] = y, z
        at += n
    return {"out": out, "lse": lse}


def _exact_tree(s):
    c = s["case"]
    Hkv, G, d = c["Hkv"], c["G"], c["d"]
    T, g, cnt, _, n = _tree_sizes(c)
    sel = s["sel"].cpu().numpy()
    mask = s["seen"].cpu().numpy().view(np.uint64)
    out, lse = torch.zeros_like(s["out"], dtype=torch.float64), torch.zeros_like(s["lse"], dtype=torch.float64)
    at = 0
    for b in range(c["B"]):
        nb = int(n[b])
        new = s["kv_new"][at:at + nb].double().view(nb, 2, Hkv, d)
        q = s["q"][at:at + nb].double().view(nb, Hkv, G, d)
        bits = np.array([[(int(mask[at + i]) >> j) & 1 for j in range(nb)] for i in range(nb)], bool).reshape(nb, nb)
        for h in range(Hkv if nb else 0):
            u = b * Hkv + h
            t = np.concatenate([np.arange(k * g[u], min((k + 1) * g[u], T[u])) for k in sel[u, :cnt[u]]])
            K, V = _unit_kv(s, u, torch.as_tensor(t, device=_dev()))
            seen = torch.as_tensor(np.concatenate([np.ones((nb, len(t)), bool), bits], 1), device=_dev())
            y, z = _exact_rows(q[:, h], torch.cat([K, new[:, 0, h]]), torch.cat([V, new[:, 1, h]]), seen)
            out[at:at + nb, h * G:(h + 1) * G], lse[at:at + nb, h * G:(h + 1) * G] = y, z
        at += nb
    return {"out": out, "lse": lse}


def _nearest_e4m3(y):
    """y rounded to the nearest E4M3 value, ties to the even mantissa (float64)."""
    a = np.minimum(np.abs(y), E4M3_MAX)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6.0)
    step = 2.0 ** (e - 3)
    return np.copysign(np.minimum(np.round(a / step) * step, E4M3_MAX), y)


def _exact_commit(s):
    c = s["case"]
    Hkv, d = c["Hkv"], c["d"]
    old, lens, row0, path, table = (s[n].cpu().numpy().astype(np.int64) for n in ("old", "lens", "row0", "path", "table"))
    new = s["kv_new"].double().cpu().numpy()
    done = {}
    for name, sname, side in (("k", "ks", 0), ("v", "vs", 1)):
        val = s[name].float().cpu().numpy().astype(np.float64)
        scl = s[sname].cpu().numpy().astype(np.float64)
        for b in range(c["B"]):
            for lp in range(old[b] // PAGE, -(-lens[b] // PAGE) if lens[b] > old[b] else 0):
                t0, t1 = max(lp * PAGE, old[b]), min((lp + 1) * PAGE, lens[b])
                rows = new[row0[b] + path[b, t0 - old[b]:t1 - old[b]], side * Hkv * d:(side + 1) * Hkv * d]
                for h in range(Hkv):
                    ph, kept = table[b * Hkv + h, lp], t0 - lp * PAGE
                    x = rows[:, h * d:(h + 1) * d]
                    if c["code"] != "e4m3":
                        val[ph, kept:kept + len(x)] = x
                        continue
                    big = np.abs(x).max()
                    need = 2.0 ** max(math.ceil(math.log2(big / E4M3_MAX)), -126) if big > 0 else 0.0
                    to = max(scl[ph], need) if kept else need
                    if kept and to > scl[ph]:
                        val[ph, :kept] = _nearest_e4m3(val[ph, :kept] * scl[ph] / to)
                    val[ph, kept:kept + len(x)] = _nearest_e4m3(x / to) if to > 0 else 0.0
                    scl[ph] = to
        done[name] = torch.as_tensor(val)
        if c["code"] == "e4m3":
            done[name + "_scale"] = torch.as_tensor(scl)
    return done
