"""The operators of the 8-bit paged KV cache, as a serving loop calls them: their cases,
their plain forms and their definition in 64 bits.

    attend    block-sparse decode attention over a cache of E4M3 or INT8 codes with one
              fp32 scale per page (16 tokens of one KV head) for K and one for V
    append    new tokens' K and V quantised into their pages (a page's scale grows with its
              largest value; codes already in the page are rounded again when it does)
    fork      beams take over their parents' pages: the children's old pages are freed, full
              pages are shared, partial last pages are copied
    turnover  finished sequences give their pages back, new ones reserve theirs
    compact   live pages move into the holes below the live count

With `own` false, run() computes them with elementary torch operations; with `own` true
it calls the framework.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
E4M3_MAX = 448.0
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "bf16": torch.bfloat16}
ACTS = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _cdiv(a, b):
    return -(-a // b)


# ----------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------
def listed():
    return [
        # A first token answered on one small unit: latency alone.
        dict(name="attend_first_token", op="attend", B=1, Hkv=1, G=4, d=64, T_lo=1, T_hi=1, g="64", frac=0.05,
             streaming=0, code="int8", act="fp32", bias=False),
        # One 32K sequence, half streaming and half retrieval heads: an interactive session.
        dict(name="attend_32k", op="attend", B=1, Hkv=8, G=4, d=128, T_lo=32768, T_hi=32768, g="32", frac=0.05,
             streaming=4, code="e4m3", act="bf16", bias=False),
        # Four 128K sequences, a granularity of its own for each head: the long-context batch.
        dict(name="attend_128k_mixed", op="attend", B=4, Hkv=8, G=4, d=128, T_lo=131069, T_hi=131069, g="16,32,64,128",
             frac=0.08, streaming=2, code="e4m3", act="bf16", bias=False),
        # A ragged batch with groups of seven and block logits (the eviction head's) in INT8.
        dict(name="attend_ragged_bias", op="attend", B=8, Hkv=4, G=7, d=128, T_lo=32769, T_hi=65533, g="64", frac=0.05,
             streaming=0, code="int8", act="bf16", bias=True),
        # One decode token for each of 64 sequences.
        dict(name="append_decode", op="append", B=64, Hkv=8, d=128, old_lo=5, old_hi=127, new_lo=1, new_hi=1,
             code="e4m3", act="bf16"),
        # Prompts of many lengths written at once, behind prefixes that end inside a page.
        dict(name="append_prefill", op="append", B=6, Hkv=8, d=128, old_lo=0, old_hi=100, new_lo=1501, new_hi=16384,
             code="int8", act="bf16"),
        # Four beams of one short answer.
        dict(name="fork_beams_short", op="fork", B=4, Hkv=2, d=64, T_lo=17, T_hi=90, parents=1, code="bf16"),
        # Sixteen of 24 sequences are beams over 8 parents of about 8K tokens.
        dict(name="fork_beams", op="fork", B=24, Hkv=8, d=128, T_lo=7000, T_hi=8200, parents=8, code="e4m3"),
        # One short sequence leaves a small cache and another enters.
        dict(name="turnover_one", op="turnover", B=4, Hkv=2, T_lo=30, T_hi=200, leave=1, slack=1.5),
        # A third of 64 sequences leaves, as many prompts enter.
        dict(name="turnover_batch", op="turnover", B=64, Hkv=8, T_lo=2000, T_hi=16384, leave=21, slack=1.3),
        # A small cache after a few departures.
        dict(name="compact_small", op="compact", B=3, Hkv=2, d=64, T_lo=50, T_hi=300, live=0.6, code="int8"),
        # A large cache with two fifths of its pages free, scattered.
        dict(name="compact_large", op="compact", B=16, Hkv=8, d=128, T_lo=6000, T_hi=8192, live=0.6, code="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "append", "fork", "turnover", "compact"])
    if op == "attend":
        B, Hkv = _log_int(rng, 1, 64), rng.choice([1, 2, 4, 5, 8])
        d = rng.choice([64, 128])
        most = min(131072, 4 * 8 * 131069 // (B * Hkv))
        hi = _log_int(rng, 1, most)
        lo = rng.randint(max(1, hi // 2), hi)
        return dict(op=op, B=B, Hkv=Hkv, G=rng.randint(1, 8), d=d, T_lo=lo, T_hi=hi,
                    g=rng.choice(["16", "32", "64", "128", "48", "16,32,64,128"]), frac=rng.uniform(0.02, 0.08),
                    streaming=rng.randint(0, 1), code=rng.choice(["e4m3", "int8"]), act=rng.choice(["bf16", "fp32"]),
                    bias=rng.random() < 0.4)
    if op == "append":
        B, Hkv = _log_int(rng, 1, 64), rng.choice([1, 2, 4, 5, 8])
        hi = _log_int(rng, 1, max(1, min(16384, 6 * 8 * 8000 // (B * Hkv))))
        return dict(op=op, B=B, Hkv=Hkv, d=rng.choice([64, 128]), old_lo=0, old_hi=rng.randint(0, 200),
                    new_lo=rng.randint(0, hi), new_hi=hi, code=rng.choice(["e4m3", "int8"]),
                    act=rng.choice(["bf16", "fp32"]))
    B, Hkv = rng.randint(2, 24), rng.choice([1, 2, 4, 5, 8])
    hi = _log_int(rng, 2, 8192)
    lo = rng.randint(1, hi)
    if op == "fork":
        return dict(op=op, B=B, Hkv=Hkv, d=rng.choice([64, 128]), T_lo=lo, T_hi=hi, parents=rng.randint(1, B - 1),
                    code=rng.choice(["e4m3", "int8", "bf16"]))
    if op == "turnover":
        hi = _log_int(rng, 256, 16384)
        return dict(op=op, B=B, Hkv=Hkv, T_lo=rng.randint(hi // 4, hi), T_hi=hi, leave=rng.randint(1, B - 1),
                    slack=rng.uniform(1.1, 2.0))
    return dict(op=op, B=min(B, 16), Hkv=Hkv, d=rng.choice([64, 128]), T_lo=lo, T_hi=hi,
                live=rng.uniform(0.1, 0.95), code=rng.choice(["e4m3", "int8", "bf16"]))


# ----------------------------------------------------------------------------------
# Sizes that a case fixes (the same for every seed)
# ----------------------------------------------------------------------------------
def _lens(case, lo, hi, n):
    """n lengths spread over [lo, hi], both ends among them where n allows."""
    if n == 1:
        return np.array([hi], np.int64)
    return np.array([lo + (hi - lo) * i // (n - 1) for i in range(n)], np.int64)


def _attend_sizes(case):
    """Per unit: T, g, selected blocks, and whether the unit streams."""
    B, Hkv = case["B"], case["Hkv"]
    gs = [int(x) for x in case["g"].split(",")]
    T = np.repeat(_lens(case, case["T_lo"], case["T_hi"], B), Hkv)
    U = B * Hkv
    g = np.array([gs[(u * 5 + u // Hkv) % len(gs)] for u in range(U)], np.int64)
    n_blk = -(-T // g)
    streams = np.array([(u % Hkv) < case["streaming"] for u in range(U)])
    # one sink block, a local window (2048 tokens on streaming heads, one block otherwise)
    n_loc = np.where(streams, -(-2048 // g), 1)
    k = np.where(streams, 0, np.maximum(1, (case["frac"] * n_blk).astype(np.int64)))
    cnt = np.minimum(n_blk, 1 + n_loc + k)
    return T, g, cnt, streams


def _unit_tokens(T, g, cnt):
    """Tokens that a selection of cnt blocks, the last one among them, covers."""
    return (cnt - 1) * g + (T - (-(-T // g) - 1) * g)


def work(case):
    op = case["op"]
    if op == "attend":
        T, g, cnt, _ = _attend_sizes(case)
        tok = _unit_tokens(T, g, cnt)
        pages = -(-tok // PAGE)
        U, G, d = len(T), case["G"], case["d"]
        act = 2 if case["act"] == "bf16" else 4
        nbytes = int(tok.sum()) * d * 2 + int(pages.sum()) * 12 + int(cnt.sum()) * (8 if case["bias"] else 4)
        nbytes += U * G * (d * act + d * 4 + 4)
        return {"bytes": nbytes, "flops": int(tok.sum()) * G * d * 4}
    if op == "append":
        old, new = _append_lens(case)
        act = 2 if case["act"] == "bf16" else 4
        tok = int(new.sum()) * case["Hkv"]
        pages = int((-(-(old + new) // PAGE) - old // PAGE)[new > 0].sum()) * case["Hkv"]
        kept = int((old % PAGE)[new > 0].sum()) * case["Hkv"]
        return {"bytes": 2 * case["d"] * (tok * (act + 1) + 2 * kept) + pages * 20, "flops": 4 * tok * case["d"]}
    if op == "turnover":
        lens, new, P, n_pages = _turnover_sizes(case)
        left = int((-(-lens[:case["leave"]] // PAGE)).sum()) * case["Hkv"]
        came = int((-(-new[:case["leave"]] // PAGE)).sum()) * case["Hkv"]
        # a row entry read and written and a count changed for each page, and every count looked at once
        return {"bytes": 16 * left + 12 * came + 4 * n_pages, "flops": 0}
    page = 2 * PAGE * case["d"] * (2 if case["code"] == "bf16" else 1)
    if op == "fork":
        lens, parent, n_pages = _fork_sizes(case)
        kids = lens[parent] if len(parent) else lens[:0]
        full, tails = int((kids // PAGE).sum()) * case["Hkv"], int((kids % PAGE > 0).sum()) * case["Hkv"]
        return {"bytes": 28 * full + tails * (2 * page + 40) + 4 * n_pages, "flops": 0}
    n_pages, live = _compact_sizes(case)
    moves = int(live * (1 - live / n_pages))   # live pages above the live count, on average
    return {"bytes": moves * (2 * page + 24) + live * 4 + 4 * n_pages, "flops": 0}


# ----------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------
def _dev():
    return torch.device("cuda")


def _gen(seed):
    return torch.Generator(device=_dev()).manual_seed(int(seed) * 7919 + 17)


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


def _random_pool(n_pages, d, code, gen):
    """A pool of pages of normal values, a spread of its own for each page; its codes and scales."""
    pool = torch.empty((n_pages, PAGE, d), dtype=CODES[code], device=_dev())
    scale = torch.zeros(n_pages, dtype=torch.float32, device=_dev())
    for a in range(0, n_pages, 65536):
        b = min(n_pages, a + 65536)
        x = torch.randn((b - a, PAGE, d), generator=gen, device=_dev())
        x *= torch.exp(0.5 * torch.randn((b - a, 1, 1), generator=gen, device=_dev()))
        if code == "bf16":
            pool[a:b] = x.bfloat16()
        else:
            s = _page_scale(x.abs().amax((1, 2)), code)
            pool[a:b] = _encode(x, s.view(-1, 1, 1), code)
            scale[a:b] = s
    return pool, scale


def prepare(case, seed):
    case = dict(case)
    return {"attend": _prep_attend, "append": _prep_append, "fork": _prep_fork, "turnover": _prep_turnover,
            "compact": _prep_compact}[case["op"]](case, int(seed))


def _prep_attend(case, seed):
    gen, rng = _gen(seed), np.random.default_rng(seed)
    B, Hkv, G, d = case["B"], case["Hkv"], case["G"], case["d"]
    T, g, cnt, streams = _attend_sizes(case)
    U = B * Hkv
    pages = -(-T // PAGE)
    P = int(pages.max())
    n_pages = int(pages.sum()) + 3
    perm = rng.permutation(n_pages)
    table = np.full((U, P), -1, np.int32)
    n_blk = -(-T // g)
    S = int(cnt.max())
    sel = np.full((U, S), -1, np.int32)
    at = 0
    for u in range(U):
        table[u, :pages[u]] = perm[at:at + pages[u]]
        at += pages[u]
        c, nb = int(cnt[u]), int(n_blk[u])
        loc = min(nb, int(-(-2048 // g[u]))) if streams[u] else 1
        forced = np.union1d([0], np.arange(nb - loc, nb))
        rest = np.setdiff1d(np.arange(nb), forced)
        pick = rng.choice(rest, size=max(0, c - len(forced)), replace=False) if c > len(forced) else rest[:0]
        mine = np.sort(np.concatenate([forced, pick]))
        mine = np.concatenate([mine[:c - 1], mine[-1:]]) if len(mine) > c else mine
        sel[u, :c] = mine
    kp, ks = _random_pool(n_pages, d, case["code"], gen)
    vp, vs = _random_pool(n_pages, d, case["code"], gen)
    q = torch.randn((B, Hkv * G, d), generator=gen, device=_dev()).to(ACTS[case["act"]])
    MB = int(n_blk.max())
    bias = None
    if case["bias"]:
        bias = torch.randn((U, MB), generator=gen, device=_dev())
        if MB >= 4:                        # blocks that the eviction head dropped
            bias[torch.rand((U, MB), generator=gen, device=_dev()) < 0.09] = -math.inf
        if U > 1:                          # and a unit that keeps none
            bias[1] = -math.inf
    lens = T.reshape(B, Hkv)[:, 0]
    mg = int((cnt * g // PAGE).max())
    return dict(case=case, k=kp, v=vp, ks=ks, vs=vs, table=_i32(table), lens=_i32(lens), g=_i32(g), sel=_i32(sel),
                cnt=_i32(cnt), q=q, bias=bias, max_blocks=MB, max_gather=mg,
                out=torch.zeros((B, Hkv * G, d), dtype=torch.float32, device=_dev()),
                lse=torch.zeros((B, Hkv * G), dtype=torch.float32, device=_dev()),
                status=torch.zeros(1, dtype=torch.int32, device=_dev()))


def _append_lens(case):
    B = case["B"]
    old = _lens(case, case["old_lo"], case["old_hi"], B)
    new = _lens(case, case["new_lo"], case["new_hi"], B)[::-1].copy()
    return old, new


def _prep_append(case, seed):
    gen, rng = _gen(seed), np.random.default_rng(seed)
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    old, new = _append_lens(case)
    pages = np.repeat(-(-(old + new) // PAGE), Hkv)
    P = max(1, int(pages.max()))
    n_pages = int(pages.sum()) + 2
    perm = rng.permutation(n_pages)
    table = np.full((B * Hkv, P), -1, np.int32)
    at = 0
    for u in range(B * Hkv):
        table[u, :pages[u]] = perm[at:at + pages[u]]
        at += pages[u]
    kp, ks = _random_pool(n_pages, d, case["code"], gen)
    vp, vs = _random_pool(n_pages, d, case["code"], gen)
    # K and V of the new tokens as the model's fused projection leaves them: one row per
    # token, K heads then V heads.
    rows = int(new.sum())
    kv_new = torch.randn((max(rows, 1), 2 * Hkv * d), generator=gen, device=_dev())
    kv_new *= torch.exp(torch.randn((max(rows, 1), 1), generator=gen, device=_dev()))
    kv_new = kv_new.to(ACTS[case["act"]])
    row0 = np.concatenate([[0], np.cumsum(new)[:-1]])
    return dict(case=case, k=kp, v=vp, ks=ks, vs=vs, table=_i32(table), old=_i32(old), lens=_i32(old + new),
                row0=_i32(row0), kv_new=kv_new, rows=rows, max_new=int(new.max()),
                status=torch.zeros(1, dtype=torch.int32, device=_dev()))


def _fork_sizes(case):
    """Lengths of the parents (slots 0 .. parents-1) and the parent of each child (the other slots)."""
    n = case["parents"]
    lens = _lens(case, case["T_lo"], case["T_hi"], n)
    parent = np.array([(3 * i + 1) % n for i in range(case["B"] - n)], np.int64)
    n_pages = (int((-(-lens // PAGE)).sum()) + (case["B"] - n)) * case["Hkv"] * 9 // 8 + 5
    return lens, parent, n_pages


def _prep_fork(case, seed):
    gen, rng = _gen(seed), np.random.default_rng(seed)
    B, Hkv, d, n = case["B"], case["Hkv"], case["d"], case["parents"]
    lens, parent, n_pages = _fork_sizes(case)
    P = int(-(-lens.max() // PAGE)) + 2
    perm = rng.permutation(n_pages)
    table = np.full((B, Hkv, P), -1, np.int32)
    ref = np.zeros(n_pages, np.int32)
    at = 0
    for b in range(n):
        np_b = int(-(-lens[b] // PAGE))
        for h in range(Hkv):
            table[b, h, :np_b] = perm[at:at + np_b]
            at += np_b
    seq = np.zeros(B, np.int64)
    seq[:n] = lens
    for i in range(B - n):                     # the beams so far: children of other parents
        p = int(rng.integers(n))
        full = int(lens[p] // PAGE)
        table[n + i, :, :full] = table[p, :, :full]
        seq[n + i] = lens[p]
        if lens[p] % PAGE:
            table[n + i, :, full] = perm[at:at + Hkv]
            at += Hkv
    np.add.at(ref, table[table >= 0], 1)
    src = parent[rng.permutation(len(parent))]
    kp, ks = _random_pool(n_pages, d, case["code"], gen)
    vp, vs = _random_pool(n_pages, d, case["code"], gen)
    return dict(case=case, k=kp, v=vp, ks=ks, vs=vs, table=_i32(table.reshape(B * Hkv, P)), ref=_i32(ref),
                lens=_i32(seq), src=_i32(src), dst=_i32(np.arange(n, B)), n=B - n,
                pairs=torch.zeros((max(1, (B - n) * Hkv), 2), dtype=torch.int32, device=_dev()),
                n_pairs=torch.zeros(1, dtype=torch.int32, device=_dev()),
                status=torch.zeros(1, dtype=torch.int32, device=_dev()))


def _turnover_sizes(case):
    lens = _lens(case, case["T_lo"], case["T_hi"], case["B"])
    lens = np.roll(lens, case["B"] // 3)
    new = _lens(case, case["T_lo"], case["T_hi"], case["B"])[::-1]
    P = int(-(-case["T_hi"] // PAGE)) + 1
    both = max(int((-(-lens // PAGE)).sum()), int((-(-np.concatenate([new[:case["leave"]], lens[case["leave"]:]]) // PAGE)).sum()))
    return lens, new, P, int(both * case["Hkv"] * case["slack"]) + 3


def _prep_turnover(case, seed):
    rng = np.random.default_rng(seed)
    B, Hkv = case["B"], case["Hkv"]
    lens, new, P, n_pages = _turnover_sizes(case)
    perm = rng.permutation(n_pages)
    table = np.full((B, Hkv, P), -1, np.int32)
    at = 0
    for b in range(B):
        np_b = int(-(-lens[b] // PAGE))
        for h in range(Hkv):
            table[b, h, :np_b] = perm[at:at + np_b]
            at += np_b
    ref = np.zeros(n_pages, np.int32)
    ref[table[table >= 0]] = 1
    # slots 0 .. leave-1 are given up, in an order of the scheduler's, and taken again
    want = lens.copy()
    want[:case["leave"]] = new[:case["leave"]]
    return dict(case=case, table=_i32(table.reshape(B * Hkv, P)), ref=_i32(ref), lens=_i32(lens),
                seqs=_i32(rng.permutation(case["leave"])), want=_i32(want), n_pages=n_pages,
                status=torch.zeros(1, dtype=torch.int32, device=_dev()))


def _compact_sizes(case):
    lens = _lens(case, case["T_lo"], case["T_hi"], case["B"])
    live = int((-(-lens // PAGE)).sum()) * case["Hkv"]
    return int(live / case["live"]) + 1, live


def _prep_compact(case, seed):
    gen, rng = _gen(seed), np.random.default_rng(seed)
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    lens = _lens(case, case["T_lo"], case["T_hi"], B)
    n_pages, live = _compact_sizes(case)
    P = int(-(-lens.max() // PAGE)) + 1
    perm = rng.permutation(n_pages)
    table = np.full((B, Hkv, P), -1, np.int32)
    at = 0
    for b in range(B):
        np_b = int(-(-lens[b] // PAGE))
        for h in range(Hkv):
            table[b, h, :np_b] = perm[at:at + np_b]
            at += np_b
    ref = np.zeros(n_pages, np.int32)
    ref[table[table >= 0]] = 1
    kp, ks = _random_pool(n_pages, d, case["code"], gen)
    vp, vs = _random_pool(n_pages, d, case["code"], gen)
    first = _i32(table.reshape(B * Hkv, P))
    return dict(case=case, k=kp, v=vp, ks=ks, vs=vs, table0=first, ref0=_i32(ref), table=first.clone(), ref=_i32(ref),
                lens=_i32(lens), pairs=torch.zeros((n_pages // 2 + 1, 2), dtype=torch.int32, device=_dev()),
                n_pairs=torch.zeros(1, dtype=torch.int32, device=_dev()),
                n_live=torch.zeros(1, dtype=torch.int32, device=_dev()),
                status=torch.zeros(1, dtype=torch.int32, device=_dev()))


# ----------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _own_attend, "append": _own_append, "fork": _own_fork, "turnover": _own_turnover,
                "compact": _own_compact}[op](state)
    return {"attend": _plain_attend, "append": _plain_append, "fork": _plain_fork, "turnover": _plain_turnover,
            "compact": _plain_compact}[op](state)


def _pools_out(s):
    out = {"k": s["k"], "v": s["v"]}
    if s["case"]["code"] != "bf16":
        out.update(k_scale=s["ks"], v_scale=s["vs"])
    return out


# -- plain forms -------------------------------------------------------------------
def _plain_attend(s):
    c = s["case"]
    B, Hkv, G, d = c["B"], c["Hkv"], c["G"], c["d"]
    U, P = s["table"].shape
    ppb = (s["g"].long() // PAGE).view(U, 1)
    T = s["lens"].long().repeat_interleave(Hkv).view(U, 1)
    i = torch.arange(s["max_gather"], device=_dev()).view(1, -1)
    blk_at = i // ppb
    blk = torch.gather(s["sel"].long(), 1, blk_at.clamp(max=s["sel"].shape[1] - 1))
    page = blk * ppb + i % ppb
    used = (blk_at < s["cnt"].long().view(U, 1)) & (page * PAGE < T)
    phys = torch.gather(s["table"].long(), 1, page.clamp(0, P - 1))
    phys = torch.where(used, phys, torch.zeros_like(phys))
    tok = page.unsqueeze(2) * PAGE + torch.arange(PAGE, device=_dev())
    seen = (used.unsqueeze(2) & (tok < T.unsqueeze(2))).view(U, 1, -1)
    K = (s["k"][phys].float() * s["ks"][phys].view(U, -1, 1, 1)).view(U, -1, d)
    q = s["q"].float().view(U, G, d)
    x = torch.matmul(q, K.transpose(1, 2)) * (1.0 / math.sqrt(d))
    if s["bias"] is not None:
        e = torch.gather(s["bias"], 1, blk.clamp(0, s["max_blocks"] - 1))
        x = x + e.repeat_interleave(PAGE, 1).view(U, 1, -1)
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    m = x.amax(2, keepdim=True)
    base = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - base)
    l = p.sum(2, keepdim=True)
    V = (s["v"][phys].float() * s["vs"][phys].view(U, -1, 1, 1)).view(U, -1, d)
    o = torch.matmul(p, V) / torch.where(l > 0, l, torch.ones_like(l))
    s["out"].copy_(o.view(B, Hkv * G, d))
    s["lse"].copy_((base + torch.log(l)).view(B, Hkv * G))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_append(s):
    c = s["case"]
    B, Hkv, d, code = c["B"], c["Hkv"], c["d"], c["code"]
    R = s["rows"]
    if R == 0:
        return _pools_out(s)
    old, row0 = s["old"].long(), s["row0"].long()
    row = torch.arange(R, device=_dev())
    # the sequence of each row, its position, and its page (and slot there) for each head
    new = s["lens"].long() - old
    b = torch.repeat_interleave(torch.arange(B, device=_dev()), new, output_size=R)
    t = old[b] + row - row0[b]
    u = b.view(-1, 1) * Hkv + torch.arange(Hkv, device=_dev())
    phys = s["table"].long()[u, (t // PAGE).view(-1, 1)]                       # [rows, Hkv]
    slot = (t % PAGE).view(-1, 1).expand(-1, Hkv)
    # pages that held tokens before: the page of position old, where it ends inside a page
    first = (old // PAGE).clamp(max=s["table"].shape[1] - 1)
    keeps = ((old % PAGE > 0) & (new > 0)).repeat_interleave(Hkv)
    ub = torch.arange(B * Hkv, device=_dev())
    head_page = s["table"].long()[ub, first.repeat_interleave(Hkv)][keeps]
    n_old = (old % PAGE).repeat_interleave(Hkv)[keeps]
    for pool, scale, x in ((s["k"], s["ks"], s["kv_new"][:R, :Hkv * d]), (s["v"], s["vs"], s["kv_new"][:R, Hkv * d:])):
        x = x.float().reshape(R, Hkv, d)
        size = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(2)
        amax = torch.zeros(scale.shape[0], device=_dev()).scatter_reduce_(0, phys.reshape(-1), size.reshape(-1), "amax")
        need = _page_scale(amax, code)
        had = torch.zeros_like(scale)
        had[head_page] = scale[head_page]
        to = torch.maximum(had, need)
        # codes already there, at the page's new scale
        at, was = to[head_page], scale[head_page]
        page = pool[head_page].float() * was.view(-1, 1, 1)
        again = _encode(page, at.view(-1, 1, 1), code)
        keep = (torch.arange(PAGE, device=_dev()).view(1, -1) < n_old.view(-1, 1)) & (at > was).view(-1, 1)
        raw = pool.view(torch.uint8)
        raw[head_page] = torch.where(keep.unsqueeze(2), again.view(torch.uint8), raw[head_page])
        raw[phys, slot] = _encode(x, to[phys].unsqueeze(2), code).view(torch.uint8)
        scale[phys.reshape(-1)] = to[phys.reshape(-1)]
    return _pools_out(s)


def _plain_free(s, seqs):
    c = s["case"]
    B, Hkv = c["B"], c["Hkv"]
    table = s["table"].view(B, Hkv, -1)
    rows = table[seqs.long()]
    s["ref"].index_add_(0, rows[rows >= 0].long(), torch.full_like(rows[rows >= 0], -1))
    table[seqs.long()] = -1
    s["lens"][seqs.long()] = 0


def _plain_fork(s):
    c = s["case"]
    B, Hkv = c["B"], c["Hkv"]
    _plain_free(s, s["dst"])
    table = s["table"].view(B, Hkv, -1)
    P = table.shape[2]
    T = s["lens"].long()[s["src"].long()]
    rows = table[s["src"].long()]                                               # [n, Hkv, P]
    j = torch.arange(P, device=_dev()).view(1, 1, -1)
    full = j < (T // PAGE).view(-1, 1, 1)
    tail = ((j == (T // PAGE).view(-1, 1, 1)) & (T % PAGE > 0).view(-1, 1, 1)).expand_as(rows)
    shared = rows[full.expand_as(rows)].long()
    s["ref"].index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    old = rows[tail].long()
    free = torch.nonzero(s["ref"] == 0).view(-1)[:old.numel()]
    mine = torch.where(full, rows, torch.full_like(rows, -1))
    mine[tail] = free.int()
    table[s["dst"].long()] = mine
    s["ref"][free] = 1
    s["lens"][s["dst"].long()] = T.int()
    for pool in (s["k"], s["v"], s["ks"], s["vs"]):
        raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        raw[free] = raw[old]
    return {"table": s["table"], "ref": s["ref"], "lens": s["lens"], **_pools_out(s)}


def _plain_turnover(s):
    _plain_free(s, s["seqs"])
    want = s["want"].long().repeat_interleave(s["case"]["Hkv"]).view(-1, 1)
    j = torch.arange(s["table"].shape[1], device=_dev()).view(1, -1)
    lacks = (s["table"] < 0) & (j * PAGE < want)
    n = lacks.sum()
    free = torch.nonzero(s["ref"] == 0).view(-1)[:n]
    s["table"][lacks] = free.int()
    s["ref"][free] = 1
    return {"table": s["table"], "ref": s["ref"], "lens": s["lens"]}


def _plain_compact(s):
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    live = s["ref"] > 0
    n = live.sum()
    at = torch.arange(s["ref"].numel(), device=_dev())
    src = at[live & (at >= n)]
    dst = at[~live & (at < n)]
    to = at.int()
    to[src] = dst.int()
    table = s["table"]
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    s["ref"][dst] = s["ref"][src]
    s["ref"][src] = 0
    for pool in (s["k"], s["v"], s["ks"], s["vs"]):
        raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        raw[dst] = raw[src]
    s["n_live"].copy_(n.view(1))
    return {"table": table, "ref": s["ref"], "n_live": s["n_live"], **_pools_out(s)}


# -- the framework's calls -----------------------------------------------------------
def _handle(s):
    """What a program keeps between calls: the dims, the pointer structs, the workspaces."""
    h = s.get("handle")
    if h is not None:
        return h
    from long_context_serving_gb300 import bsattn as A

    c = s["case"]
    kv = {"e4m3": A.BS_E4M3, "int8": A.BS_INT8, "bf16": A.BS_BF16}[c.get("code", "bf16")]
    pool_pages = s["k"].shape[0] if "k" in s else s["n_pages"]
    dims = A.Dims(batch=c["B"], n_q_heads=c["Hkv"] * c.get("G", 1), n_kv_heads=c["Hkv"], head_dim=c.get("d", 128),
                  page_size=PAGE, max_pages_per_unit=s["table"].shape[1], max_blocks_per_unit=s.get("max_blocks", 1),
                  max_sel_per_unit=s["sel"].shape[1] if "sel" in s else 1, max_subs_per_unit=1,
                  max_gather_pages_per_unit=s.get("max_gather", 1), n_pages=pool_pages, kv_dtype=kv,
                  q_dtype=A.BS_FP32 if c.get("act") == "fp32" else A.BS_BF16)
    h = dict(A=A, dims=dims)
    p = lambda t: t.data_ptr()  # noqa: E731
    if c["op"] == "attend":
        h["kv"] = A.KV(k_pool=p(s["k"]), v_pool=p(s["v"]), page_table=p(s["table"]), seq_lens=p(s["lens"]),
                       k_scale=p(s["ks"]), v_scale=p(s["vs"]))
        h["cfg"] = A.HeadCfg(block_tokens=p(s["g"]))
        h["ws"] = torch.zeros(A.workspace_size(dims) // 4, dtype=torch.float32, device=_dev())
    else:
        if "k" in s:
            eight = c["code"] != "bf16"
            h["pools"] = A.Pools(k_pool=p(s["k"]), v_pool=p(s["v"]), k_scale=p(s["ks"]) if eight else 0,
                                 v_scale=p(s["vs"]) if eight else 0)
        if "ref" in s:
            h["map"] = A.PageMap(page_table=p(s["table"]), ref_count=p(s["ref"]), seq_lens=p(s["lens"]))
            h["ws"] = torch.zeros(A.pages_workspace_size(dims) // 4, dtype=torch.int32, device=_dev())
        if "pairs" in s:
            h["copies"] = A.PageCopies(pairs=p(s["pairs"]), count=p(s["n_pairs"]), capacity=s["pairs"].shape[0])
        if c["op"] == "append":
            h["k_new"], h["v_new"] = s["kv_new"][:, :c["Hkv"] * c["d"]], s["kv_new"][:, c["Hkv"] * c["d"]:]
    s["handle"] = h
    return h


def _own_attend(s):
    h = _handle(s)
    h["A"].sparse_decode_attn(h["dims"], s["q"], h["kv"], h["cfg"], s["sel"], s["cnt"], s["out"], s["lse"], h["ws"],
                              s["status"], evict_bias=s["bias"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_append(s):
    h = _handle(s)
    if s["rows"] > 0:
        h["A"].quant_append(h["dims"], h["pools"], s["table"], s["lens"], s["old"], s["row0"], h["k_new"], h["v_new"],
                            s["kv_new"].stride(0), s["rows"], s["max_new"], s["status"])
    return _pools_out(s)


def _own_fork(s):
    h = _handle(s)
    A = h["A"]
    A.pages_free(h["dims"], h["map"], s["dst"], s["status"])
    A.pages_fork(h["dims"], h["map"], s["src"], s["dst"], h["copies"], h["ws"], s["status"])
    A.pages_copy(h["dims"], h["pools"], h["copies"], s["status"])
    return {"table": s["table"], "ref": s["ref"], "lens": s["lens"], **_pools_out(s)}


def _own_turnover(s):
    h = _handle(s)
    A = h["A"]
    A.pages_free(h["dims"], h["map"], s["seqs"], s["status"])
    A.pages_reserve(h["dims"], h["map"], s["want"], h["ws"], s["status"])
    return {"table": s["table"], "ref": s["ref"], "lens": s["lens"]}


def _own_compact(s):
    h = _handle(s)
    A = h["A"]
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    A.pages_compact(h["dims"], h["map"], h["copies"], s["n_live"], h["ws"], s["status"])
    A.pages_copy(h["dims"], h["pools"], h["copies"], s["status"])
    return {"table": s["table"], "ref": s["ref"], "n_live": s["n_live"], **_pools_out(s)}


# ----------------------------------------------------------------------------------
# The definition in 64 bits
# ----------------------------------------------------------------------------------
def exact(case, seed):
    """Attention unit by unit in float64; E4M3 append value by value (its scales are powers of
    two, so every quotient is a float64 and each code is the nearest one). The page calls move
    whole numbers and bytes, and INT8 codes are of quotients rounded to fp32: no such value."""
    if case["op"] == "attend":
        return _exact_attend(prepare(case, seed))
    if case["op"] == "append" and case["code"] == "e4m3":
        return _exact_append(prepare(case, seed))
    return None


def _exact_attend(s):
    c = s["case"]
    Hkv, G, d = c["Hkv"], c["G"], c["d"]
    sel, cnt, g, table = (s[n].cpu().numpy() for n in ("sel", "cnt", "g", "table"))
    lens = s["lens"].cpu().numpy()
    out, lse = torch.zeros_like(s["out"], dtype=torch.float64), torch.zeros_like(s["lse"], dtype=torch.float64)
    for u in range(c["B"] * Hkv):
        b, h = divmod(u, Hkv)
        t = np.concatenate([np.arange(k * g[u], min((k + 1) * g[u], lens[b])) for k in sel[u, :cnt[u]]])
        where = torch.as_tensor(table[u, t // PAGE].astype(np.int64), device=_dev())
        at = torch.as_tensor(t % PAGE, device=_dev())
        K = s["k"].view(torch.uint8)[where, at].view(s["k"].dtype).double() * s["ks"].double()[where, None]
        V = s["v"].view(torch.uint8)[where, at].view(s["v"].dtype).double() * s["vs"].double()[where, None]
        x = s["q"][b, h * G:(h + 1) * G].double() @ K.T / math.sqrt(d)
        if s["bias"] is not None:
            x = x + s["bias"][u].double()[torch.as_tensor(t // g[u], device=_dev())]
        top = torch.logsumexp(x, 1)
        w = torch.where(top[:, None] == -math.inf, torch.zeros_like(x), torch.exp(x - top[:, None]))
        out[b, h * G:(h + 1) * G] = w @ V
        lse[b, h * G:(h + 1) * G] = top
    return {"out": out, "lse": lse}


def _nearest_e4m3(y):
    """y rounded to the nearest E4M3 value, ties to the even mantissa (float64)."""
    a = np.minimum(np.abs(y), E4M3_MAX)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6.0)
    step = 2.0 ** (e - 3)
    return np.copysign(np.minimum(np.round(a / step) * step, E4M3_MAX), y)


def _exact_append(s):
    c = s["case"]
    Hkv, d = c["Hkv"], c["d"]
    old, lens, row0, table = (s[n].cpu().numpy().astype(np.int64) for n in ("old", "lens", "row0", "table"))
    new = s["kv_new"].double().cpu().numpy()
    done = {}
    for name, sname, side in (("k", "ks", 0), ("v", "vs", 1)):
        val = s[name].float().cpu().numpy().astype(np.float64)
        scl = s[sname].cpu().numpy().astype(np.float64)
        for b in range(c["B"]):
            for lp in range(old[b] // PAGE, -(-lens[b] // PAGE) if lens[b] > old[b] else 0):
                t0, t1 = max(lp * PAGE, old[b]), min((lp + 1) * PAGE, lens[b])
                rows = new[row0[b] + t0 - old[b]:row0[b] + t1 - old[b], side * Hkv * d:(side + 1) * Hkv * d]
                for h in range(Hkv):
                    ph = table[b * Hkv + h, lp]
                    x = rows[:, h * d:(h + 1) * d]
                    big = np.abs(x).max()
                    need = 2.0 ** max(math.ceil(math.log2(big / E4M3_MAX)), -126) if big > 0 else 0.0
                    kept = t0 - lp * PAGE
                    to = max(scl[ph], need) if kept else need
                    if kept and to > scl[ph]:
                        val[ph, :kept] = _nearest_e4m3(val[ph, :kept] * scl[ph] / to)
                    val[ph, kept:kept + len(x)] = _nearest_e4m3(x / to) if to > 0 else 0.0
                    scl[ph] = to
        done[name], done[name + "_scale"] = torch.as_tensor(val), torch.as_tensor(scl)
    return done
