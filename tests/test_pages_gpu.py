"""Pages handed out, shared, taken back, moved and copied on the GPU, against a plain model
of the page table and counts on the host; every call's refusals that only the device can
see; and a serving run of all of them over an 8-bit cache."""
import numpy as np
import pytest
import torch

import _quant as Q
from long_context_serving_gb300 import bsattn as B
from long_context_serving_gb300.build import build
from oracle import bsattn_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build()
    B.lib()


def i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device="cuda")


class Model:
    """The page table, counts and lengths on the host, and the rules as plain loops."""

    def __init__(self, B_, H, P, n_pages):
        self.B, self.H, self.P, self.n = B_, H, P, n_pages
        self.table = np.full((B_ * H, P), -1, np.int64)
        self.ref = np.zeros(n_pages, np.int64)
        self.lens = np.zeros(B_, np.int64)

    def _free(self):
        return np.flatnonzero(self.ref == 0)

    def reserve(self, new_lens):
        want = [(u, j) for u in range(self.B * self.H) for j in range(-(-max(int(new_lens[u // self.H]), 0) // 16))]
        if any(j >= self.P for _, j in want):
            return B.BS_ERR_CAPACITY
        want = [(u, j) for u, j in want if self.table[u, j] < 0]
        free = self._free()
        if len(want) > len(free):
            return B.BS_ERR_CAPACITY
        for (u, j), p in zip(want, free):
            self.table[u, j] = p
            self.ref[p] = 1
        return 0

    def fork(self, src, dst):
        """(status, pairs)"""
        free = list(self._free())
        jobs = [(s, d) for s, d in zip(src, dst) if s >= 0 and d >= 0]
        tails = []
        for s, d in jobs:
            T = int(self.lens[s])
            for h in range(self.H):
                if T % 16 and self.table[s * self.H + h, T // 16] >= 0:
                    tails.append((s, d, h))
        if len(tails) > len(free):
            return B.BS_ERR_CAPACITY, []
        pairs = []
        for s, d in jobs:
            T = int(self.lens[s])
            for h in range(self.H):
                a, b = s * self.H + h, d * self.H + h
                for j in range(T // 16):
                    p = self.table[a, j]
                    self.table[b, j] = p
                    if p >= 0:
                        self.ref[p] += 1
                if (s, d, h) in tails:
                    p = free.pop(0)
                    self.table[b, T // 16] = p
                    self.ref[p] = 1
                    pairs.append((self.table[a, T // 16], p))
            self.lens[d] = T
        return 0, pairs

    def free(self, seqs):
        for s in dict.fromkeys(int(x) for x in seqs if x >= 0):
            for h in range(self.H):
                row = self.table[s * self.H + h]
                for p in row[row >= 0]:
                    self.ref[p] -= 1
                row[:] = -1
            self.lens[s] = 0

    def compact(self):
        n_live = int((self.ref > 0).sum())
        src = [p for p in range(n_live, self.n) if self.ref[p] > 0]
        dst = [p for p in range(n_live) if self.ref[p] == 0]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.ref[d], self.ref[s] = self.ref[s], 0
        for i in np.ndindex(self.table.shape):
            if self.table[i] in to:
                self.table[i] = to[self.table[i]]
        return n_live, list(zip(src, dst))


class Map:
    """The same on the device."""

    def __init__(self, m: Model, Hq=None, d=64, kv=B.BS_BF16, capacity=None):
        self.table, self.ref, self.lens = i32(m.table), i32(m.ref), i32(m.lens)
        self.dims = B.Dims(batch=m.B, n_q_heads=Hq or m.H, n_kv_heads=m.H, head_dim=d, page_size=16,
                           max_pages_per_unit=m.P, max_blocks_per_unit=m.P, max_sel_per_unit=m.P, max_subs_per_unit=1,
                           max_gather_pages_per_unit=m.P, n_pages=m.n, kv_dtype=kv, q_dtype=B.BS_BF16)
        self.ptrs = B.PageMap(page_table=self.table.data_ptr(), ref_count=self.ref.data_ptr(), seq_lens=self.lens.data_ptr())
        cap = capacity or max(m.n // 2, m.B * m.H, 1)
        self.pairs, self.count = torch.zeros((cap, 2), dtype=torch.int32, device="cuda"), i32([77])
        self.copies = B.PageCopies(pairs=self.pairs.data_ptr(), count=self.count.data_ptr(), capacity=cap)
        # a workspace of noise: nothing may rest on its contents
        self.ws = torch.randint(-2 ** 31, 2 ** 31 - 1, (B.pages_workspace_size(self.dims) // 4,), dtype=torch.int32,
                                device="cuda")
        self.n_live, self.status = i32([0]), i32([0])

    def reserve(self, lens):
        B.pages_reserve(self.dims, self.ptrs, i32(lens), self.ws, self.status)

    def fork(self, src, dst):
        B.pages_fork(self.dims, self.ptrs, i32(src), i32(dst), self.copies, self.ws, self.status)

    def free(self, seqs):
        B.pages_free(self.dims, self.ptrs, i32(seqs), self.status)

    def compact(self):
        B.pages_compact(self.dims, self.ptrs, self.copies, self.n_live, self.ws, self.status)

    def listed(self):
        return [tuple(x) for x in self.pairs[:int(self.count)].tolist()]

    def take_status(self):
        torch.cuda.synchronize()
        code = int(self.status)
        self.status.zero_()
        return code

    def check(self, m: Model):
        torch.cuda.synchronize()
        assert np.array_equal(self.table.cpu().numpy(), m.table)
        assert np.array_equal(self.ref.cpu().numpy(), m.ref)
        assert np.array_equal(self.lens.cpu().numpy(), m.lens)


@pytest.mark.parametrize("seed,Bn,H,P,n_pages", [(1, 1, 1, 1, 1), (2, 3, 1, 4, 40), (3, 5, 3, 9, 97), (4, 9, 2, 300, 4097),
                                                 (5, 20, 8, 40, 5000), (6, 6, 4, 700, 8192), (7, 40, 16, 3, 2100),
                                                 (8, 400, 8, 2, 9000)])   # (more units than CTAs)
def test_random_runs_equal_the_model(seed, Bn, H, P, n_pages):
    """Sixty random calls each; after every one the table, counts, lengths and copy list are the model's."""
    rng = np.random.default_rng(seed)
    m = Model(Bn, H, P, n_pages)
    g = Map(m)
    seen = set()
    for _ in range(60):
        op = rng.choice(["reserve", "reserve", "fork", "free", "compact"])
        if op == "reserve":
            grow = np.where(rng.random(Bn) < 0.4, rng.integers(0, 16 * P + 1, Bn) * (rng.random(Bn) ** 2), 0).astype(int)
            want = np.minimum(m.lens + grow, 16 * P)
            want[rng.random(Bn) < 0.1] = -5
            code = m.reserve(want)
            g.reserve(want)
            if code == 0:       # the caller's lengths, part of what was reserved
                m.lens = np.where(want > m.lens, rng.integers(m.lens, np.maximum(want, m.lens) + 1), m.lens)
                g.lens.copy_(i32(m.lens))
        elif op == "fork":
            empty = [b for b in range(Bn) if m.lens[b] == 0 and (m.table[b * H:(b + 1) * H] < 0).all()]
            rng.shuffle(empty)
            dst = empty[:int(rng.integers(0, len(empty) + 1))]
            parents = [b for b in range(Bn) if b not in dst]
            if not dst or not parents:
                continue
            src = rng.choice(parents, len(dst))
            holes = rng.random(len(dst)) < 0.15
            src, dst = np.where(holes, -1, src), np.array(dst)
            code, pairs = m.fork(src, dst)
            g.fork(src, dst)
            assert g.listed() == [tuple(int(x) for x in p) for p in pairs]
        elif op == "free":
            seqs = rng.integers(-1, Bn, int(rng.integers(1, Bn + 1)))      # repeats and skips among them
            code = 0
            m.free(seqs)
            g.free(seqs)
        else:
            code = 0
            n_live, pairs = m.compact()
            g.compact()
            assert g.listed() == [tuple(int(x) for x in p) for p in pairs]
            assert int(g.n_live) == n_live
        assert g.take_status() == code, op
        seen.add((op, code))
        g.check(m)
    assert Bn == 1 or {o for o, _ in seen} == {"reserve", "fork", "free", "compact"}


@pytest.mark.parametrize("n_pages", [1, 31, 32, 33, 4095, 4096, 4097, 300_001, 5_000_011])
def test_lowest_free_pages_in_pools_of_any_size(n_pages):
    """Counts with holes anywhere, across words, tiles and (from 2^22 pages) larger tiles."""
    rng = np.random.default_rng(n_pages)
    m = Model(3, 2, 200, n_pages)
    m.ref = (rng.random(n_pages) < 0.7).astype(np.int64)
    m.ref[: n_pages // 3] = 1                              # a long run without a free page
    g = Map(m)
    lens = [1500, 0, 3197] if n_pages > 4000 else [1, 0, 0]
    code = m.reserve(lens)
    g.reserve(lens)
    assert g.take_status() == code
    g.check(m)
    # pages in use that no table names move all the same
    n_live, pairs = m.compact() if n_pages < 10000 else (None, None)
    if pairs is not None:
        g.compact()
        assert g.take_status() == 0 and int(g.n_live) == n_live and g.listed() == [tuple(map(int, p)) for p in pairs]
        g.check(m)


def test_compact_a_large_pool():
    """Larger tiles (above 2^22 pages), against array operations."""
    n = 5_000_011
    rng = np.random.default_rng(3)
    m = Model(2, 1, 3000, n)
    m.table[:] = rng.permutation(n)[:6000].reshape(2, 3000)
    m.table[1, 2500:] = -1
    m.ref = (rng.random(n) < 0.45).astype(np.int64) * 3
    m.ref[m.table[m.table >= 0]] = 1
    g = Map(m)
    n_live = int((m.ref > 0).sum())
    at = np.arange(n)
    src, dst = at[(m.ref > 0) & (at >= n_live)], at[(m.ref == 0) & (at < n_live)]
    to = at.copy()
    to[src] = dst
    m.table = np.where(m.table >= 0, to[m.table], m.table)
    m.ref[dst], m.ref[src] = m.ref[src], 0
    g.compact()
    assert g.take_status() == 0 and int(g.n_live) == n_live and int(g.count) == len(src)
    assert np.array_equal(g.pairs[:len(src)].cpu().numpy(), np.stack([src, dst], 1))
    g.check(m)


def filled(Bn=4, H=2, P=8, n_pages=64, lens=(40, 16, 0, 0)):
    m = Model(Bn, H, P, n_pages)
    m.reserve(lens)
    m.lens[:] = lens
    return m, Map(m)


def test_refusals_change_nothing():
    cases = [("fork", lambda g: g.fork([0, 0], [2, 2]), B.BS_ERR_INVALID_ARG),           # a slot named twice
             ("fork", lambda g: g.fork([0, 0], [2, 1]), B.BS_ERR_INVALID_ARG),           # a slot that holds pages
             ("fork", lambda g: g.fork([0, 2], [2, 3]), B.BS_ERR_INVALID_ARG),           # a slot that is a source too
             ("fork", lambda g: g.fork([0], [0]), B.BS_ERR_INVALID_ARG),
             ("fork", lambda g: g.fork([4], [2]), B.BS_ERR_INVALID_ARG),                 # out of the batch
             ("fork", lambda g: g.fork([0], [4]), B.BS_ERR_INVALID_ARG),
             ("reserve", lambda g: g.reserve([0, 0, 129, 16]), B.BS_ERR_CAPACITY)]        # longer than the row
    for op, call, code in cases:
        m, g = filled()
        call(g)
        assert g.take_status() == code, op
        if op == "fork":
            assert int(g.count) == 0
        g.check(m)
    # too few free pages: 8 in use of 9
    m, g = filled(n_pages=9)
    g.fork([0, 0], [2, 3])                                # 4 tails, 1 free page
    assert g.take_status() == B.BS_ERR_CAPACITY and int(g.count) == 0
    g.check(m)
    g.reserve([40, 32, 0, 0])                             # 2 pages, 1 free
    assert g.take_status() == B.BS_ERR_CAPACITY
    g.check(m)
    # damaged maps: entries outside the pool or on free pages, lengths outside the row
    for what in ("entry", "free", "length", "negative"):
        m, g = filled()
        if what == "entry":
            m.table[1, 1] = 64
        elif what == "free":
            m.ref[m.table[1, 1]] = 0
        else:
            m.lens[0] = 129 if what == "length" else -1
        g = Map(m)
        g.fork([1, 0], [2, 3])
        assert g.take_status() == {"entry": B.BS_ERR_DEVICE_BOUNDS, "free": B.BS_ERR_DEVICE_BOUNDS,
                                   "length": B.BS_ERR_CAPACITY, "negative": B.BS_ERR_INVALID_ARG}[what]
        g.check(m)
    # compact into a list that is too short
    m = Model(2, 1, 8, 64)
    m.ref[40:50] = 1
    m.table[0, :8], m.table[1, :2] = np.arange(40, 48), (48, 49)
    g = Map(m, capacity=9)
    g.compact()
    assert g.take_status() == B.BS_ERR_CAPACITY and int(g.count) == 0 and int(g.n_live) == 10
    g.check(m)


def test_damaged_entries_are_dropped_or_left():
    m, g = filled()
    m.table[0, 0], m.table[1, 0] = 64, m.table[1, 0]
    m.ref[m.table[1, 0]] = 0
    g = Map(m)
    g.free([0, 9, -1])
    assert g.take_status() in (B.BS_ERR_DEVICE_BOUNDS, B.BS_ERR_INVALID_ARG)
    want = m
    for h in range(2):
        for p in m.table[h][m.table[h] >= 0]:
            if p < 64 and m.ref[p] > 0:
                want.ref[p] -= 1
        want.table[h] = -1
    want.lens[0] = 0
    g.check(want)
    # compact: an entry outside the pool, and one at or above the live count on a free page, stay
    m = Model(2, 1, 8, 64)
    m.ref[40:50] = 1
    m.table[0, :8], m.table[1, :2] = np.arange(40, 48), (48, 49)
    m.table[1, 5], m.table[1, 6] = 1000, 60
    g = Map(m)
    g.compact()
    assert g.take_status() == B.BS_ERR_DEVICE_BOUNDS
    m.compact()
    g.check(m)


@pytest.mark.parametrize("kv,dt", [(B.BS_BF16, torch.int16), (B.BS_FP32, torch.int32), (B.BS_E4M3, torch.uint8),
                                   (B.BS_INT8, torch.uint8)])
@pytest.mark.parametrize("d", [64, 128])
def test_copy_moves_whole_pages_and_scales(kv, dt, d):
    rng = np.random.default_rng(d)
    m = Model(1, 1, 1, 300)
    g = Map(m, d=d, kv=kv, capacity=120)
    k, v = (torch.randint(0, 100, (300, 16, d), device="cuda").to(dt) for _ in range(2))
    ks, vs = (torch.rand(300, device="cuda") for _ in range(2))
    want = [x.clone() for x in (k, v, ks, vs)]
    pages = rng.permutation(300)[:200]
    pairs = np.stack([pages[:100], pages[100:]], 1)
    quant = kv in (B.BS_E4M3, B.BS_INT8)
    pools = B.Pools(k_pool=k.data_ptr(), v_pool=v.data_ptr(), k_scale=ks.data_ptr() if quant else 0,
                    v_scale=vs.data_ptr() if quant else 0)
    g.pairs[:100] = i32(pairs)
    for n in (0, 1, 57, 100):
        g.count.fill_(n)
        B.pages_copy(g.dims, pools, g.copies, g.status)
        src, dst = (torch.as_tensor(pairs[:n, i].copy(), device="cuda") for i in (0, 1))
        for x in want[:4 if quant else 2]:
            x[dst] = x[src]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((k, v, ks, vs), want)), n
    assert g.take_status() == 0
    # a pair outside the pool is skipped, a count above the capacity is cut to it
    g.pairs[:3] = i32([[0, 300], [-1, 5], [pages[0], pages[150]]])
    g.count.fill_(3)
    B.pages_copy(g.dims, pools, g.copies, g.status)
    want[0][int(pages[150])] = want[0][int(pages[0])]
    assert g.take_status() == B.BS_ERR_DEVICE_BOUNDS and torch.equal(k, want[0])
    g.pairs.zero_()
    g.pairs[:, 1] = 1
    g.count.fill_(10 ** 9)
    B.pages_copy(g.dims, pools, g.copies, g.status)
    assert g.take_status() == 0 and torch.equal(k[1], k[0])


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_serving_run(kind):
    """Prompts are reserved and appended, beams fork and diverge token by token, beams die and the
    cache is compacted, all on the device; at every step each live sequence's attention over the
    whole of its tokens is that of a cache of its own."""
    rng = np.random.default_rng(41)
    Bn, H, G, d, P = 6, 2, 3, 64, 12
    kv = B.BS_E4M3 if kind == "e4m3" else B.BS_INT8
    m = Model(Bn, H, P, 90)
    g = Map(m, Hq=H * G, d=d, kv=kv)
    n_pages = m.n
    k, v = (torch.full((n_pages, 16, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((n_pages,), float("nan"), device="cuda") for _ in range(2))
    pools = B.Pools(k_pool=k.data_ptr(), v_pool=v.data_ptr(), k_scale=ks.data_ptr(), v_scale=vs.data_ptr())
    # each sequence's own cache, page by page: (codes, scale) of K and V per head
    own = [[[[], []] for _ in range(H)] for _ in range(Bn)]
    lens = np.zeros(Bn, np.int64)
    ws = torch.zeros(B.workspace_size(g.dims) // 4, device="cuda")

    def append(new):
        new = np.asarray(new)
        want = lens + new
        B.pages_reserve(g.dims, g.ptrs, i32(np.where(new > 0, want, 0)), g.ws, g.status)
        x = torch.as_tensor(rng.normal(size=(int(new.sum()), 2 * H * d)) * 1.5 ** rng.integers(0, 6), device="cuda").bfloat16()
        row0 = np.cumsum(new) - new
        B.quant_append(g.dims, pools, g.table, i32(want), i32(lens), i32(row0), x[:, :H * d], x[:, H * d:], 2 * H * d,
                       int(new.sum()), int(new.max()), g.status)
        xs = x.float().cpu().numpy()
        for b in range(Bn):
            for i in range(int(new[b])):
                t = int(lens[b]) + i
                for h in range(H):
                    for side in range(2):
                        pages = own[b][h][side]
                        if t % 16 == 0:
                            pages.append((np.zeros((16, d), np.uint8), np.float32(0)))
            for h in range(H):
                for side in range(2):
                    rows = xs[row0[b]:row0[b] + new[b], side * H * d + h * d:side * H * d + (h + 1) * d]
                    t = int(lens[b])
                    while len(rows):
                        take = min(len(rows), 16 - t % 16)
                        c, s = own[b][h][side][t // 16]
                        own[b][h][side][t // 16] = Q.append_page(c, s, t % 16, rows[:take], kind)
                        rows, t = rows[take:], t + take
        lens[:] = want
        g.lens.copy_(i32(lens))

    def attend():
        q = torch.as_tensor(rng.normal(size=(Bn, H * G, d)), device="cuda").bfloat16()
        nb = -(-lens // 16)
        sel = np.where(np.arange(P) < nb[:, None], np.arange(P), -1).repeat(H, 0)
        gs = i32([16] * (Bn * H))
        out, lse = torch.zeros((Bn, H * G, d), device="cuda"), torch.zeros((Bn, H * G), device="cuda")
        safe = i32(np.maximum(lens, 1))         # (an empty slot: one token nobody reads, count 0)
        kvp = B.KV(k_pool=k.data_ptr(), v_pool=v.data_ptr(), page_table=g.table.data_ptr(), seq_lens=safe.data_ptr(),
                   k_scale=ks.data_ptr(), v_scale=vs.data_ptr())
        B.sparse_decode_attn(g.dims, q, kvp, B.HeadCfg(block_tokens=gs.data_ptr()), i32(sel), i32(nb.repeat(H)), out, lse,
                             ws, g.status)
        assert g.take_status() == 0
        for b in range(Bn):
            for h in range(H):
                if lens[b] == 0:
                    assert (out[b, h * G:(h + 1) * G] == 0).all()
                    continue
                K, V = (np.concatenate([Q.decode(c, kind) * float(s) for c, s in own[b][h][side]])[:lens[b]]
                        for side in range(2))
                want, _ = O.sparse_attention(q[b, h * G:(h + 1) * G].double().cpu().numpy(), K, V, list(range(nb[b])), 16,
                                             int(lens[b]))
                err = np.abs(out[b, h * G:(h + 1) * G].cpu().numpy() - want).max()
                # scores to (d 2^-23 + 2^-21) A, A < 4 |q||K| / 8 here; see the attention tests
                A = float((np.abs(q[b, h * G:(h + 1) * G].double().cpu().numpy()) @ np.abs(K).T).max()) / np.sqrt(d)
                assert err <= (2 * (d * 2.0 ** -23 + 2.0 ** -21) * A + 2.0 ** -18) * np.abs(V).max(), (b, h)

    def fork(src, dst):
        B.pages_fork(g.dims, g.ptrs, i32(src), i32(dst), g.copies, g.ws, g.status)
        B.pages_copy(g.dims, pools, g.copies, g.status)
        for s, t in zip(src, dst):
            lens[t] = lens[s]
            own[t] = [[[(c.copy(), sc) for c, sc in own[s][h][side]] for side in range(2)] for h in range(H)]

    def free(seqs):
        B.pages_free(g.dims, g.ptrs, i32(seqs), g.status)
        for s in seqs:
            lens[s] = 0
            own[s] = [[[], []] for _ in range(H)]

    append([37, 16, 0, 0, 0, 0])
    attend()
    fork([0, 0, 1], [2, 3, 4])
    attend()
    for _ in range(13):
        append([1, 1, 1, 1, 1, 0])
    attend()
    free([0, 3])
    B.pages_compact(g.dims, g.ptrs, g.copies, g.n_live, g.ws, g.status)
    B.pages_copy(g.dims, pools, g.copies, g.status)
    attend()
    fork([2, 4], [0, 3])
    append([3, 0, 20, 1, 1, 31])
    attend()
    free([0, 1, 2, 3, 4, 5])
    torch.cuda.synchronize()
    assert int((g.ref != 0).sum()) == 0 and int((g.table >= 0).sum()) == 0 and g.take_status() == 0


def test_calls_in_a_captured_graph():
    """free, fork and copy captured once and replayed: each replay takes over the parents as they are then."""
    m, g = filled(lens=(40, 16, 40, 0))
    # slot 2 is a beam of slot 0 for now
    m2 = Model(4, 2, 8, 64)
    m2.reserve([40, 16, 0, 0])
    m2.lens[:] = [40, 16, 0, 0]
    _, _ = m2.fork([0], [2])
    g = Map(m2)
    src, dst = i32([1, 0]), i32([2, 3])

    def step():
        B.pages_free(g.dims, g.ptrs, dst, g.status)
        B.pages_fork(g.dims, g.ptrs, src, dst, g.copies, g.ws, g.status)

    def model():
        m2.free([2, 3])
        return m2.fork(src.tolist(), dst.tolist())

    step()
    model()
    g.check(m2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for a in ([0, 0], [1, 1], [0, 1], [-1, 0]):
        src.copy_(i32(a))
        graph.replay()
        code, pairs = model()
        assert g.take_status() == code == 0
        assert g.listed() == [tuple(map(int, p)) for p in pairs]
        g.check(m2)
