"""Attention over 8-bit caches at the ends of its inputs' range, against float64 over the
dequantised values.

Bound, element by element, derived: a score of D terms is within (D 2^-23 + 2^-21) A of its
value, A = max_t sum_i |q_i K_ti| / sqrt(d) (codes exact, fp32 sums), so every weight is
within e^that; its exponent (x - m) log2 e is rounded twice at up to 2^7 (2^-16), its fp16
parts keep 2^-22, or 2^-38 of its page's largest weight; sums over N pages and the merges add
N 2^-23 + 2^-19. So an element is within
    (2 (D 2^-23 + 2^-21) A + 2^-15 + N 2^-23 + 2^-19) S + 16 2^-38 R,
S = sum_t w_t |V_t| and R = sum over pages of (largest w) (largest |V|), both over the sum of
weights, and where the result is not far above 2^-126 each addition is within 2^-149."""
import numpy as np
import pytest
import torch

from test_quant_gpu import Cache, i32
from long_context_serving_gb300 import bsattn as B
from long_context_serving_gb300.build import build

pytestmark = pytest.mark.gpu
LOWEST = float(np.finfo(np.float32).min)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build()
    B.lib()


def attend_all(c, g, q, bias=None):
    """out and lse of every block of every unit (g tokens each)."""
    U, nb = c.B * c.Hkv, -(-c.T // g)
    d = c.dims
    d.max_sel_per_unit = d.max_blocks_per_unit = int(nb.max())
    d.max_gather_pages_per_unit = int(nb.max()) * g // 16
    sel = np.where(np.arange(nb.max()) < nb[:, None], np.arange(nb.max()), -1)
    t_g, t_sel, t_cnt = i32([g] * U), i32(sel), i32(nb)
    out = torch.full((c.B, c.G * c.Hkv, c.d), float("nan"), device="cuda")
    lse = torch.full((c.B, c.G * c.Hkv), float("nan"), device="cuda")
    e = None if bias is None else torch.as_tensor(np.ascontiguousarray(bias, dtype=np.float32), device="cuda")
    ws = torch.zeros(B.workspace_size(d) // 4, device="cuda")
    B.sparse_decode_attn(d, q, c.kv, B.HeadCfg(block_tokens=t_g.data_ptr()), t_sel, t_cnt, out, lse, ws, c.status,
                         evict_bias=e)
    torch.cuda.synchronize()
    assert int(c.status) == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def definition(c, u, g, q, bias=None):
    """(out, lse, S, R, A) of unit u in float64; see the module's text."""
    b, h = divmod(u, c.Hkv)
    K, V = c.unit(u)
    t = np.arange(len(K))
    qh = q[b, h * c.G:(h + 1) * c.G].double().cpu().numpy()
    x = qh @ K.T / np.sqrt(c.d)
    A = float((np.abs(qh) @ np.abs(K).T).max()) / np.sqrt(c.d)
    if bias is not None:
        x = x + np.asarray(bias, dtype=np.float32)[u, t // g].astype(np.float64)
    m = x.max(1, keepdims=True)
    w = np.exp(x - m)
    l = w.sum(1, keepdims=True)
    R = np.zeros((len(qh), c.d))
    for p in range(0, len(K), 16):
        R += w[:, p:p + 16].max(1, keepdims=True) * np.abs(V[p:p + 16]).max(0, keepdims=True).max()
    return w @ V / l, (m + np.log(l))[:, 0], w @ np.abs(V) / l, R / l, A


def within(got, want, S, R, A, d, pages, tiny=0.0):
    eps = 2 * (d * 2.0 ** -23 + 2.0 ** -21) * A + 2.0 ** -15 + pages * 2.0 ** -23 + 2.0 ** -19
    return (np.abs(got - want) <= eps * S + 16 * 2.0 ** -38 * R + tiny).all()


PLANS = {"cluster": (4, [300, 100]), "workspace": (8, [6000, 5000, 4700])}


@pytest.mark.parametrize("q32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("plan", sorted(PLANS))
def test_block_logits_of_the_largest_magnitudes(plan, kind, q32):
    """Every finite block logit counts, the type's lowest too: a unit whose blocks are all at it has
    the mean of its values and its logit plus log of its tokens as lse."""
    Hkv, lens = PLANS[plan]
    rng = np.random.default_rng(51)
    c = Cache(lens, Hkv, 64, kind, rng, G=2, q32=q32)
    g = 32
    U, nb = c.B * Hkv, -(-c.T // g)
    bias = np.zeros((U, int(nb.max())), np.float32)
    bias[0] = LOWEST                                   # nothing left but lowest
    bias[1] = LOWEST                                   # one block left
    bias[1, 1] = 0.5
    bias[2] = LOWEST                                   # lowest beside dropped
    bias[2, ::2] = -np.inf
    bias[3, 2] = -LOWEST                               # one block above all
    bias[4] = np.linspace(LOWEST, -LOWEST, int(nb.max()))
    bias[5] = -3e38
    q = torch.as_tensor(rng.normal(size=(c.B, 2 * Hkv, 64)).astype(np.float32), device="cuda")
    q = q if q32 else q.bfloat16()
    out, lse = attend_all(c, g, q, bias)
    for u in range(U):
        b, h = divmod(u, Hkv)
        want, want_l, S, R, A = definition(c, u, g, q, bias)
        assert within(out[b, 2 * h:2 * h + 2], want, S, R, A, 64, nb[u] * g / 16), u
        tol = (64 * 2.0 ** -23 + 2.0 ** -21) * A + 2.0 ** -15 + nb[u] * 2.0 ** -22 + 2.0 ** -19
        # (a logit of 2^127 and the score beside it: the sum's last place, twice)
        assert (np.abs(lse[b, 2 * h:2 * h + 2] - want_l) <= tol + 2.0 ** -23 * np.abs(want_l)).all(), u


@pytest.mark.parametrize("exponent", [-126, -122, -118])
@pytest.mark.parametrize("d", [64, 128])
def test_v_scales_near_the_smallest_normal(d, exponent):
    """INT8 page scales are any fp32 from 2^-126 up: no bit of them is lost on the way. The same
    cache with its V scales 2^60 larger gives the same results, 2^60 larger, but for what is
    rounded below 2^-126: each page's sum, rescaling and merge by half of 2^-149, and with it the
    last place of the result."""
    rng = np.random.default_rng(52)
    c = Cache([100, 700], 2, d, "int8", rng, G=3)
    sc = (2.0 ** exponent * rng.uniform(1, 2, c.n_pages)).astype(np.float32)
    c.vs.copy_(torch.as_tensor(sc))
    q = torch.as_tensor(rng.normal(size=(2, 6, d)).astype(np.float32), device="cuda").bfloat16()
    out, _ = attend_all(c, 32, q)
    low = (4 * 44 + 64) * 2.0 ** -149                # 44 pages
    for u in range(4):
        b, h = divmod(u, 2)
        want, _, S, R, A = definition(c, u, 32, q)
        assert within(out[b, 3 * h:3 * h + 3], want, S, R, A, d, -(-c.T[u] // 16), tiny=low), u
    c.vs.mul_(2.0 ** 60)
    big, _ = attend_all(c, 32, q)
    big *= 2.0 ** -60
    assert (np.abs(out - big) <= 2.0 ** -22 * np.abs(big) + low).all() and np.abs(big).max() > 2.0 ** -122


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("order", ["falling", "rising", "mixed"])
def test_small_weights_of_pages_with_large_scales(order, kind):
    """Blocks whose weights fall by e^-11 each while their V scales grow by 2^16 each count alike:
    the V products keep a page's weights relative to that page's largest."""
    rng = np.random.default_rng(53)
    c = Cache([640, 640], 1, 64, kind, rng, G=4)
    g, nb = 32, 20
    step = {"falling": np.arange(nb) % 8, "rising": 7 - np.arange(nb) % 8, "mixed": rng.integers(0, 8, nb)}[order]
    bias = np.tile(-11.0 * step, (2, 1)).astype(np.float32)
    vs = c.vs.cpu().numpy()
    for u in range(2):
        pages = c.table[u, :nb * 2]
        vs[pages] *= np.exp2(16.0 * np.repeat(step, 2) - 60).astype(np.float32)
    c.vs.copy_(torch.as_tensor(vs))
    q = torch.as_tensor(rng.normal(size=(2, 4, 64)).astype(np.float32), device="cuda").bfloat16()
    out, _ = attend_all(c, g, q, bias)
    for u in range(2):
        want, _, S, R, A = definition(c, u, g, q, bias)
        assert within(out[u], want, S, R, A, 64, nb * 2), u
