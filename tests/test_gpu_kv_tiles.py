"""The tile kernel of omq_kv_attn (requests of more than 512 query rows per kv head) within the
bound of its float16 operands."""
import ctypes

import numpy as np
import pytest
import torch

from tests import kv_common as kc
from tests import kv_kernels as kk
from tests.test_gpu_kv_attn import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def omq(cuda_device):
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


def refill(s, w, x, b=0):
    """Request b's keys (w = 0) or values (1): the rows x [n, Hkv, D]."""
    pos = np.arange(len(x))
    s.kv[b][w] = kk.encode(x.astype(np.float32))
    s.put(s.pool_np, s.table[b, pos // s.page] * s.page + pos % s.page, w, *s.kv[b][w])
    s.pool.copy_(torch.from_numpy(s.pool_np))


NARROW = [(0.01, 2e-4), (0.0, 1e-4), (9e-6, 0.0), (9.075e-4, 1.5e-5), (-9.075e-4, 1.5e-5), (0.0, 1.5e-5), (-0.4, 0.01),
          (0.05, 0.03), (3.0, 0.1), (700.0, 900.0)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mid,spread", NARROW)
def test_value_rows_of_any_spread(omq, cuda_device, mid, spread, D):
    """Values mid +- spread / 2 under equal weights (queries of zeros): no more than the float16
    rounding of each value, whatever its row's step."""
    s = Setup(cuda_device, [600], [520], 1, 1, D, 16, "f16", seed=97)
    rng = np.random.default_rng(97)
    refill(s, 1, mid + spread * (rng.random((1, 1, D)) - 0.5) + np.zeros((600, 1, 1)))
    s.args[0].zero_()
    s.q.zero_()
    for causal in (True, False):
        out = omq.kv_attn(*s.args, s.max_q, causal=causal)
        omq.sync_check()
        kk.check(s, out, causal=causal, every=71)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mid,spread", [(8.6e-3, 1.43e-4), (-8.6e-3, 1.43e-4), (9e-6, 0.0), (0.3, 4.9e-3), (0.0, 0.1), (40.0, 3.0)])
def test_key_rows_of_any_spread(omq, cuda_device, mid, spread, D):
    """Keys mid +- spread / 2 that all queries meet with elements of one sign: the scores, seen in
    the log-sum-exp, are off by no more than the float16 rounding of each key's elements."""
    s = Setup(cuda_device, [600], [520], 1, 1, D, 16, "bf16", seed=101)
    rng = np.random.default_rng(101)
    refill(s, 0, mid + spread * (rng.random((1, 1, D)) - 0.5) + np.zeros((600, 1, 1)))
    s.args[0].fill_(96.0 if abs(mid) < 1 else 0.5)
    s.q.copy_(s.args[0])
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    kk.check(s, out, lse, every=71)


def test_narrow_rows_among_others(omq, cuda_device):
    """Every third row of k and v narrow, keys shared between pairs: rows of both kinds in every
    run of 16 tokens."""
    n = 5000
    s = Setup(cuda_device, [n], [300], 1, 2, 128, 64, "f16", seed=103)
    rng = np.random.default_rng(103)
    for w in range(2):
        x = kc.values(*s.kv[0][w])
        x[::3] = (1e-2 * rng.choice([-1, 1], (len(x[::3]), 1, 1)) + 1e-4 * rng.standard_normal(x[::3].shape))
        refill(s, w, x)
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    kk.check(s, out, lse, every=59)


SHAPES = [  # lens, new, Hkv, G, D, page, dtype; every call has a request of more than 512 rows
    ([520], [513], 1, 1, 128, 16, "f16"),
    ([700, 66, 80, 3], [600, 64, 65, 1], 2, 1, 64, 32, "bf16"),
    ([1200, 20, 300], [130, 16, 17], 2, 4, 128, 48, "f16"),
    ([900, 1, 0, 257], [300, 1, 0, 257], 1, 2, 64, 16, "f16"),
    ([260, 1030], [33, 1025], 1, 1, 128, 128, "bf16"),
    ([129, 75], [74, 75], 1, 7, 128, 64, "f16"),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,new,Hkv,G,D,page,dt", SHAPES)
def test_chunks_and_single_tokens_together(omq, cuda_device, lens, new, Hkv, G, D, page, dt, causal):
    """Requests of either kernel in one call, on both sides of 64 rows."""
    s = Setup(cuda_device, lens, new, Hkv, G, D, page, dt, seed=107 + D)
    out, lse = omq.kv_attn(*s.args, s.max_q, causal=causal, lse=True)
    omq.sync_check()
    kk.check(s, out, lse, causal, every=67)


def split(omq, s):
    """Whether a single request's keys are shared between pairs: its parts need a workspace."""
    assert len(s.lens) == 1
    d, q, pool = s.D, s.args[0], s.pool
    a = omq.KvAttnArgs(omq.KvPool(pool.data_ptr(), pool.shape[0], s.page, s.Hkv, d), 1, s.T, s.Hkv * s.G, q.data_ptr(),
                       s.Hkv * s.G * d, omq._dt(q), s.args[2].data_ptr(), s.args[2].shape[1], s.args[3].data_ptr(),
                       s.args[4].data_ptr(), s.max_q, d ** -0.5, 1, 1 << 40, omq._dt(q), None)
    return omq._lib.omq_kv_attn_workspace_bytes(ctypes.byref(a)) > 0


SHARED = [(600, 600, 20, False), (5000, 520, 1, True)]      # keys, queries, kv heads, shared


@pytest.mark.parametrize("n,new,Hkv,shared", SHARED)
@pytest.mark.parametrize("what", [0, 128])
def test_a_nan_step_reaches_only_rows_that_see_it(omq, cuda_device, n, new, Hkv, shared, what):
    """A NaN step of a key (0) or a value (128) in the last tile of keys but one."""
    s = Setup(cuda_device, [n], [new], Hkv, 1, 64, 16, "f16", seed=109)
    assert split(omq, s) == shared
    clean = omq.kv_attn(*s.args, s.max_q)
    at = n - 200
    page, off = divmod(at, 16)
    cell = s.pool[s.table[0, page], Hkv - 1, 0]
    cell[kc.CELL * 64 + what + 4 * off:kc.CELL * 64 + what + 4 * off + 4] = 255
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    first = at - (n - new)
    assert bool(torch.isnan(out[first:, -1]).all()) and bool(torch.isnan(lse[first:, -1]).all())
    assert torch.equal(out[:first], clean[:first]) and torch.equal(out[:, :-1], clean[:, :-1])


@pytest.mark.parametrize("n,new,Hkv,shared", SHARED)
def test_pages_that_are_not_there(omq, cuda_device, n, new, Hkv, shared):
    """Single pages, and so many in a row that tiles of keys and whole shares are empty, are no keys;
    neither is a table without a page."""
    s = Setup(cuda_device, [n], [new], Hkv, 1, 64, 16, "bf16", seed=113)
    assert split(omq, s) == shared
    pages = n // 16
    hidden = [(0, p) for p in [0, 3, *range(pages // 3, 2 * pages // 3), pages - 1]]
    for (_, p), bad in zip(hidden, [-1, s.pool.shape[0], 2 ** 30, *[-5] * pages]):
        s.args[2][0, p] = bad
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    kk.check(s, out, lse, hidden=hidden, every=131)
    s.args[2].fill_(-1)
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    assert not out.any() and bool((lse == -np.inf).all())


@pytest.mark.parametrize("n,new,Hkv,shared", [(90, 600, 20, False), (90, 600, 1, True)])
def test_more_queries_than_keys_and_rows_behind_the_last(omq, cuda_device, n, new, Hkv, shared):
    """The first rows see nothing; rows of q and out behind the request stay as they were, and a
    NaN there goes nowhere. (The table allows more keys than there are: the keys are shared.)"""
    s = Setup(cuda_device, [n], [new], Hkv, 1, 128, 16, "bf16", seed=127, extra_rows=9)
    table = torch.full((1, 400 if shared else 6), -1, dtype=torch.int32, device=cuda_device)
    table[:, :6] = s.args[2][:, :6]
    s.args[2] = table
    assert split(omq, s) == shared
    s.args[0][-9:] = float("nan")
    out = torch.full_like(s.args[0], 3.0)
    got, lse = omq.kv_attn(*s.args, s.max_q, out=out, lse=True)
    omq.sync_check()
    assert got is out and bool((out[-9:] == 3.0).all())
    kk.check(s, out[:-9], lse[:-9], every=37)


@pytest.mark.parametrize("n,new,Hkv,shared", [(900, 600, 20, False), (5000, 520, 1, True)])
def test_captured_chunks_in_two_graphs(omq, cuda_device, n, new, Hkv, shared):
    """Captured twice, replayed in turn; lengths and queries change between replays."""
    s = Setup(cuda_device, [n], [new], Hkv, 1, 128, 16, "f16", seed=131)
    assert split(omq, s) == shared
    lens = s.args[3].clone()
    graphs, outs = [], []
    omq.kv_attn(*s.args, s.max_q)
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(omq.kv_attn(s.args[0], s.args[1], s.args[2], lens, s.args[4], s.max_q, lse=True))
        graphs.append(g)
    for m in (n, n - 111, 200, 0):
        lens.fill_(m)
        s.args[0].mul_(0.75)
        want = omq.kv_attn(s.args[0], s.args[1], s.args[2], lens, s.args[4], s.max_q, lse=True)
        for g in graphs * 2:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[i], want[i]) for o in outs for i in range(2))
    omq.sync_check()


@pytest.mark.parametrize("D", [64, 128])
def test_query_rows_of_very_different_size(omq, cuda_device, D):
    """Rows of 2^-40 to 2^15 times ordinary ones next to each other, which are staged by powers of
    two of their own; another output type; a given scale; values far from zero."""
    s = Setup(cuda_device, [700], [600], 1, 1, D, 16, "bf16", seed=137, spread=2.0 ** -11, shift=6.0)
    gen = torch.Generator().manual_seed(137)
    e = torch.tensor([-40.0, -12.0, 4.0, 15.0])[torch.randint(0, 4, (600, 1, 1), generator=gen)]
    s.q *= torch.exp2(e).to(s.q.dtype)
    s.args[0].copy_(s.q)
    out, lse = omq.kv_attn(*s.args, s.max_q, scale=0.07, out_dtype=torch.float16, lse=True)
    omq.sync_check()
    assert out.dtype == torch.float16
    kk.check(s, out, lse, scale=0.07, every=7)


@pytest.mark.parametrize("shared", [False, True])
def test_weights_far_below_the_largest(omq, cuda_device, shared):
    """One key that all queries prefer by 2^25.5 over each of 60000 others, whose weights sum to a
    part of the result that float16 outputs show. The values are float16 numbers (steps of 2^-4),
    so the bound on o is: the others' share sum p_j |v_j - o| by what their scores (2 e) and the
    rounding of their weights allow (2^-18.5 as float16 subnormals: 2^-6.5 of each), the float32
    sums, the half step of the output. Weights lost below 2^-25 would lose the whole share."""
    n, D, new, Hkv = 60000, 64, 513, 1 if shared else 80
    s = Setup(cuda_device, [n], [new], 1, 1, D, 64, "f16", seed=139)
    rng = np.random.default_rng(139)
    r0, r1 = rng.standard_normal((2, 1, 1, D)).astype(np.float32)
    k = np.broadcast_to(r0, (n, 1, D)).copy()
    k[7] = r1
    v = 2 + rng.integers(0, 16, (n, 1, D)) / 16
    v[:, :, 0], v[:, :, 1] = 2, 2 + 15 / 16
    v[7] -= 2.5
    refill(s, 0, k)
    refill(s, 1, v)
    assert np.array_equal(kc.values(*s.kv[0][1]), v)
    d = kc.values(*s.kv[0][0])[:, 0]
    d = d[7] - d[8]
    s.q = torch.from_numpy(np.broadcast_to(d * (25.5 * np.log(2) * D ** 0.5 / (d @ d)), (new, 1, D)).copy()).half()
    s.args[0] = s.q.to(cuda_device)
    if not shared:                                        # the same head many times: items for all pairs
        s.args[0] = s.args[0].expand(new, Hkv, D).contiguous()
        s.args[1] = s.pool = s.pool.expand(-1, Hkv, -1, -1).contiguous()
        s.Hkv = Hkv
    assert split(omq, s) == shared
    out = omq.kv_attn(*s.args, s.max_q)
    omq.sync_check()
    assert torch.equal(out, out[:, :1].expand_as(out))
    kd = kc.values(*s.kv[0][0])[:, 0]
    for i in (0, new - 1):
        seen = np.arange(n) <= n - new + i
        o, _, _, ltol = kk.attend_tiles(s.q[i, 0].double().numpy(), kd[seen], v[seen, 0], D ** -0.5, 2.0 ** -11)
        sc = kd[seen] @ s.q[i, 0].double().numpy() * D ** -0.5
        p = np.exp(sc - sc.max()) / np.exp(sc - sc.max()).sum()
        rest = np.arange(len(p)) != 7
        share = p[rest] @ np.abs(v[seen, 0][rest] - o)
        tol = (ltol + 2.0 ** -6.5) * share + (n / 16 + 64) * 2.0 ** -22 * (p @ np.abs(v[seen, 0])) + \
            2.0 ** -11 * (np.abs(o) + share) + 2.0 ** -25
        assert np.all(np.abs(out[i, 0].double().cpu().numpy() - o) <= tol)
        assert np.median(share / tol) > 1.3               # the bound tells the share from nothing


@pytest.mark.parametrize("new,cut,G", [(700, 520, 1), (400, 300, 2)])
def test_max_q_leaves_the_rows_behind_it(omq, cuda_device, new, cut, G):
    """Rows from max_q on stay as they were, the others see what they see without it."""
    s = Setup(cuda_device, [800, 310], [new, 2], 1, G, 64, 16, "f16", seed=149)
    out = torch.full_like(s.args[0], 5.0)
    omq.kv_attn(*s.args, cut, out=out)
    omq.sync_check()
    assert bool((out[cut:new] == 5.0).all())
    s.new = np.array([cut, 2])
    s.lens = np.array([800 - new + cut, 310])
    s.kv = [[tuple(x[:n] for x in w) for w in r] for r, n in zip(s.kv, s.lens)]
    kk.check(s, out, every=61)


def kernel_of(omq, s):
    """The kernel of each request, seen in its log-sum-exp under keys that are all one row whose
    elements, times scale log2(e), lie half a float16 step beside 2^-3, and queries of ones: the tile
    kernel's operand is off by 2^-11 of the score, the row kernel's score by (D + 8) 2^-22."""
    scale = s.D ** -0.5
    kappa = 0.125 * (1 + 0.98 * 2.0 ** -11) / (scale * 1.4426950408889634)
    kv = s.kv, s.pool_np.copy(), s.args[0].clone()
    s.kv = [list(r) for r in s.kv]
    for b, n in enumerate(s.lens):
        refill(s, 0, np.full((int(n), s.Hkv, s.D), kappa), b)
    s.args[0].fill_(1)
    _, lse = omq.kv_attn(*s.args, s.max_q, causal=False, lse=True)
    omq.sync_check()
    tiles = []
    for b, n in enumerate(s.lens):
        score = scale * kc.values(*[x[0, 0] for x in s.kv[b][0]]).sum()
        err = np.abs(lse[int(s.cu[b]):int(s.cu[b + 1])].double().cpu().numpy() - score - np.log(float(n))) / score
        assert err.size == 0 or err.max() < 2.0 ** -13 or err.min() > 2.0 ** -12, (b, err.min(), err.max())
        tiles.append(bool(err.size and err.min() > 2.0 ** -12))
    s.kv, s.pool_np = kv[0], kv[1]
    s.args[0].copy_(kv[2])
    s.pool.copy_(torch.from_numpy(s.pool_np))
    return tiles


@pytest.mark.parametrize("lens,new,Hkv,G,D,dt,tiles", [
    ([512], [512], 8, 1, 128, "bf16", [False]),                     # one short prompt: rows
    ([512], [512], 8, 1, 128, "f16", [False]),
    ([513], [513], 8, 1, 128, "bf16", [True]),                      # a row more
    ([600, 90], [128, 1], 1, 4, 128, "f16", [False, False]),        # 512 rows, and 516
    ([600, 90], [129, 1], 1, 4, 128, "f16", [True, False]),
    ([124] * 39, [124] * 39, 8, 1, 64, "bf16", [False] * 39),
    ([65536], [64], 1, 1, 64, "bf16", [False]),                     # 64 rows at most: rows, always
    ([65536], [65], 1, 1, 64, "bf16", [False]),                     # estimates of 25 us and 32
    ([8192, 700], [16, 17], 4, 4, 128, "f16", [False, False]),      # 25 and 30
    ([65536], [65], 8, 1, 128, "bf16", [False]),                    # 115 and 128
    ([65536], [128], 8, 1, 128, "bf16", [True]),                    # 178 and 128
    ([4096] * 8, [32] * 4 + [16] * 4, 8, 4, 128, "bf16", [True] * 4 + [False] * 4),   # 182 and 74
    ([8192], [200], 8, 1, 128, "f16", [True]),                      # 46 and 30
])
def test_which_kernel_a_request_takes(omq, cuda_device, lens, new, Hkv, G, D, dt, tiles):
    """Both sides of the limits of 64 and 512 rows and of the estimate between them, each within the
    bound of the kernel that it takes."""
    s = Setup(cuda_device, lens, new, Hkv, G, D, 64, dt, seed=151)
    assert kernel_of(omq, s) == tiles
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    kk.check(s, out, lse, every=1000, tiles=tiles)         # the first row of a request and the last
