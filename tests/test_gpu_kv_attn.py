"""omq_kv_attn against the binary64 attention over the stored values, element by element within
the error bound of tests/kv_common.py:attend (derived there, before any run): every shape class
the entry point takes (single rows, drafted tokens, chunks, whole prompts; ragged lengths from
0 on; pages that end inside a tile; rows without a key), with the pool's unused slots full of
NaN steps."""
import numpy as np
import pytest
import torch

from tests import kv_common as kc

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def omq(cuda_device):
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


class Setup:
    """Requests with lens keys and new queries each over a shuffled table; slots no request owns
    (and those behind a request's last token) hold 0xFF bytes: codes 15, steps NaN."""

    def __init__(self, dev, lens, new, Hkv, G, D, page, dt, seed=0, far=None, spread=1.0, extra_rows=0,
                 shift=0.0):
        rng = np.random.default_rng(seed)
        self.lens, self.new = np.asarray(lens), np.asarray(new)
        self.Hkv, self.G, self.D, self.page = Hkv, G, D, page
        need = -(-np.maximum(self.lens, 0) // page)
        width = max(1, int(need.max()) + 1)
        n_pages = int(need.sum()) + 2
        ids = rng.permutation(n_pages)
        self.table = np.full((len(lens), width), -1, np.int32)
        self.kv = []
        pool = np.full((n_pages, Hkv, page // 16, kc.cell_bytes(D)), 255, np.uint8)
        at = 0
        for b, n in enumerate(self.lens):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
            k = rng.standard_normal((n, Hkv, D)) * np.exp(0.5 * rng.standard_normal((Hkv, D))) * spread
            v = rng.standard_normal((n, Hkv, D)) * np.exp(rng.standard_normal((n, 1, 1))) + shift
            rows = [kc.encode(x.astype(np.float32)) for x in (k, v)]
            pos = np.arange(n)
            slots = self.table[b, pos // page] * page + pos % page
            for w in range(2):
                self.put(pool, slots, w, *rows[w])
            self.kv.append(rows)
        self.cu = np.concatenate(([0], np.cumsum(self.new))).astype(np.int32)
        self.T = int(self.cu[-1]) + extra_rows
        gen = torch.Generator().manual_seed(seed)
        self.q = torch.randn(max(self.T, 1), Hkv * G, D, generator=gen).to(DT[dt])
        if far is not None:                       # rows of very different size
            self.q *= torch.exp2(torch.randint(-far, far, (max(self.T, 1), Hkv * G, 1), generator=gen)).to(self.q.dtype)
        self.dev, self.pool_np = dev, pool
        self.pool = torch.from_numpy(pool).to(dev)
        i = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)  # noqa: E731
        self.args = [self.q.to(dev), self.pool, i(self.table), i(self.lens), i(self.cu)]
        self.max_q = max(1, int(self.new.max()))

    def put(self, pool, slots, w, c, h, z):
        """kc.put, vectorised."""
        D, half = self.D, kc.CELL * self.D // 2
        p, off = np.divmod(slots, self.page)
        cell, r = np.divmod(off, kc.CELL)
        code = c.astype(np.uint8)
        by = code[..., 0::2] | (code[..., 1::2] << 4)
        codes = pool[..., w * half:(w + 1) * half].reshape(*pool.shape[:3], kc.CELL, D // 2)
        codes[p, :, cell, r] = by
        pool[..., w * half:(w + 1) * half] = codes.reshape(*pool.shape[:3], half)
        for off_, x, t in ((0, h, np.float32), (64, z, np.int32)):
            a = 2 * half + 128 * w + off_
            m = np.ascontiguousarray(pool[..., a:a + 64]).view(t)
            m[p, :, cell, r] = x[..., 0].astype(t)
            pool[..., a:a + 64] = m.view(np.uint8).reshape(*pool.shape[:3], 64)

    def check(self, out, lse=None, causal=True, scale=None, rows=None, hidden=(), far=None, tiny=-25):
        """Every row (or every `rows`-th of a request) of every head against the statement.
        hidden: (request, page index) pairs whose table entries are not pages."""
        scale = self.D ** -0.5 if scale is None else scale
        eps = torch.finfo(out.dtype).eps / 2
        got = out.double().cpu().numpy()
        got_l = None if lse is None else lse.double().cpu().numpy()
        worst = 0.0
        # a request of more than 32 query rows per kv head takes k and v as float16 operands
        step = [2.0 ** -11 if n * self.G > 32 else 0.0 for n in self.new]
        for b in range(len(self.lens)):
            n, m = int(self.lens[b]), int(self.new[b])
            there = np.ones(n, bool)
            for rb, pg in hidden:
                if rb == b:
                    there[pg * self.page:(pg + 1) * self.page] = False
            pick = range(m) if rows is None else sorted({0, m - 1, *range(0, m, rows)} if m else ())
            for i in pick:
                seen = there & (np.arange(n) <= n - m + i) if causal else there
                t = int(self.cu[b]) + i
                for h in range(self.Hkv * self.G):
                    kh = h // self.G
                    (a, ah, az), (c, ch, cz) = self.kv[b]
                    o, l, tol, ltol = kc.attend(self.q[t, h].double().numpy(), a[:, kh], ah[:, kh], az[:, kh],
                                                c[:, kh], ch[:, kh], cz[:, kh], seen, scale, eps, step[b], far, tiny)
                    err = np.abs(got[t, h] - o)
                    assert np.all(err <= tol), (b, i, h, float((err - tol).max()), float(err.max()))
                    worst = max(worst, float((err / np.maximum(tol, 1e-30)).max()))
                    if got_l is not None:
                        assert (got_l[t, h] == l) if np.isinf(l) else abs(got_l[t, h] - l) <= ltol, (b, i, h)
        return worst


SMALL = [  # lens, new, Hkv, G, D, page, dtype
    ([1], [1], 1, 1, 128, 16, "f16"),
    ([0, 1, 2], [0, 1, 1], 2, 1, 64, 16, "bf16"),
    ([15, 16, 17, 63, 64, 65], [1] * 6, 2, 4, 128, 16, "bf16"),
    ([47, 48, 49, 96, 200, 1], [1] * 6, 1, 8, 128, 48, "f16"),
    ([130, 7, 300, 257], [1] * 4, 3, 7, 64, 64, "f16"),
    ([1023, 31], [1, 1], 1, 3, 128, 128, "bf16"),
    ([5, 64, 130], [5, 5, 5], 2, 2, 64, 32, "f16"),
    ([5, 64, 130, 9], [3, 1, 8, 0], 2, 4, 128, 16, "bf16"),
    ([20, 33, 150], [20, 17, 40], 1, 1, 128, 16, "f16"),
    ([129, 300], [129, 130], 2, 4, 128, 64, "bf16"),
    ([260, 140, 3], [259, 33, 3], 1, 7, 64, 48, "f16"),
    ([600], [1], 2, 16, 128, 64, "bf16"),
    ([400, 128], [70, 128], 1, 16, 64, 16, "bf16"),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,new,Hkv,G,D,page,dt", SMALL)
def test_attention(omq, cuda_device, lens, new, Hkv, G, D, page, dt, causal):
    s = Setup(cuda_device, lens, new, Hkv, G, D, page, dt, seed=len(lens) + D)
    out, lse = omq.kv_attn(*s.args, s.max_q, causal=causal, lse=True)
    omq.sync_check()
    s.check(out, lse, causal, rows=None if sum(new) * Hkv * G < 400 else 13)


@pytest.mark.parametrize("lens,new,Hkv,G,D,page,dt", [
    ([4099, 2000], [1, 1], 2, 4, 128, 64, "bf16"),
    ([20011], [1], 1, 8, 128, 16, "f16"),
    ([9000], [4], 1, 2, 64, 128, "f16"),
    ([3000, 5], [700, 5], 1, 4, 128, 64, "bf16"),
    ([2048], [2048], 2, 1, 128, 16, "bf16"),
    ([1500, 1411, 2047], [500, 1, 257], 1, 2, 64, 32, "f16")])
def test_long_contexts(omq, cuda_device, lens, new, Hkv, G, D, page, dt):
    s = Setup(cuda_device, lens, new, Hkv, G, D, page, dt, seed=7)
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    s.check(out, lse, rows=97)


@pytest.mark.parametrize("n_req,Hkv,G,new,wide", [(40, 8, 1, 1, 9600), (150, 3, 6, 2, 12000),
                                                  (300, 2, 1, 1, 9000)])
def test_ragged_requests_under_a_wide_table(omq, cuda_device, n_req, Hkv, G, new, wide):
    """Lengths far below what the table allows, one far above the others: the blocks share one
    line of all requests' runs (300 requests: found over several chunks of the block)."""
    rng = np.random.default_rng(n_req)
    lens = rng.integers(new, 90, n_req)
    lens[3], lens[n_req - 2] = 3000, 0
    cnt = np.minimum(np.full(n_req, new), lens)
    s = Setup(cuda_device, lens, cnt, Hkv, G, 64, 16, "f16", seed=5)
    table = torch.full((n_req, wide // 16), -1, dtype=torch.int32, device=cuda_device)
    table[:, :s.table.shape[1]] = s.args[2]
    s.args[2] = table
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    s.check(out, lse)


@pytest.mark.parametrize("new", [1, 6, 150])
def test_other_types_scales_and_sizes(omq, cuda_device, new):
    """Output of another type, a given scale, queries of very different size, values far from
    zero (zero points outside the codes' range), peaked scores."""
    s = Setup(cuda_device, [200, 333], [new, new], 2, 2, 128, 16, "bf16", seed=11, far=3, spread=2.0, shift=6.0)
    out, lse = omq.kv_attn(*s.args, s.max_q, scale=0.2, out_dtype=torch.float16, lse=True)
    omq.sync_check()
    assert out.dtype == torch.float16
    s.check(out, lse, scale=0.2, rows=11)


@pytest.mark.parametrize("new", [1, 40, 300])
def test_missing_pages_hold_no_keys(omq, cuda_device, new):
    s = Setup(cuda_device, [300, 320, 301], [new, new, new], 2, 1, 64, 32, "f16", seed=13)
    hidden = [(0, 2), (1, 0), (1, 9), *[(2, p) for p in range(10)]]
    for (b, p), bad in zip(hidden, [-1, s.pool.shape[0], 2 ** 30, *[-5] * 10]):
        s.args[2][b, p] = bad
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    s.check(out, lse, hidden=hidden, rows=17)
    mine = slice(int(s.cu[2]), int(s.cu[3]))
    assert not out[mine].any() and bool((lse[mine] == -np.inf).all())


@pytest.mark.parametrize("new", [1, 30, 200])
def test_rows_without_keys_and_rows_behind_the_last(omq, cuda_device, new):
    """A request with more queries than keys: its first rows see nothing. Rows of q and out
    behind the last request stay as they were, and a NaN there goes nowhere."""
    s = Setup(cuda_device, [max(1, new // 2), 90], [new, new], 2, 2, 128, 16, "bf16", seed=17, extra_rows=9)
    s.lens = s.lens.copy()
    s.args[0][-9:] = float("nan")
    out = torch.full_like(s.args[0], 3.0)
    got, lse = omq.kv_attn(*s.args, s.max_q, out=out, lse=True)
    omq.sync_check()
    assert got is out and bool((out[-9:] == 3.0).all())
    s.check(out[:-9], lse[:-9], rows=7)


@pytest.mark.parametrize("new", [1, 64])
def test_nan_keys_and_values_reach_only_rows_that_see_them(omq, cuda_device, new):
    s = Setup(cuda_device, [100, 80], [new, min(new, 80)], 1, 2, 128, 16, "f16", seed=19)
    clean = omq.kv_attn(*s.args, s.max_q)
    half = kc.CELL * 64
    for pos, at in ((99, 2 * half), (70, 2 * half + 128)):          # a key step, a value step
        page, off = divmod(pos, 16)
        cell = s.pool[s.table[0, page], 0, 0]
        cell[at + 4 * off: at + 4 * off + 4] = 255
    out = omq.kv_attn(*s.args, s.max_q)
    omq.sync_check()
    first = 70 - (100 - new)                                        # the first row that sees one
    assert bool(torch.isnan(out[max(first, 0):new]).all())
    assert torch.equal(out[:max(first, 0)], clean[:max(first, 0)])
    assert torch.equal(out[new:], clean[new:])


def test_strided_queries_and_repeatability(omq, cuda_device):
    for new in (1, 5, 300):
        s = Setup(cuda_device, [400, 77, 310], [new, min(new, 77), new], 2, 4, 128, 64, "bf16", seed=23)
        q = s.args[0]
        wide = torch.full((q.shape[0], q.shape[1] * 128 + 256), float("nan"), dtype=q.dtype, device=q.device)
        wide[:, 128:128 + q.shape[1] * 128] = q.flatten(1)
        view = wide[:, 128:128 + q.shape[1] * 128].unflatten(1, (q.shape[1], 128))
        want = omq.kv_attn(*s.args, s.max_q)
        for _ in range(3):
            assert torch.equal(omq.kv_attn(view, *s.args[1:], s.max_q), want)


def test_max_q_cuts_a_request(omq, cuda_device):
    for new, cut in ((7, 3), (300, 140)):
        s = Setup(cuda_device, [400, 310], [new, 2], 1, 2, 64, 16, "f16", seed=29)
        out = torch.full_like(s.args[0], 5.0)
        omq.kv_attn(*s.args, cut, out=out)
        assert bool((out[cut:new] == 5.0).all())


def test_pool_beyond_32_bit_byte_offsets(omq, cuda_device):
    page, Hkv = 64, 8
    n_pages = (5 << 30) // (Hkv * page // 16 * 2304)
    big = omq.kv_pool(n_pages, Hkv, 128, page, cuda_device)
    for new in (1, 100):
        s = Setup(cuda_device, [130, 190], [new, new], Hkv, 1, 128, page, "bf16", seed=31)
        n = s.pool.shape[0]
        big[n_pages - n:] = s.pool
        table = torch.where(s.args[2] >= 0, s.args[2] + (n_pages - n), s.args[2]).int()
        got = omq.kv_attn(s.args[0], big, table, s.args[3], s.args[4], s.max_q)
        assert torch.equal(got, omq.kv_attn(*s.args, s.max_q))


@pytest.mark.parametrize("D,G,dt", [(128, 4, "bf16"), (64, 2, "f16"), (128, 1, "f16")])
def test_requests_of_64_and_65_rows(omq, cuda_device, D, G, dt):
    """Both sides of the row count at which a request changes its kernel, together in one call;
    G = 4 has no request of 65 rows, but of 64 and 68."""
    s = Setup(cuda_device, [700, 65, 1200, 66, 90], [64 // G, 64 // G + 1, 64 // G + 1, 64 // G, 1], 2, G, D, 16, dt,
              seed=37 + G)
    for causal in (True, False):
        out, lse = omq.kv_attn(*s.args, s.max_q, causal=causal, lse=True)
        omq.sync_check()
        s.check(out, lse, causal, rows=9)


@pytest.mark.parametrize("lens,new,Hkv,G,D", [
    ([5000], [300], 1, 2, 128),          # one request: its keys shared by many pairs
    ([2600, 140, 2500], [260, 140, 1], 1, 2, 64),
    ([4097, 0, 130], [80, 0, 130], 2, 1, 128),
    ([900, 1300], [700, 1100], 1, 1, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_keys_shared_between_pairs(omq, cuda_device, lens, new, Hkv, G, D, causal):
    """Few row tiles under long contexts; a request far shorter than the table, whose later
    shares are empty; first rows that see only the first shares. Twice, to the bit."""
    s = Setup(cuda_device, lens, new, Hkv, G, D, 32, "bf16", seed=41)
    out, lse = omq.kv_attn(*s.args, s.max_q, causal=causal, lse=True)
    again, lse2 = omq.kv_attn(*s.args, s.max_q, causal=causal, lse=True)
    omq.sync_check()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    s.check(out, lse, causal, rows=83)


def test_shared_keys_missing_pages_nan_and_empty_rows(omq, cuda_device):
    """More queries than keys in a request whose keys are shared; pages that are not there make
    whole shares empty; a NaN key in the last share reaches only the rows that see it."""
    s = Setup(cuda_device, [4000, 30], [200, 200], 1, 1, 128, 16, "f16", seed=43)
    hidden = [(0, p) for p in range(40, 200)]
    for b, p in hidden:
        s.args[2][b, p] = -1
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    s.check(out, lse, hidden=hidden, rows=29)
    assert not out[200:370].any() and bool((lse[200:370] == -np.inf).all())
    page, off = divmod(3950, 16)
    cell = s.pool[s.table[0, page], 0, 0]
    cell[2 * kc.CELL * 64 + 4 * off: 2 * kc.CELL * 64 + 4 * off + 4] = 255
    bad = omq.kv_attn(*s.args, s.max_q)
    omq.sync_check()
    first = 3950 - (4000 - 200)
    assert bool(torch.isnan(bad[first:200]).all())
    assert torch.equal(bad[:first], out[:first]) and torch.equal(bad[200:], out[200:])


@pytest.mark.parametrize("n_req", [40, 600, 1100])
def test_one_chunk_among_many_single_tokens(omq, cuda_device, n_req):
    """A step of a serving batch: single tokens, two chunks at any place of the batch (found
    over several rounds of the block's scan), requests without new tokens."""
    rng = np.random.default_rng(n_req)
    lens = rng.integers(1, 40, n_req)
    new = rng.integers(0, 2, n_req)
    for at, (n, m) in zip((n_req // 3, n_req - 1), ((700, 90), (260, 150))):
        lens[at], new[at] = n, m
    s = Setup(cuda_device, lens.tolist(), new.tolist(), 1, 1, 64, 16, "bf16", seed=47, extra_rows=5)
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    n = int(s.cu[-1])
    s.check(out[:n], lse[:n], rows=37)


@pytest.mark.parametrize("n,new,G,D,dt", [(70, 1, 4, 128, "bf16"), (300, 1, 1, 64, "f16"), (150, 9, 2, 128, "f16"),
                                          (200, 90, 1, 128, "bf16"), (900, 1, 4, 128, "f16")])
def test_constant_value_rows_among_others(omq, cuda_device, n, new, G, D, dt):
    """Value rows that are constant, or nearly, have steps of 1e-8 and zero points of up to 2^30:
    beside ordinary rows their weights are below float16's, their values are not."""
    s = Setup(cuda_device, [n, n - 1], [new, new], 1, G, D, 16, dt, seed=53)
    rng = np.random.default_rng(53)
    for b, m in enumerate(s.lens):
        pos = np.arange(b, m, 5)
        x = np.broadcast_to(rng.choice([5.0, -3.0, 0.25, 8.0, -0.001], (len(pos), 1, 1)), (len(pos), 1, D))
        x = (x + rng.choice([0.0, 2e-6, 1e-4], (len(pos), 1, 1)) * rng.standard_normal((len(pos), 1, D))).astype(np.float32)
        c, h, z = kc.encode(x)
        for have, got in zip(s.kv[b][1], (c, h, z)):
            have[pos] = got
        s.put(s.pool_np, s.table[b, pos // 16] * 16 + pos % 16, 1, c, h, z)
    s.pool.copy_(torch.from_numpy(s.pool_np))
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    s.check(out, lse, rows=11, far=64)


def test_side_stream_owns_what_the_call_allocates(omq, cuda_device):
    """With stream=, results and workspace belong to that stream: while the current stream is
    busy with memory it has already given back, calls on the side stream do not get that memory."""
    s = Setup(cuda_device, [5000, 3000, 900], [3, 3, 3], 2, 4, 128, 64, "bf16", seed=59)
    want = omq.kv_attn(*s.args, s.max_q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        busy = [torch.empty(1 << 20, device=cuda_device) for _ in range(12)]
        torch.cuda._sleep(2_000_000)
        for t in busy:
            t.fill_(float("nan"))
        del t, busy                                         # still being written by this stream
        got = [omq.kv_attn(*s.args, s.max_q, stream=side) for _ in range(3)]
        side.synchronize()
        assert all(torch.equal(g, want) for g in got)
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got)


def test_two_streams_at_once(omq, cuda_device):
    """Calls that overlap on two streams, single tokens and chunks with shared keys, each with its
    own workspace: the results of the same calls alone."""
    a = Setup(cuda_device, [9000, 5000], [1, 4], 2, 4, 128, 64, "bf16", seed=61)
    b = Setup(cuda_device, [6000, 700], [200, 300], 2, 4, 128, 64, "bf16", seed=67)
    want = [omq.kv_attn(*s.args, s.max_q) for s in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate((a, b)):
            got[i].append(omq.kv_attn(*s.args, s.max_q, stream=streams[i]))
    torch.cuda.synchronize()
    omq.sync_check()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])


def test_captured_chunks_and_a_second_graph(omq, cuda_device):
    """Chunks with shared keys captured twice in two graphs, replayed in turn while eager calls run
    between them; lengths and queries change between replays."""
    s = Setup(cuda_device, [4000, 300], [200, 100], 1, 2, 128, 16, "f16", seed=71)
    lens = s.args[3].clone()
    graphs, outs = [], []
    omq.kv_attn(*s.args, s.max_q)
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(omq.kv_attn(s.args[0], s.args[1], s.args[2], lens, s.args[4], s.max_q))
        graphs.append(g)
    for n in (4000, 3111, 200):
        lens.copy_(torch.tensor([n, 300], dtype=torch.int32))
        s.args[0].mul_(0.75)
        want = omq.kv_attn(s.args[0], s.args[1], s.args[2], lens, s.args[4], s.max_q)
        for g in graphs * 2:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    omq.sync_check()


@pytest.mark.parametrize("new,G,D,dt", [(1, 2, 128, "f16"), (5, 4, 64, "f16"), (90, 1, 128, "f16")])
def test_many_weights_far_below_the_largest(omq, cuda_device, new, G, D, dt):
    """One key that all queries prefer by 2^25.5 over each of 60000 others, whose weights sum to a
    part of the result that float16 outputs show. The bound: the others' share of o may change
    by what their scores and the rounding of their weights (the first one's is exact) allow,
    (4 e_s + 2^-11) sum p_j |v_j - o|; the float32 sums, n/16 + 64 of terms p h (c + |z|); the
    output's half step. Weights below float16's numbers would lose the whole share."""
    n = 60000
    s = Setup(cuda_device, [n], [new], 1, G, D, 64, dt, seed=73, shift=2.0)
    rng = np.random.default_rng(73)
    r0, r1 = rng.standard_normal((2, 1, 1, D)).astype(np.float32)
    k = np.broadcast_to(r0, (n, 1, D)).copy()
    k[7] = r1
    v = np.full((n, 1, D), 2.0, np.float32) + rng.random((n, 1, D), np.float32)
    v[7] -= 2.5
    pos = np.arange(n)
    for w, x in enumerate((k, v)):
        rows = kc.encode(x)
        s.put(s.pool_np, s.table[0, pos // 64] * 64 + pos % 64, w, *rows)
        s.kv[0][w] = rows
    d = kc.values(*s.kv[0][0])[:, 0]
    d = d[7] - d[8]
    s.q = torch.from_numpy(np.broadcast_to(d * (25.5 * np.log(2) * D ** 0.5 / (d @ d)), (new, G, D)).copy()).half()
    s.args[0] = s.q.to(cuda_device)
    s.pool.copy_(torch.from_numpy(s.pool_np))
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    s.check(out, lse, rows=31, far=64, tiny=-40 if new * G <= 64 else -32)
    (a, ah, az), (c, ch, cz) = s.kv[0]
    seen = pos <= n - new
    o, _, _, ltol = kc.attend(s.q[0, 0].double().numpy(), a[:, 0], ah[:, 0], az[:, 0], c[:, 0], ch[:, 0], cz[:, 0],
                              seen, D ** -0.5, 2.0 ** -12, 0.0 if new * G <= 64 else 2.0 ** -11)
    val = kc.values(c, ch, cz)[seen, 0]
    sc = kc.values(a, ah, az)[seen, 0] @ s.q[0, 0].double().numpy() * D ** -0.5
    p = np.exp(sc - sc.max()) / np.exp(sc - sc.max()).sum()
    rest = np.arange(len(p)) != 7
    share = p[rest] @ np.abs(val[rest] - o)
    sums = (n / 16 + 64) * 2.0 ** -22 * (p @ (ch * (c + np.abs(cz)))[seen, 0])
    tol = (2 * ltol + 2.0 ** -11) * share + sums + 2.0 ** -11 * (np.abs(o) + share) + 2.0 ** -25
    if new * G > 64:
        tol = tol + 2.0 ** -11 * np.abs(val).max(0)       # v itself, rounded to float16
    assert np.all(np.abs(out[0, 0].double().cpu().numpy() - o) <= tol)
    if new * G <= 64:
        assert np.median(share / tol) > 1.3               # the bound tells the share from nothing


@pytest.mark.parametrize("n_req,Hkv,G,new,D", [(1, 32, 1, 1, 128), (9, 8, 2, 1, 64), (20, 3, 4, 2, 128), (12, 8, 3, 5, 64),
                                               (50, 4, 1, 1, 128), (3, 1, 8, 7, 128)])
def test_shares_joined_by_their_blocks(omq, cuda_device, n_req, Hkv, G, new, D):
    """Two to eight blocks an item; requests far shorter than the table, whose later shares are
    empty, of one token, without any, or without a query."""
    rng = np.random.default_rng(n_req)
    lens = rng.integers(1, 700, n_req)
    lens[0] = 1500
    lens[1::4] = rng.integers(0, 3, len(lens[1::4]))
    new = np.full(n_req, new)
    new[2::5] = 0
    s = Setup(cuda_device, lens.tolist(), new.tolist(), Hkv, G, D, 16, "f16", seed=79)
    for causal in (True, False):
        out, lse = omq.kv_attn(*s.args, s.max_q, causal=causal, lse=True)
        omq.sync_check()
        s.check(out, lse, causal, rows=3)


@pytest.mark.parametrize("new,cut,G", [(7, 3, 2), (300, 140, 2), (40, 33, 4)])
def test_rows_below_max_q_do_not_depend_on_it(omq, cuda_device, new, cut, G):
    """Rows that a smaller max_q leaves in see the keys they see without it."""
    s = Setup(cuda_device, [400, 310], [new, 2], 1, G, 64, 16, "f16", seed=83)
    out = torch.zeros_like(s.args[0])
    omq.kv_attn(*s.args, cut, out=out)
    omq.sync_check()
    s.new = np.array([cut, 2])                              # the rows to look at, and their keys
    s.lens = np.array([400 - new + cut, 310])
    s.kv = [[tuple(x[:n] for x in w) for w in r] for r, n in zip(s.kv, s.lens)]
    s.check(out, rows=9)

