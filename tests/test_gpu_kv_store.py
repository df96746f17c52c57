"""omq_kv_append and omq_kv_read against the numpy statement of the store: the pool's bytes, the
queries and the values read back must match bit for bit (every operation is one binary32
rounding), with everything that was not to be written left as it was."""
import numpy as np
import pytest
import torch

from tests import kv_common as kc

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def omq(cuda_device):
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


def store(case, q, k, v, cos, sin, sa, so, dl, abits):
    """(q~, (codes, h, z) of k~, of v~) of float32 arrays."""
    if cos is not None:
        q, k = kc.rotate(q, cos, sin), kc.rotate(k, cos, sin)
    if sa is not None:
        q, k = (q / np.repeat(sa, max(1, case["G"]), 0)).astype(np.float32), (k * sa).astype(np.float32)
    if so is not None:
        v = v if dl is None else (v - dl).astype(np.float32)
        v = (v / so).astype(np.float32)
    if abits < 16:
        q = kc.values(*kc.encode(q, 2 ** abits - 1), np.float32)
    return q, kc.encode(k), kc.encode(v)


CASES = [
    dict(T=1, Hkv=1, G=1, D=128, page=16, dt="f32", q_dt="f16", abits=16, rope=True, let=True),
    dict(T=5, Hkv=2, G=4, D=128, page=48, dt="bf16", q_dt="bf16", abits=16, rope=True, let=False),
    dict(T=33, Hkv=3, G=1, D=128, page=16, dt="f16", q_dt="f32", abits=4, rope=True, let=True),
    dict(T=77, Hkv=1, G=8, D=64, page=64, dt="bf16", q_dt="f16", abits=8, rope=True, let=True),
    dict(T=18, Hkv=4, G=7, D=64, page=32, dt="f32", q_dt="f16", abits=2, rope=False, let=False),
    dict(T=300, Hkv=5, G=3, D=128, page=128, dt="f32", q_dt="f16", abits=16, rope=True, let=True),
    dict(T=300, Hkv=8, G=0, D=64, page=16, dt="f16", q_dt="f16", abits=16, rope=True, let=True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T{T}_H{Hkv}x{G}_D{D}_{dt}".format(**c))
def test_store_and_read(omq, cuda_device, case):
    dev = cuda_device
    T, Hkv, G, D, page = (case[n] for n in ("T", "Hkv", "G", "D", "page"))
    Hq = Hkv * G
    rng = np.random.default_rng(T * 7 + D)
    gen = torch.Generator().manual_seed(T + D)
    fused = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen) * torch.exp(
        torch.randn(T, 1, generator=gen))
    fused[T // 2] += 25.0                       # rows far from zero: zero points outside 0 .. 15
    fused[T // 3] = 0.0                         # rows without a range
    fused = fused.to(DT[case["dt"]])
    parts = [fused[:, a * D:b * D].unflatten(1, (b - a, D)) if b > a else None
             for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv))]
    n_pages = -(-T // page) + 3
    slots = rng.permutation(n_pages * page)[:T].astype(np.int32)
    n_pos = 5000
    pos = rng.integers(0, n_pos, T).astype(np.int32)
    skipped = [t for t, s in ((T - 1, -1), (T // 4, n_pages * page), (T // 5, None)) if T > 9]
    if skipped:                                 # no slot, a slot past the pool, a bad position
        slots[skipped[0]], slots[skipped[1]] = -1, n_pages * page
        if case["rope"]:
            pos[skipped[2]] = n_pos
        else:
            slots[skipped[2]] = -5
    live = np.array([t for t in range(T) if t not in skipped])
    sa = so = dl = None
    if case["let"]:
        sa, so = (np.exp(0.4 * rng.standard_normal((Hkv, D))).astype(np.float32) for _ in range(2))
        dl = (0.3 * rng.standard_normal((Hkv, D))).astype(np.float32)
    rope = omq.rope_table(n_pos, D, 10000.0, dev) if case["rope"] else None
    cos = sin = None
    if rope is not None:
        want_cos, want_sin = kc.rope_rows(np.arange(n_pos), D)
        # the device's binary64 functions may differ from numpy's in the last place, which
        # moves a result across a binary32 rounding once in about 2^28
        off = np.abs(rope[0].cpu().numpy() - want_cos).max(), np.abs(rope[1].cpu().numpy() - want_sin).max()
        assert max(off) <= 2.0 ** -24
        cos, sin = (rope[i].cpu().numpy()[np.minimum(pos, n_pos - 1)] for i in (0, 1))
    host = [None if p is None else p.float().numpy() for p in parts]
    wq, wk, wv = store(case, host[0] if G else host[1], host[1], host[2], cos, sin,
                       sa, so, dl, case["abits"] if G else 16)
    pool = np.full((n_pages, Hkv, page // 16, kc.cell_bytes(D)), 0xA5, np.uint8)
    t_pool = torch.from_numpy(pool).to(dev)
    d = lambda a: None if a is None else (torch.from_numpy(a) if isinstance(a, np.ndarray) else a).to(dev)  # noqa: E731
    on_dev = fused.to(dev)
    views = [on_dev[:, a * D:b * D].unflatten(1, (b - a, D)) if b > a else None
             for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv))]
    q_out = torch.full((T, Hq, D), 7.0, dtype=DT[case["q_dt"]], device=dev) if G else None
    got_q = omq.kv_append(t_pool, d(slots), views[1], views[2], q=views[0], positions=d(pos), rope=rope,
                          s_a=d(sa), s_o=d(so), delta_o=d(dl), abits=case["abits"], q_out=q_out)
    k, v = omq.kv_read(t_pool, d(slots), torch.float32)
    torch.cuda.synchronize()
    kc.put(pool, page, np.where(np.isin(np.arange(T), live), slots, -1), 0, *wk)
    kc.put(pool, page, np.where(np.isin(np.arange(T), live), slots, -1), 1, *wv)
    assert np.array_equal(t_pool.cpu().numpy(), pool)
    for got, want in ((k, wk), (v, wv)):
        assert np.array_equal(got.cpu().numpy()[live], kc.values(*want, np.float32)[live])
    if skipped:
        assert not k[skipped[0]].any() and not v[skipped[1]].any()
    if G:
        want = torch.from_numpy(wq.astype(np.float32)).to(DT[case["q_dt"]])
        assert torch.equal(got_q.cpu()[live], want[live])
        if skipped:
            assert bool((got_q[skipped] == 7.0).all())
    k16, _ = omq.kv_read(t_pool, d(slots), torch.float16)
    assert torch.equal(k16.cpu()[live], torch.from_numpy(kc.values(*wk, np.float32)).to(torch.float16)[live])


def test_rows_that_are_not_finite_read_as_nan(omq, cuda_device):
    gen = torch.Generator().manual_seed(3)
    k = torch.randn(6, 2, 128, generator=gen)
    v = torch.randn(6, 2, 128, generator=gen)
    k[0, 0, 5], k[1, 1, 127], v[2, 0, 64], v[3, 1, 0] = np.nan, np.inf, -np.inf, np.nan
    k[4, 0, 0], k[4, 0, 1] = 3e38, -3e38                 # finite, but its range is not
    pool = omq.kv_pool(2, 2, 128, 16, cuda_device)
    slots = torch.arange(6, dtype=torch.int32, device=cuda_device)
    omq.kv_append(pool, slots, k.to(cuda_device), v.to(cuda_device))
    gk, gv = (t.cpu().numpy() for t in omq.kv_read(pool, slots))
    bad_k, bad_v = np.zeros((6, 2), bool), np.zeros((6, 2), bool)
    bad_k[0, 0] = bad_k[1, 1] = bad_k[4, 0] = bad_v[2, 0] = bad_v[3, 1] = True
    for g, x, bad in ((gk, k, bad_k), (gv, v, bad_v)):
        assert np.isnan(g[bad]).all()
        want = kc.values(*kc.encode(x.numpy()), np.float32)
        assert np.array_equal(g[~bad], want[~bad])


def test_slots_beyond_32_bit_byte_offsets(omq, cuda_device):
    """A pool of more than 4 GiB, written and read at its two ends only."""
    page, Hkv = 64, 8
    n_pages = (5 << 30) // (Hkv * page // 16 * 2304)
    pool = omq.kv_pool(n_pages, Hkv, 128, page, cuda_device)
    gen = torch.Generator().manual_seed(4)
    k = torch.randn(4, Hkv, 128, generator=gen)
    slots = torch.tensor([0, 3, n_pages * page - 1, n_pages * page - 40], dtype=torch.int32,
                         device=cuda_device)
    omq.kv_append(pool, slots, k.to(cuda_device), (2 * k).to(cuda_device))
    gk, gv = omq.kv_read(pool, slots)
    assert np.array_equal(gk.cpu().numpy(), kc.values(*kc.encode(k.numpy()), np.float32))
    assert np.array_equal(gv.cpu().numpy(), kc.values(*kc.encode(2 * k.numpy()), np.float32))


def test_cache_holds_what_the_block_calibrates(omq, cuda_device):
    """The block step's fake-quantized q, k and v (4-bit activations, affinity and V / o
    transforms) equal what the store puts in the cache and into q_out, bit for bit."""
    from tests.test_gpu_block import Run
    M, H = 136, 2
    blk = Run(omq, cuda_device, M, H, 160, 0, 4, 4).blk
    qkv = blk.buffer("qkv").view(M, 3, H, 128)
    want = blk.buffer("qqkv").view(M, 3, H, 128)
    pool = omq.kv_pool(3, H, 128, 64, cuda_device)
    slots = torch.arange(M, dtype=torch.int32, device=cuda_device)
    rope = omq.rope_table(M, 128, 10000.0, cuda_device)
    part = lambda n: blk.theta_part(n).clone()  # noqa: E731
    q = omq.kv_append(pool, slots, qkv[:, 1], qkv[:, 2], q=qkv[:, 0], positions=slots, rope=rope,
                      s_a=part("s_a"), s_o=part("s_o"), delta_o=part("delta_o"), abits=4)
    k, v = omq.kv_read(pool, slots, torch.float16)
    assert torch.equal(q, want[:, 0]) and torch.equal(k, want[:, 1]) and torch.equal(v, want[:, 2])
