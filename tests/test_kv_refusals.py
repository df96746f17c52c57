"""Host-side refusals of the 4-bit paged cache's entry points (no CUDA work is enqueued) and the
checks of their Python binding, on the CPU; and the plain statements of tests/kv_common.py
against each other."""
import ctypes

import numpy as np
import pytest
import torch

from tests import kv_common as kc

P = 1 << 20                      # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def omq():
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


NULL, SHAPE, DTYPE, ALIGN, BITS = 1, 2, 3, 4, 5


def pool_of(omq, **kw):
    return omq.KvPool(**{**dict(data=P, n_pages=10, page=64, Hkv=2, D=128), **kw})


BAD_POOLS = [(dict(data=None), NULL), (dict(data=P + 8), ALIGN), (dict(D=96), SHAPE),
             (dict(page=24), SHAPE), (dict(page=0), SHAPE), (dict(page=8192), SHAPE),
             (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 26), SHAPE), (dict(Hkv=0), SHAPE)]


def test_cell_bytes(omq):
    assert omq.kv_cell_bytes(128) == kc.cell_bytes(128) == 2304
    assert omq.kv_cell_bytes(64) == kc.cell_bytes(64) == 1280
    assert omq.kv_cell_bytes(96) == 0 and omq.kv_cell_bytes(-1) == 0


def plan_args(omq, **kw):
    d = dict(lens=P, new_tokens=P, n_req=4, table=P, width=8, page=64, free_pages=P, n_pages=32,
             n_free=P, lens_out=P, n_free_out=P, cu=P, slots=P, positions=P, requests=P,
             capacity=16)
    return omq.KvPlanArgs(**{**d, **kw})


@pytest.mark.parametrize("kw,want", [
    *[({n: None}, NULL) for n in ("lens", "new_tokens", "table", "free_pages", "n_free",
                                  "lens_out", "n_free_out", "cu", "slots", "positions",
                                  "requests")],
    (dict(n_req=0), SHAPE), (dict(n_req=65537), SHAPE), (dict(page=17), SHAPE),
    (dict(page=8192), SHAPE), (dict(width=0), SHAPE), (dict(width=1 << 25), SHAPE),
    (dict(n_pages=0), SHAPE), (dict(capacity=0), SHAPE), (dict(capacity=1 << 31), SHAPE)])
def test_plan_refuses(omq, kw, want):
    assert omq._lib.omq_kv_plan(ctypes.byref(plan_args(omq, **kw)), None) == want


def append_args(omq, pool=None, **kw):
    d = dict(pool=pool or pool_of(omq), T=3, Hq=4, dt=omq.OMQ_BF16, q=P, k=P, v=P, q_ld=512,
             k_ld=256, v_ld=256, slots=P, positions=P, rope=P, n_pos=100, s_a=None, s_o=None,
             delta_o=None, abits=16, q_out=P, q_dt=omq.OMQ_F16)
    return omq.KvAppendArgs(**{**d, **kw})


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(q_out=None), NULL),
    (dict(delta_o=P), NULL), (dict(T=0), SHAPE), (dict(T=1 << 31), SHAPE), (dict(Hq=3), SHAPE),
    (dict(Hq=0), SHAPE), (dict(q_ld=511), SHAPE), (dict(k_ld=255), SHAPE), (dict(v_ld=0), SHAPE),
    (dict(n_pos=0), SHAPE), (dict(dt=7), DTYPE), (dict(q_dt=7), DTYPE), (dict(abits=5), BITS),
    (dict(k=P + 8), ALIGN), (dict(q=P + 2), ALIGN), (dict(v_ld=257), ALIGN), (dict(q_out=P + 4), ALIGN),
    (dict(rope=P + 4), ALIGN), (dict(s_a=P + 4), ALIGN)])
def test_append_refuses(omq, kw, want):
    assert omq._lib.omq_kv_append(ctypes.byref(append_args(omq, **kw)), None) == want


@pytest.mark.parametrize("kw,want", BAD_POOLS)
def test_every_entry_refuses_a_bad_pool(omq, kw, want):
    pool = pool_of(omq, **kw)
    assert omq._lib.omq_kv_append(ctypes.byref(append_args(omq, pool)), None) == want
    assert omq._lib.omq_kv_attn(ctypes.byref(attn_args(omq, pool)), None, 0, None) == want
    assert omq._lib.omq_kv_read(ctypes.byref(pool), 3, P, P, P, 0, None) == want


def attn_args(omq, pool=None, **kw):
    d = dict(pool=pool or pool_of(omq), n_req=4, T=16, Hq=8, q=P, q_ld=1024, dt=omq.OMQ_BF16,
             table=P, width=8, lens=P, cu=P, max_q=4, scale=0.1, causal=1, out=P,
             out_dt=omq.OMQ_BF16, lse=None)
    return omq.KvAttnArgs(**{**d, **kw})


@pytest.mark.parametrize("kw,want", [
    *[({n: None}, NULL) for n in ("q", "table", "lens", "cu", "out")],
    (dict(dt=0), DTYPE), (dict(out_dt=0), DTYPE), (dict(n_req=0), SHAPE), (dict(T=0), SHAPE),
    (dict(Hq=9), SHAPE), (dict(Hq=0), SHAPE), (dict(width=0), SHAPE), (dict(width=1 << 25), SHAPE),
    (dict(max_q=0), SHAPE), (dict(max_q=17), SHAPE), (dict(q_ld=1023), SHAPE),
    (dict(q_ld=1028), ALIGN), (dict(q=P + 8), ALIGN), (dict(out=P + 8), ALIGN),
    (dict(T=1 << 30, max_q=1 << 30), SHAPE), (dict(n_req=65536, T=1 << 20, max_q=1 << 20), SHAPE)])
def test_attn_refuses(omq, kw, want):
    assert omq._lib.omq_kv_attn(ctypes.byref(attn_args(omq, **kw)), None, 0, None) == want


def test_read_and_rope_refuse(omq):
    pool = pool_of(omq)
    read = omq._lib.omq_kv_read
    assert read(None, 3, P, P, P, 0, None) == NULL
    assert read(ctypes.byref(pool), 3, None, P, P, 0, None) == NULL
    assert read(ctypes.byref(pool), 3, P, None, P, 0, None) == NULL
    assert read(ctypes.byref(pool), 0, P, P, P, 0, None) == SHAPE
    assert read(ctypes.byref(pool), 3, P, P, P, 9, None) == DTYPE
    assert read(ctypes.byref(pool), 3, P, P + 4, P, 0, None) == ALIGN
    rope = omq._lib.omq_rope_table
    assert rope(16, 128, 1e4, None, None) == NULL
    assert rope(0, 128, 1e4, P, None) == SHAPE
    assert rope(16, 96, 1e4, P, None) == SHAPE
    assert rope(16, 128, 1.0, P, None) == SHAPE
    assert rope(16, 128, float("nan"), P, None) == SHAPE
    assert rope(16, 128, 1e4, P + 4, None) == ALIGN


def test_binding_refuses_host_tensors(omq):
    pool = torch.zeros(2, 1, 4, 2304, dtype=torch.uint8)
    i = torch.zeros(4, dtype=torch.int32)
    kv = torch.zeros(4, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        omq.kv_append(pool, i, kv, kv)
    with pytest.raises(ValueError):
        omq.kv_read(pool, i)
    with pytest.raises(ValueError):
        omq.kv_attn(kv, pool, i.view(4, 1), i, torch.zeros(5, dtype=torch.int32), 1)
    with pytest.raises(ValueError):
        omq.kv_plan(i, i, i.view(4, 1), i, i[:1], 64, 4)
    with pytest.raises(ValueError):
        omq.kv_pool(2, 1, 96, 64, device="cpu")


def test_pool_layout_round_trip():
    rng = np.random.default_rng(0)
    for D, page in ((64, 48), (128, 16)):
        pool = np.full((5, 3, page // 16, kc.cell_bytes(D)), 255, np.uint8)
        slots = rng.permutation(5 * page)[:9]
        rows = [kc.encode(rng.standard_normal((9, 3, D)).astype(np.float32) + s) for s in (0, 40)]
        for w in range(2):
            kc.put(pool, page, slots, w, *rows[w])
        for w in range(2):
            for a, b in zip(kc.get(pool, page, slots, w), rows[w]):
                assert np.array_equal(a, b)


def test_quantizer_statement_is_the_oracle_encoder():
    """The cache's rows use the per-token activation quantizer's rule: codes, step and zero
    point agree bit for bit with the oracle's."""
    from oracle import omniquant as om
    rng = np.random.default_rng(1)
    X = (rng.standard_normal((40, 128)) * np.exp(rng.standard_normal((40, 1)))).astype(np.float32)
    X[3] += 30
    X[5] = 0
    want = om.act_quant(X, 4)
    c, h, z = kc.encode(X)
    assert c.min() >= 0 and c.max() <= 15
    # within half a step of the row wherever the code is not clamped
    v = kc.values(c, h, z)
    free = (c > 0) & (c < 15)
    assert np.all(np.abs(v - X)[free] <= (h * (0.5 + 1e-5)).astype(np.float64).repeat(128, 1)[free])
    assert np.array_equal(c, want.codes) and np.array_equal(h, want.h)
    assert np.array_equal(z.astype(np.int32), want.z_i32)
    assert np.array_equal(kc.values(c, h, z, np.float32), want.deq)


FAR = P + (1 << 30)


@pytest.mark.parametrize("kw", [dict(out=P), dict(out=P + 2048 * 15 + 2032), dict(q=FAR, out=FAR - 16 * 2048 + 16)])
def test_attn_refuses_out_over_q(omq, kw):
    a = attn_args(omq, **kw)
    assert omq._lib.omq_kv_attn(ctypes.byref(a), None, 0, None) == 8
    assert omq._lib.omq_kv_attn_workspace_bytes(ctypes.byref(a)) == 0


@pytest.mark.parametrize("kw", [dict(q=FAR, k=FAR + 4096, v=FAR + 8192, q_out=FAR), dict(q_out=P + 512, q=FAR, v=FAR),
                                dict(q_out=P + 512, q=FAR, k=FAR)])
def test_append_refuses_q_out_over_its_inputs(omq, kw):
    assert omq._lib.omq_kv_append(ctypes.byref(append_args(omq, **kw)), None) == 8
