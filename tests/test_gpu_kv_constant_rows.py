"""Constant rows of any size in the 4-bit cache: their step is the floor of 1e-8, so that from
10.7 on their zero point is beyond the integers the cache stores. What is read back, and what is
made of the queries, is the quantizer's (c - z) h with its zero point as it is."""
import numpy as np
import pytest
import torch

from oracle import omniquant as om
from tests import kv_common as kc

pytestmark = pytest.mark.gpu

SIZES = [0.0, 1e-9, 0.3, -3.0, 10.5, 10.7374, 10.7375, -10.7374, -10.74, 10.8, 20.0, -20.0, 333.3, -6e4, 1e9, -1.5e20, 3e30]


@pytest.fixture(scope="module")
def omq(cuda_device):
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


def rows(D, heads=3):
    """[T, heads, D] float32: a constant row of each size on one head, ordinary ones on the others."""
    rng = np.random.default_rng(D)
    x = rng.standard_normal((len(SIZES), heads, D)).astype(np.float32)
    for t, c in enumerate(SIZES):
        x[t, t % heads] = c
    return x


def simulated(x, bits=4):
    """The calibration's per-row fake-quantized values, float32."""
    return om.act_quant(x.reshape(-1, x.shape[-1]), bits).deq.reshape(x.shape)


@pytest.mark.parametrize("D", [64, 128])
def test_constant_rows_read_back_as_calibrated(omq, cuda_device, D):
    x = rows(D)
    pool = omq.kv_pool(3, 3, D, 16, cuda_device)
    slots = torch.arange(len(x), dtype=torch.int32, device=cuda_device)
    t = torch.from_numpy(x).to(cuda_device)
    q = omq.kv_append(pool, slots, t, -t, q=t, abits=4, q_dtype=torch.float32)
    k, v = omq.kv_read(pool, slots)
    omq.sync_check()
    assert np.array_equal(k.cpu().numpy(), simulated(x))
    assert np.array_equal(v.cpu().numpy(), simulated(-x))
    assert np.array_equal(q.cpu().numpy(), simulated(x))
    # to the quantizer's half step, for a constant row the rounding of z and of the product
    at = np.arange(len(x))
    err = np.abs(k.cpu().numpy().astype(np.float64) - x)[at, at % 3]
    size = np.abs(np.array(SIZES))[:, None]
    assert np.all(err <= 0.5e-8 + 2.0 ** -22 * size)


def test_a_constant_row_without_a_finite_zero_point_is_nan(omq, cuda_device):
    x = np.ones((3, 1, 64), np.float32)
    x[0], x[1] = 3.5e30, -1e38
    pool = omq.kv_pool(1, 1, 64, 16, cuda_device)
    slots = torch.arange(3, dtype=torch.int32, device=cuda_device)
    t = torch.from_numpy(x).to(cuda_device)
    q = omq.kv_append(pool, slots, t, t, q=t, abits=8, q_dtype=torch.float32)
    for g in (q, *omq.kv_read(pool, slots)):
        assert torch.isnan(g[:2]).all() and bool((g[2] - 1).abs().max() < 1e-6)


@pytest.mark.parametrize("new", [1, 600])
def test_attention_over_constant_rows(omq, cuda_device, new):
    """Values of 20 and -500 in turn, keys of 30 and -30 (both kernels): the weights are those of
    the keys' scores, 0 and 1 to within 2^-30, so the result is the seen value."""
    n, D = 700, 64
    pool = omq.kv_pool(44, 1, D, 16, cuda_device)
    sign = torch.ones(n, 1, 1, device=cuda_device)
    sign[1::2] = -1
    k = (30 * sign).expand(n, 1, D).contiguous()
    v = torch.where(sign > 0, 20.0, -500.0).expand(n, 1, D).contiguous()
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda_device)  # noqa: E731
    omq.kv_append(pool, torch.arange(n, dtype=torch.int32, device=cuda_device), k, v)
    q = torch.full((new, 1, D), 0.5, dtype=torch.float16, device=cuda_device)
    q[1::2] = -0.5
    table = torch.arange(44, dtype=torch.int32, device=cuda_device)[None]
    out = omq.kv_attn(q, pool, table, i(n), i(0, new), new)
    omq.sync_check()
    want = torch.full_like(out, 20.0)
    want[1::2] = -500.0
    # half a step of k, v, the weights and the result each, of equal values: 4 x 2^-11
    assert bool(((out - want).abs() <= 2.0 ** -9 * want.abs()).all())
