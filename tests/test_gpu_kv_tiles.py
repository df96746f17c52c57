"""The tile kernel of omq_kv_attn (requests of more than 512 query rows per kv head) within the
bound of its float16 operands."""
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
    s.kv[b][w] = kc.encode(x.astype(np.float32))
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
