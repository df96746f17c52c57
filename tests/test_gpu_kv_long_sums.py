"""The row kernel's sums over long contexts whose blocks share nothing: the codes' part of the
result and the zero points' part are large and cancel."""
import numpy as np
import pytest
import torch

from tests import kv_common as kc
from tests.test_gpu_kv_attn import Setup
from tests.test_gpu_kv_tiles import refill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def omq(cuda_device):
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


@pytest.mark.parametrize("D,Hkv,G", [(64, 240, 1), (64, 150, 16), (128, 240, 1), (128, 150, 16)])
def test_sums_of_codes_are_not_cut_off(omq, cuda_device, D, Hkv, G):
    """Equal softmax weights (queries of zeros) of n values (c - z) h, z 7 or 8, h from 1/16 to 1/8, so w = p h
    is a weight of float16's full length; as many items as blocks, so a warp sums n / 4 tokens. The
    error's mean over the columns but the two that fix the rows' steps, in units of s = sum p h c (7.5 of the mean h):
      weights   rounded to float16, 2^-11 of each, independent: of n D terms p h 8 at most, by
                Hoeffding's inequality below 2^-10 (n D)^-1/2 5 of 8 / 7.5 s in all but 1e-10
      o         n / 256 additions a warp, half an ulp of the sum so far each: n / 256 2^-25 of s
      runs      4 steps of the matrix unit, 2^-22 each: 2^-20 of s
      zero      n / 128 additions a lane: n / 128 2^-25 of 8 / 7.5 s
      joins     16 additions: 2^-20 of s; the output's half step 2^-11 |o|, 2^-25
    Cut off towards zero step by step by the matrix unit, n / 64 times, s lost n / 64 2^-24 and more."""
    n = 100000
    s = Setup(cuda_device, [n], [1], 1, G, D, 64, "f16", seed=181)
    rng = np.random.default_rng(181)
    c = rng.integers(0, 16, (n, 1, D))
    c[:, :, 0], c[:, :, 1] = 0, 15
    mid = 7 + np.arange(n)[:, None, None] % 2                   # zero points of 7 and 8: the mean is near zero
    refill(s, 1, (c - mid) * (1 + rng.random((n, 1, 1))) / 16)
    codes, h, z = s.kv[0][1]
    want = kc.values(codes, h, z)[:, 0].mean(0)
    pool = s.pool.expand(-1, Hkv, -1, -1).contiguous()
    q = torch.zeros(1, Hkv * G, D, dtype=torch.float16, device=cuda_device)
    out = omq.kv_attn(q, pool, *s.args[2:], 1)
    omq.sync_check()
    assert torch.equal(out, out[:, :1].expand_as(out))
    size = float((codes * h.astype(np.float64))[:, 0].mean())
    tol = size * (2.0 ** -10 * (n * D) ** -0.5 * 5 * 8 / 7.5 + n / 256 * 2.0 ** -25 + 2.0 ** -20 + n / 128 * 2.0 ** -25 * 8 / 7.5 +
                  2.0 ** -20) + 2.0 ** -11 * np.abs(want[2:]).mean() + 2.0 ** -25
    assert tol < size * n / 64 * 2.0 ** -24 / 2               # the bound tells them apart
    assert abs(float((out[0, 0].double().cpu().numpy() - want)[2:].mean())) <= tol
