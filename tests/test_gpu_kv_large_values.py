"""Values and keys beyond float16 in the tile kernel, whose operands are float16: the rows that see
such a value are NaN, the others do not notice; a key beyond it is met only by its own column."""
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


@pytest.mark.parametrize("n,new", [(600, 600), (5000, 520)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("which,size", [(1, 7e4), (1, 1e9), (1, 1e30), (0, 1e7), (0, 1e30)])
def test_rows_that_do_not_see_a_large_row(omq, cuda_device, n, new, D, which, size):
    """One element, or all, of a row of values (1) or keys (0) of `size`, 200 tokens before the last."""
    s = Setup(cuda_device, [n], [new], 1, 1, D, 16, "bf16", seed=173)
    clean, clean_l = omq.kv_attn(*s.args, s.max_q, lse=True)
    x = kc.values(*s.kv[0][which])
    at = n - 200
    first = at - (n - new)
    for where in (slice(3, 4), slice(0, D), slice(D - 1, D)):
        y = x.copy()
        y[at, 0, where] = -size if where.start == D - 1 else size
        refill(s, which, y)
        out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
        omq.sync_check()
        assert torch.equal(out[:first], clean[:first]) and torch.equal(lse[:first], clean_l[:first])
        if which == 1:
            assert bool(torch.isnan(out[first:]).all())


def test_values_up_to_float16_s_largest(omq, cuda_device):
    """Constant values of 65504 and -65504, whose steps are the values: the result is theirs."""
    s = Setup(cuda_device, [600], [600], 1, 1, 64, 16, "bf16", seed=179)
    v = np.full((600, 1, 64), 65504.0)
    for sign in (1, -1):
        pos = torch.arange(600, dtype=torch.int32, device=cuda_device)
        slots = s.args[2][0, (pos // 16).long()] * 16 + pos % 16
        k, _ = omq.kv_read(s.pool, slots)
        omq.kv_append(s.pool, slots, k, torch.from_numpy(sign * v).float().to(cuda_device))
        out = omq.kv_attn(*s.args, s.max_q)
        omq.sync_check()
        # half a step of the weights and of the output: 2^-11 + 2^-9, of each sum's terms
        assert bool(((out.float() - sign * 65504).abs() <= 65504 * (2.0 ** -11 + 2.0 ** -9 + 2.0 ** -13)).all())
