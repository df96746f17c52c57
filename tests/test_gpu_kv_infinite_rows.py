"""A query row that holds infinities or NaN next to others of the same request: only its own
result changes. (Rows are processed together and scaled by their largest element.)"""
import pytest
import torch

from tests.test_gpu_kv_attn import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def omq(cuda_device):
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


@pytest.mark.parametrize("new,G,dt", [(1, 4, "bf16"), (8, 1, "bf16"), (5, 4, "bf16"), (16, 1, "f16"), (600, 1, "bf16"), (600, 1, "f16")])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 18, 2.0 ** -22])
def test_an_infinite_row_leaves_the_others(omq, cuda_device, new, G, dt, bad, size):
    if dt == "f16" and size > 1:
        size = 2.0 ** 10                                   # within float16
    s = Setup(cuda_device, [700], [new], 1, G, 128, 16, dt, seed=167, spread=min(1.0, 1 / size))
    q = s.args[0]
    q.mul_(size)
    t, h = new // 2, G - 1
    q[t, h] = 0                                            # an ordinary row in its place
    want, want_l = omq.kv_attn(*s.args, s.max_q, lse=True)
    q[t, h, ::3] = bad
    got, got_l = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    assert bool(torch.isnan(got[t, h]).all())
    for a, b in ((got, want), (got_l, want_l)):
        a[t, h] = b[t, h]
        assert not torch.isnan(a).any() and torch.equal(a, b)
