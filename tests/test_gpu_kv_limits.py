"""Requests that grow to the end of their block table, where that is past max_len: every token
the plan grants is stored and attended, and what the table has no room for is refused."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kv_step import Server

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def omq(cuda_device):
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


@pytest.mark.parametrize("max_len,page,G,D", [(100, 64, 4, 128), (33, 48, 1, 64), (100, 16, 2, 128)])
def test_requests_that_reach_the_table_s_end(omq, cuda_device, max_len, page, G, D):
    """A prompt of max_len - 2 tokens, single tokens past max_len to the end of the last page, and
    one more, which is refused; the pool's pages held other tokens before."""
    s = Server(omq, cuda_device, 2, 40, 2, G, D, page, 16, max_len=max_len)
    room = -(-max_len // page) * page
    s.cache.pool.fill_(0x5A)                 # codes, steps and zero points of an earlier request
    new = [[max_len - 2, 3]] + [[1, 1]] * (room - max_len + 2) + [[1, 1]]
    for i, n in enumerate(new):
        x = s.qkv(sum(n))
        step, qt, out = s.device_step(torch.tensor(n, dtype=torch.int32, device=cuda_device), x.to(cuda_device), max(n))
        omq.sync_check()
        granted = np.diff(step["cu"].cpu().numpy())
        assert np.array_equal(granted, n if i < len(new) - 1 else [0, 1]), i
        s.note(step, x)
        s.check(step, qt, out, every=1 if i else 13)
    assert s.cache.lens.cpu().tolist() == [room, len(new) + 2]
