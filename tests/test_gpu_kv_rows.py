"""The row kernel of omq_kv_attn (few query rows a request) within the bound of its exact
operands, where the lanes of a warp share their work most unevenly."""
import pytest
import torch

from tests import kv_kernels as kk
from tests.test_gpu_kv_attn import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def omq(cuda_device):
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


@pytest.mark.parametrize("G,D,dt", [(1, 128, "f16"), (4, 128, "bf16"), (3, 64, "f16"), (16, 64, "bf16")])
def test_runs_that_end_at_every_token(omq, cuda_device, G, D, dt):
    """Contexts of 1 to 130 tokens, and with pages that are not there: the tokens of a 64-token run
    that are there, whose steps the warp's lanes read for one another, are any subset of its
    cells and any part of the last. Repeated to the bit."""
    lens = list(range(1, 131))
    s = Setup(cuda_device, lens, [1] * 130, 2, G, D, 16, dt, seed=89 + G)
    hidden = [(b, p) for b in range(40, 130) for p in range(len(range(0, lens[b], 16)) - 1) if (b >> p) & 1]
    for with_holes in (False, True):
        if with_holes:
            for b, p in hidden:
                s.args[2][b, p] = -1
        out, lse = omq.kv_attn(*s.args, 1, lse=True)
        for _ in range(20):
            again, lse2 = omq.kv_attn(*s.args, 1, lse=True)
            assert torch.equal(out, again) and torch.equal(lse, lse2)
        omq.sync_check()
        kk.check(s, out, lse, hidden=hidden if with_holes else ())
