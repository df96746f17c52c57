"""The row kernel of omq_kv_attn (few query rows a request) within the bound of its exact
operands, where the lanes of a warp share their work most unevenly."""
import numpy as np
import pytest
import torch

from tests import kv_kernels as kk
from tests.test_gpu_kv_attn import SMALL, Setup

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


LONG = [([4099, 2000], [1, 1], 2, 4, 128, 64, "bf16"), ([20011], [1], 1, 8, 128, 16, "f16"), ([9000], [4], 1, 2, 64, 128, "f16"),
        ([5000, 333, 0], [8, 8, 0], 2, 8, 128, 32, "f16")]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,new,Hkv,G,D,page,dt", [c for c in SMALL if max(c[1]) * c[3] <= 64] + LONG)
def test_exact_operands(omq, cuda_device, lens, new, Hkv, G, D, page, dt, causal):
    """Up to 64 rows a request: the codes and the queries are exact, whatever the length."""
    s = Setup(cuda_device, lens, new, Hkv, G, D, page, dt, seed=157 + D)
    out, lse = omq.kv_attn(*s.args, s.max_q, causal=causal, lse=True)
    omq.sync_check()
    kk.check(s, out, lse, causal)


@pytest.mark.parametrize("n_req,Hkv,G,new,wide", [(40, 8, 1, 1, 9600), (150, 3, 6, 2, 12000), (20, 3, 4, 2, 0)])
def test_exact_operands_of_many_requests(omq, cuda_device, n_req, Hkv, G, new, wide):
    """On the even line of all requests' runs (a wide table), and shared by blocks of a cluster."""
    rng = np.random.default_rng(n_req)
    lens = rng.integers(new, 90, n_req)
    lens[3], lens[n_req - 2] = 1500, 0
    s = Setup(cuda_device, lens, np.minimum(new, lens), Hkv, G, 64, 16, "f16", seed=163)
    if wide:
        table = torch.full((n_req, wide // 16), -1, dtype=torch.int32, device=cuda_device)
        table[:, :s.table.shape[1]] = s.args[2]
        s.args[2] = table
    out, lse = omq.kv_attn(*s.args, s.max_q, lse=True)
    omq.sync_check()
    kk.check(s, out, lse)
