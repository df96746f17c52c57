"""omq_kv_plan against the documented rules stated request by request: every output, the block
table and the free stack must match exactly."""
import numpy as np
import pytest
import torch

from tests import kv_common as kc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def omq(cuda_device):
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


def make(rng, lens, new, width, page, spare):
    """A consistent state: distinct pages for what the lengths hold, the rest on the stack."""
    lens, new = np.asarray(lens, np.int32), np.asarray(new, np.int32)
    held = -(-lens // page)
    n_pages = int(held.sum()) + spare
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    free = np.concatenate((ids[at:], np.full(at, -7, np.int32)))
    return lens, new, table, free, np.array([spare], np.int32)


def check(omq, dev, state, page, capacity, in_place=False):
    want = kc.plan(*state, page, capacity)
    t = [torch.from_numpy(a.copy()).to(dev) for a in state]
    got = omq.kv_plan(*t, page, capacity, in_place=in_place)
    torch.cuda.synchronize()
    got = {**got, "table": t[2], "free": t[3]}
    if in_place:
        assert got["lens"] is t[0] and got["n_free"] is t[4]
    for k, v in want.items():
        assert np.array_equal(got[k].cpu().numpy(), v), k
    return want


CASES = [  # lens, new, width, page, spare pages, capacity
    ([0], [1], 1, 16, 1, 1),
    ([0, 0, 0], [0, 0, 0], 4, 16, 3, 5),                     # nothing asked
    ([15, 16, 17, 31, 32, 0], [1, 1, 1, 1, 1, 16], 4, 16, 10, 64),
    ([5, 40, 64, 0, 33], [3, -1, 1, 70, -5], 8, 16, 2, 100),  # released pages are used at once
    ([16, 16, 16, 16], [1, 1, 1, 1], 4, 16, 2, 8),           # pages for two only
    ([16, 20, 16, 21], [1, 1, 1, 1], 4, 16, 1, 8),           # refused, yet room in its page later
    ([3, 3, 3, 3], [5, 5, 5, 5], 4, 16, 8, 11),              # capacity for two
    ([3, 3, 3, 3], [5, 9, 1, 0], 4, 16, 8, 6),               # refused by capacity, and all behind it
    ([60, 10], [10, 2], 4, 16, 9, 16),                       # longer than the table
    ([47, 100], [2, 30], 4, 48, 3, 40),                      # a page that is no power of two
    ([-1, -2], [-1, -1], 2, 16, 4, 3),                       # lengths out of range, released
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,new,width,page,spare,capacity", CASES)
def test_small(omq, cuda_device, lens, new, width, page, spare, capacity, in_place):
    lens = np.asarray(lens)
    state = make(np.random.default_rng(1), np.maximum(lens, 0), new, width, page, spare)
    state = (lens.astype(np.int32), *state[1:])
    check(omq, cuda_device, state, page, capacity, in_place)


@pytest.mark.parametrize("n_req,page,share,capacity", [
    (511, 16, 1.0, 5000), (512, 64, 0.5, 600), (513, 128, 0.3, 9000), (1500, 32, 0.7, 20000),
    (5000, 16, 0.6, 7000)])
def test_many_requests(omq, cuda_device, n_req, page, share, capacity):
    """Several chunks of requests, refusals by pages and by capacity, releases, and (past 4096
    requests) the bisection over the offsets in global memory."""
    rng = np.random.default_rng(n_req)
    width = 20
    lens = rng.integers(0, width * page + 1, n_req)
    new = rng.choice([1, 1, 1, 0, -1, 30], n_req)
    need = np.where((new > 0) & (lens + new <= width * page),
                    -(-(lens + new) // page) - -(-lens // page), 0).sum()
    back = np.where(new < 0, -(-lens // page), 0).sum()
    spare = max(0, int(need * share) - int(back))
    want = check(omq, cuda_device, make(rng, lens, new, width, page, spare), page, capacity)
    assert 0 < want["cu"][-1] <= capacity


def test_a_full_stack_takes_no_more(omq, cuda_device):
    state = list(make(np.random.default_rng(2), [40, 40], [-1, -1], 4, 16, 2))
    state[4] = np.array([6], np.int32)          # 8 pages, 6 already said to be free
    state[3] = np.arange(8, dtype=np.int32)
    check(omq, cuda_device, state, 16, 4)
    state[4] = np.array([99], np.int32)         # a count above the pool
    check(omq, cuda_device, state, 16, 4)
    state[4] = np.array([-3], np.int32)
    check(omq, cuda_device, state, 16, 4)


def test_out_of_place_plan_repeats(omq, cuda_device):
    state = make(np.random.default_rng(3), [5, 40, 64, 0, 33], [3, -1, 1, 70, -5], 8, 16, 20)
    t = [torch.from_numpy(a.copy()).to(cuda_device) for a in state]
    a = omq.kv_plan(*t, 16, 100)
    b = omq.kv_plan(*t, 16, 100)
    for k in a:
        assert torch.equal(a[k], b[k]), k
