"""omq_kv_plan with page ids that no pool has, in the table and on the stack: their tokens have
no slot, and the others theirs."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def omq(cuda_device):
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


@pytest.mark.parametrize("page,bad", [(16, (1 << 28) + 3), (64, (1 << 26) + 2), (64, 1 << 25), (4096, 1 << 19), (48, 2 ** 31 - 1), (16, -7)])
def test_ids_beyond_any_pool_give_no_slot(omq, cuda_device, page, bad):
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda_device)  # noqa: E731
    table = torch.full((3, 2), -1, dtype=torch.int32, device=cuda_device)
    table[0, 0], table[1, 0] = bad, 1                # a held page; a good one
    step = omq.kv_plan(i(3, 5, 0), i(1, 2, 2), table, i(0, 2, bad), i(3), page, 6)
    omq.sync_check()
    assert table[2, 0] == bad                        # the top of the stack
    assert step["slots"].tolist() == [-1, page + 5, page + 6, -1, -1, -1]
    assert step["positions"].tolist() == [3, 5, 6, 0, 1, -1]
