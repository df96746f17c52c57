"""The largest tables omq_kv_plan takes, by its host checks alone: nothing is launched."""
import ctypes

import pytest

from tests.test_kv_refusals import SHAPE, omq, plan_args  # noqa: F401


@pytest.mark.parametrize("n_req,width", [(512, 1 << 22), (65536, 1 << 22), (512, (1 << 26) - 1), (100, (1 << 25)), (64, 1 << 25)])
def test_tables_whose_pages_pass_32_bits_are_refused(omq, n_req, width):  # noqa: F811
    """A chunk of 512 requests counts its pages in 32 bits."""
    a = plan_args(omq, n_req=n_req, width=width, page=16)
    assert omq._lib.omq_kv_plan(ctypes.byref(a), None) == SHAPE
