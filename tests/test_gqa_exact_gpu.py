"""GQA tree attention where it is easily wrong: waits that run out behind another error."""

import pytest

from speculative_decoding_tree_mla_gb300 import kdtv
from tests.test_gqa_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_a_wait_that_runs_out_behind_another_error(cache, d):
    """The loads never start (a test flag; every wait has a limit) in a call whose batch has a bad
    prefix as well, or whose status word holds an earlier error: the timeout is reported and no row
    is written, whatever the workspace held."""
    for earlier in (0, kdtv.STATUS_CODE["KDTV_ERR_BAD_TREE"]):
        x = Case(3, 9, 8, 2, d, cache, 16, [700, 300, 20], seed=24)
        good = x.prefix.copy()
        if not earlier:
            x.prefix[1] = -1
        op = x.op(kdtv.KDTV_FLAG_TEST_STALL)
        op.workspace.zero_()                       # what was not written looks like partial rows
        op._status.fill_(earlier)
        out = op()
        assert kdtv.STATUS[op.status()] == "KDTV_ERR_DEVICE_TIMEOUT"
        assert (out == 9.0).all()
        assert op.status() == 0
        x.prefix = good
        again = x.op()
        x.check(again(), True)
        assert again.status() == 0
