"""The chunked scan's bounded waits, made to run out at many places: the CTAs that gave up end behind their copies, and what the next
call on the stream computes is right."""
import pytest
import torch

from gpu_util import library
from test_gpu_ssm import check, make, prefill, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    yield g
    g.set_prefill_wait_limit(0)


def limited(gdn, s, polls, **kw):
    try:
        gdn.set_prefill_wait_limit(polls)
        return prefill(gdn, s, **kw)
    finally:
        gdn.set_prefill_wait_limit(0)


@pytest.mark.parametrize("lens,H,P,S,gated", [([700, 40, 513], 5, 64, 128, True), ([900], 2, 128, 64, False), ([5000, 300], 2, 64, 64, True),
                                              ([4500], 2, 128, 128, True)])
def test_ctas_that_give_up_leave_nothing_behind(gdn, lens, H, P, S, gated):
    """CTAs that follow on the same SMs, ended early or not, find their barriers and shared memory to themselves."""
    s = make(21, lens, H, P, 1, S, gated)
    want = reference(s)
    timeouts = 0
    for polls in (1, 17, 33, 65, 129, 257, 513, 1025, 4097):
        _, _, status = limited(gdn, s, polls)
        assert status in (0, gdn.STATUS_TIMEOUT)
        timeouts += status != 0
        y, state, status = prefill(gdn, s)
        assert status == 0
        check(s, y, state, want, True)
    assert timeouts > 0
