"""Windows of few tokens on a state pool that is 16-byte aligned, as single tokens may have it."""
import pytest
import torch

from gpu_util import library
from test_gpu_ssm import check, make, prefill, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


def test_windows(gdn):
    s = make(61, [5, 16, 0, 1], 2, 64, 1, 128)
    ref = reference(s)
    n = s["state"].numel()
    pool = torch.empty(n + 4, device="cuda")[4:].view(s["state"].shape)
    assert pool.data_ptr() % 32 == 16
    pool.copy_(s["state"])
    y = gdn.ssm_prefill_chunked(s["x"], s["dt"], s["B"], s["C"], s["A_log"], s["dt_bias"], pool, s["slots"], s["cu"], 16, D=s["D"], z=s["z"])
    check(s, y, pool, ref, False)
    with pytest.raises(gdn.GdnError, match="32-byte"):
        gdn.ssm_prefill_chunked(s["x"], s["dt"], s["B"], s["C"], s["A_log"], s["dt_bias"], pool, s["slots"], s["cu"], 17, D=s["D"], z=s["z"])
