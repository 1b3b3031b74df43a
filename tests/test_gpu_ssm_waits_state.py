"""The state pool after a chunked scan whose waits ran out: each head of each slot is as it was, or right.  The workspace holds large numbers
ahead of the call, so that a state that was never formed there shows."""
import pytest
import torch

from gpu_util import library
from test_gpu_ssm import make, reference
from test_gpu_ssm_waits import limited

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    yield g
    g.set_prefill_wait_limit(0)


def sweep(gdn, s, limits, repeats):
    lens, H, P, S = s["lens"], s["x"].shape[1], s["x"].shape[2], s["B"].shape[2]
    _, want, _, size = reference(s)
    # as for the states of a call whose waits do not run out: decays and sums in fp32, dt x in two bf16 parts
    tol = ((90 + 4 * 512 + 300) * 2.0 ** -24 + 2.0 ** -16) * size + 1e-30
    need = gdn.ssm_prefill_workspace_size(len(lens), sum(lens), H, P, S)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    timeouts = kept = right = 0
    for polls in limits:
        for _ in range(repeats):
            ws = torch.full((need,), 0x71, dtype=torch.uint8, device="cuda")  # 1.2e30 in fp32
            flush.fill_(1)
            _, state, status = limited(gdn, s, polls, workspace=ws)
            assert status in (0, gdn.STATUS_TIMEOUT)
            timeouts += status != 0
            for slot in s["slots"].tolist():
                for h in range(H):
                    same = torch.equal(state[slot, h], s["state"][slot, h])
                    err = (state[slot, h].double() - want[slot, h]).abs()
                    good = bool((err <= tol[slot, h]).all())
                    assert same or good, (polls, slot, h, float(err.max()))
                    assert good or status
                    kept, right = kept + same, right + good
    assert timeouts > 0 and kept > 0 and right > 0


@pytest.mark.parametrize("lens,H,P,S", [([9000, 200, 4000], 4, 64, 128), ([6000], 3, 64, 64), ([5000, 17], 2, 128, 64), ([7000], 2, 128, 128)])
def test_each_state_is_as_it_was_or_right(gdn, lens, H, P, S):
    s = make(23, lens, H, P, 1, S, dt=(0.0003, 0.01))
    sweep(gdn, s, (1, 17, 33, 49, 65, 97, 129, 193, 257, 385, 513, 769, 1025, 2049), 1)


@pytest.mark.parametrize("H,P,S,stride", [(2, 64, 64, 1 << 18), (2, 128, 64, 1 << 18), (8, 64, 64, 1 << 16)])
def test_states_ahead_that_were_not_formed(gdn, H, P, S, stride):
    """The last segment has one token, and dt's rows are far apart: the states ahead wait for a thousand of them, it for one, so that
    there are limits at which only those give up."""
    s = make(23, [2049], H, P, 1, S, dt=(0.0003, 0.01))
    wide = torch.empty((2049, stride), dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = s["dt"]
    s["dt"] = wide[:, :H]
    sweep(gdn, s, (1, 17, 33, 49, 65, 81, 97, 129, 513), 6)
