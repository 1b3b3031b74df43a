"""Single tokens with large steps among small ones: what stands behind such a token keeps its digits, in chunks as token by token."""
import math

import pytest
import torch

from gpu_util import library
from test_gpu_ssm import check, make, prefill
from test_gpu_ssm import reference as full_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


def jumps(lens, P, S, large, at, **kw):
    """dt 0.003 with a decay of 16 per unit, but for the tokens `at`, whose dt is `large`; those tokens add nothing of their own."""
    s = make(41, lens, 2, P, 1, S, **kw)
    s["A_log"].fill_(math.log(16.0))
    s["dt_bias"].fill_(math.log(math.expm1(0.003)))
    s["dt"].fill_(0.0)
    at = torch.tensor(at, device="cuda")
    s["dt"][at] = large
    s["x"][at] = 0.0
    return s


def reference(s):
    """The 64-bit form takes softplus by way of e^raw, which is no number beyond 709.  With steps of at most 600 it is the same: the decay
    e^(-16 * 600) is zero in 64 bits already, and x is zero where the steps are larger."""
    return full_reference(dict(s, dt=s["dt"].clamp(max=600.0)))


@pytest.mark.parametrize("large", [30.0, 300.0, 3000.0, 30000.0, 1e6, 3e38])
@pytest.mark.parametrize("P,S", [(64, 128), (128, 64)])
def test_outputs_behind_a_large_step(gdn, large, P, S):
    s = jumps([300], P, S, large, [0, 5, 40, 41, 42, 70, 127, 128, 200, 255])
    ref = reference(s)
    for max_len in (300, 1):  # in chunks, token by token
        y, state, status = prefill(gdn, s, max_len=max_len)
        assert status == 0 and bool(y.isfinite().all()) and bool(state.isfinite().all())
        check(s, y, state, ref, max_len > 1)
        # Weights and the state's copy in bf16 are off by 2^-9 of their norm in the mean at most (a third of the half step's square is
        # (2^-8)^2 / 3, over a factor of two in size less); the difference of sums adds at most 2^-11 ln 2, the output's rounding 2^-9.
        err = (y.double() - ref[0]).norm() / ref[0].norm()
        assert float(err) <= math.hypot(2.0 ** -9, 2.0 ** -9) + 2.0 ** -11, float(err)


def test_large_steps_in_every_block(gdn):
    """Every third token of a block is a large step: the sums within a block grow to their limit."""
    s = jumps([640, 256], 64, 128, 1e4, [t for t in range(896) if t % 3 == 0])
    ref = reference(s)
    y, state, status = prefill(gdn, s, max_len=640)
    assert status == 0
    check(s, y, state, ref, True)
    err = (y.double() - ref[0]).norm() / ref[0].norm()
    assert float(err) <= math.hypot(2.0 ** -9, 2.0 ** -9) + 2.0 ** -11, float(err)


def test_a_large_step_in_a_cut_sequence(gdn):
    """The states that segments start from, and their decays, with steps whose decay leaves nothing."""
    s = jumps([5000], 64, 128, 3e38, [1, 1000, 2500, 4095, 4999])
    s["x"][::7] = 1.0
    s["x"][torch.tensor([1, 1000, 2500, 4095, 4999], device="cuda")] = 0.0
    ref = reference(s)
    y, state, status = prefill(gdn, s, max_len=5000)
    assert status == 0
    check(s, y, state, ref, True)


@pytest.mark.parametrize("max_len", [3000, 1])
@pytest.mark.parametrize("name", ["A_log", "dt_bias", "dt"])
def test_what_is_no_number_shows(gdn, name, max_len):
    """One head's decay, or one token's step, is no number: the head's outputs from there on are none, and the other head's are as they were."""
    s = make(42, [3000], 2, 64, 1, 128)
    clean = prefill(gdn, s, max_len=max_len)
    s[name] = s[name].clone()
    first = 1500 if name == "dt" else 0
    s[name][(slice(1500, 1501), 1) if name == "dt" else 1] = float("nan")
    y, state, status = prefill(gdn, s, max_len=max_len)
    slot = int(s["slots"][0])
    assert status == 0 and bool(y[first:, 1].isnan().all()) and bool(state[slot, 1].isnan().all())
    assert torch.equal(y[:, 0], clean[0][:, 0]) and torch.equal(state[slot, 0], clean[1][slot, 0])
    assert torch.equal(y[:first // 128 * 128], clean[0][:first // 128 * 128])
