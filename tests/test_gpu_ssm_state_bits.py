"""The chunked scan's states to fp32: their error's norm, where each holds few tokens, so that nothing but the chunk's own arithmetic counts."""
import pytest
import torch

from gpu_util import library
from test_gpu_ssm import make, prefill, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


@pytest.mark.parametrize("lens,H,P,G,S", [([640, 300, 129], 4, 64, 2, 128), ([640, 300, 129], 3, 64, 1, 64), ([500], 2, 128, 1, 128), ([640, 17, 300], 4, 128, 2, 64),
                                          ([2100], 2, 64, 1, 128), ([2100], 2, 64, 1, 64), ([2100], 2, 128, 1, 128), ([2100], 2, 128, 1, 64)])
def test_norm_of_the_states_error(gdn, lens, H, P, G, S):
    s = make(71, lens, H, P, G, S, dt=(0.02, 0.1))
    _, want, _, _ = reference(s)
    _, state, status = prefill(gdn, s, max_len=max(lens))
    assert status == 0
    # A token's weight: softplus, the exponential and the sums of the steps behind it, 2^-21 together where it still counts.  Its product with
    # three bf16 parts: nothing.  24 accumulations of a chunk (8 of 16 tokens, three parts), each of which may cut off 2^-23 of a sum that grows
    # to its size: half of that in the mean, of half the size.
    used = s["slots"]
    err = float((state[used].double() - want[used]).norm() / want[used].norm())
    assert err <= 2.0 ** -21 + 24 * 2.0 ** -25, err
