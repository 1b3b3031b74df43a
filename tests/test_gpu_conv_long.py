"""short_conv's kernel for long calls, directly against the definition, and with waits for its copies that run out."""
import pytest
import torch

import layer_reference as lr
from gpu_util import library
from test_gpu_conv import close, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    yield g
    g.set_prefill_wait_limit(0)


def long_call(seed, C, taps, dtype, tail):
    """Sequences of odd lengths around one that makes the call long on this GPU: three tiles of 128 tokens per SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lens = [1, 2, 3, 131, 0, 128, 3 * sms * 128 - 700, 127, 0, 1, 1, 257, tail]
    s = make(seed, lens, C, taps, dtype)
    tiles, blocks = -(-s["x"].shape[0] // 128), -(-C // 1024)
    assert tiles * blocks >= 2 * sms + 16  # that kernel's calls, with room
    return s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("taps,C,tail", [(2, 8, 1), (3, 24, 64), (4, 16, 130)])
def test_against_the_definition(gdn, taps, C, tail, dtype):
    s = long_call(taps, C, taps, dtype, tail)
    T = sum(s["lens"])
    y, hist, status = run(gdn, s, [C])
    assert status == 0 and bool((y[T:] == 9.0).all())
    at = 0
    for n, k in enumerate(s["lens"]):  # the long one's first and last tokens, of which the definition needs the taps - 1 ahead
        x = s["x"][at:at + k].double()
        for a, b in ((0, k),) if k < 1000 else ((0, 700), (k - 700, k)):
            past = s["hist"].double() if a == 0 else s["hist"].double().clone()
            if a > 0:
                past[s["slots"][n]] = x[a - taps + 1:a].T
            ref, mag, new = lr.conv(x[a:b], s["w"].double(), s["bias"].double(), past, s["slots"][n:n + 1].tolist(), [b - a], True)
            close(y[at + a:at + b], ref, mag, dtype)
        slot = s["slots"][n]
        assert torch.equal(hist[slot].double(), new[slot] if k else s["hist"][slot].double())
        at += k


@pytest.mark.parametrize("polls", [1, 2, 5, 20, 100])
def test_copies_that_come_late_are_done_without(gdn, polls):
    s = long_call(5, 1032, 4, torch.bfloat16, 77)
    want, hist, _ = run(gdn, s, [1024, 8])
    try:
        gdn.set_prefill_wait_limit(polls)
        for _ in range(3):
            got, h, status = run(gdn, s, [1024, 8])
            assert status == 0 and torch.equal(got.view(torch.int16), want.view(torch.int16)) and torch.equal(h, hist)
    finally:
        gdn.set_prefill_wait_limit(0)
    got, h, status = run(gdn, s, [1024, 8])
    assert status == 0 and torch.equal(got.view(torch.int16), want.view(torch.int16)) and torch.equal(h, hist)
