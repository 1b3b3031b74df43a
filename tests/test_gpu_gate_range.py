"""z / (1 + e^-z) over the whole range of the types, in the convolution's activation and in the scan's gate."""
import pytest
import torch

import layer_reference as lr
import test_gpu_conv
import test_gpu_ssm
from gpu_util import library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


def spread(n, dtype):
    """Both signs of n / 2 magnitudes from 2^-10 to the type's largest value."""
    top = torch.finfo(dtype).max
    size = torch.logspace(-10, torch.tensor(top, dtype=torch.float64).log2().item(), n // 2, base=2.0, dtype=torch.float64).clamp(max=top)
    return torch.stack([size, -size], 1).flatten().to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens", [[40], [1] * 40])
def test_activation(gdn, lens, dtype):
    C = 32
    s = test_gpu_conv.make(31, lens, C, 2, dtype, pad=0)
    s["w"][:, 0], s["w"][:, 1], s["bias"][:] = 0.0, 1.0, 0.0  # y is the token itself
    s["wide"][:, 8:8 + C] = spread(40 * C, dtype).reshape(40, C)
    y, _, status = test_gpu_conv.run(gdn, s, [C], step=len(lens) == 40)
    ref, _, _ = lr.conv(s["x"].double(), s["w"].double(), s["bias"].double(), s["hist"].double(), s["slots"].tolist(), lens, True)
    assert status == 0 and bool(y.isfinite().all())
    # One rounding (half a step), the exponential and the quotient 2^-20 of the value.  e^z is taken as zero below 2^-126, where what is
    # left is at most 88 * 2^-126; and the type's own smallest steps.
    tol = (lr.HALF[dtype] * 1.01 + 2.0 ** -20) * ref.abs() + lr.TINY[dtype] + 100 * 2.0 ** -126
    assert bool(((y.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("lens,max_len", [([3] * 20, 3), ([40, 20], 40), ([1] * 60, None)])
@pytest.mark.parametrize("P,S", [(64, 128), (128, 64)])
def test_gate(gdn, lens, max_len, P, S):
    """Windows token by token, prompts in chunks, single tokens.  D x is a power of two and the state adds nothing to it, so that the
    output is the gate's value times it, exactly."""
    H, T = 2, sum(lens)
    s = test_gpu_ssm.make(32, lens, H, P, 1, S)
    s["x"].fill_(0.5), s["B"].fill_(0.0), s["state"].fill_(0.0), s["D"].fill_(0.25)
    s["z"].copy_(spread(T * H * P, torch.bfloat16).reshape(T, H, P))
    if max_len is None:
        y = gdn.ssm_decode_step(s["x"], s["dt"], s["B"], s["C"], s["A_log"], s["dt_bias"], s["state"], s["slots"], D=s["D"], z=s["z"])
    else:
        y, _, status = test_gpu_ssm.prefill(gdn, s, max_len=max_len)
        assert status == 0
    z = s["z"].double()
    ref = z * torch.sigmoid(z) / 8
    assert bool(y.isfinite().all())
    tol = (2.0 ** -8 * 1.01 + 2.0 ** -20) * ref.abs() + 100 * 2.0 ** -126
    assert bool(((y.double() - ref).abs() <= tol).all())
