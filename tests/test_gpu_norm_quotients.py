"""add_rms_norm to e4m3 next to the middles between two values.  Rows of ones have a root mean square of one, so that y is the weight itself, which
may be any fp32 number: quotients are put on either side of every middle."""
import pytest
import torch

from gpu_util import library

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("C,group", [(256, 0), (1024, 0), (1024, 256), (8192, 128), (20480, 64)])
def test_next_to_the_middles(gdn, C, group, dtype):
    n = group or C
    g = torch.Generator().manual_seed(C + group)
    values = torch.arange(1, 127, dtype=torch.uint8).view(F8).double()  # 2^-9 .. 448
    middles = (values[1:] + values[:-1]) / 2
    groups = C // n
    top = torch.exp2(3 * torch.rand((groups, 1), generator=g, dtype=torch.float64)).float()  # each group's largest
    scale = top / 448
    pick = middles[torch.randint(len(middles), (groups, n), generator=g)]
    off = torch.exp2(-torch.randint(18, 23, (groups, n), generator=g).double()) * (torch.randint(2, (groups, n), generator=g) * 2 - 1)
    weight = (pick * (1 + off) * scale.double()).float()
    weight[:, n // 2] = top[:, 0]
    weight *= torch.randint(2, weight.shape, generator=g) * 2 - 1
    x = torch.ones((3, C), dtype=dtype, device="cuda")
    out, s = gdn.add_rms_norm(x, weight.flatten().cuda(), eps=0.0, e4m3=True, group=group)
    assert torch.equal(s.cpu(), scale.T.expand(3, groups))  # the largest over 448, to fp32
    quotient = weight.double() / scale.double()
    size = quotient.abs()
    step = torch.exp2(torch.floor(torch.log2(size.clamp(min=2.0 ** -6))) - 3)
    want = torch.round(size / step) * step * quotient.sign()
    # fp32's quotient is off by 2^-24: nearer to a middle either value is right
    apart = ((size / step - torch.floor(size / step) - 0.5).abs() * step / size) > 1.01 * 2.0 ** -24
    assert float(apart.double().mean()) > 0.9
    got = out.float().cpu().double().reshape(3, groups, n)
    assert bool(((got == want) | ~apart).all()), int(((got != want) & apart).sum())
