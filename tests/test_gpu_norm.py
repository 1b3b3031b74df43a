"""add_rms_norm on the GPU against the definition in 64 bits, the residual bit for bit."""
import pytest
import torch

import layer_reference as lr
from gpu_util import library

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
# the sum of squares: at most 32 terms in a row and 10 levels of pairs; the mean, root and two products: 50 roundings of 2^-24
FP32 = 50 * 2.0 ** -24


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


def make(seed, T, C, dtype, wide=8):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, C + wide), generator=g)).to(dtype)
    res = (3 * torch.randn((T, C), generator=g) * torch.exp(torch.randn(C, generator=g))).to(dtype)
    return x[:, :C], res, 1.0 + 0.3 * torch.randn(C, generator=g)


def reference(x, res, w, eps, dtype):
    r = x if res is None else (x.float() + res.float()).to(dtype)
    d = r.double()
    return r, d * torch.rsqrt(d.square().mean(-1, keepdim=True) + eps) * w.double()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,C", [(1, 8), (5, 64), (3, 264), (9, 1024), (2, 2048), (3, 2056), (7, 4096), (2, 5120), (1, 16384), (2, 16392), (1, 32768)])
def test_sixteen_bits(gdn, T, C, dtype):
    x, res, w = make(T + C, T, C, dtype)
    for with_res in (True, False):
        cres = res.cuda() if with_res else None
        y = gdn.add_rms_norm(x.cuda() if C % 16 else x.cuda().contiguous(), w.cuda(), residual=cres, eps=1e-5)
        r, ref = reference(x, res if with_res else None, w, 1e-5, dtype)
        if with_res:
            assert torch.equal(cres.cpu().view(torch.int16), r.view(torch.int16))
        err = (y.cpu().double() - ref).abs()
        assert bool((err <= (lr.HALF[dtype] * 1.01 + FP32) * ref.abs() + lr.TINY[dtype]).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,C,group", [(1, 8, 0), (5, 64, 32), (5, 64, 64), (3, 264, 0), (4, 512, 256), (3, 1024, 128), (9, 5120, 128), (2, 5120, 0), (3, 2304, 64),
                                       (1, 16384, 0), (2, 20480, 128), (1, 32768, 0)])
def test_eight_bits(gdn, T, C, group, dtype):
    x, res, w = make(T + C + group, T, C, dtype)
    if T > 2:
        res[1] = -x[1]           # a row of zeros
    cres = res.cuda()
    y, scale = gdn.add_rms_norm(x.cuda(), w.cuda(), residual=cres, e4m3=True, group=group)
    r, ref = reference(x, res, w, 1e-6, dtype)
    assert y.dtype == F8 and scale.shape == (T, C // group if group else 1)
    assert torch.equal(cres.cpu().view(torch.int16), r.view(torch.int16))
    parts = ref.reshape(T, scale.shape[1], -1)
    amax = parts.abs().amax(-1)
    want = torch.where(amax > 0, amax / 448.0, 1.0)
    s = scale.cpu().double()
    assert bool(((s - want).abs() <= (FP32 + 2.0 ** -23) * want).all())
    got = y.cpu().float().double().reshape(parts.shape) * s[..., None]
    # half a step of e4m3, 2^-4 of the value or 2^-10 of the scale among its subnormal numbers
    tol = (2.0 ** -4 * 1.001 + 2 * FP32) * parts.abs() + 2.0 ** -10 * s[..., None]
    assert bool(((got - parts).abs() <= tol).all())
    assert bool((y.cpu().float().abs() <= 448).all())


def test_out_may_be_x(gdn):
    x, res, w = make(1, 6, 512, torch.bfloat16, wide=0)
    a = gdn.add_rms_norm(x.cuda(), w.cuda(), residual=res.cuda())
    b = x.cuda()
    assert gdn.add_rms_norm(b, w.cuda(), residual=res.cuda(), out=b) is b
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_rows_do_not_touch_each_other(gdn):
    x, res, w = make(2, 9, 136, torch.float16)
    res[4, 7] = float("inf")
    res[2, 3] = float("nan")
    y = gdn.add_rms_norm(x.cuda(), w.cuda(), residual=res.cuda()).cpu()
    rows = [t for t in range(9) if t not in (2, 4)]
    _, ref = reference(x, res, w, 1e-6, torch.float16)
    assert bool(((y[rows].double() - ref[rows]).abs() <= (2.0 ** -11 * 1.01 + FP32) * ref[rows].abs() + 2.0 ** -25).all())
    assert bool(y[2].isnan().all())


def test_many_rows_and_no_rows(gdn):
    T, C = 70001, 16
    x, _, w = make(3, T, C, torch.bfloat16, wide=0)
    y = gdn.add_rms_norm(x.cuda(), w.cuda())
    _, ref = reference(x, None, w, 1e-6, torch.bfloat16)
    assert bool(((y.cpu().double() - ref).abs() <= (2.0 ** -8 * 1.01 + FP32) * ref.abs()).all())
    assert gdn.add_rms_norm(x[:0].cuda(), w.cuda()).shape == (0, C)


def test_refuses_from_python(gdn):
    x, res, w = make(4, 4, 64, torch.bfloat16, wide=0)
    x, res, w = x.cuda(), res.cuda(), w.cuda()
    for kw, err in ((dict(residual=res.half()), TypeError), (dict(residual=res[:2]), ValueError), (dict(group=32), ValueError), (dict(e4m3=True, group=48), ValueError),
                    (dict(e4m3=True, group=16), gdn.GdnError), (dict(residual=x), gdn.GdnError), (dict(out=res, residual=res), gdn.GdnError),
                    (dict(out=x.float()), TypeError), (dict(scale=w), ValueError)):
        with pytest.raises(err):
            gdn.add_rms_norm(x, w, **kw)
    with pytest.raises(TypeError):
        gdn.add_rms_norm(x.float(), w)
    with pytest.raises(gdn.GdnError):
        gdn.add_rms_norm(x[:, :12], w[:12].contiguous())
    with pytest.raises(ValueError):
        gdn.add_rms_norm(x.T, w)
