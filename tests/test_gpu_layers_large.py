"""Offsets past 32 bits in the convolution, the scan, the append and the norm: rows far apart, slots at the end of large pools and caches, against
the same rows close together, bit for bit."""
import pytest
import torch

from gpu_util import library

pytestmark = pytest.mark.gpu
B16 = torch.bfloat16


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


def rnd(*s, seed=0):
    return torch.randn(s, generator=torch.Generator().manual_seed(seed)).cuda()


def apart(x, stride):
    """The rows of x [T, C] in a buffer of T * stride elements."""
    wide = torch.empty(x.shape[0] * stride, dtype=x.dtype, device="cuda").as_strided(x.shape, (stride, 1))
    wide.copy_(x)
    return wide


@pytest.mark.parametrize("T,C,stride", [(300, 16, 1 << 23), (40000, 1024, 1 << 17)])
def test_conv(gdn, T, C, stride):
    assert T * stride > 1 << 31
    x, w = rnd(T, C).to(B16), rnd(C, 4, seed=1)
    cu = torch.tensor([0, T - 5, T], device="cuda")
    pool = torch.empty(((1 << 31) // (3 * C) + 10, C, 3), device="cuda")
    idx = torch.tensor([pool.shape[0] - 1, pool.shape[0] - 7], device="cuda")
    small = rnd(2, C, 3, seed=2)
    pool[idx] = small
    far, = gdn.short_conv(apart(x, stride), w, pool, idx, cu)
    near, = gdn.short_conv(x, w, small, torch.arange(2, device="cuda"), cu)
    assert torch.equal(far, near) and torch.equal(pool[idx], small)


@pytest.mark.parametrize("T,max_len", [(300, 300), (9, 9)])
def test_scan(gdn, T, max_len):
    H, P, S = 16, 64, 128
    stride = (1 << 31) // T // 8 * 8 + 64
    x, B, C, z = (rnd(T, n, seed=i).to(B16) for i, n in enumerate((H * P, S, S, H * P)))
    dt, A, b = rnd(T, H, seed=5).to(B16), rnd(H, seed=6), rnd(H, seed=7) - 4
    cu = torch.tensor([0, T], device="cuda")
    pool = torch.empty(((1 << 31) // (H * P * S) + 3, H, P, S), device="cuda")
    small = rnd(1, H, P, S, seed=8)
    idx = torch.tensor([pool.shape[0] - 1], device="cuda")
    pool[idx] = small

    def run(f, state, at):
        X, Z = (f(t).unflatten(1, (H, P)) for t in (x, z))
        return gdn.ssm_prefill_chunked(X, f(dt), f(B).unflatten(1, (1, S)), f(C).unflatten(1, (1, S)), A, b, state, at, cu, max_len, z=Z)
    far = run(lambda t: apart(t, stride), pool, idx)
    near = run(lambda t: t, small, torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert torch.equal(far, near) and torch.equal(pool[idx], small)


@pytest.mark.parametrize("f8", [False, True])
def test_append(gdn, f8):
    T, H, D, page = 50, 8, 128, 64
    pages = (1 << 32) // (H * page * D) + 5
    kind = torch.float8_e4m3fn if f8 else B16
    large = [torch.empty((pages, H, page, D), dtype=torch.uint8 if f8 else B16, device="cuda") for _ in range(2)]
    large = [c.view(kind) if f8 else c for c in large]
    small = [torch.zeros((1, H, page, D), dtype=torch.uint8, device="cuda").view(kind) if f8 else torch.zeros((1, H, page, D), dtype=B16, device="cuda")
             for _ in range(2)]
    scales = [[torch.ones((n, H, page), device="cuda") if f8 else None for _ in range(2)] for n in (pages, 1)]
    q, k, v = (rnd(T, n, D, seed=i).to(B16) for i, n in enumerate((16, H, H)))
    angle = rnd(T, D // 2, seed=4)
    rot, at = torch.cat([angle.cos(), angle.sin()], 1), torch.arange(T, device="cuda")
    far = gdn.attn_cache_append(q, k, v, rot, at, at + (pages - 1) * page, *large, *scales[0])
    near = gdn.attn_cache_append(q, k, v, rot, at, at, *small, *scales[1])
    assert torch.equal(far, near)
    for c, d, s, r in zip(large, small, *scales):
        assert torch.equal(c[-1, :, :T].view(torch.uint8), d[0, :, :T].view(torch.uint8))
        assert s is None or torch.equal(s[-1], r[0])


@pytest.mark.parametrize("e4m3", [False, True])
def test_norm(gdn, e4m3):
    C, T = 32768, 70000
    assert T * C > 1 << 31
    x, res, w = rnd(3, C).to(B16), rnd(3, C, seed=1).to(B16), rnd(C, seed=2)
    X, R = (torch.zeros((T, C), dtype=B16, device="cuda") for _ in range(2))
    X[-3:], R[-3:] = x, res
    far = gdn.add_rms_norm(X, w, R, e4m3=e4m3, group=128 if e4m3 else 0)
    near = gdn.add_rms_norm(x, w, res, e4m3=e4m3, group=128 if e4m3 else 0)
    assert torch.equal(R[-3:], res)
    for a, b in zip(far, near) if e4m3 else [(far, near)]:
        assert torch.equal(a[-3:].view(torch.uint8), b.view(torch.uint8))
