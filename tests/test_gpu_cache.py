"""attn_cache_write and attn_cache_read on the GPU.  Quantisation by a power of two is exact up to the one
rounding to e4m3, so every comparison here is of equal numbers."""
import numpy as np
import pytest
import torch

import attn_reference as ar
from gpu_util import library

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


def same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=12345.0), torch.nan_to_num(b, nan=12345.0)) and torch.equal(a.isnan(), b.isnan())


def rows(seed, T, H, D, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, D), generator=g) * torch.exp(2 * torch.randn((T, H, 1), generator=g))
    x = x.to(dtype)
    if T > 3:
        x[0] = 0                                   # a row of zeros
        x[1, :, 0] = 448.0 * 2.0 ** -5             # largest element exactly 448 times a power of two
        x[1, :, 1:] = x[1, :, 1:].clamp(-1, 1)
        x[2, 0, 0], x[2, 0, 1], x[2, 0, 2] = float("inf"), float("-inf"), float("nan")
        x[3] = (x[3].float() * (2.0 ** -120 if dtype == torch.bfloat16 else 2.0 ** -22)).to(dtype)  # tiny, subnormal
    return x


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 64, 16), (5, 3, 128, 7), (17, 2, 256, 1), (200, 4, 128, 64), (2500, 2, 64, 48),
                                        (2049, 1, 256, 100)])
def test_write_and_read_back(gdn, T, H, D, page, dtype, f8):
    k, v = rows(T, T, H, D, dtype), rows(T + 1, T, H, D, dtype)
    pages = -(-T // page) + 2
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[T // 2] = -1                              # a token that is left out
    ct = F8 if f8 else dtype
    caches, scales = [], []
    for _ in range(2):
        caches.append(torch.full((pages, H, page, D), 3.0).to(ct).cuda())
        scales.append(torch.full((pages, H, page), 7.0, device="cuda") if f8 else None)
    # the sources are slices of one wider row per token
    wide = torch.zeros((T, 2 * H + 1, D), dtype=dtype)
    wide[:, :H], wide[:, H + 1:] = k, v
    wide = wide.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.attn_cache_write(wide[:, :H], wide[:, H + 1:], slots.cuda(), *caches, *scales, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for x, c, s in zip((k, v), caches, scales):
        want = torch.full((pages, H, page, D), 3.0).to(ct).float()
        wscale = torch.full((pages, H, page), 7.0)
        val, sc = (torch.from_numpy(a).float() for a in ar.quantise(x.double().numpy())) if f8 else (x.float(), None)
        for t in range(T):
            if slots[t] >= 0:
                want[slots[t] // page, :, slots[t] % page] = val[t]
                if f8:
                    wscale[slots[t] // page, :, slots[t] % page] = sc[t]
        assert same(c.float().cpu(), want)
        if f8:
            assert torch.equal(s.cpu(), wscale)
    # read back by a page table: pages in order, as two sequences
    table = torch.arange(pages).repeat(2, 1)
    total = pages * page
    a = total // 3
    cu = torch.tensor([0, a, total])
    rk, rv = gdn.attn_cache_read(*caches, table.cuda(), cu.cuda(), total, dtype=dtype, k_scale=scales[0], v_scale=scales[1],
                                 dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for got, c, s in zip((rk, rv), caches, scales):
        flat = c.float().cpu() * (s.cpu()[..., None] if f8 else 1.0)
        flat = flat.transpose(1, 2).reshape(total, H, D).to(dtype)
        assert same(got.float().cpu(), torch.cat([flat[:a], flat[:total - a]]).float())


def test_written_values_round_to_even(gdn):
    # every positive bf16 of some binades in one row each with a 448: scale 1, so the values are the roundings
    x = torch.cat([torch.arange(i * 64, (i + 1) * 64).float()[None] for i in range(0, 400)]).reshape(400, 64)
    bits = (x.reshape(-1)[: 400 * 63].to(torch.int32) + (100 << 7)).to(torch.int16).view(torch.bfloat16).float()
    bits = torch.where(bits <= 448, bits, torch.tensor(1.0)).reshape(400, 63)
    x = torch.cat([torch.full((400, 1), 448.0), bits], 1).reshape(400, 1, 64).bfloat16()
    kc = torch.zeros((400, 1, 1, 64), device="cuda").to(F8)
    vc = kc.clone()
    ks, vs = torch.zeros((400, 1, 1), device="cuda"), torch.zeros((400, 1, 1), device="cuda")
    gdn.attn_cache_write(x.cuda(), x.cuda(), torch.arange(400).cuda(), kc, vc, ks, vs)
    want = ar.e4m3_round(x.double().numpy()).reshape(400, 1, 1, 64)
    assert np.array_equal(kc.float().cpu().double().numpy(), want) and torch.equal(kc.float(), vc.float())
    assert bool((ks == 1).all())


def test_out_of_range_is_reported_and_not_written(gdn):
    kc = torch.zeros((4, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.attn_cache_write(x, x, torch.tensor([0, 32, 1 << 40]).cuda(), kc, vc, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == gdn.STATUS_BAD_CACHE_INDEX
    assert float(kc.float().sum()) == 2 * 64 and float(vc.float().sum()) == 2 * 64
    # reading: a page outside the cache, and a sequence longer than its table
    status.zero_()
    out = [torch.full((10, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gdn.attn_cache_read(kc, vc, torch.tensor([[0, 4]]).cuda(), torch.tensor([0, 10]).cuda(), 10, k=out[0], v=out[1], dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == gdn.STATUS_BAD_CACHE_INDEX
    assert bool((out[0][8:] == 5).all()) and bool((out[0][0] == 1).all())
    status.zero_()
    gdn.attn_cache_read(kc, vc, torch.tensor([[0]]).cuda(), torch.tensor([0, 10]).cuda(), 10, k=out[0], v=out[1], dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == gdn.STATUS_BAD_SEQLENS


def test_large_offsets(gdn):
    pages, H, page, D = 2200, 16, 512, 256      # over 2^32 elements
    kc = torch.empty((pages, H, page, D), dtype=torch.uint8, device="cuda").view(F8)
    vc = torch.empty((pages, H, page, D), dtype=torch.uint8, device="cuda").view(F8)
    ks, vs = (torch.empty((pages, H, page), device="cuda") for _ in range(2))
    x = rows(2, 3, H, D, torch.bfloat16)
    slots = torch.tensor([pages * page - 1, 0, (pages - 1) * page + 5])
    gdn.attn_cache_write(x.cuda(), (-x).cuda(), slots.cuda(), kc, vc, ks, vs)
    table = (slots // page)[:, None]
    for t in range(3):
        off = int(slots[t] % page)
        k, v = gdn.attn_cache_read(kc, vc, table[t:t + 1].cuda(), torch.tensor([0, off + 1]).cuda(), off + 1, k_scale=ks, v_scale=vs)
        val, sc = ar.quantise(x[t].double().numpy())
        want = torch.from_numpy(val * sc[..., None]).float()
        assert torch.equal(k[off].float().cpu(), want) and torch.equal(v[off].float().cpu(), -want)


def test_no_tokens_and_refusals(gdn):
    kc = torch.zeros((4, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    gdn.attn_cache_write(none, none, torch.empty(0, dtype=torch.int64, device="cuda"), kc, vc)
    x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.arange(3).cuda()
    with pytest.raises(TypeError):
        gdn.attn_cache_write(x.half(), x.half(), s, kc, vc)
    with pytest.raises(ValueError):
        gdn.attn_cache_write(x, x, s[:2], kc, vc)
    with pytest.raises(gdn.GdnError):
        gdn.attn_cache_write(x, x, s, kc, kc)
    with pytest.raises(gdn.GdnError):  # 96 features
        gdn.attn_cache_write(torch.ones((3, 2, 96), dtype=torch.bfloat16, device="cuda"),
                             torch.ones((3, 2, 96), dtype=torch.bfloat16, device="cuda"), s,
                             *(torch.zeros((4, 2, 8, 96), dtype=torch.bfloat16, device="cuda") for _ in range(2)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_at_the_top_of_the_range(gdn, dtype):
    # 256 times the largest scale is past the type's range: what would round to it becomes 240 times it, and what
    # comes back, and what is computed with it, is finite
    big = torch.finfo(dtype).max
    s = 2.0 ** (8 if dtype == torch.float16 else 120)
    f = torch.tensor([255.0, 248.0, 247.0, 240.0, 232.0, 225.0, 224.5, 224.0]) * s
    x = torch.randn((16, 2, 64), generator=torch.Generator().manual_seed(9)) * 8 * s
    x = x.clamp(-0.5 * big, 0.5 * big)
    for i in range(8):
        x[i, 0, 3], x[8 + i, 1, 5] = f[i], -f[i]
    x[0, 1, 7], x[1, 1, 7], x[2, 1, 7], x[3, 1, 7] = big, -big, float("inf"), float("nan")
    x[2, 1, 8] = big
    x = x.to(dtype)
    kc, vc = (torch.zeros((2, 2, 8, 64), device="cuda").to(F8) for _ in range(2))
    ks, vs = (torch.ones((2, 2, 8), device="cuda") for _ in range(2))
    gdn.attn_cache_write(x.cuda(), x.cuda(), torch.arange(16).cuda(), kc, vc, ks, vs)
    val, sc = ar.quantise(x.double().numpy())       # to nearest, and at the top scale 240 in the place of 256
    val = np.where((sc[..., None] == s) & (np.abs(val) == 256), np.sign(val) * 240, val)
    want = torch.from_numpy(val * sc[..., None]).float()
    assert int((torch.from_numpy(sc) == s).sum()) >= 10
    table, cu = torch.tensor([[0, 1]]).cuda(), torch.tensor([0, 16]).cuda()
    k, v = gdn.attn_cache_read(kc, vc, table, cu, 16, dtype=dtype, k_scale=ks, v_scale=vs)
    assert same(k.float().cpu(), want) and same(v.float().cpu(), want)
    assert bool(torch.isfinite(k)[x.cuda().isfinite()].all())
    assert float(((k.double().cpu() - x.double()).abs() / x.double().abs().clamp(min=s))[x.isfinite()].max()) <= 2.0 ** -4
    # a token whose one key is such a row: the output is that row
    for t in (0, 1, 5):
        one = torch.tensor([[0]]).cuda()
        kc1, vc1 = (c.view(torch.uint8)[:, :, t:t + 1].contiguous().view(F8) for c in (kc, vc))
        ks1, vs1 = (c[:, :, t:t + 1].contiguous() for c in (ks, vs))
        q = torch.zeros((40, 2, 64), dtype=dtype, device="cuda")
        for T in (1, 40):
            lens, n = torch.ones(T, dtype=torch.int64).cuda(), torch.arange(T + 1).cuda()
            out = gdn.attn_paged(q[:T], kc1, vc1, one.expand(T, 1).contiguous(), lens, n, 1, k_scale=ks1, v_scale=vs1)
            assert torch.equal(out.float().cpu(), want[t].expand(T, 2, 64)), (t, T)


@pytest.mark.parametrize("cu", [[0, 10, 5, 12], [0, 12, 11, 12], [0, 5, 40, 12], [-3, 4, 8, 12], [0, 4, 8, 13], [20, 20, 12, 12]])
def test_malformed_bounds_are_reported(gdn, cu):
    # a sequence that ends before it begins, begins below 0 or ends past T, whether or not a row falls to it
    kc = torch.ones((4, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 1], [2, 3], [1, 2]]).cuda()
    for bounds, bad in ((cu, True), ([0, 4, 4, 12], False)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.attn_cache_read(kc, kc.clone(), table, torch.tensor(bounds).cuda(), 12, dev_status=status)
        assert status.item() == (gdn.STATUS_BAD_SEQLENS if bad else 0)
