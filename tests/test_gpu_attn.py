"""attn_paged on the GPU against the plain 64-bit form (tests/attn_reference.py), through the binding.

Bounds, derived from the arithmetic (u = 2^-8 for bf16 and 2^-11 for binary16 is the rounding of the
output, up that of the weights: 2^-11 where an 8-bit cache makes the products binary16):
  out   |x - ref| <= u |ref| + (up + e) sum_j w_j |v_j| + n 2^-25 max |v|,  e = 8e-6 (1 + A):
        the output's rounding, one relative rounding per weight, the scores' f32 error (A the largest
        sum |q_i k_i| scale, so a score is off by a few 2^-24 A sqrt(D), and 2^y by as much relatively),
        and the weights that are below binary16's smallest step (n keys);
  lse   |x - ref| <= e + 2^-22 |ref|."""
import numpy as np
import pytest
import torch

import attn_reference as ar
from gpu_util import library

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


def make(seed, new, kv, hq, hkv, dim, page, dtype, f8, spread=1.0, pad=3, garbage=float("nan")):
    """A cache of shuffled pages, garbage where nothing was written, table entries past the end -1."""
    g = torch.Generator().manual_seed(seed)
    pages_of = [-(-k // page) for k in kv]
    total = sum(pages_of) + pad
    perm = torch.randperm(total, generator=g)
    table = torch.full((len(kv), max(max(pages_of, default=0), 1)), -1, dtype=torch.int64)
    at = 0
    for n, c in enumerate(pages_of):
        table[n, :c] = perm[at:at + c]
        at += c
    x = {"table": table, "kv": kv, "cu": np.concatenate([[0], np.cumsum(new)]).tolist()}
    for name, shift in (("k", 0.0), ("v", 0.25)):
        vals = torch.randn((total, hkv, page, dim), generator=g) * spread + shift
        live = torch.zeros((total, page), dtype=torch.bool)
        for n, L in enumerate(kv):
            for t in range(L):
                live[table[n, t // page], t % page] = True
        live = live[:, None, :]
        if f8:
            q, s = ar.quantise(vals.to(dtype).double().numpy())
            q = torch.from_numpy(q).float()
            q[~live.expand(q.shape[:3])] = garbage
            s = torch.from_numpy(s).float()
            s[~live.expand(s.shape)] = garbage
            x[name], x[name + "_scale"] = q.to(F8), s
        else:
            v = vals.to(dtype)
            v[~live.expand(v.shape[:3])] = garbage
            x[name], x[name + "_scale"] = v, None
    x["q"] = (torch.randn((sum(new), hq, dim), generator=g) * 1.5).to(dtype)
    return x


def call(gdn, x, scale, max_q=None, **kw):
    new = np.diff(x["cu"])
    c = {k: (None if x[k] is None else x[k].cuda()) for k in ("k", "v", "k_scale", "v_scale", "table", "q")}
    T, hq, _ = x["q"].shape
    lse = torch.full((T, hq), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gdn.attn_paged(c["q"], c["k"], c["v"], c["table"], torch.tensor(x["kv"], dtype=torch.int64).cuda(),
                         torch.tensor(x["cu"], dtype=torch.int64).cuda(),
                         int(new.max(initial=0)) if max_q is None else max_q, scale=scale, k_scale=c["k_scale"],
                         v_scale=c["v_scale"], lse=lse, dev_status=status, **kw)
    torch.cuda.synchronize()
    return out.cpu().double(), lse.cpu().double(), int(status.item())


def check(x, out, lse, scale):
    dt = x["q"].dtype
    f8 = x["k"].dtype == F8
    ref, rlse, wabs, size, keys, vmax = ar.attention(x["q"], x["k"], x["v"], x["k_scale"], x["v_scale"], x["table"],
                                                     x["kv"], x["cu"], scale)
    e = 8e-6 * (1 + size)
    tol = UNIT[dt] * ref.abs() + ((2.0 ** -11 if f8 else UNIT[dt]) + e) * wabs + keys * 2.0 ** -25 * vmax
    assert bool(((out - ref).abs() <= tol).all()), float(((out - ref).abs() / tol.clamp(min=1e-30)).max())
    none = torch.isinf(rlse)
    assert bool((torch.isinf(lse) == none).all()) and bool((lse[none] < 0).all())
    assert bool((out[none] == 0).all())
    off = (lse - rlse)[~none].abs() - 2.0 ** -22 * rlse[~none].abs()
    assert off.numel() == 0 or float(off.max()) <= e, float(off.max())


FORMS = [
    # new, kv, hq, hkv
    ([1], [1], 4, 4),                                  # one key
    ([1], [63], 8, 2),
    ([1, 1, 1], [64, 65, 1000], 8, 1),                 # tile borders, several CTAs per unit
    ([1, 0, 1, 1], [17, 0, 0, 5], 6, 2),               # empty sequences; a query without a key; G = 3
    ([4, 8, 3], [4, 200, 77], 8, 2),                   # drafted windows; one of them a whole prompt
    ([5, 2], [3, 40], 4, 2),                           # more queries than cached keys: empty rows first
    ([33, 1, 70], [33, 500, 130], 4, 1),               # chunks of several query tiles beside a single token
    ([130, 257], [300, 257], 6, 2),                    # long chunks
    ([3], [90], 16, 1), ([2], [300], 40, 2),           # wide groups: 16 and 20 heads on a key head
    ([2, 1], [70, 9], 128, 1),                         # the widest
]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_against_plain_form(gdn, form, dim, dtype, f8):
    new, kv, hq, hkv = FORMS[form]
    page = (16, 48, 7, 64, 1, 32, 100, 128, 24, 16, 33)[form]
    x = make(1000 * form + dim, new, kv, hq, hkv, dim, page, dtype, f8)
    scale = dim ** -0.5
    out, lse, status = call(gdn, x, scale)
    assert status == 0
    check(x, out, lse, scale)
    # the kernel choice is only a hint: either gives the result
    for max_q in (1, 1000):
        out, lse, status = call(gdn, x, scale, max_q=max_q)
        assert status == 0
        check(x, out, lse, scale)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("max_q", [1, 64])
def test_sharp_and_flat_scores(gdn, f8, max_q):
    # scores over hundreds (the running reference has to move, weights underflow) and all equal
    x = make(5, [1, 9], [700, 260], 4, 2, 128, 16, torch.bfloat16, f8, spread=6.0)
    for scale in (1.0, 0.0, -0.25):
        out, lse, _ = call(gdn, x, scale, max_q=max_q)
        check(x, out, lse, scale)


@pytest.mark.parametrize("max_q", [1, 64])
def test_rising_scores(gdn, max_q):
    # keys ordered so that every tile raises the maximum
    x = make(6, [2], [900], 2, 1, 64, 32, torch.bfloat16, False)
    x["q"][:] = 0
    x["q"][:, :, 0] = 1.0
    for t in range(900):
        x["k"][x["table"][0, t // 32], 0, t % 32] = 0
        x["k"][x["table"][0, t // 32], 0, t % 32, 0] = t / 8
    out, lse, _ = call(gdn, x, 1.0, max_q=max_q)
    check(x, out, lse, 1.0)


@pytest.mark.parametrize("max_q", [1, 64])
@pytest.mark.parametrize("size", [1e-6, 1e4])
def test_scales_of_any_size(gdn, size, max_q):
    # an 8-bit cache whose values, and queries whose elements, are very small or very large
    x = make(7, [1, 3], [130, 70], 4, 2, 128, 16, torch.bfloat16, True)
    x["v_scale"] = x["v_scale"] * 2.0 ** round(np.log2(size))
    x["k_scale"] = x["k_scale"] * 2.0 ** round(np.log2(size))
    x["q"] = (x["q"].float() * 2.0 ** -round(np.log2(size))).bfloat16()
    # rows whose value scales differ by 2^40 within one sequence
    x["v_scale"][:, :, ::2] *= 2.0 ** -40
    out, lse, _ = call(gdn, x, 128 ** -0.5, max_q=max_q)
    check(x, out, lse, 128 ** -0.5)


@pytest.mark.parametrize("max_q", [1, 64])
@pytest.mark.parametrize("garbage", [float("inf"), -3.0e38])
def test_memory_past_the_end_is_not_used(gdn, garbage, max_q):
    x = make(8, [1, 2], [33, 100], 4, 2, 128, 64, torch.bfloat16, False, garbage=garbage)
    out, lse, _ = call(gdn, x, 0.1, max_q=max_q)
    check(x, out, lse, 0.1)


@pytest.mark.parametrize("max_q", [1, 64])
def test_strided_queries_other_stream_given_buffers(gdn, max_q):
    x = make(9, [3, 20], [50, 90], 4, 2, 64, 16, torch.float16, False)
    wide = torch.randn((23, 11, 64)).half()
    wide[:, 2:6] = x["q"]
    y = dict(x, q=wide.cuda()[:, 2:6])
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.empty((23, 4, 64), dtype=torch.float16, device="cuda")
    ws = torch.full((gdn.attn_paged_workspace_size(64),), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        got, lse, status = call(gdn, y, 0.125, max_q=max_q, out=out, workspace=ws)
    assert status == 0 and torch.equal(out.cpu().double(), got)
    check(x, got, lse, 0.125)


@pytest.mark.parametrize("max_q", [1, 64])
def test_repeats_bit_for_bit(gdn, max_q):
    x = make(10, [1, 40, 2], [3000, 1500, 10], 8, 2, 128, 16, torch.bfloat16, False)
    a = call(gdn, x, 0.09, max_q=max_q)
    for _ in range(3):
        b = call(gdn, x, 0.09, max_q=max_q)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("max_q", [1, 64])
def test_same_bits_with_cold_and_warm_caches(gdn, max_q, dim, f8):
    # copies that come late or early, and in another order, change no bit
    x = make(15, [8, 8, 30], [900, 1500, 300], 8, 2, dim, 64, torch.bfloat16, f8)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    first = call(gdn, x, 0.07, max_q=max_q)
    check(x, first[0], first[1], 0.07)
    for i in range(24):
        if i % 2 == 0:
            flush.fill_(i)
        again = call(gdn, x, 0.07, max_q=max_q)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1]), i


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_no_wait_runs_out_at_the_ends_of_units(gdn, dim, f8):
    # many units of one to five key tiles, so that every wait at a unit's end meets early and late arrivals
    kv = [40 + 7 * n for n in range(40)]
    x = make(16, [min(k, 40) for k in kv], kv, 16, 4, dim, 64, torch.bfloat16, f8)
    first = call(gdn, x, 0.06, max_q=64)
    assert first[2] == 0
    check(x, first[0], first[1], 0.06)
    for i in range(100):
        again = call(gdn, x, 0.06, max_q=64)
        assert again[2] == 0, i
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1]), i


@pytest.mark.parametrize("max_q", [1, 64])
def test_many_sequences(gdn, max_q):
    # more sequences than a block has threads, most of them tiny
    kv = [(7 * n) % 40 for n in range(300)]
    new = [min(1 + n % 3, 2) for n in range(300)]
    x = make(11, new, kv, 2, 1, 64, 16, torch.bfloat16, False)
    out, lse, status = call(gdn, x, 0.125, max_q=max_q)
    assert status == 0
    check(x, out, lse, 0.125)


@pytest.mark.parametrize("max_q", [1, 64])
def test_malformed_bounds_are_reported(gdn, max_q):
    x = make(12, [2, 2, 2], [20, 30, 40], 4, 2, 64, 16, torch.bfloat16, False)
    good, glse, _ = call(gdn, x, 0.125, max_q=max_q)
    # a length beyond the page table: that sequence is skipped, the others are not
    y = dict(x, kv=[20, 16 * x["table"].shape[1] + 1, 40])
    keep = torch.full((6, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    out, lse, status = call(gdn, y, 0.125, max_q=max_q, out=keep)
    assert status == gdn.STATUS_BAD_SEQLENS
    assert torch.equal(out[[0, 1, 4, 5]], good[[0, 1, 4, 5]]) and bool((out[2:4] == 5.0).all())
    # a page outside the cache: reported, nothing read there, other sequences unharmed
    t = x["table"].clone()
    t[1, 0] = x["k"].shape[0]
    out, lse, status = call(gdn, dict(x, table=t), 0.125, max_q=max_q)
    assert status == gdn.STATUS_BAD_CACHE_INDEX
    assert torch.equal(out[[0, 1, 4, 5]], good[[0, 1, 4, 5]])


@pytest.mark.parametrize("max_q", [1, 64])
def test_offsets_beyond_32_bits(gdn, max_q):
    # a cache of more than 2^32 bytes and 2^31 elements, the sequence in its last pages
    pages, hkv, page, dim = 2200, 16, 512, 128
    kc = torch.empty((pages, hkv, page, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty((pages, hkv, page, dim), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[pages - 1, pages - 3]])
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((2, hkv, page, dim), generator=g).bfloat16() for _ in range(2))
    kc[table[0].cuda()], vc[table[0].cuda()] = k.cuda(), v.cuda()
    x = {"q": torch.randn((3, hkv, dim), generator=g).bfloat16(), "k": k, "v": v, "k_scale": None, "v_scale": None,
         "table": torch.tensor([[0, 1]]), "kv": [600], "cu": [0, 3]}
    lse = torch.empty((3, hkv), device="cuda")
    out = gdn.attn_paged(x["q"].cuda(), kc, vc, table.cuda(), torch.tensor([600]).cuda(), torch.tensor([0, 3]).cuda(),
                         max_q, lse=lse)
    check(x, out.cpu().double(), lse.cpu().double(), dim ** -0.5)


def test_no_work(gdn):
    x = make(13, [0, 0], [5, 0], 2, 1, 64, 16, torch.bfloat16, False)
    out, lse, status = call(gdn, x, 1.0)
    assert out.numel() == 0 and status == 0


def test_refusals(gdn):
    x = make(14, [1], [8], 4, 2, 64, 16, torch.bfloat16, True)
    c = {k: x[k].cuda() for k in ("k", "v", "k_scale", "v_scale", "table", "q")}
    kv, cu = torch.tensor([8]).cuda(), torch.tensor([0, 1]).cuda()
    sc = dict(k_scale=c["k_scale"], v_scale=c["v_scale"])
    with pytest.raises(TypeError):
        gdn.attn_paged(c["q"].float(), c["k"], c["v"], c["table"], kv, cu, 1, **sc)
    with pytest.raises(TypeError):
        gdn.attn_paged(c["q"].half(), c["k"].to(torch.bfloat16), c["v"].to(torch.bfloat16), c["table"], kv, cu, 1)
    with pytest.raises(TypeError):  # an 8-bit cache without scales
        gdn.attn_paged(c["q"], c["k"], c["v"], c["table"], kv, cu, 1)
    with pytest.raises(ValueError):  # scales on a 16-bit cache
        gdn.attn_paged(c["q"], c["k"].to(torch.bfloat16), c["v"].to(torch.bfloat16), c["table"], kv, cu, 1, **sc)
    with pytest.raises(ValueError):  # tokens whose heads are not contiguous
        gdn.attn_paged(torch.zeros((1, 64, 4), dtype=torch.bfloat16, device="cuda").transpose(1, 2), c["k"], c["v"], c["table"], kv, cu,
                       1, **sc)
    with pytest.raises(gdn.GdnError):  # 3 heads over 2
        gdn.attn_paged(c["q"][:, :3].contiguous(), c["k"], c["v"], c["table"], kv, cu, 1, **sc)
    with pytest.raises(gdn.GdnError):  # workspace too small
        gdn.attn_paged(c["q"], c["k"], c["v"], c["table"], kv, cu, 1, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"), **sc)


def test_workspace_refusals(gdn):
    x = make(17, [1], [8], 4, 2, 64, 16, torch.bfloat16, False)
    size = gdn.attn_paged_workspace_size(64)
    for ws, err in ((torch.empty(size, dtype=torch.uint8), ValueError), (torch.empty(2 * size, dtype=torch.uint8, device="cuda")[::2], ValueError),
                    (0, TypeError)):
        with pytest.raises(err, match="workspace"):
            call(gdn, x, 1.0, workspace=ws)
    # any element type will do; without a workspace, an unsupported head width is still the library's to refuse
    a, b = call(gdn, x, 1.0), call(gdn, x, 1.0, workspace=torch.empty(size // 4, device="cuda"))
    assert torch.equal(a[0], b[0])
    with pytest.raises(gdn.GdnError, match="64, 128 or 256"):
        call(gdn, make(18, [1], [8], 4, 2, 96, 16, torch.bfloat16, False), 1.0)


@pytest.mark.parametrize("new", [[1, 3], [20, 30]])  # the row kernel, the tile kernel
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("power", [120, 100, -100, -125])
def test_queries_of_any_finite_size(gdn, power, dim, new):
    # an 8-bit cache: queries close to the largest and the smallest numbers, keys that bring the scores back
    x = make(19, new, [130, 70], 8, 2, dim, 16, torch.bfloat16, True)
    x["q"] = (x["q"].float() * 2.0 ** power).bfloat16()
    x["k_scale"] = (x["k_scale"].double() * 2.0 ** -power).float()
    out, lse, status = call(gdn, x, dim ** -0.5)
    assert status == 0
    check(x, out, lse, dim ** -0.5)
