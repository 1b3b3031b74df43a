"""attn_paged's tile kernel (tcgen05) on the GPU: calls with more rows per key head than the row kernel takes.

The caches are made on the GPU and are larger than those of test_gpu_attn.py, so that a CTA walks many key
tiles and units.  The plain form is in 64 bits; its bounds are those of test_gpu_attn.py."""
import math

import pytest
import torch

from gpu_util import library

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


def make(seed, new, kv, hq, hkv, dim, page, dtype, f8, spread=1.0):
    """A cache of shuffled pages; NaN where no token was written, table entries past a sequence's pages -1."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages_of = [-(-k // page) for k in kv]
    total = sum(pages_of) + 3
    perm = torch.randperm(total, generator=g, device="cuda")
    table = torch.full((len(kv), max(max(pages_of), 1)), -1, dtype=torch.int64, device="cuda")
    live = torch.zeros((total, page), dtype=torch.bool, device="cuda")
    at = 0
    for n, c in enumerate(pages_of):
        table[n, :c] = perm[at:at + c]
        at += c
        t = torch.arange(kv[n], device="cuda")
        live[table[n, t // page], t % page] = True
    live = live[:, None, :].expand(total, hkv, page)
    x = {"table": table, "kv": kv, "cu": [sum(new[:n]) for n in range(len(new) + 1)]}
    for name, shift in (("k", 0.0), ("v", 0.25)):
        vals = torch.randn((total, hkv, page, dim), generator=g, device="cuda") * spread + shift
        if f8:
            scale = torch.exp2(torch.randint(-7, -3, (total, hkv, page), generator=g, device="cuda").float())
            vals = (vals / scale[..., None]).clamp(-448, 448)
            x[name + "_scale"] = torch.where(live, scale, math.nan)
        else:
            x[name + "_scale"] = None
        vals[~live] = math.nan
        x[name] = vals.to(F8 if f8 else dtype)
    x["q"] = (torch.randn((sum(new), hq, dim), generator=g, device="cuda") * 1.5).to(dtype)
    return x


def call(gdn, x, scale, **kw):
    """(out, lse, status) of one call that reaches the tile kernel."""
    T, hq, _ = x["q"].shape
    assert T * (hq // x["k"].shape[1]) > 64, "the row kernel would take this call"
    lse = torch.full((T, hq), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gdn.attn_paged(x["q"], x["k"], x["v"], x["table"], torch.tensor(x["kv"]).cuda(), torch.tensor(x["cu"]).cuda(), T,
                         scale=scale, k_scale=x["k_scale"], v_scale=x["v_scale"], lse=lse, dev_status=status, **kw)
    torch.cuda.synchronize()
    return out, lse, int(status.item())


def rows_of(x, which, n):
    """Sequence n's cached rows in 64 bits: [H, L, D]."""
    c, s, L = x[which], x[which + "_scale"], x["kv"][n]
    pages = x["table"][n, :-(-L // c.shape[2])]
    r = (c.view(torch.uint8)[pages].view(F8) if s is not None else c[pages]).double()
    if s is not None:
        r = r * s[pages].double()[..., None]
    return r.transpose(0, 1).reshape(c.shape[1], -1, c.shape[3])[:, :L]


def check(x, out, lse, scale, seqs=None):
    """out and lse of the sequences `seqs` (all of them) against the definition."""
    u = UNIT[x["q"].dtype]
    up = 2.0 ** -11 if x["k"].dtype == F8 else u
    hq, hkv = x["q"].shape[1], x["k"].shape[1]
    for n in range(len(x["kv"])) if seqs is None else seqs:
        a, b, L = x["cu"][n], x["cu"][n + 1], x["kv"][n]
        m = b - a
        if m == 0:
            continue
        k, v = rows_of(x, "k", n), rows_of(x, "v", n)
        q = x["q"][a:b].double().reshape(m, hkv, hq // hkv, -1).transpose(0, 1)        # [hkv, m, G, D]
        s = torch.einsum("hmgd,hld->hmgl", q, k) * scale
        sees = torch.arange(L, device="cuda") <= torch.arange(m, device="cuda")[:, None] + (L - m)
        s = s.masked_fill(~sees[None, :, None], -math.inf)
        z = torch.logsumexp(s, -1)
        none = z == -math.inf
        w = torch.exp(s - torch.where(none, 0.0, z)[..., None])
        ref, wabs = torch.einsum("hmgl,hld->hmgd", w, v), torch.einsum("hmgl,hld->hmgd", w, v.abs())
        e = 8e-6 * (1 + float(torch.einsum("hmgd,hld->hmgl", q.abs(), k.abs()).max()) * abs(scale) if L else 1)
        got = out[a:b].double().reshape(m, hkv, hq // hkv, -1).transpose(0, 1)
        glse = lse[a:b].double().reshape(m, hkv, hq // hkv).transpose(0, 1)
        tol = u * ref.abs() + (up + e) * wabs + L * 2.0 ** -25 * (float(v.abs().max()) if L else 0.0)
        assert bool(((got - ref).abs() <= tol).all()), (n, float(((got - ref).abs() / tol.clamp(min=1e-30)).max()))
        assert bool((torch.isinf(glse) == none).all()) and bool((glse[none] < 0).all()) and bool((got[none] == 0).all())
        off = (glse - z)[~none].abs() - 2.0 ** -22 * z[~none].abs()
        assert off.numel() == 0 or float(off.max()) <= e, (n, float(off.max()))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_bad_page_amid_a_sequence(gdn, dim, f8):
    # about ten key tiles per CTA (20 of 64 keys), the bad entries anywhere among them; page and box of 16 rows
    kv, new = [9000, 14000, 70], [20, 20, 20]
    x = make(21, new, kv, 32, 8, dim, 16, torch.bfloat16, f8)
    good, glse, status = call(gdn, x, 0.07)
    assert status == 0
    check(x, good, glse, 0.07)
    others = [i for i in range(60) if not 20 <= i < 40]
    for seed in range(12):
        g = torch.Generator().manual_seed(seed)
        t = x["table"].clone()
        for i in torch.randint(0, 14000 // 16, (1 + seed,), generator=g).tolist():
            t[1, i] = x["k"].shape[0] if i % 2 else -1
        out, lse, status = call(gdn, dict(x, table=t), 0.07)
        assert status == gdn.STATUS_BAD_CACHE_INDEX, (seed, status)
        assert torch.equal(out[others], good[others]) and torch.equal(lse[others], glse[others]), seed


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_short_prompts(gdn, dim, f8):
    # some forty units per CTA, of one to four key tiles and of few or many rows, so that a unit's roles are in
    # step with those of the units before and behind it, or out of step as far as the barriers let them
    kv = [20 + (53 * n) % 231 for n in range(1500)]
    x = make(22, kv, kv, 8, 2, dim, 32, torch.bfloat16, f8)
    first = call(gdn, x, 0.08)
    assert first[2] == 0
    check(x, first[0], first[1], 0.08, range(0, 1500, 31))
    for i in range(40):
        again = call(gdn, x, 0.08)
        assert again[2] == 0, i
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1]), i


FORMS = [
    # new, kv, hq, hkv, page
    ([70], [70], 4, 4, 16),                              # one prompt, a row per token
    ([65, 0, 2], [63, 0, 5], 2, 2, 7),                   # more queries than keys; an empty sequence; a page with no factor of 8
    ([1] * 70, [(37 * n) % 260 for n in range(70)], 8, 2, 1),   # single tokens, one of them without a key; pages of one token
    ([9, 33, 1], [400, 1000, 129], 6, 2, 48),            # groups of 3
    ([130, 257], [300, 257], 12, 2, 100),                # groups of 6; a page of 100
    ([8] * 12, [128 * n + 1 for n in range(1, 13)], 32, 2, 24),  # windows that end one key into a tile; 8 rows to a box
    ([40], [5000], 20, 1, 128),                          # a group of 20
    ([3, 1], [900, 64], 128, 1, 64),                     # the widest
    ([200, 1], [3000, 3000], 16, 1, 256),
]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_forms(gdn, form, dim, dtype, f8):
    new, kv, hq, hkv, page = FORMS[form]
    x = make(100 * form + dim, new, kv, hq, hkv, dim, page, dtype, f8)
    out, lse, status = call(gdn, x, dim ** -0.5)
    assert status == 0
    check(x, out, lse, dim ** -0.5)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_sharp_flat_and_negative_scores(gdn, dim, f8):
    # scores over hundreds (the running reference has to move, weights underflow), all equal, and of the other sign
    x = make(23, [25, 90], [1700, 260], 8, 2, dim, 16, torch.bfloat16, f8, spread=6.0)
    for scale in (1.0, 0.0, -0.25):
        out, lse, status = call(gdn, x, scale)
        assert status == 0
        check(x, out, lse, scale)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rising_scores(gdn, dim, f8):
    # keys in an order in which every tile raises the maximum
    x = make(24, [80], [3500], 1, 1, dim, 32, torch.bfloat16, f8)
    t = torch.arange(3500, device="cuda")
    page, off = x["table"][0, t // 32], t % 32
    k = torch.zeros((3500, dim), device="cuda")
    k[:, 0] = t / 8
    if f8:
        x["k_scale"][page, 0, off] = torch.exp2(torch.floor(t / 256))
        k[:, 0] = 8 + t % 8
        x["k"].view(torch.uint8)[page, 0, off] = k.to(F8).view(torch.uint8)
    else:
        x["k"][page, 0, off] = k.bfloat16()
    x["q"][:] = 0
    x["q"][:, :, 0] = 1.0
    out, lse, status = call(gdn, x, 0.125 if f8 else 1.0)
    assert status == 0
    check(x, out, lse, 0.125 if f8 else 1.0)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("power", [-20, 13])
def test_scales_of_any_size(gdn, power, dim):
    # an 8-bit cache whose values are very small or very large, their scales 2^40 apart within a sequence
    x = make(25, [20, 30], [400, 170], 8, 2, dim, 16, torch.bfloat16, True)
    x["v_scale"] = x["v_scale"] * 2.0 ** power
    x["k_scale"] = x["k_scale"] * 2.0 ** power
    x["q"] = (x["q"].float() * 2.0 ** -power).bfloat16()
    x["v_scale"][:, :, ::2] *= 2.0 ** -40
    out, lse, status = call(gdn, x, dim ** -0.5)
    assert status == 0
    check(x, out, lse, dim ** -0.5)


@pytest.mark.parametrize("garbage", [math.inf, -3.0e38, math.nan])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_memory_past_the_end_is_not_used(gdn, dim, f8, garbage):
    x = make(26, [20, 40], [33, 300], 8, 2, dim, 64, torch.bfloat16, f8)
    good = call(gdn, x, 0.1)
    check(x, good[0], good[1], 0.1)
    for name in ("k", "v"):
        if f8:  # 8-bit values have no infinity
            x[name + "_scale"] = torch.where(x[name + "_scale"].isnan(), garbage, x[name + "_scale"])
        else:
            x[name] = torch.where(x[name].isnan(), torch.tensor(garbage, dtype=torch.bfloat16, device="cuda"), x[name])
    again = call(gdn, x, 0.1)
    assert again[2] == 0 and torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_malformed_bounds_are_reported(gdn, dim, f8):
    x = make(27, [20, 20, 20], [200, 300, 400], 8, 2, dim, 16, torch.bfloat16, f8)
    good = call(gdn, x, 0.1)[0]
    for bad in (16 * x["table"].shape[1] + 1, -1, 1 << 40):
        keep = torch.full_like(good, 5.0)
        out, lse, status = call(gdn, dict(x, kv=[200, bad, 400]), 0.1, out=keep)
        assert status == gdn.STATUS_BAD_SEQLENS
        check(x, out, lse, 0.1, (0, 2))
        assert bool((out[20:40] == 5).all()) and bool((lse[20:40] == 7).all())
    # bounds that begin below 0, decrease or pass T: those sequences are skipped, the others are not
    for cu, rest, untouched in (([0, 20, 61, 60], (0,), range(20, 60)), ([0, 20, 10, 10], (0,), range(20, 60)),
                                ([-1, 20, 40, 60], (1, 2), range(20))):
        keep = torch.full_like(good, 5.0)
        out, lse, status = call(gdn, dict(x, cu=cu), 0.1, out=keep)
        assert status == gdn.STATUS_BAD_SEQLENS
        check(x, out, lse, 0.1, rest)
        assert bool((out[list(untouched)] == 5).all()) and bool((lse[list(untouched)] == 7).all())


@pytest.mark.parametrize("f8", [False, True])
def test_offsets_beyond_32_bits(gdn, f8):
    # a cache of over 2^31 bytes (2^32 in 16 bits), the sequence in its last pages
    pages, hkv, page, dim = 2200, 16, 512, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    x = {"kv": [900], "cu": [0, 70], "table": torch.tensor([[pages - 1, pages - 3]]).cuda(), "k_scale": None, "v_scale": None,
         "q": torch.randn((70, hkv, dim), generator=g, device="cuda").bfloat16()}
    for name in ("k", "v"):
        c = torch.empty((pages, hkv, page, dim * (1 if f8 else 2)), dtype=torch.uint8, device="cuda").view(F8 if f8 else torch.bfloat16)
        rows = torch.randn((2, hkv, page, dim), generator=g, device="cuda").to(c.dtype)
        c.view(torch.uint8)[x["table"][0]] = rows.view(torch.uint8)
        x[name] = c
        if f8:
            x[name + "_scale"] = torch.full((pages, hkv, page), 0.5, device="cuda")
    out, lse, status = call(gdn, x, dim ** -0.5)
    assert status == 0
    check(x, out, lse, dim ** -0.5)


def test_rows_past_the_coordinates_of_a_box(gdn):
    # over 2^31 rows of 64 bytes: too many for a box's coordinates, so the copies go without
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 150 GB")
    pages, hkv, page, dim = 16500, 8, 16384, 64
    x = {"kv": [20000], "cu": [0, 20], "table": torch.tensor([[pages - 1, 1]]).cuda()}
    g = torch.Generator(device="cuda").manual_seed(4)
    x["q"] = torch.randn((20, 4 * hkv, dim), generator=g, device="cuda").bfloat16()
    one = torch.empty((pages, hkv, page, dim), dtype=torch.uint8, device="cuda").view(F8)
    rows = torch.randn((2, hkv, page, dim), generator=g, device="cuda").to(F8)
    one.view(torch.uint8)[x["table"][0]] = rows.view(torch.uint8)
    scale = torch.ones((pages, hkv, page), device="cuda")
    out, lse = torch.empty_like(x["q"]), torch.empty((20, 4 * hkv), device="cuda")
    # keys and values in one buffer: 138 GB of it
    for max_q in (1, 20):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.attn_paged(x["q"], one, one, x["table"], torch.tensor(x["kv"]).cuda(), torch.tensor(x["cu"]).cuda(), max_q, scale=0.125,
                       k_scale=scale, v_scale=scale, out=out, lse=lse, dev_status=status)
        assert status.item() == 0
        check(dict(x, k=one, v=one, k_scale=scale, v_scale=scale), out, lse, 0.125)
    del one, scale
    torch.cuda.empty_cache()


def test_other_stream_strided_queries_given_buffers(gdn):
    x = make(28, [30, 50], [90, 700], 8, 2, 64, 16, torch.float16, False)
    wide = torch.randn((80, 15, 64), device="cuda").half()
    wide[:, 2:10] = x["q"]
    y = dict(x, q=wide[:, 2:10])
    out = torch.empty((80, 8, 64), dtype=torch.float16, device="cuda")
    ws = torch.full((gdn.attn_paged_workspace_size(64),), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got, lse, status = call(gdn, y, 0.125, out=out, workspace=ws)
    assert status == 0 and got.data_ptr() == out.data_ptr()
    check(x, got, lse, 0.125)
