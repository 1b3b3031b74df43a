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
