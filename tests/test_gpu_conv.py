"""short_conv on the GPU against the definition in 64 bits, the history bit for bit."""
import pytest
import torch

import layer_reference as lr
from gpu_util import library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


def make(seed, lens, C, taps, dtype, extra=2, pad=8):
    """Inputs as slices of wider rows, and `pad` rows of no sequence behind the last."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    s = {"wide": (2.0 * torch.randn((T + pad, C + 16), generator=g)).to(dtype)}
    s["x"] = s["wide"][:, 8:8 + C]
    s["w"], s["bias"] = torch.randn((C, taps), generator=g), torch.randn(C, generator=g)
    s["hist"] = torch.randn((len(lens) + extra, C, taps - 1), generator=g)
    s["slots"] = torch.randperm(len(lens) + extra, generator=g)[:len(lens)]
    s["cu"], s["lens"] = lr.ragged(lens), list(lens)
    return s


def close(got, ref, mag, dtype):
    # the sums: taps products and sums in fp32, each off by 2^-24 of the magnitudes; the activation's slope is at most 1.1 and its
    # exponential and quotient are good to 2^-21 of its value; one rounding of the result
    tol = lr.HALF[dtype] * ref.abs() * 1.01 + lr.TINY[dtype] + 1.2 * 6 * 2.0 ** -24 * mag + 2.0 ** -20 * ref.abs()
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got.double() - ref).abs() / tol).max()))


def run(gdn, s, splits, silu=True, bias=True, step=False):
    dtype = s["x"].dtype
    wide, hist = s["wide"].cuda(), s["hist"].cuda()
    x = wide[:, 8:8 + s["x"].shape[1]]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.full((x.shape[0], w), 9.0, dtype=dtype, device="cuda") for w in splits]
    got = gdn.short_conv(x, s["w"].cuda(), hist, s["slots"].cuda(), None if step else s["cu"].cuda(), bias=s["bias"].cuda() if bias else None,
                         splits=splits, silu=silu, outs=outs, dev_status=status)
    torch.cuda.synchronize()
    assert [o.data_ptr() for o in got] == [o.data_ptr() for o in outs]
    return torch.cat(outs, 1).cpu(), hist.cpu(), status.item()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("lens,splits", [([1], [8]), ([1, 2, 3, 4], [64]), ([5, 0, 16, 1, 0, 17, 15], [24, 8, 40]), ([100, 33], [1024, 8, 128]),
                                         ([0, 48], [1032, 16]), ([3, 1, 1, 1, 1, 1, 2, 1, 30], [96])])
def test_prompts(gdn, lens, splits, taps, dtype):
    s = make(sum(lens) + taps, lens, sum(splits), taps, dtype)
    T = sum(lens)
    for silu, bias in ((True, True), (False, False)):
        y, hist, status = run(gdn, s, splits, silu, bias)
        ref, mag, new = lr.conv(s["x"][:T].double(), s["w"].double(), s["bias"].double() if bias else None, s["hist"].double(), s["slots"].tolist(), lens, silu)
        assert status == 0
        close(y[:T], ref, mag, dtype)
        assert bool((y[T:] == 9.0).all())           # rows of no sequence stay
        assert torch.equal(hist.double(), new)       # the inputs themselves; other slots stay


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("taps,N,splits", [(4, 1, [8]), (4, 65, [256, 16, 16]), (2, 5, [1032]), (3, 7, [64, 64])])
def test_single_tokens(gdn, taps, N, splits, dtype):
    s = make(N, [1] * N, sum(splits), taps, dtype, pad=0)
    y, hist, status = run(gdn, s, splits, step=True)
    ref, mag, new = lr.conv(s["x"].double(), s["w"].double(), s["bias"].double(), s["hist"].double(), s["slots"].tolist(), [1] * N, True)
    assert status == 0
    close(y, ref, mag, dtype)
    assert torch.equal(hist.double(), new)
    again, hist2, _ = run(gdn, s, splits)            # the same by way of bounds
    assert torch.equal(again.view(torch.int16), y.view(torch.int16)) and torch.equal(hist2, hist)


def test_a_prompt_in_pieces(gdn):
    lens, C, taps = [70, 41], 48, 4
    whole = make(1, lens, C, taps, torch.bfloat16, pad=0)
    y, hist, _ = run(gdn, whole, [C])
    now = whole["hist"]
    parts = [[] for _ in lens]
    for a, b in (((0, 0), (1, 2)), ((1, 2), (17, 2)), ((17, 2), (70, 41))):
        piece = dict(whole, lens=[j - i for i, j in zip(a, b)], hist=now)
        rows = torch.cat([torch.arange(whole["cu"][n] + a[n], whole["cu"][n] + b[n]) for n in range(2)])
        piece["wide"] = whole["wide"][rows]
        piece["x"], piece["cu"] = piece["wide"][:, 8:8 + C], lr.ragged(piece["lens"])
        got, now, status = run(gdn, piece, [C])
        assert status == 0
        for n in range(2):
            parts[n].append(got[piece["cu"][n]:piece["cu"][n + 1]])
    assert torch.equal(torch.cat(parts[0] + parts[1]).view(torch.int16), y.view(torch.int16)) and torch.equal(now, hist)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("taps,splits", [(4, [16]), (2, [8]), (3, [1032, 8])])
def test_long_calls(gdn, taps, splits, dtype):
    """Calls of so many tokens that another kernel takes them, against the same sequences in calls of a few, bit for bit."""
    lens = [1, 2, 3, 500, 0, 128, 129, 127, 1, 1, 1, 9000, 7, 64, 8, 8, 8, 8, 8000, 31, 33, 6000, 5, 0, 12001, 3000, 1]
    s = make(taps, lens, sum(splits), taps, dtype)
    y, hist, status = run(gdn, s, splits)
    assert status == 0 and bool((y[sum(lens):] == 9.0).all())
    at, now = 0, s["hist"]
    for n, k in enumerate(lens):
        for a in range(0, k, 4000):
            m = min(4000, k - a)
            part = dict(s, wide=s["wide"][at + a:at + a + m], lens=[m], slots=s["slots"][n:n + 1], hist=now, cu=torch.tensor([0, m]))
            part["x"] = part["wide"][:, 8:8 + sum(splits)]
            got, now, status = run(gdn, part, splits)
            assert status == 0 and torch.equal(got.view(torch.int16), y[at + a:at + a + m].view(torch.int16)), (n, a)
        at += k
    assert torch.equal(now, hist)


def test_large_and_small_activations(gdn):
    s = make(2, [40], 16, 2, torch.bfloat16, pad=0)
    s["w"][:, 0], s["w"][:, 1], s["bias"][:] = 0.0, 1.0, 0.0
    s["wide"][:, 8:24] = torch.linspace(-2000, 2000, 640).reshape(40, 16).to(torch.bfloat16)
    y, _, _ = run(gdn, s, [16])
    ref, mag, _ = lr.conv(s["x"].double(), s["w"].double(), s["bias"].double(), s["hist"].double(), s["slots"].tolist(), [40], True)
    # below -87 e^z is no longer a normal number: what is left is off by less than 2000 e^-80
    assert bool(((y.double() - ref).abs() <= 2.0 ** -8 * 1.01 * ref.abs() + 2000 * 1.9e-35).all())


def test_malformed_sequences_are_skipped(gdn):
    lens = [20, 30, 10]
    s = make(3, lens, 32, 4, torch.bfloat16, pad=0)
    good, hist, _ = run(gdn, s, [32])
    bad = dict(s, slots=s["slots"].clone())
    bad["slots"][1] = 5
    y, h, status = run(gdn, bad, [32])
    assert status == gdn.STATUS_BAD_CACHE_INDEX
    assert bool((y[20:50] == 9.0).all()) and torch.equal(y[:20], good[:20]) and torch.equal(y[50:], good[50:])
    assert torch.equal(h[s["slots"][1]], s["hist"][s["slots"][1]]) and torch.equal(h[s["slots"][2]], hist[s["slots"][2]])
    bad = dict(s, cu=torch.tensor([0, 20, 50, 61]))  # the last ends behind T
    y, h, status = run(gdn, bad, [32])
    assert status == gdn.STATUS_BAD_SEQLENS
    assert bool((y[50:] == 9.0).all()) and torch.equal(y[:50], good[:50]) and torch.equal(h[s["slots"][2]], s["hist"][s["slots"][2]])
    y, h, status = run(gdn, dict(s, slots=torch.tensor([-1, 0, 1])), [32], step=False)
    assert status == gdn.STATUS_BAD_CACHE_INDEX and bool((y[:20] == 9.0).all())


def test_feeds_the_window(gdn):
    """The history that a prompt leaves is the one that gdn_window_fused reads: its next token's channels agree."""
    h_k, h_v, N = 1, 2, 2
    C = (2 * h_k + h_v) * 128
    s = make(4, [9, 2], C, 4, torch.bfloat16, extra=0, pad=0)
    s["slots"] = torch.arange(N)
    _, hist, _ = run(gdn, s, [C], bias=False)
    g = torch.Generator().manual_seed(5)
    nxt = torch.randn((N, C), generator=g).to(torch.bfloat16)
    pool = hist.cuda()
    y, = gdn.short_conv(nxt.cuda(), s["w"].cuda(), pool, torch.arange(N, device="cuda"))
    # the window with a zero state, beta 1 and no decay commits k v^T; the history it commits is the convolution's
    out = torch.empty_like(pool)
    state = torch.zeros((N, 128, h_v, 128), device="cuda")
    one = torch.ones((N, 1, h_v), device="cuda")
    gdn.gdn_window_fused(state, hist.cuda(), out, nxt.float().reshape(N, 1, C).cuda(), one, one, torch.ones((N, 1, h_v, 128), device="cuda"), s["w"].cuda(),
                         torch.zeros(h_v, device="cuda"), -torch.ones(h_v, device="cuda"), torch.ones(128, device="cuda"), h_k, 1)
    assert torch.equal(out, pool)
    # the state it wrote is k v^T / |k| sigmoid(beta) with the convolution's k and v: rank one along both
    k, v = y[:, 128:256].double(), y[:, 256:].double().reshape(N, h_v, 128)
    want = torch.einsum("ni,nhj->nihj", k / k.norm(dim=1, keepdim=True), v)
    got = state.double() * (want.norm(dim=(1, 3), keepdim=True) / state.double().norm(dim=(1, 3), keepdim=True))
    assert float((got - want).abs().max()) <= 2.0 ** -6 * float(want.abs().max())


def test_refuses_from_python(gdn):
    s = make(6, [4], 16, 4, torch.bfloat16, pad=0)
    x, w, h, i, cu = s["wide"].cuda()[:, 8:24], s["w"].cuda(), s["hist"].cuda(), s["slots"].cuda(), s["cu"].cuda()
    for args, err in (((x.float(), w, h, i, cu), TypeError), ((x, w[:, :3], h, i, cu), ValueError), ((x, w[:8], h, i, cu), ValueError),
                      ((x, w, h[:, :8], i, cu), ValueError), ((x, w, h, i.int(), cu), TypeError), ((x, w, h, i, cu[:1]), ValueError),
                      ((x, w, h, i), gdn.GdnError), ((x[:, 4:], w[4:].contiguous(), h[:, 4:].contiguous(), i, cu), gdn.GdnError)):
        with pytest.raises(err):
            gdn.short_conv(*args)
    with pytest.raises(ValueError):
        gdn.short_conv(x, w, h, i, cu, splits=[8, 4])
    with pytest.raises(gdn.GdnError):
        gdn.short_conv(x, w, h, i, cu, splits=[12, 4])
    with pytest.raises(gdn.GdnError):
        gdn.short_conv(x, w, h, i, cu, outs=[h.view(torch.bfloat16).flatten()[:64].reshape(4, 16)])
