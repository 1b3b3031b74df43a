"""attn_cache_append on the GPU: the rotated queries against the formula with each rounding where the header puts it, the
cache against attn_cache_write of the rotated rows, both bit for bit."""
import pytest
import torch

import layer_reference as lr
from gpu_util import library

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


def bits(t):
    return t.view(torch.uint8) if t.dtype == F8 else t.view(torch.int16 if t.element_size() == 2 else torch.int32)


def table(positions, turned, base=10000.0):
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-2.0 * torch.arange(turned // 2) / turned)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def make(seed, T, Hq, H, D, turned, page, dtype, f8, positions=300):
    g = torch.Generator().manual_seed(seed)
    s = {"wide": (torch.randn((T, Hq + 2 * H + 1, D), generator=g) * torch.exp(torch.randn((T, 1, 1), generator=g))).to(dtype).cuda()}
    s["q"], s["k"], s["v"], _ = s["wide"].split([Hq, H, H, 1], 1)
    s["rot"] = table(positions, turned).cuda()
    s["pos"] = torch.randint(0, positions, (T,), generator=g).cuda()
    pages = -(-T // page) + 2
    s["slots"] = torch.randperm(pages * page, generator=g)[:T].cuda()
    s["caches"] = [torch.full((pages, H, page, D), 3.0).to(F8 if f8 else dtype).cuda() for _ in range(4)]
    s["scales"] = [torch.full((pages, H, page), 7.0, device="cuda") if f8 else None for _ in range(4)]
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def check(gdn, s, neighbours, q_out=None, kept=None):
    """One call against the two steps it stands for; kept: the tokens whose positions are in the table."""
    T, table_ = s["k"].shape[0], s["rot"].cpu()
    kept = torch.arange(T) if kept is None else kept
    q0 = s["q"].clone()
    out = gdn.attn_cache_append(s["q"], s["k"], s["v"], s["rot"], s["pos"], s["slots"], s["caches"][0], s["caches"][1], s["scales"][0],
                                s["scales"][1], q_out=q_out, neighbours=neighbours, dev_status=s["status"])
    torch.cuda.synchronize()
    rows = table_[s["pos"].cpu()[kept]]
    q, k = (lr.turn(x.cpu()[kept], rows, neighbours) for x in (q0, s["k"]))
    assert torch.equal(bits(out.cpu()[kept]), bits(q))
    st = torch.zeros_like(s["status"])
    gdn.attn_cache_write(k.cuda(), s["v"][kept.cuda()].contiguous(), s["slots"][kept.cuda()], s["caches"][2], s["caches"][3], s["scales"][2],
                         s["scales"][3], dev_status=st)
    torch.cuda.synchronize()
    for i in (0, 1):
        assert torch.equal(bits(s["caches"][i]), bits(s["caches"][i + 2]))
        if s["scales"][0] is not None:
            assert torch.equal(s["scales"][i], s["scales"][i + 2])
    return out


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("dtype,f8", [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float16, False), (torch.float16, True)])
@pytest.mark.parametrize("T,Hq,H,D,turned,page", [(1, 1, 1, 64, 64, 16), (7, 6, 2, 128, 128, 5), (33, 4, 4, 64, 32, 16), (150, 5, 1, 256, 64, 48),
                                                  (9, 3, 3, 256, 256, 1), (65, 2, 1, 128, 16, 7), (40, 1, 2, 128, 112, 64), (2051, 9, 3, 64, 64, 16), (2048, 10, 1, 128, 96, 48),
                                                  (2500, 1, 9, 256, 128, 64)])
def test_rotates_and_appends(gdn, T, Hq, H, D, turned, page, dtype, f8, neighbours):
    s = make(T, T, Hq, H, D, turned, page, dtype, f8)
    s["slots"][T // 2] = -1  # this token is not kept; its query is rotated
    check(gdn, s, neighbours)
    assert s["status"].item() == 0


@pytest.mark.parametrize("D,turned", [(64, 64), (128, 64), (256, 256)])
def test_queries_in_place(gdn, D, turned):
    s = make(3, 50, 7, 2, D, turned, 16, torch.bfloat16, True)
    before = s["wide"].clone()
    out = check(gdn, s, False, q_out=s["q"])
    assert out.data_ptr() == s["wide"].data_ptr() and torch.equal(bits(s["wide"][:, 7:]), bits(before[:, 7:]))


def test_keys_and_values_alone(gdn):
    s = make(4, 21, 3, 2, 128, 128, 16, torch.float16, False)
    assert gdn.attn_cache_append(None, s["k"], s["v"], s["rot"], s["pos"], s["slots"], *s["caches"][:2], dev_status=s["status"]) is None
    k = lr.turn(s["k"].cpu(), s["rot"].cpu()[s["pos"].cpu()], False).cuda()
    gdn.attn_cache_write(k, s["v"].contiguous(), s["slots"], *s["caches"][2:], dev_status=s["status"])
    assert torch.equal(bits(s["caches"][0]), bits(s["caches"][2])) and torch.equal(bits(s["caches"][1]), bits(s["caches"][3]))


def test_positions_and_slots_outside(gdn):
    s = make(5, 30, 4, 2, 64, 64, 16, torch.bfloat16, True)
    s["pos"][3], s["pos"][17] = -1, 300
    out = torch.full((30, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    kept = torch.tensor([t for t in range(30) if t not in (3, 17)])
    check(gdn, s, False, q_out=out, kept=kept)
    assert s["status"].item() == gdn.STATUS_BAD_POSITION
    assert bool((out[[3, 17]] == 5.0).all())
    s = make(6, 30, 4, 2, 64, 64, 16, torch.bfloat16, False)
    s["slots"][11] = s["caches"][0].shape[0] * 16
    good = s["slots"].clone()
    gdn.attn_cache_append(s["q"], s["k"], s["v"], s["rot"], s["pos"], s["slots"], *s["caches"][:2], dev_status=s["status"])
    good[11] = -1
    gdn.attn_cache_append(s["q"], s["k"], s["v"], s["rot"], s["pos"], good, *s["caches"][2:])
    assert s["status"].item() == gdn.STATUS_BAD_CACHE_INDEX
    assert torch.equal(bits(s["caches"][0]), bits(s["caches"][2]))


def test_infinities_and_nan_stay_in_their_pairs(gdn):
    s = make(7, 5, 1, 1, 64, 32, 16, torch.bfloat16, True)
    s["k"][1, 0, 40], s["k"][2, 0, 0], s["v"][3, 0, 5] = float("inf"), float("nan"), float("-inf")
    check(gdn, s, False)
    got = s["caches"][0].float().cpu().permute(0, 2, 1, 3).reshape(-1, 64)[s["slots"].cpu()]
    assert got[1].isnan().nonzero().flatten().tolist() == [40] and got[2].isnan().nonzero().flatten().tolist() == [0, 16]


def test_captured_and_on_another_stream(gdn):
    s = make(8, 64, 8, 2, 128, 128, 16, torch.bfloat16, True)
    out = torch.empty((64, 8, 128), dtype=torch.bfloat16, device="cuda")
    call = lambda: gdn.attn_cache_append(s["q"], s["k"], s["v"], s["rot"], s["pos"], s["slots"], *s["caches"][:2], *s["scales"][:2], q_out=out,  # noqa: E731
                                         dev_status=s["status"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    s["wide"].copy_(torch.randn_like(s["wide"].float()))
    s["pos"].add_(1).clamp_(max=299)
    graph.replay()
    torch.cuda.synchronize()
    q = lr.turn(s["q"].cpu(), s["rot"].cpu()[s["pos"].cpu()], False)
    assert torch.equal(bits(out.cpu()), bits(q))


def test_refuses_from_python(gdn):
    s = make(9, 4, 2, 1, 64, 64, 16, torch.bfloat16, False)
    args = [s["q"], s["k"], s["v"], s["rot"], s["pos"], s["slots"], *s["caches"][:2]]
    for i, bad, err in ((0, s["q"].half(), TypeError), (3, s["rot"][0], ValueError), (4, s["pos"].int(), TypeError), (4, s["pos"][:3], ValueError),
                        (3, s["rot"][:, :24].contiguous(), gdn.GdnError), (6, s["caches"][0].half(), TypeError), (1, s["k"].cpu(), ValueError)):
        with pytest.raises(err):
            gdn.attn_cache_append(*[bad if j == i else a for j, a in enumerate(args)])
    with pytest.raises(gdn.GdnError):  # overlaps the sources, and is not q
        gdn.attn_cache_append(*args, q_out=s["wide"][:, 1:3])
