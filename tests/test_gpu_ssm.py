"""ssm_decode_step and ssm_prefill_chunked on the GPU against the recurrence in 64 bits."""
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


def make(seed, lens, H, P, G, S, gated=True, extra=2, pad=0, dt=(0.001, 0.1), strided=True):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + pad
    bf = torch.bfloat16
    inner, e = H * P, 8 if strided else 0

    def rows(n, h, d):
        return torch.randn((T, n + e), generator=g).to(bf).cuda()[:, e:].unflatten(1, (h, d))
    s = {"x": rows(inner, H, P), "B": rows(G * S, G, S), "C": rows(G * S, G, S), "z": rows(inner, H, P) if gated else None,
         "dt": torch.randn((T, H + 3), generator=g).to(bf).cuda()[:, 3:]}
    step = torch.exp(torch.rand(H, generator=g) * (torch.tensor(dt[1]).log() - torch.tensor(dt[0]).log()) + torch.tensor(dt[0]).log())
    s["dt_bias"] = (step + torch.log(-torch.expm1(-step))).cuda()
    s["A_log"] = torch.log(1 + 15 * torch.rand(H, generator=g)).cuda()
    s["D"] = torch.randn(H, generator=g).cuda()
    s["state"] = torch.randn((len(lens) + extra, H, P, S), generator=g).cuda()
    s["slots"] = torch.randperm(len(lens) + extra, generator=g)[:len(lens)].cuda()
    s["cu"], s["lens"] = lr.ragged(lens).cuda(), list(lens)
    return s


def reference(s):
    d = lambda t: None if t is None else t.double()  # noqa: E731
    D = torch.zeros_like(s["A_log"]) if s["D"] is None else s["D"]
    return lr.scan(d(s["x"]), d(s["dt"]), d(s["B"]), d(s["C"]), d(s["z"]), d(s["A_log"]), d(D), d(s["dt_bias"]), d(s["state"]), s["slots"].tolist(), s["lens"])


def check(s, y, state, ref, chunked):
    """The tolerances.  The decay e^(A dt) is off by |A dt| 2^-22 (its argument, rounded, times its size) and some 2^-22, once
    for each of the steps that a state element goes through; over those steps A dt sums to at most some 90 before nothing is
    left.  fp32 sums: 2^-24 each.  The chunked kernels round the weights of a chunk's pairs, or the state that
    a chunk begins with, to bf16 (2^-8 of the magnitudes summed), and hold dt x in two bf16 parts (2^-16)."""
    yr, sr, ym, sm = ref
    T = sum(s["lens"])
    longest = max(s["lens"] + [1])
    fp32 = (90 + 4 * min(longest, 512) + 300) * 2.0 ** -24
    tol = 2.0 ** -8 * 1.01 * yr.abs() + (fp32 + (2.0 ** -8 if chunked else 0.0)) * (ym + yr.abs()) + 1e-30
    err = (y.double() - yr).abs()[:T]
    assert bool((err <= tol[:T]).all()), float((err / tol[:T]).max())
    err = (state.double() - sr).abs()
    tol = (fp32 + (2.0 ** -16 if chunked else 0.0)) * sm + 1e-30
    assert bool((err <= tol).all()), float((err / tol).max())
    spare = [i for i in range(state.shape[0]) if i not in s["slots"].tolist()]
    assert torch.equal(state[spare], s["state"][spare])


def prefill(gdn, s, **kw):
    state = s["state"].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(s["x"].shape, 9.0, dtype=torch.bfloat16, device="cuda")
    kw.setdefault("cu", s["cu"])
    gdn.ssm_prefill_chunked(s["x"], s["dt"], s["B"], s["C"], s["A_log"], s["dt_bias"], state, kw.pop("slots", s["slots"]), kw.pop("cu"),
                            kw.pop("max_len", max(s["lens"] + [0])), D=s["D"], z=s["z"], out=out, dev_status=status, **kw)
    torch.cuda.synchronize()
    return out, state, status.item()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N,H,P,G,S", [(1, 1, 64, 1, 64), (3, 4, 64, 2, 128), (65, 3, 128, 1, 128), (5, 6, 128, 3, 64)])
def test_single_tokens(gdn, N, H, P, G, S, gated):
    s = make(N, [1] * N, H, P, G, S, gated)
    state = s["state"].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = gdn.ssm_decode_step(s["x"], s["dt"], s["B"], s["C"], s["A_log"], s["dt_bias"], state, s["slots"], D=s["D"], z=s["z"], dev_status=status)
    assert status.item() == 0
    check(s, y, state, reference(s), False)


@pytest.mark.parametrize("H,P,G,S", [(2, 64, 1, 128), (3, 64, 1, 64), (1, 128, 1, 128), (4, 128, 2, 64)])
@pytest.mark.parametrize("lens", [[1], [7], [8, 0, 9, 1], [16, 3, 17], [127], [128], [129, 1, 64], [300, 0, 255, 31], [700, 513]])
def test_prompts(gdn, lens, H, P, G, S):
    s = make(sum(lens) + H, lens, H, P, G, S, gated=H != 2, pad=5)
    ref = reference(s)
    for max_len in (max(lens), 1, 1 << 40):  # whatever the caller says of the longest, the result is the same to rounding
        y, state, status = prefill(gdn, s, max_len=max_len)
        assert status == 0
        check(s, y, state, ref, True)
        assert bool((y[sum(lens):] == 9.0).all())
        empty = [int(s["slots"][n]) for n, k in enumerate(lens) if k == 0]
        assert torch.equal(state[empty], s["state"][empty])


def test_without_d(gdn):
    s = make(1, [140, 20], 2, 64, 1, 128)
    s["D"] = None
    y, state, _ = prefill(gdn, s)
    check(s, y, state, reference(s), True)


@pytest.mark.parametrize("lens,H,P,G,S", [([2500, 5, 1400], 1, 64, 1, 128), ([1025], 3, 128, 1, 64), ([0, 4097, 1024, 1300], 2, 64, 2, 64),
                                          ([3000], 2, 128, 2, 128)])
def test_segments(gdn, lens, H, P, G, S):
    """Sequences long enough to be cut: the states of pieces are formed ahead, the pool's state is replaced meanwhile."""
    s = make(sum(lens), lens, H, P, G, S, pad=3, dt=(0.0003, 0.01))
    assert gdn.ssm_prefill_workspace_size(len(lens), sum(lens), H, P, S) > 0
    ref = reference(s)
    for max_len in (max(lens), 100):  # cut, and not
        y, state, status = prefill(gdn, s, max_len=max_len)
        assert status == 0
        check(s, y, state, ref, True)
        assert bool((y[sum(lens):] == 9.0).all())


def test_strong_decays_keep_their_digits(gdn):
    """Steps of up to 60 units of decay: sums of hundreds within a chunk, of which a pair of near tokens sees the difference."""
    s = make(11, [400, 130], 4, 64, 1, 128, dt=(0.5, 4.0))
    y, state, status = prefill(gdn, s, max_len=400)
    assert status == 0
    check(s, y, state, reference(s), True)
    s["A_log"].fill_(30.0)  # nothing is left of what came before
    y, state, status = prefill(gdn, s, max_len=400)
    check(s, y, state, reference(s), True)


def test_tokens_behind_a_sequence_may_hold_anything(gdn):
    """A chunk's tile reaches into the next sequence's rows, and behind the last sequence into what memory holds."""
    lens = [100, 40, 129, 3]
    s = make(12, lens, 3, 64, 1, 128, pad=200)
    clean = prefill(gdn, s, max_len=129)
    for n in (0, 2):  # sequences 1 and 3 hold no numbers, and the rows behind the last neither
        cut = dict(s, lens=lens[:n + 1])
        for name in ("x", "B", "C", "z", "dt"):
            cut[name] = s[name].clone()
            cut[name][sum(lens[:n + 1]):] = float("nan")
        y, state, status = prefill(gdn, cut, cu=s["cu"][:n + 2].contiguous(), slots=s["slots"][:n + 1].contiguous(), max_len=129)
        assert status == 0
        T = sum(lens[:n + 1])
        assert torch.equal(y[:T], clean[0][:T]) and bool((y[T:] == 9.0).all())
        assert torch.equal(state[s["slots"][:n + 1]], clean[1][s["slots"][:n + 1]])


def test_malformed_sequences_are_skipped(gdn):
    lens = [60, 200, 30]
    s = make(13, lens, 2, 64, 1, 64, pad=10)
    for max_len in (8, 200):
        good, gstate, _ = prefill(gdn, s, max_len=max_len)
        slots = s["slots"].clone()
        slots[1] = 5
        y, state, status = prefill(gdn, s, slots=slots, max_len=max_len)
        assert status == gdn.STATUS_BAD_CACHE_INDEX
        assert bool((y[60:260] == 9.0).all()) and torch.equal(y[:60], good[:60]) and torch.equal(y[260:290], good[260:290])
        assert torch.equal(state[s["slots"][1]], s["state"][s["slots"][1]]) and torch.equal(state[s["slots"][2]], gstate[s["slots"][2]])
        y, state, status = prefill(gdn, s, cu=torch.tensor([0, 60, 260, 301], device="cuda"), max_len=max_len)
        assert status == gdn.STATUS_BAD_SEQLENS
        assert bool((y[260:] == 9.0).all()) and torch.equal(y[:260], good[:260]) and torch.equal(state[s["slots"][2]], s["state"][s["slots"][2]])


def test_a_prompt_in_pieces_and_single_tokens(gdn):
    """A prompt at once, in two pieces, and its last tokens one by one."""
    s = make(14, [300], 4, 64, 2, 128)
    ref = reference(s)
    state = s["state"].clone()
    outs = []
    for a, b in ((0, 150), (150, 297), (297, 298), (298, 299), (299, 300)):
        part = [s[k][a:b] for k in ("x", "dt", "B", "C")]
        kw = dict(D=s["D"], z=s["z"][a:b])
        if b - a > 1:
            outs.append(gdn.ssm_prefill_chunked(*part, s["A_log"], s["dt_bias"], state, s["slots"], torch.tensor([0, b - a], device="cuda"), b - a, **kw))
        else:
            outs.append(gdn.ssm_decode_step(*part, s["A_log"], s["dt_bias"], state, s["slots"], **kw))
    check(s, torch.cat(outs), state, ref, True)


def test_captured_with_two_workspaces(gdn):
    """Two captured calls, replayed on streams of their own at once: each has its own workspace and answers as alone."""
    calls = []
    for seed in (15, 16):
        s = make(seed, [1500, 700], 2, 64, 1, 128)
        state, out, status = s["state"].clone(), torch.empty_like(s["x"].contiguous()), torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = torch.empty(gdn.ssm_prefill_workspace_size(2, 2200, 2, 64, 128), dtype=torch.uint8, device="cuda")
        go = lambda s=s, state=state, out=out, ws=ws, status=status: gdn.ssm_prefill_chunked(  # noqa: E731
            s["x"], s["dt"], s["B"], s["C"], s["A_log"], s["dt_bias"], state, s["slots"], s["cu"], 1500, D=s["D"], z=s["z"], out=out, workspace=ws, dev_status=status)
        go()
        torch.cuda.synchronize()
        want = out.clone(), state.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            state.copy_(s["state"])
            go()
        calls.append((graph, out, state, want, status, go))  # go keeps what the graph reads
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        for st, (graph, *_r) in zip(streams, calls):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, state, want, status, _ in calls:
        assert status.item() == 0 and torch.equal(out, want[0]) and torch.equal(state, want[1])


def test_a_wait_that_runs_out_reports_and_the_next_call_is_right(gdn):
    s = make(17, [1400], 2, 64, 1, 128)
    try:
        gdn.set_prefill_wait_limit(1)
        _, _, status = prefill(gdn, s)
    finally:
        gdn.set_prefill_wait_limit(0)
    assert status & gdn.STATUS_TIMEOUT
    y, state, status = prefill(gdn, s)
    assert status == 0
    check(s, y, state, reference(s), True)


@pytest.mark.parametrize("P,S", [(64, 128), (128, 64)])
def test_a_wait_that_runs_out_in_a_cut_sequence(gdn, P, S):
    s = make(19, [6000, 200], 2, P, 1, S)
    try:
        gdn.set_prefill_wait_limit(1)
        _, _, status = prefill(gdn, s)
    finally:
        gdn.set_prefill_wait_limit(0)
    assert status & gdn.STATUS_TIMEOUT
    y, state, status = prefill(gdn, s)
    assert status == 0
    check(s, y, state, reference(s), True)


def test_bounds_that_go_back_stay_in_the_workspace(gdn):
    """cu_seqlens that falls: every second sequence is malformed, the others have the same tokens, and more segments than T tokens do."""
    T, n = 6000, 9
    s = make(20, [T] + [0] * (n - 1), 2, 64, 1, 128)
    need = gdn.ssm_prefill_workspace_size(n, T, 2, 64, 128)
    ws = torch.full((need + 65536,), 85, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, T] * 5, device="cuda")
    _, state, status = prefill(gdn, s, cu=cu, max_len=T, workspace=ws)
    assert status == gdn.STATUS_BAD_SEQLENS and bool((ws[need:] == 85).all())
    odd = s["slots"][1::2]  # the sequences that end before they begin, and the slots of none
    spare = [i for i in range(state.shape[0]) if i not in s["slots"].tolist()]
    assert torch.equal(state[odd], s["state"][odd]) and torch.equal(state[spare], s["state"][spare])


def test_refuses_from_python(gdn):
    s = make(18, [2, 2], 2, 64, 1, 64, strided=False)
    args = [s["x"], s["dt"], s["B"], s["C"], s["A_log"], s["dt_bias"], s["state"], s["slots"], s["cu"], 2]
    for i, bad, err in ((0, s["x"].half(), TypeError), (1, s["dt"].T, ValueError), (2, s["B"][:3], ValueError), (3, s["C"][..., ::2], ValueError),
                        (4, s["A_log"][:1], ValueError), (6, s["state"][..., :32], ValueError), (6, s["state"].double(), TypeError), (7, s["slots"].int(), TypeError),
                        (8, s["cu"][:2], ValueError), (9, -1, gdn.GdnError)):
        with pytest.raises(err):
            gdn.ssm_prefill_chunked(*[bad if j == i else a for j, a in enumerate(args)])
    with pytest.raises(ValueError):  # four tokens, two sequences
        gdn.ssm_decode_step(*args[:8])
    with pytest.raises(gdn.GdnError):
        gdn.ssm_prefill_chunked(*args, out=s["x"])
