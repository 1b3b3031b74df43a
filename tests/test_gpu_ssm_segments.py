"""The chunked scan where sequences are cut, shown by what the call leaves in its workspace: segments of more than one batch of chunks, many
segments, every head width and state width, two captured calls at once; and the norm of its outputs' error."""
import math

import pytest
import torch

from gpu_util import library
from test_gpu_ssm import check, make, prefill, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


def workspace(gdn, s):
    lens, H, P, S = s["lens"], s["x"].shape[1], s["x"].shape[2], s["B"].shape[2]
    ws = torch.full((gdn.ssm_prefill_workspace_size(len(lens), sum(lens), H, P, S),), 0x71, dtype=torch.uint8, device="cuda")
    return ws, H * P * S * 4


def states_left(ws, state_bytes):
    """How many states the call wrote to its workspace: for a sequence of n > 1 segments its first one and n - 1 more."""
    n = ws.numel() // (state_bytes + state_bytes // 4096)
    return int((ws[:n * state_bytes].reshape(n, state_bytes)[:, :4096] != 0x71).any(1).sum())


def close_in_norm(y, ref, chunked):
    # Half a step of bf16 is 2^-8 of the least value with an exponent, so an output's rounding is 2^-8 / sqrt(3) / 1.3 or so of the outputs'
    # norm, 2^-9; the rounding of M's weights, or of the state's copy, to bf16 likewise of the norm of the terms that they weigh.
    err = float((y.double() - ref).norm() / ref.norm())
    assert err <= (math.hypot(2.0 ** -9, 2.0 ** -9) if chunked else 2.0 ** -9), err


@pytest.mark.parametrize("lens,H,P,G,S,most", [([4096], 64, 128, 2, 64, 3), ([16300], 32, 128, 2, 64, 8), ([6200, 130], 96, 64, 1, 128, None), ([40000], 1, 64, 1, 64, None),
                                                   ([2049], 3, 128, 1, 64, None), ([2049], 3, 128, 1, 128, None), ([2049, 1, 3000], 3, 64, 1, 64, None)])
def test_cut_sequences(gdn, lens, H, P, G, S, most):
    """most: segments, where they are to be of more than one batch of eight chunks."""
    s = make(51 + H, lens, H, P, G, S, dt=(0.0003, 0.01), pad=3)
    ws, state_bytes = workspace(gdn, s)
    y, state, status = prefill(gdn, s, workspace=ws)
    assert status == 0 and bool((y[sum(lens):] == 9.0).all())
    assert 2 <= states_left(ws, state_bytes) <= (most or math.inf)
    ref = reference(s)
    check(s, y, state, ref, True)
    close_in_norm(y[:sum(lens)], ref[0][:sum(lens)], True)
    # the same from states that were not formed ahead, within the same bounds
    y, state, status = prefill(gdn, s, workspace=ws, max_len=200)
    assert status == 0
    check(s, y, state, ref, True)
    close_in_norm(y[:sum(lens)], ref[0][:sum(lens)], True)


@pytest.mark.parametrize("H,P,G,S", [(4, 64, 1, 128), (6, 64, 2, 64), (3, 128, 1, 128), (2, 128, 2, 64)])
def test_norm_of_the_error(gdn, H, P, G, S):
    s = make(52, [700, 17, 300, 128], H, P, G, S)
    ref = reference(s)
    for max_len in (700, 1):
        y, state, status = prefill(gdn, s, max_len=max_len)
        assert status == 0
        close_in_norm(y, ref[0], max_len > 16)


def test_captured_with_two_workspaces_that_both_use(gdn):
    """Two captured calls whose sequences are cut, replayed on streams of their own at once."""
    calls = []
    for seed in (53, 54):
        s = make(seed, [5000, 700], 4, 64, 1, 128, dt=(0.0003, 0.01))
        state, out, status = s["state"].clone(), torch.empty_like(s["x"].contiguous()), torch.zeros(1, dtype=torch.int32, device="cuda")
        ws, state_bytes = workspace(gdn, s)
        go = lambda s=s, state=state, out=out, ws=ws, status=status: gdn.ssm_prefill_chunked(  # noqa: E731
            s["x"], s["dt"], s["B"], s["C"], s["A_log"], s["dt_bias"], state, s["slots"], s["cu"], 5000, D=s["D"], z=s["z"], out=out, workspace=ws, dev_status=status)
        go()
        torch.cuda.synchronize()
        assert states_left(ws, state_bytes) >= 5
        want = out.clone(), state.clone()
        check(s, want[0], want[1], reference(s), True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ws.fill_(0x71)
            state.copy_(s["state"])
            go()
        calls.append((graph, out, state, want, status, ws, state_bytes, go))  # go keeps what the graph reads
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        for st, (graph, *_r) in zip(streams, calls):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, state, want, status, ws, state_bytes, _ in calls:
        assert status.item() == 0 and torch.equal(out, want[0]) and torch.equal(state, want[1])
        assert states_left(ws, state_bytes) >= 5


def test_long_prompts_have_few_segments(gdn):
    """A segment starts from the sum of the states of all segments ahead of it: in 64 segments these sums took two thirds of the call."""
    T, H, P, S = 65536, 64, 64, 64
    z = lambda *d: torch.zeros(d, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    s = {"lens": [T], "x": z(T, H, P), "B": z(T, 1, S)}
    ws, state_bytes = workspace(gdn, s)
    state, status = torch.ones((1, H, P, S), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    y = gdn.ssm_prefill_chunked(s["x"], z(T, H), s["B"], z(T, 1, S), torch.full((H,), -30.0, device="cuda"), torch.full((H,), -30.0, device="cuda"), state,
                                torch.zeros(1, dtype=torch.int64, device="cuda"), torch.tensor([0, T], device="cuda"), T, workspace=ws, dev_status=status)
    assert status.item() == 0 and not bool(y.any()) and bool((state == 1).all())  # steps of e^-30, of which nothing is seen in fp32
    assert 2 <= states_left(ws, state_bytes) <= 24
