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
