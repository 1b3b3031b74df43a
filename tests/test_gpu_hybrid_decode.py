"""The drafted decode step of examples/hybrid_decode.py: window, cache, attention and verification
together.  Rejected drafts must leave no trace, and the accepted prefix must count in full."""
import os
import sys

import pytest
import torch

from gpu_util import library

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def hd():
    library()
    import hybrid_decode
    return hybrid_decode


def test_rejected_drafts_leave_no_trace(hd):
    T = 4
    a, b = hd.HybridModel(seed=3), hd.HybridModel(seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    last = torch.randint(a.vocab, (a.N,), generator=g, device="cuda")
    for _ in range(5):
        p = a.probabilities(last[:, None])
        draft_p = (0.6 * p + 0.4 / a.vocab).expand(-1, T, -1).contiguous()
        drafts = torch.multinomial(draft_p.reshape(-1, a.vocab), 1, generator=g).reshape(a.N, T)
        u, us = torch.rand((a.N, T), generator=g, device="cuda"), torch.rand(a.N, generator=g, device="cuda")
        accepted, tokens = a.step(last, drafts, draft_p, u, us)
        # the other model sees the tokens that stand, one at a time, and no drafts
        for n, c in enumerate(accepted.tolist()):
            assert tokens[n, :c].tolist() == drafts[n, :c].tolist() and tokens[n, c + 1:].tolist() == [-1] * (T - c)
        window = torch.cat([last[:, None], drafts], 1)
        for i in range(int(accepted.max()) + 1):
            b.probabilities(window[:, i:i + 1])
            on = (accepted >= i).tolist()
            for n in range(b.N):
                if on[n]:
                    b._recurrent(window[n:n + 1, i:i + 1], 1, slice(n, n + 1))
            b.lens += torch.tensor(on, device="cuda").long()
        last = tokens.gather(1, accepted[:, None]).squeeze(1)
        assert a.lens.tolist() == b.lens.tolist()
        # the window in one chunk and token by token agree to the order of fp32 sums (the window's bound, 1e-4)
        assert float((a.state - b.state).abs().max()) <= 1e-4 * float(b.state.abs().max())
        assert torch.equal(a.hist, b.hist)
        pa = a.probabilities(last[:, None])
        pb = b.probabilities(last[:, None])
        # keys and values one bf16 rounding apart may fall on neighbouring 8-bit values (a step of 2^-3): a few
        # of them, weighted, move a logit by less than a few hundredths
        assert float((pa.log() - pb.log()).abs().max()) <= 0.05
    assert int(a.status.item()) == 0 and int(b.status.item()) == 0


def test_example_runs(hd, capsys):
    hd.main(steps=2)
    assert "accepted" in capsys.readouterr().out
