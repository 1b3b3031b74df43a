"""The state space layer and the attention layer of examples/hybrid_prompt.py together: a prompt at once, in pieces and token by
token, eager and from a CUDA graph, must leave the same."""
import os
import sys

import pytest
import torch

from gpu_util import library

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def hp():
    library()
    import hybrid_prompt
    return hybrid_prompt


def tokens_of(model, counts, seed=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randint(model.vocab, (c,), generator=g, device="cuda") for c in counts]


def rel(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm())


# Between two ways through the same tokens these roundings differ, each of at most 2^-8 of a value, 2^-8 / sqrt(3) in the mean square:
# in the scan M, the state's copy and the output, in the attention the weights and the output, and behind either the products'
# results, the residual stream and the norm's rows (of one way each, so twice): 16 in all.  Relative to sums of products of
# independent signs they stay what they are: sqrt(16) 2^-8 / sqrt(3) = 0.009 of a row's norm.  2^-5 leaves a factor of three.
CLOSE = 2.0 ** -5


@pytest.mark.parametrize("cuts", [[(200, 1, 64)], [(1, 1, 1), (128, 0, 40), (71, 0, 23)], [(199, 1, 1), (1, 0, 63)]])
def test_pieces_against_steps(hp, cuts):
    counts = [200, 1, 64]
    a, b = hp.HybridModel(seed=4), hp.HybridModel(seed=4)
    toks = tokens_of(a, counts)
    rows = [[] for _ in counts]
    done = [0] * 3
    for piece in cuts:
        packed = torch.cat([toks[n][done[n]:done[n] + c] for n, c in enumerate(piece)])
        h, _ = a.prompt(packed, list(piece))
        for n, part in enumerate(h.split(list(piece))):
            rows[n].append(part)
            done[n] += piece[n]
    # the same token by token: a sequence that has no more is stepped on a model whose state is put back
    steps = [[] for _ in counts]
    for t in range(max(counts)):
        keep = b.hist.clone(), b.state.clone(), b.lens.clone()
        h, _ = b.step(torch.stack([toks[n][min(t, c - 1)] for n, c in enumerate(counts)]))
        for n, c in enumerate(counts):
            if t < c:
                steps[n].append(h[n])
            else:
                b.hist[n], b.state[n], b.lens[n] = (k[n] for k in keep)
    assert a.lens.tolist() == b.lens.tolist() == counts
    for n in range(3):
        assert rel(torch.cat(rows[n]), torch.stack(steps[n])) <= CLOSE
    assert rel(a.hist, b.hist) <= 2.0 ** -7  # rows of a product in another order of sums: at most a step of bf16 apart
    assert rel(a.state, b.state) <= CLOSE
    assert int(a.status.item()) == 0 and int(b.status.item()) == 0


def test_captured_steps(hp):
    counts = [40, 3, 17]
    a, b = hp.HybridModel(seed=6), hp.HybridModel(seed=6)
    toks = torch.cat(tokens_of(a, counts))
    a.prompt(toks, counts)
    b.prompt(toks, counts)
    fed = torch.stack(tokens_of(a, [6] * 3, seed=9), 1)
    at = fed[0].clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        c = hp.HybridModel(seed=6)  # the first calls of a process load kernels, which a capture must not
        c.prompt(toks, counts)
        c.step(at)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, logits = a.step(at)
    for t in range(6):
        at.copy_(fed[t])
        graph.replay()
        hb, logits_b = b.step(fed[t])
        # the library's products may take another form inside a capture: the same bound
        assert rel(h, hb) <= CLOSE and rel(logits, logits_b) <= CLOSE
    assert torch.equal(a.lens, b.lens) and rel(a.state, b.state) <= CLOSE and rel(a.hist, b.hist) <= 2.0 ** -7
    assert rel(a.cache[0], b.cache[0]) <= CLOSE and rel(a.cache[1], b.cache[1]) <= CLOSE
    assert int(a.status.item()) == 0 and int(b.status.item()) == 0


def test_history_of_the_fused_window(hp):
    """The convolution's history is the fused decode window's: a prompt's last inputs, where the window goes on."""
    import gated_deltanet_delta_gb300 as gdn
    h_k, h_v, D, N, T, W = 1, 2, 128, 2, 9, 3
    C = (2 * h_k + h_v) * D
    g = torch.Generator(device="cuda").manual_seed(8)

    def r(*s):
        return torch.randn(s, generator=g, device="cuda")
    x = r(N, T + W, C).to(torch.bfloat16)  # what both take: the window has its rows in fp32
    w = r(C, 4) * 0.5
    hist = torch.zeros((N, C, 3), device="cuda")
    cu = torch.arange(0, N * T + 1, T, device="cuda")
    idx = torch.arange(N, device="cuda")
    gdn.short_conv(x[:, :T].reshape(N * T, C), w, hist, idx, cu)
    other = hist.clone()
    gdn.short_conv(x[:, T:].reshape(N * W, C), w, other, idx, torch.arange(0, N * W + 1, W, device="cuda"))
    out = torch.empty_like(hist)
    gdn.gdn_window_fused(torch.zeros((N, D, h_v, D), device="cuda"), hist, out, x[:, T:].float().contiguous(), r(N, W, h_v), r(N, W, h_v),
                         r(N, W, h_v, D), w, r(h_v), -torch.rand(h_v, device="cuda") - 0.5, torch.ones(D, device="cuda"), h_k, 1)
    assert torch.equal(out, other)


def test_example_runs(hp, capsys):
    hp.main(steps=2)
    assert "lengths" in capsys.readouterr().out
