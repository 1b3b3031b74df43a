"""draft_verify on the GPU against exact integer arithmetic: counts and tokens are equal numbers."""
import numpy as np
import pytest
import torch

import attn_reference as ar
from gpu_util import library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    library()
    import gated_deltanet_delta_gb300 as g
    return g


def make(seed, N, T, V, noise):
    g = np.random.default_rng(seed)

    def soft(z):
        z = np.exp(z - z.max(-1, keepdims=True))
        return (z / z.sum(-1, keepdims=True)).astype(np.float32)
    logits = g.standard_normal((N, T + 1, V)) * 2
    p = soft(logits)
    q = soft(logits[:, :T] + noise * g.standard_normal((N, T, V)))
    x = np.array([[g.choice(V, p=q[n, t].astype(np.float64) / q[n, t].astype(np.float64).sum()) for t in range(T)]
                  for n in range(N)], np.int64).reshape(N, T)
    return p, q, x, g.random((N, T), np.float32), g.random(N, np.float32)


def call(gdn, p, q, x, u, us, nd=None):
    d = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (p, q, x, u, us)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, t = gdn.draft_verify(*d, num_drafts=None if nd is None else torch.tensor(nd).cuda(), dev_status=status)
    torch.cuda.synchronize()
    return a.cpu().numpy(), t.cpu().numpy(), int(status.item())


@pytest.mark.parametrize("N,T,V,noise", [(1, 1, 1, 0.0), (3, 4, 7, 1.0), (40, 3, 257, 0.7), (5, 8, 2048, 0.3), (2, 40, 300, 0.05),
                                         (3, 2, 20011, 1.0), (2, 3, 70000, 2.0), (6, 0, 500, 0.0)])
def test_against_integer_form(gdn, N, T, V, noise):
    p, q, x, u, us = make(N + V, N, T, V, noise)
    a, t, status = call(gdn, p, q, x, u, us)
    ra, rt = ar.verify(p, q, x, u, us)
    assert status == 0 and np.array_equal(a, ra) and np.array_equal(t, rt)


def test_fewer_drafts_in_some_sequences(gdn):
    p, q, x, u, us = make(3, 6, 5, 100, 0.1)
    nd = [0, 1, 5, 3, 99, -2]
    a, t, status = call(gdn, p, q, x, u, us, nd)
    ra, rt = ar.verify(p, q, x, u, us, nd)
    assert status == 0 and np.array_equal(a, ra) and np.array_equal(t, rt)


def test_marks_at_the_ends(gdn):
    # uniform numbers 0, the largest below 1, and (as if) 1 and NaN; mass in the first and last entry only
    p, q, x, u, us = make(4, 4, 1, 1000, 0.5)
    p[:] = 0
    p[:, :, 0] = 0.25
    p[:, :, 999] = 0.75
    x[:] = 5                                       # target probability 0: always rejected
    us[:] = [0.0, np.float32(1 - 2.0 ** -24), 1.0, np.nan]
    q[:] = 0
    a, t, _ = call(gdn, p, q, x, u, us)
    assert a.tolist() == [0] * 4 and t[:, 0].tolist() == [0, 999, 999, 0] and bool((t[:, 1] == -1).all())


def test_draft_covers_target(gdn):
    # nothing left of max(p - q, 0): the token comes from p
    p, q, x, u, us = make(5, 3, 2, 600, 0.0)
    q[:] = p[:, :2]
    u[:] = 1.0                                     # u q < p fails where p = q
    a, t, status = call(gdn, p, q, x, u, us)
    ra, rt = ar.verify(p, q, x, u, us)
    assert status == 0 and a.tolist() == [0, 0, 0] and np.array_equal(t, rt) and np.array_equal(a, ra)


def test_no_mass_and_bad_tokens_are_reported(gdn):
    p, q, x, u, us = make(6, 3, 2, 50, 0.1)
    p[1] = 0
    a, t, status = call(gdn, p, q, x, u, us)
    assert status == gdn.STATUS_BAD_PROBS and a[1] == 0 and t[1].tolist() == [0, -1, -1]
    p, q, x, u, us = make(7, 3, 2, 50, 0.1)
    x[0, 0], x[2, 0] = 50, -1
    a, t, status = call(gdn, p, q, x, u, us)
    ra, rt = ar.verify(p, q, x, u, us)
    assert status == gdn.STATUS_BAD_TOKEN and np.array_equal(a, ra) and np.array_equal(t, rt)


def test_nan_and_unnormalised_rows(gdn):
    p, q, x, u, us = make(8, 2, 1, 300, 0.1)
    p[0, :, 7] = np.nan
    p[1] *= 37.0
    p[1, :, 3] = np.inf
    x[:] = 9
    u[:] = 1e30
    a, t, _ = call(gdn, p, q, x, u, us)
    ra, rt = ar.verify(p, q, x, u, us)
    assert np.array_equal(a, ra) and np.array_equal(t, rt)


def test_distribution_of_what_comes_out(gdn):
    # whatever the draft, the first token is distributed as the target: chi-square over 40000 draws of 8
    # outcomes; with 7 degrees of freedom 40 is exceeded with probability 1e-6
    g = np.random.default_rng(1)
    N, V = 40000, 8
    p1 = np.array([0.3, 0.2, 0.15, 0.1, 0.1, 0.08, 0.05, 0.02], np.float32)
    q1 = np.array([0.05, 0.3, 0.05, 0.2, 0.1, 0.1, 0.1, 0.1], np.float32)
    p, q = np.broadcast_to(p1, (N, 2, V)), np.broadcast_to(q1, (N, 1, V))
    x = g.choice(V, size=(N, 1), p=q1.astype(np.float64) / q1.astype(np.float64).sum())
    a, t, _ = call(gdn, p, q, x, g.random((N, 1), np.float32), g.random(N, np.float32))
    got = np.bincount(t[:, 0], minlength=V)
    want = N * p1.astype(np.float64) / p1.astype(np.float64).sum()
    assert float(((got - want) ** 2 / want).sum()) < 40


def test_refusals(gdn):
    p, q, x, u, us = (torch.from_numpy(a).cuda() for a in make(9, 2, 2, 20, 0.1))
    with pytest.raises(TypeError):
        gdn.draft_verify(p.half(), q, x, u, us)
    with pytest.raises(ValueError):
        gdn.draft_verify(p, q[:, :1].contiguous(), x, u, us)
    with pytest.raises(ValueError):
        gdn.draft_verify(p, q, x, u[:1], us)
    with pytest.raises(gdn.GdnError):
        big = torch.zeros((1, 1, (1 << 20) + 1), device="cuda")
        gdn.draft_verify(big, torch.empty((1, 0, (1 << 20) + 1), device="cuda"), torch.empty((1, 0), dtype=torch.int64, device="cuda"),
                         torch.empty((1, 0), device="cuda"), us[:1].contiguous())


@pytest.mark.parametrize("N,V", [(76, 16384), (600, 8192), (3000, 4096), (4001, 900)])
def test_short_rows_of_many_clusters(gdn, N, V):
    # clusters of 8, 4, 2 CTAs and single ones with the least work per CTA, in many waves: a CTA's sum reaches
    # another soon after, or before, that one has begun
    g = torch.Generator(device="cuda").manual_seed(N)
    p = torch.softmax(2 * torch.randn((N, 2, V), generator=g, device="cuda"), -1)
    q = torch.softmax(2 * torch.randn((N, 1, V), generator=g, device="cuda"), -1)
    x = torch.randint(V, (N, 1), generator=g, device="cuda")
    u, us = torch.rand((N, 1), generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    stands = u[:, 0] * q[:, 0].gather(1, x)[:, 0] < p[:, 0].gather(1, x)[:, 0]
    row = torch.where(stands[:, None], p[:, 1], p[:, 0])
    whole = (row.double() * 2.0 ** 36).long()
    units = torch.where(stands[:, None], whole, (whole - (q[:, 0].double() * 2.0 ** 36).long()).clamp(min=0))
    mark = units.sum(1) * (us.double() * 2 ** 24).long() >> 24
    token = (units.cumsum(1) <= mark[:, None]).sum(1)
    for i in range(20):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        accepted, tokens = gdn.draft_verify(p, q, x, u, us, dev_status=status)
        assert status.item() == 0 and torch.equal(accepted, stands.long()), i
        assert torch.equal(tokens.gather(1, stands.long()[:, None])[:, 0], token), i
