"""attn_paged at the longest lengths that 32-bit key positions allow.  The page table names one page over and
over, so the cache is small: a sequence's keys are those of the page, each as often as the length says."""
import math

import pytest
import torch

from test_gpu_attn_tiles import F8, gdn

pytestmark = pytest.mark.gpu
PAGE, PAGES = 38464, 55831  # 2^31 - 64 tokens


def call(gdn, lens, new, G, f8):
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn((1, 1, PAGE, 64), generator=g, device="cuda") for _ in range(2))
    one = torch.ones((1, 1, PAGE), device="cuda") if f8 else None
    k, v = (x.to(F8 if f8 else torch.bfloat16) for x in (k, v))
    T = sum(new)
    q = torch.randn((T, G, 64), generator=g, device="cuda").bfloat16()
    table = torch.zeros((len(lens), PAGES), dtype=torch.int64, device="cuda")
    cu = torch.tensor([sum(new[:n]) for n in range(len(new) + 1)]).cuda()
    out, lse = torch.full((T, G, 64), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, G), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.attn_paged(q, k, v, table, torch.tensor(lens).cuda(), cu, max(new), scale=0.125, k_scale=one, v_scale=one, out=out, lse=lse,
                   dev_status=status)
    torch.cuda.synchronize()
    return q, k, out, lse, int(status.item())


def want_lse(q, k, length):
    """ln of the sum over the first `length` keys of the repeated page, per head of a token q [G, D]."""
    times = torch.full((PAGE,), length // PAGE, dtype=torch.float64, device="cuda")
    times[:length % PAGE] += 1
    return torch.logsumexp(q.double() @ k[0, 0].double().T * 0.125 + times.log(), -1)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("new,G", [(1, 8), (12, 8)])  # the row kernel, the tile kernel
def test_the_longest_length(gdn, new, G, f8):
    # a thread adds at most 2^31 / 152 / 4 terms to a sum in fp32, each rounding within 2^-24 of it: 2^31 / 608 2^-24
    # = 0.21 in the worst case; dropped keys (the length past 32 bits) would miss by more than 10
    L = 2 ** 31 - 1024
    q, k, out, lse, status = call(gdn, [L], [new], G, f8)
    assert status == 0
    for i in range(new):
        assert float((lse[i].double() - want_lse(q[i], k, L - new + i + 1)).abs().max()) <= 0.21
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("new,G", [(1, 8), (12, 8)])
@pytest.mark.parametrize("length", [2 ** 31 - 1023, 2 ** 31 - 64])
def test_a_longer_one_is_refused(gdn, length, new, G, f8):
    q, k, out, lse, status = call(gdn, [100, length, 70], [new] * 3, G, f8)
    assert status == gdn.STATUS_BAD_SEQLENS
    assert bool((out[new:2 * new] == 5).all()) and bool((lse[new:2 * new] == 7).all())
    for n, L in ((0, 100), (2, 70)):
        for i in range(new):
            row = n * new + i
            # the scores' fp32 error, a few 2^-24 sqrt(D) of at most 16
            assert float((lse[row].double() - want_lse(q[row], k, L - new + i + 1)).abs().max()) <= 1e-4
