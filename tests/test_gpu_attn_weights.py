"""Small weights of attn_paged: many keys whose weights are far below the largest one's still count together.

The cache names two pages: one with 16 keys that take most of the weight and have no value, then many times a
page whose keys have 2^-26 of such a key's weight each, and the value 1.  With n of those the output is
m / (1 + m), m = n 2^-30, and lse = ln(16 e^s (1 + m)).

Bounds: weights and values are powers of two, so what is left is the output's rounding u, the exponents' error
(three roundings of a number of at most 26: 78 2^-24 ln 2 < 2^-18 of the weight) and the rounding of fp32 sums
to which a thread adds n / 16 times at most, 2^-24 of the sum each."""
import math

import pytest
import torch

from test_gpu_attn_tiles import F8, UNIT, gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 80])  # the row kernel, the tile kernel
def test_many_small_weights(gdn, dim, new, cache):
    dtype = torch.float16 if cache == "f16" else torch.bfloat16
    page, pages, seqs = 256, 512, 170         # a CTA's stretch is about one sequence: the large key and the small ones meet
    n = page * (pages - 1)
    k = torch.zeros((2, 1, page, dim), device="cuda")
    v = torch.zeros((2, 1, page, dim), device="cuda")
    k[0, 0, :, 0] = -64                       # no weight
    k[0, 0, ::16, 0] = 2                      # where every warp of a CTA, and either half of the tile kernel's softmax, has some
    k[1, :, :, 0] = -24
    v[1] = 1
    scale = math.log(2.0)                     # so that the weights are 2^k
    q = torch.zeros((seqs * new, 1, dim), dtype=dtype, device="cuda")
    q[:, :, 0] = 1
    one = torch.ones((2, 1, page), device="cuda") if cache == "e4m3" else None
    k, v = (t.to(F8 if cache == "e4m3" else dtype) for t in (k, v))
    table = torch.ones((seqs, pages), dtype=torch.int64, device="cuda")
    table[:, 0] = 0
    lens = torch.full((seqs,), page * pages, device="cuda")
    lse = torch.empty((seqs * new, 1), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gdn.attn_paged(q, k, v, table, lens, torch.arange(0, seqs * new + 1, new).cuda(), new, scale=scale, k_scale=one, v_scale=one,
                         lse=lse, dev_status=status)
    assert status.item() == 0
    seen = (n - torch.arange(new - 1, -1, -1, device="cuda")).double().repeat(seqs)  # small keys that a query sees
    mass = seen * 2.0 ** -30
    want = mass / (1 + mass)
    e = 2.0 ** -18 + n / 16 * 2.0 ** -24
    tol = UNIT[dtype] + e
    assert float(((out.double()[:, 0] - want[:, None]).abs() / want[:, None]).max()) <= tol
    off = lse.double()[:, 0] - (math.log(2.0) * 6 + torch.log1p(mass))
    assert float(off.abs().max()) <= e
