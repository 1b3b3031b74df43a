"""attn_paged's bounded device-side waits, made to run out on purpose.

Every barrier wait of the tile kernel and of the 8-bit row kernel gives up after a bounded number of polls,
sets GDN_STATUS_TIMEOUT and stops its CTA once its copies and products in flight have ended.
attn_set_wait_limit(1) makes the limits small enough to run out on a healthy GPU: the call must return and
report it, and the next call on the same stream, with the built-in limits, must be right.  No fault, trap or
hang is involved: the kernels stop by themselves."""
import pytest
import torch

from test_gpu_attn_tiles import call, check, gdn, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built_in_limits(gdn):
    yield
    gdn.set_attn_wait_limit(0)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_tile_kernel(gdn, dim, f8):
    x = make(31, [20, 20, 20], [9000, 3000, 100], 32, 8, dim, 64, torch.bfloat16, f8)
    good = call(gdn, x, 0.07)
    check(x, good[0], good[1], 0.07)
    for _ in range(5):
        gdn.set_attn_wait_limit(1)
        assert call(gdn, x, 0.07)[2] == gdn.STATUS_TIMEOUT
        gdn.set_attn_wait_limit(0)
        again = call(gdn, x, 0.07)
        assert again[2] == 0 and torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_row_kernel(gdn, dim):
    # one poll may last as long as a copy, so the wait runs out in most calls on a cold cache, not in every one
    kv = [8192 - 100 * n for n in range(64)]
    x = make(32, [1] * 64, kv, 64, 8, dim, 64, torch.bfloat16, True)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")

    def one():
        lse, status = torch.empty((64, 64), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        out = gdn.attn_paged(x["q"], x["k"], x["v"], x["table"], torch.tensor(kv).cuda(), torch.tensor(x["cu"]).cuda(), 1, scale=0.07,
                             k_scale=x["k_scale"], v_scale=x["v_scale"], lse=lse, dev_status=status)
        return out, lse, int(status.item())
    good = one()
    assert good[2] == 0
    check(x, good[0], good[1], 0.07, (0, 31, 63))
    seen = 0
    for _ in range(50):
        flush.fill_(1)
        gdn.set_attn_wait_limit(1)
        status = one()[2]
        assert status in (0, gdn.STATUS_TIMEOUT)
        seen += status != 0
        gdn.set_attn_wait_limit(0)
        again = one()
        assert again[2] == 0 and torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])
    assert seen > 0
