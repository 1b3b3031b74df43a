"""attn_paged's tile kernel where a wait runs out behind the last copy that is issued: calls of a tile or two, whose loaders come to
their end while others give up.  The CTA still gives those copies a millisecond before it ends."""
import pytest
import torch

from test_gpu_attn_tiles import call, check, gdn, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built_in_limits(gdn):  # noqa: F811
    yield
    gdn.set_attn_wait_limit(0)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_short_call_that_gives_up(gdn, dim, f8):  # noqa: F811
    x = make(41, [20, 20], [60, 100], 32, 8, dim, 64, torch.bfloat16, f8)
    good = call(gdn, x, 0.07)
    assert good[2] == 0
    check(x, good[0], good[1], 0.07)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    kv, cu = torch.tensor(x["kv"]).cuda(), torch.tensor(x["cu"]).cuda()
    ws = torch.empty(gdn.attn_paged_workspace_size(dim), dtype=torch.uint8, device="cuda")
    out, status = torch.empty_like(x["q"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    seen = 0
    for _ in range(20):
        flush.fill_(1)
        status.zero_()
        gdn.set_attn_wait_limit(1)
        begin.record()
        gdn.attn_paged(x["q"], x["k"], x["v"], x["table"], kv, cu, 20, scale=0.07, k_scale=x["k_scale"], v_scale=x["v_scale"], out=out, workspace=ws,
                       dev_status=status)
        end.record()
        gdn.set_attn_wait_limit(0)
        again = call(gdn, x, 0.07)
        assert again[2] == 0 and torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])
        assert status.item() in (0, gdn.STATUS_TIMEOUT)
        if status.item():
            seen += 1
            assert begin.elapsed_time(end) >= 0.98  # ms: the event clock ticks in half microseconds
    assert seen > 0
