"""Host-side refusals of buffers that a call both writes and reads: the scan's workspace and state pool, the append's scales (no GPU)."""
import pytest

import gated_deltanet_delta_gb300 as gdn
from test_abi_layers import APPEND, E4M3, INVALID, SCAN, SCAN_ORDER, STEP, at, call, lib  # noqa: F401


@pytest.mark.parametrize("name", ["x", "dt", "B", "C", "z", "A", "D", "bias", "state", "idx", "cu", "out", "st"])
def test_workspace(lib, name):  # noqa: F811
    long = dict(SCAN, T=5000, max_len=5000)
    assert call(lib.ssm_prefill_chunked, long, SCAN_ORDER, dict(ws=long[name])) == INVALID
    assert gdn.last_error().startswith("ssm_prefill_chunked: workspace overlaps")


@pytest.mark.parametrize("name", ["A", "D", "bias"])
def test_state_pool(lib, name):  # noqa: F811
    assert call(lib.ssm_decode_step, STEP, STEP, dict(state=STEP[name])) == INVALID
    assert "state_pool overlaps" in gdn.last_error()


@pytest.mark.parametrize("scale", ["ksc", "vsc"])
@pytest.mark.parametrize("name", ["q", "k", "v", "rot", "qo", "kc", "vc"])
def test_scales(lib, name, scale):  # noqa: F811
    kw = dict(cdt=E4M3, ksc=at(10), vsc=at(11))
    kw[scale] = APPEND[name]
    assert call(lib.attn_cache_append, APPEND, APPEND, kw) == INVALID
    assert gdn.last_error() == "attn_cache_append: a scale overlaps another buffer"
