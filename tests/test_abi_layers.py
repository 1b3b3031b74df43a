"""Host-side refusals of the rotation with the append, the short convolution, the state space scan and the norm (no GPU:
every call here is rejected, or has nothing to do, before the first CUDA call)."""
import ctypes

import pytest

import gated_deltanet_delta_gb300 as gdn
from gated_deltanet_delta_gb300 import build as gbuild

N, BF16, F32, F16, E4M3 = None, 0, 1, 2, 3
INVALID, UNSUPPORTED, OK = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_OK


def at(i, off=0):  # addresses far apart, never dereferenced
    return ctypes.c_void_p(((i + 1) << 44) + off)


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load()


def call(f, defaults, order, kw):
    a = dict(defaults)
    a.update(kw)
    return f(*[a[k] for k in order], N)


APPEND = dict(q=at(0), k=at(1), v=at(2), qs=1024, ks=256, vs=256, dt=BF16, rot=at(3), maxpos=100, R=128, nb=0, pos=at(4), slots=at(5), T=3,
              qo=at(6), qos=1024, kc=at(7), vc=at(8), ksc=N, vsc=N, cdt=BF16, pages=10, page=16, hq=8, h=2, D=128, st=at(9))


@pytest.mark.parametrize("kw,want", [
    (dict(k=at(0), ks=1024), INVALID), (dict(k=at(0, 512), ks=1024), INVALID), (dict(k=at(0, 2 * 1024), ks=1536), INVALID),
    (dict(v=at(0, 2 * 1400), vs=1536, qs=1536, qos=1536), INVALID), (dict(k=at(0, 2 * 1024), ks=1536, qs=1536, qos=1536, T=0), OK),
])
def test_append_in_place_refuses_rows_that_overlap(lib, kw, want):
    """q_out is q: the keys and values may stand behind the queries in the same rows, not among them."""
    assert call(lib.attn_cache_append, APPEND, APPEND, dict(kw, qo=at(0))) == want
    if want != OK:
        assert "overlap" in gdn.last_error()


@pytest.mark.parametrize("kw,want,word", [
    (dict(D=96), UNSUPPORTED, "64, 128 or 256"), (dict(R=8), UNSUPPORTED, "rotary_dim"), (dict(R=144), UNSUPPORTED, "rotary_dim"),
    (dict(R=24), UNSUPPORTED, "rotary_dim"), (dict(dt=F32), INVALID, "dtype"), (dict(cdt=F16), INVALID, "cache_dtype"), (dict(cdt=E4M3), INVALID, "k_scale"),
    (dict(q=N), INVALID, "null"), (dict(qo=N), INVALID, "null"), (dict(rot=N), INVALID, "null"), (dict(pos=N), INVALID, "null"),
    (dict(ks=252), INVALID, "strides"), (dict(qs=1000), INVALID, "strides"), (dict(qos=1020), INVALID, "strides"),
    (dict(q=at(0, 8)), INVALID, "aligned"), (dict(rot=at(3, 4)), INVALID, "aligned"), (dict(kc=at(8)), INVALID, "overlap"),
    (dict(qo=at(1)), INVALID, "overlap"), (dict(qo=at(0, 2048)), INVALID, "overlap"), (dict(qo=at(0), qos=2048), INVALID, "overlap"),
    (dict(qo=at(3)), INVALID, "overlap"), (dict(qo=at(7)), INVALID, "overlap"), (dict(k=at(7)), INVALID, "overlap"),
    (dict(cdt=E4M3, ksc=at(10), vsc=at(10)), INVALID, "overlap"), (dict(T=-1), INVALID, "sizes"), (dict(page=0), INVALID, "sizes"),
    (dict(hq=-1), INVALID, "sizes"), (dict(T=1 << 31), UNSUPPORTED, "2^31"), (dict(maxpos=1 << 50), UNSUPPORTED, "max_positions"),
    (dict(hq=70000, qs=70000 * 128, qos=70000 * 128), UNSUPPORTED, "65535"),
])
def test_append_refuses(lib, kw, want, word):
    assert call(lib.attn_cache_append, APPEND, APPEND, kw) == want
    assert gdn.last_error().startswith("attn_cache_append:") and word in gdn.last_error()


def test_append_without_work(lib):
    assert call(lib.attn_cache_append, APPEND, APPEND, dict(T=0, q=N, kc=N)) == OK


CONV = dict(x=at(0), xs=512, dt=BF16, w=at(1), b=at(2), hist=at(3), pool=5, idx=at(4), cu=at(5), n=2, T=9, C=256, taps=4, silu=1, o0=at(6), c0=128,
            o1=at(7), c1=64, o2=at(8), c2=64, st=at(9))


@pytest.mark.parametrize("kw,want,word", [
    (dict(taps=1), UNSUPPORTED, "taps"), (dict(taps=5), UNSUPPORTED, "taps"), (dict(dt=E4M3), INVALID, "dtype"), (dict(c0=120), INVALID, "add up"),
    (dict(c0=192, c1=0), INVALID, "add up"), (dict(c0=132, c1=60), UNSUPPORTED, "multiples of 8"), (dict(cu=N), INVALID, "num_seqs"),
    (dict(x=N), INVALID, "null"), (dict(o1=N), INVALID, "null"), (dict(idx=N), INVALID, "null"), (dict(st=N), INVALID, "null"),
    (dict(xs=255), INVALID, "x_stride"), (dict(xs=260), INVALID, "x_stride"), (dict(xs=1 << 31), INVALID, "x_stride"),
    (dict(x=at(0, 8)), INVALID, "aligned"), (dict(w=at(1, 4)), INVALID, "aligned"), (dict(hist=at(3, 8)), INVALID, "aligned"), (dict(o2=at(8, 2)), INVALID, "aligned"),
    (dict(o0=at(0)), INVALID, "overlap"), (dict(o1=at(6)), INVALID, "overlap"), (dict(o2=at(3)), INVALID, "overlap"), (dict(hist=at(0)), INVALID, "overlap"),
    (dict(T=-1), INVALID, "sizes"), (dict(C=0), INVALID, "sizes"), (dict(T=1 << 31), UNSUPPORTED, "2^31"),
])
def test_conv_refuses(lib, kw, want, word):
    assert call(lib.short_conv, CONV, CONV, kw) == want
    assert gdn.last_error().startswith("short_conv:") and word in gdn.last_error()


def test_conv_without_work(lib):
    assert call(lib.short_conv, CONV, CONV, dict(T=0, x=N)) == OK and call(lib.short_conv, CONV, CONV, dict(n=0, cu=N, x=N)) == OK


def strides(*s):
    return (ctypes.c_int64 * 5)(*s)


STEP = dict(x=at(0), dt=at(1), B=at(2), C=at(3), z=at(4), strides=strides(512, 9, 256, 256, 512), A=at(5), D=at(6), bias=at(7), state=at(8), pool=4, idx=at(9),
            n=3, H=8, P=64, G=2, S=128, out=at(10), st=at(11))
SCAN = dict(STEP, cu=at(12), T=50, max_len=20, ws=at(13), wsz=1 << 40)
SCAN_ORDER = ("x", "dt", "B", "C", "z", "strides", "A", "D", "bias", "state", "pool", "idx", "cu", "n", "T", "max_len", "H", "P", "G", "S", "out", "ws", "wsz", "st")
BOTH = [
    (dict(H=7), INVALID, "multiple"), (dict(P=32), UNSUPPORTED, "64 or 128"), (dict(S=256), UNSUPPORTED, "64 or 128"), (dict(G=0), INVALID, "sizes"),
    (dict(x=N), INVALID, "null"), (dict(A=N), INVALID, "null"), (dict(state=N), INVALID, "null"), (dict(idx=N), INVALID, "null"), (dict(strides=N), INVALID, "null"),
    (dict(strides=strides(504, 9, 256, 256, 512)), INVALID, "strides"), (dict(strides=strides(512, 7, 256, 256, 512)), INVALID, "strides"),
    (dict(strides=strides(512, 9, 260, 256, 512)), INVALID, "strides"), (dict(strides=strides(512, 9, 256, 256, 516)), INVALID, "strides"),
    (dict(x=at(0, 8)), INVALID, "aligned"), (dict(z=at(4, 2)), INVALID, "aligned"), (dict(state=at(8, 4)), INVALID, "aligned"), (dict(out=at(10, 8)), INVALID, "aligned"),
    (dict(out=at(0)), INVALID, "overlap"), (dict(out=at(4)), INVALID, "overlap"), (dict(out=at(8)), INVALID, "overlap"), (dict(state=at(2)), INVALID, "overlap"),
    (dict(out=at(5)), INVALID, "overlap"),
]


@pytest.mark.parametrize("kw,want,word", BOTH + [(dict(n=-1), INVALID, "sizes"), (dict(n=1 << 28), UNSUPPORTED, "2^31")])
def test_step_refuses(lib, kw, want, word):
    assert call(lib.ssm_decode_step, STEP, STEP, kw) == want
    assert gdn.last_error().startswith("ssm_decode_step:") and word in gdn.last_error()


@pytest.mark.parametrize("kw,want,word", BOTH + [
    (dict(T=-1), INVALID, "sizes"), (dict(T=1 << 31), UNSUPPORTED, "2^31"), (dict(cu=N), INVALID, "cu_seqlens"), (dict(max_len=-1), INVALID, "max_len"),
    (dict(ws=at(13, 8)), INVALID, "aligned"), (dict(ws=at(13, 16)), INVALID, "32-byte"), (dict(state=at(8, 16)), INVALID, "32-byte"),
])
def test_prefill_refuses(lib, kw, want, word):
    assert call(lib.ssm_prefill_chunked, SCAN, SCAN_ORDER, kw) == want
    assert gdn.last_error().startswith("ssm_prefill_chunked:") and word in gdn.last_error()


def test_scan_without_work(lib):
    assert call(lib.ssm_decode_step, STEP, STEP, dict(n=0, x=N)) == OK
    assert call(lib.ssm_prefill_chunked, SCAN, SCAN_ORDER, dict(n=0, x=N)) == OK and call(lib.ssm_prefill_chunked, SCAN, SCAN_ORDER, dict(T=0, x=N)) == OK
    assert gdn.ssm_prefill_workspace_size(2, 100, 4, 96, 64) == 0


NORM = dict(x=at(0), xs=256, res=at(1), dt=BF16, w=at(2), eps=1e-6, T=5, C=256, out=at(3), odt=E4M3, scale=at(4), group=64)


@pytest.mark.parametrize("kw,want,word", [
    (dict(C=36), UNSUPPORTED, "multiple of 8"), (dict(C=32776), UNSUPPORTED, "32768"), (dict(dt=F32), INVALID, "dtype"), (dict(odt=F16), INVALID, "out_dtype"),
    (dict(scale=N), INVALID, "scale"), (dict(odt=BF16), INVALID, "scale"), (dict(odt=BF16, scale=N), UNSUPPORTED, "group"), (dict(group=16), UNSUPPORTED, "group"),
    (dict(C=320, xs=320, group=128), UNSUPPORTED, "group"), (dict(x=N), INVALID, "null"), (dict(w=N), INVALID, "null"), (dict(xs=248), INVALID, "x_stride"),
    (dict(xs=260), INVALID, "x_stride"), (dict(x=at(0, 2)), INVALID, "aligned"), (dict(w=at(2, 4)), INVALID, "aligned"), (dict(res=at(0)), INVALID, "overlap"),
    (dict(out=at(0)), INVALID, "overlap"), (dict(out=at(1)), INVALID, "overlap"), (dict(scale=at(3)), INVALID, "overlap"), (dict(T=-1), INVALID, "sizes"),
    (dict(out=at(0), odt=BF16, scale=N, group=0, xs=512), INVALID, "overlap"), (dict(T=1 << 31), UNSUPPORTED, "2^31"),
])
def test_norm_refuses(lib, kw, want, word):
    assert call(lib.add_rms_norm, NORM, NORM, kw) == want
    assert gdn.last_error().startswith("add_rms_norm:") and word in gdn.last_error()


def test_norm_without_work(lib):
    assert call(lib.add_rms_norm, NORM, NORM, dict(T=0, x=N)) == OK
