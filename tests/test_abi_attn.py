"""Host-side refusals of the cache, attention and verification entry points (no GPU: every call here is
rejected, or has nothing to do, before the first CUDA call)."""
import ctypes

import pytest

import gated_deltanet_delta_gb300 as gdn
from gated_deltanet_delta_gb300 import build as gbuild

N, BF16, F32, F16, E4M3 = None, 0, 1, 2, 3
INVALID, UNSUPPORTED, OK = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_OK


def at(i):  # addresses far apart, never dereferenced
    return ctypes.c_void_p((i + 1) << 44)


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load()


def test_workspace_size(lib):
    for d in (64, 128, 256):
        # headers, then two slots per CTA: 160 CTAs with 256 (128 for D = 256) rows of D + 2 floats
        rows = 160 * (128 if d == 256 else 256)
        assert gdn.attn_paged_workspace_size(d) == 608 * 24 + rows * 2 * (d + 2) * 4
    assert gdn.attn_paged_workspace_size(96) == 0


def attn(lib, **kw):
    a = dict(q=at(0), q_stride=1024, dtype=BF16, kc=at(1), vc=at(2), ks=N, vs=N, cdt=BF16, pages=10, page=16, table=at(3), maxp=4,
             kv=at(4), cu=at(5), n=2, T=3, max_q=2, hq=8, hkv=2, D=128, scale=1.0, out=at(6), lse=at(7), ws=at(8),
             wsz=gdn.attn_paged_workspace_size(128), st=at(9))
    a.update(kw)
    return lib.attn_paged(*[a[k] for k in ("q", "q_stride", "dtype", "kc", "vc", "ks", "vs", "cdt", "pages", "page", "table", "maxp",
                                           "kv", "cu", "n", "T", "max_q", "hq", "hkv", "D", "scale", "out", "lse", "ws", "wsz", "st")], N)


@pytest.mark.parametrize("kw,want,word", [
    (dict(hq=7), INVALID, "multiple"), (dict(hq=258, hkv=2), UNSUPPORTED, "128"), (dict(D=96), UNSUPPORTED, "64, 128 or 256"),
    (dict(dtype=F32), INVALID, "dtype"), (dict(cdt=F16), INVALID, "cache_dtype"), (dict(cdt=E4M3), INVALID, "k_scale"),
    (dict(ks=at(10), vs=at(11)), INVALID, "no scales"), (dict(kc=N), INVALID, "null"), (dict(q=N), INVALID, "null"),
    (dict(table=N), INVALID, "null"), (dict(st=N), INVALID, "null"), (dict(q_stride=1023), INVALID, "q_stride"),
    (dict(q_stride=1020), INVALID, "q_stride"), (dict(q=ctypes.c_void_p((1 << 44) + 8)), INVALID, "aligned"),
    (dict(kc=ctypes.c_void_p((2 << 44) + 8)), INVALID, "aligned"), (dict(ws=N), INVALID, "workspace"),
    (dict(wsz=1000), INVALID, "workspace"), (dict(ws=ctypes.c_void_p((9 << 44) + 8)), INVALID, "aligned"),
    (dict(out=at(0)), INVALID, "overlaps"), (dict(lse=at(6)), INVALID, "overlaps"), (dict(out=at(2)), INVALID, "overlaps"),
    (dict(T=-1), INVALID, "sizes"), (dict(page=0), INVALID, "sizes"), (dict(T=1 << 30), UNSUPPORTED, "2^30"),
    (dict(page=1 << 20, maxp=1 << 12, pages=1), UNSUPPORTED, "2^31"), (dict(pages=1 << 50), UNSUPPORTED, "too large"),
])
def test_attn_paged_refuses(lib, kw, want, word):
    assert attn(lib, **kw) == want
    assert gdn.last_error().startswith("attn_paged:") and word in gdn.last_error()


def test_attn_paged_without_work(lib):
    assert attn(lib, T=0, q=N, out=N) == OK and attn(lib, n=0, cu=N) == OK


def write(lib, **kw):
    a = dict(k=at(0), v=at(1), ks=256, vs=256, dtype=BF16, slots=at(2), T=5, kc=at(3), vc=at(4), ksc=at(5), vsc=at(6), cdt=E4M3, pages=4,
             page=16, h=2, D=128, st=at(7))
    a.update(kw)
    return lib.attn_cache_write(*[a[k] for k in ("k", "v", "ks", "vs", "dtype", "slots", "T", "kc", "vc", "ksc", "vsc", "cdt", "pages",
                                                 "page", "h", "D", "st")], N)


@pytest.mark.parametrize("kw,want,word", [
    (dict(D=32), UNSUPPORTED, "64, 128 or 256"), (dict(dtype=E4M3), INVALID, "dtype"), (dict(ksc=N), INVALID, "k_scale"),
    (dict(cdt=BF16), INVALID, "no scales"), (dict(slots=N), INVALID, "null"), (dict(ks=255), INVALID, "strides"),
    (dict(vs=128), INVALID, "strides"), (dict(kc=at(4)), INVALID, "overlap"), (dict(v=at(3)), INVALID, "overlap"),
    (dict(k=ctypes.c_void_p((1 << 44) + 2)), INVALID, "aligned"), (dict(h=70000), UNSUPPORTED, "65535"), (dict(T=-2), INVALID, "sizes"),
])
def test_cache_write_refuses(lib, kw, want, word):
    assert write(lib, **kw) == want
    assert gdn.last_error().startswith("attn_cache_write:") and word in gdn.last_error()


def test_cache_write_without_work(lib):
    assert write(lib, T=0, k=N, kc=N) == OK


def read(lib, **kw):
    a = dict(kc=at(3), vc=at(4), ksc=at(5), vsc=at(6), cdt=E4M3, pages=4, page=16, table=at(8), maxp=2, cu=at(9), n=1, T=5, h=2, D=128,
             k=at(0), v=at(1), dtype=F16, st=at(7))
    a.update(kw)
    return lib.attn_cache_read(*[a[k] for k in ("kc", "vc", "ksc", "vsc", "cdt", "pages", "page", "table", "maxp", "cu", "n", "T", "h",
                                                "D", "k", "v", "dtype", "st")], N)


@pytest.mark.parametrize("kw,want,word", [
    (dict(D=512), UNSUPPORTED, "64, 128 or 256"), (dict(dtype=F32), INVALID, "dtype"), (dict(cu=N), INVALID, "null"),
    (dict(table=N), INVALID, "null"), (dict(v=at(0)), INVALID, "overlap"), (dict(k=at(3)), INVALID, "overlap"),
    (dict(k=ctypes.c_void_p((1 << 44) + 8)), INVALID, "aligned"), (dict(maxp=-1), INVALID, "sizes"),
])
def test_cache_read_refuses(lib, kw, want, word):
    assert read(lib, **kw) == want
    assert gdn.last_error().startswith("attn_cache_read:") and word in gdn.last_error()


def test_cache_read_without_work(lib):
    assert read(lib, T=0, k=N) == OK and read(lib, n=0) == OK


def verify(lib, **kw):
    a = dict(p=at(0), q=at(1), x=at(2), nd=N, u=at(3), us=at(4), N=2, T=3, V=100, acc=at(5), tok=at(6), st=at(7))
    a.update(kw)
    return lib.draft_verify(*[a[k] for k in ("p", "q", "x", "nd", "u", "us", "N", "T", "V", "acc", "tok", "st")], N)


@pytest.mark.parametrize("kw,want,word", [
    (dict(V=0), INVALID, "sizes"), (dict(T=-1), INVALID, "sizes"), (dict(V=(1 << 20) + 1), UNSUPPORTED, "2^20"),
    (dict(N=1 << 28), UNSUPPORTED, "2^28"), (dict(p=N), INVALID, "null"), (dict(q=N), INVALID, "null"), (dict(st=N), INVALID, "null"),
    (dict(u=ctypes.c_void_p((4 << 44) + 2)), INVALID, "misaligned"), (dict(tok=at(2)), INVALID, "overlap"),
    (dict(acc=at(6)), INVALID, "overlap"),
])
def test_draft_verify_refuses(lib, kw, want, word):
    assert verify(lib, **kw) == want
    assert gdn.last_error().startswith("draft_verify:") and word in gdn.last_error()


def test_draft_verify_without_work(lib):
    assert verify(lib, N=0, p=N) == OK


def test_attn_wait_limit_is_a_host_setting(lib):
    gdn.set_attn_wait_limit(1)
    lib.attn_set_wait_limit(ctypes.c_uint32(0xFFFFFFFF))
    gdn.set_attn_wait_limit(0)


def test_a_workspace_off_the_device_is_refused():
    # its address would be written to by the kernels
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        gdn._want_workspace(torch.empty(64, dtype=torch.uint8), 64, "cpu")
    with pytest.raises(TypeError, match="workspace"):
        gdn._want_workspace(bytes(64), 64, "cpu")
    assert gdn._want_workspace(None, 64, "cpu").nbytes == 64 and gdn._want_workspace(None, 0, "cpu").nbytes == 0


def test_cache_write_refuses_shared_scales(lib):
    # keys and values would write their scales to the same places
    assert write(lib, vsc=at(5)) == INVALID and "k_scale and v_scale overlap" in gdn.last_error()
    assert write(lib, vsc=ctypes.c_void_p((6 << 44) + 4 * 16 * 2 * 4 - 4)) == INVALID
