"""Host-side refusals of the 8-bit step's entry points (no GPU): nothing is
enqueued, and the text names the argument."""

import ctypes

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2


def at(i):
    """Addresses that lie far apart, never dereferenced: every case fails on the host first."""
    return ctypes.c_void_p((i + 1) << 40)


ODD = ctypes.c_void_p((1 << 46) + 8)


@pytest.fixture(scope="module")
def lib():
    from hashed_gram_embedding_gb300 import build, _lib
    build.build()
    return _lib.lib()


def norm(lib, **kw):
    a = dict(x=at(0), xs=256, r=at(1), rs=256, g=at(2), eps=1e-6, T=3, C=256, so=at(3), ss=256, codes=at(4), scales=at(5))
    a.update(kw)
    return lib.ple_norm_mx8(a["x"], a["xs"], a["r"], a["rs"], a["g"], a["eps"], a["T"], a["C"], a["so"], a["ss"],
                            a["codes"], a["scales"], None)


def read(lib, **kw):
    a = dict(codes=at(0), scales=at(1), rows=3, C=256, out=at(2))
    a.update(kw)
    return lib.ple_mx8_read(a["codes"], a["scales"], a["rows"], a["C"], a["out"], None)


def gated(lib, **kw):
    a = dict(x=at(0), xs=at(1), T=3, C=256, w=at(2), ws=at(3), inner=128, act=0, codes=at(4), scales=at(5))
    a.update(kw)
    return lib.ple_gated_mx8(a["x"], a["xs"], a["T"], a["C"], a["w"], a["ws"], a["inner"], a["act"], a["codes"],
                             a["scales"], None, None)


def proj(lib, **kw):
    a = dict(x=at(0), xs=at(1), T=3, C=256, w=at(2), ws=at(3), N=77, r=at(4), rs=80, out=at(5))
    a.update(kw)
    return lib.ple_proj_mx8(a["x"], a["xs"], a["T"], a["C"], a["w"], a["ws"], a["N"], a["r"], a["rs"], a["out"],
                            None, None)


def near(p, n):
    return ctypes.c_void_p(p.value + n)


def test_scale_bytes(lib):
    f = lib.ple_mx8_scale_bytes
    assert [f(1, 128), f(128, 128), f(129, 128), f(300, 640)] == [512, 512, 1024, 3 * 5 * 512]
    assert [f(0, 128), f(-1, 128), f(5, 0), f(5, 100), f(5, -128), f(1 << 32, 128)] == [0] * 6
    assert f(2**31 - 1, 128) == (2**31 // 128) * 512


def test_norm(lib):
    for bad in (dict(T=-1), dict(T=1 << 31), dict(C=0), dict(C=-128), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(codes=None), dict(scales=None),
                dict(x=ODD), dict(r=ODD), dict(g=ODD), dict(so=ODD), dict(codes=ODD), dict(scales=ODD), dict(xs=260),
                dict(rs=260), dict(ss=260), dict(ss=248), dict(ss=0)):
        assert norm(lib, **bad) == INVALID, bad
    for bad in (dict(C=100), dict(C=16512)):
        assert norm(lib, **bad) == UNSUPPORTED, bad
        assert b"hidden" in lib.ple_last_error()
    assert norm(lib, T=0, x=None, codes=None) == OK
    # outputs on inputs or on one another; the sum in the place of an input, but by other rows
    for bad in (dict(codes=at(0)), dict(codes=near(at(1), 3 * 512 - 16)), dict(scales=at(2)), dict(scales=at(4)),
                dict(so=at(4)), dict(so=near(at(5), 496)), dict(so=at(2)), dict(so=at(0), ss=512, xs=256),
                dict(so=near(at(1), 16), rs=256), dict(x=at(3), r=near(at(3), 32))):
        assert norm(lib, **bad) == INVALID, bad
        assert b"overlap" in lib.ple_last_error()


def test_read(lib):
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(C=0), dict(codes=None), dict(scales=None), dict(out=None),
                dict(codes=ODD), dict(scales=ODD), dict(out=ODD), dict(out=at(0)), dict(out=near(at(1), 496)),
                dict(out=near(at(0), -1536 + 16))):
        assert read(lib, **bad) == INVALID, bad
    assert read(lib, C=96) == UNSUPPORTED
    assert read(lib, rows=0, codes=None) == OK


def test_gated(lib):
    for bad in (dict(T=-1), dict(T=1 << 31), dict(C=0), dict(inner=0), dict(x=None), dict(xs=None), dict(w=None),
                dict(ws=None), dict(codes=None), dict(scales=None), dict(x=ODD), dict(xs=ODD), dict(w=ODD), dict(ws=ODD),
                dict(codes=ODD), dict(scales=ODD)):
        assert gated(lib, **bad) == INVALID, bad
    for bad in (dict(C=160), dict(inner=64), dict(inner=192), dict(act=2), dict(act=-1), dict(inner=1 << 30)):
        assert gated(lib, **bad) == UNSUPPORTED, bad
    assert gated(lib, T=0, x=None) == OK
    for bad in (dict(codes=at(0)), dict(codes=near(at(1), 1008)), dict(codes=near(at(2), 65520)), dict(codes=at(3)),
                dict(scales=at(0)), dict(scales=at(1)), dict(scales=near(at(2), -496)), dict(scales=at(3)),
                dict(scales=near(at(4), 368))):
        assert gated(lib, **bad) == INVALID, bad
        assert b"overlap" in lib.ple_last_error()


def test_proj(lib):
    for bad in (dict(T=-1), dict(T=1 << 31), dict(C=0), dict(N=0), dict(x=None), dict(xs=None), dict(w=None),
                dict(ws=None), dict(out=None), dict(x=ODD), dict(xs=ODD), dict(w=ODD), dict(ws=ODD),
                dict(out=near(at(5), 1)), dict(r=near(at(4), 1))):
        assert proj(lib, **bad) == INVALID, bad
    assert proj(lib, C=64) == UNSUPPORTED and proj(lib, N=2**31 - 1) == UNSUPPORTED and proj(lib, T=5 << 20) == UNSUPPORTED
    assert proj(lib, T=0, x=None) == OK
    for bad in (dict(out=at(0)), dict(out=at(1)), dict(out=near(at(2), 77 * 256 - 16)), dict(out=at(3)),
                dict(out=at(4), rs=80), dict(out=near(at(4), 16), rs=77), dict(out=near(at(4), -16), rs=77)):
        assert proj(lib, **bad) == INVALID, bad
        assert b"overlap" in lib.ple_last_error()
