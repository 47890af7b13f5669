"""Host-side refusals of the 4-bit step's entry points (no GPU): nothing is
enqueued, and the text names the argument."""

import ctypes

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p(256)  # never dereferenced: every case fails on the host first
ODD = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def lib():
    from hashed_gram_embedding_gb300 import build, _lib
    build.build()
    return _lib.lib()


CACHE = dict(cache=P, pages=4, page=16, table=P, max_pages=2, qsl=P, R=1, lens=P)


def append(lib, **kw):
    a = dict(q=P, qs=512, k=P, ks=256, v=P, vs=256, T=2, H=4, Hk=2, D=128, cs=P, npos=10, rot=128, inter=0,
             pos=None, qo=P, qos=512, **CACHE)
    a.update(kw)
    return lib.ple_kv_append(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["T"], a["H"], a["Hk"], a["D"],
                             a["cs"], a["npos"], a["rot"], a["inter"], a["pos"], a["cache"], a["pages"], a["page"],
                             a["table"], a["max_pages"], a["qsl"], a["R"], a["lens"], a["qo"], a["qos"], None, None)


def read(lib, **kw):
    a = dict(T=2, Hk=2, D=128, ko=P, vo=P, **CACHE)
    a.update(kw)
    return lib.ple_kv_read(a["cache"], a["pages"], a["page"], a["table"], a["max_pages"], a["qsl"], a["R"],
                           a["lens"], a["T"], a["Hk"], a["D"], a["ko"], a["vo"], None, None)


def attention(lib, **kw):
    a = dict(q=P, qs=512, T=2, H=4, Hk=2, D=128, hint=0, scale=0.1, causal=1, window=0, out=P, os=512, ws=P,
             wsb=1 << 30, **CACHE)
    a.update(kw)
    return lib.ple_kv_attention(a["q"], a["qs"], a["T"], a["H"], a["Hk"], a["D"], a["cache"], a["pages"], a["page"],
                                a["table"], a["max_pages"], a["qsl"], a["R"], a["lens"], a["hint"], a["scale"],
                                a["causal"], a["window"], a["out"], a["os"], a["ws"], a["wsb"], None, None)


def proj(lib, **kw):
    a = dict(x=P, xs=256, T=2, E=256, N=10, codes=P, scales=P, zeros=None, group=64, out=P)
    a.update(kw)
    return lib.ple_proj_w4(a["x"], a["xs"], a["T"], a["E"], a["N"], a["codes"], a["scales"], a["zeros"], a["group"],
                           a["out"], None, None)


@pytest.mark.parametrize("call", [append, read, attention])
def test_cache_arguments(lib, call):
    assert call(lib, D=96) == UNSUPPORTED
    assert b"head_dim 96" in lib.ple_last_error()
    assert call(lib, page=24) == INVALID
    assert b"page_size 24" in lib.ple_last_error()
    for bad in (dict(page=0), dict(page=-16), dict(pages=-1), dict(max_pages=-1), dict(R=0), dict(Hk=0),
                dict(cache=None), dict(cache=ODD), dict(table=None), dict(qsl=None), dict(lens=None), dict(T=-1),
                dict(T=1 << 32)):
        assert call(lib, **bad) == INVALID, bad
    assert call(lib, T=0, cache=None, qsl=None) == OK  # no tokens: nothing to do


def test_append_arguments(lib):
    for bad in (dict(k=None), dict(v=None), dict(q=None), dict(qo=None), dict(H=0), dict(q=ODD), dict(k=ODD),
                dict(v=ODD), dict(qo=ODD), dict(cs=ODD), dict(qs=513), dict(ks=4), dict(vs=-3), dict(qos=2),
                dict(npos=-1)):
        assert append(lib, **bad) == INVALID, bad
    for rot in (0, 8, 24, 144, -16):
        assert append(lib, rot=rot) == UNSUPPORTED


def test_read_arguments(lib):
    assert read(lib, ko=ODD) == INVALID and read(lib, vo=ODD) == INVALID
    assert read(lib, ko=None, vo=None) == OK  # nothing wanted


def test_attention_arguments(lib):
    for bad in (dict(H=0), dict(H=5), dict(q=None), dict(out=None), dict(q=ODD), dict(out=ODD), dict(qs=516),
                dict(os=9), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(hint=-1), dict(window=-1), dict(window=4, causal=0)):
        assert attention(lib, **bad) == INVALID, bad
    need = lib.ple_kv_attention_workspace(4, 2, 128)
    assert need > 0 and need % 256 == 0
    for bad in (dict(ws=None), dict(ws=ODD), dict(wsb=need - 1)):
        assert attention(lib, **bad) == INVALID, bad
        assert b"workspace" in lib.ple_last_error()
    for heads in ((0, 2, 128), (4, 0, 128), (5, 2, 128), (4, 2, 96)):
        assert lib.ple_kv_attention_workspace(*heads) == 0


def test_block_bytes(lib):
    assert [lib.ple_kv_block_bytes(d) for d in (64, 128, 256)] == [1152, 2176, 4224]
    assert [lib.ple_kv_block_bytes(d) for d in (0, -64, 96, 512)] == [0, 0, 0, 0]


def test_proj_arguments(lib):
    for bad in (dict(x=None), dict(codes=None), dict(scales=None), dict(out=None), dict(x=ODD), dict(codes=ODD),
                dict(xs=12), dict(T=-1), dict(T=1 << 32), dict(E=0), dict(N=0)):
        assert proj(lib, **bad) == INVALID, bad
    for bad in (dict(group=16), dict(group=0), dict(group=256), dict(E=96), dict(E=96, group=128)):
        assert proj(lib, **bad) == UNSUPPORTED, bad
    assert proj(lib, T=0, x=None) == OK
