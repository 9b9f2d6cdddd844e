"""What the page operators refuse before they touch a device (CPU)."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def nsv():
    from paged_kv_decode_nsv_gb300 import build
    build.build()
    from paged_kv_decode_nsv_gb300 import nsv as mod
    return mod


P = 1 << 20     # a fake but aligned pointer: every refusal comes before its use


def _calls(nsv, shape, count=3, tokens=9, ws=P, ws_bytes=1 << 40, null=None, off=None):
    """Every operator's return code, and the names of its pointers."""
    s, lib = ctypes.byref(shape), nsv._lib

    def p(name):
        return None if name == null else P + (off[1] if off and off[0] == name else 0)

    return {
        "copy": lambda: lib.nsv_blocks_copy(s, count, p("a"), p("b"), p("k"), p("v"), None),
        "fork": lambda: lib.nsv_rows_fork(s, count, p("a"), p("b"), p("bt"), p("ctx"), p("refs"),
                                          p("k"), p("v"), ws, ws_bytes, None),
        "extend": lambda: lib.nsv_rows_extend(s, tokens, p("starts"), p("bt"), p("ctx"), p("refs"),
                                              p("slots"), ws, ws_bytes, None),
        "free": lambda: lib.nsv_rows_free(s, count, p("a"), p("bt"), p("ctx"), p("refs"), None),
        "compact": lambda: lib.nsv_blocks_compact(s, p("bt"), p("ctx"), p("refs"), p("k"), p("v"),
                                                  ws, ws_bytes, None),
    }


NAMES = {"copy": ["a", "b", "k", "v"], "fork": ["a", "b", "bt", "ctx", "refs", "k", "v"],
         "extend": ["starts", "bt", "ctx", "refs", "slots"], "free": ["a", "bt", "ctx", "refs"],
         "compact": ["bt", "ctx", "refs", "k", "v"]}


def _shape(nsv, **kw):
    d = dict(rows=4, num_heads=2, num_kv_heads=2, head_dim=128, max_blocks=64, num_blocks=200,
             dtype=nsv.BF16)
    d.update(kw)
    return nsv.make_shape(**d)


@pytest.mark.parametrize("op", list(NAMES))
def test_pointers(nsv, op):
    s = _shape(nsv)
    for name in NAMES[op]:
        assert _calls(nsv, s, null=name)[op]() == -1
        off = 8 if name in ("k", "v") else 4 if name == "slots" else 2
        assert _calls(nsv, s, off=(name, off))[op]() == -4


@pytest.mark.parametrize("op", list(NAMES))
@pytest.mark.parametrize("kw,code", [(dict(head_dim=80), -10), (dict(block_size=8), -10),
                                     (dict(dtype=2), -2), (dict(rows=9000), -3),
                                     (dict(num_blocks=0), -3), (dict(max_blocks=0), -3)])
def test_shapes(nsv, op, kw, code):
    assert _calls(nsv, _shape(nsv, **kw))[op]() == code


def test_counts(nsv):
    s = _shape(nsv)
    for op in ("copy", "fork", "free"):
        assert _calls(nsv, s, count=-1)[op]() == -3
        assert _calls(nsv, s, count=0, null="a")[op]() == 0
    assert _calls(nsv, s, count=5)["fork"]() == -3      # more forks than rows
    assert _calls(nsv, s, tokens=-1)["extend"]() == -3
    assert _calls(nsv, s, tokens=1 << 30)["extend"]() == -3
    assert _calls(nsv, s, tokens=0, null="bt")["extend"]() == 0
    assert _calls(nsv, _shape(nsv, rows=0), null="bt")["extend"]() == 0
    assert _calls(nsv, _shape(nsv, rows=0), null="bt")["free"]() == 0


@pytest.mark.parametrize("op", ["fork", "extend", "compact"])
def test_workspace(nsv, op):
    s = _shape(nsv)
    need = nsv.pages_workspace_bytes(4, 200)
    for kw in (dict(ws=None), dict(ws=P + 128), dict(ws_bytes=need - 1)):
        assert _calls(nsv, s, **kw)[op]() == -8
    # fork: two int2 per row and the free blocks; compact: map, holes, movers
    assert need == 256 + max(4 * 16 + 200 * 4, 200 * 4 + 2 * 101 * 4)
    assert nsv.pages_workspace_bytes(8192, 10) == 256 + 8192 * 20


def test_blocks_too_large_to_count(nsv):
    s = _shape(nsv, num_heads=1 << 20, num_kv_heads=1 << 20)
    for op in ("copy", "fork", "compact"):
        assert _calls(nsv, s)[op]() == -3
