"""What the chunk attention refuses before it touches a device (CPU), and its
workspace sizes."""

import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def nsv():
    from paged_kv_decode_nsv_gb300 import build
    build.build()
    from paged_kv_decode_nsv_gb300 import nsv as mod
    return mod


def _shape(nsv, **kw):
    d = dict(rows=4, num_heads=8, num_kv_heads=2, head_dim=128, max_blocks=64, num_blocks=200,
             dtype=nsv.BF16, query_len=1)
    d.update(kw)
    return nsv.make_shape(**d)


@pytest.mark.parametrize("kw,tokens,code", [
    (dict(head_dim=96), 10, -10), (dict(block_size=32), 10, -10), (dict(dtype=3), 10, -2),
    (dict(num_heads=7), 10, -3), (dict(rows=8193), 10, -3), (dict(rows=-1), 10, -3),
    (dict(query_len=2), 10, -3), (dict(), -1, -3), (dict(), 1 << 30, -3),
    (dict(num_blocks=(1 << 29)), 10, -3), (dict(num_heads=130), 10, -3),
])
def test_bad_sizes(nsv, kw, tokens, code):
    with pytest.raises(nsv.NsvError) as e:
        nsv.chunk_workspace_bytes(_shape(nsv, **kw), tokens, num_sms=152)
    assert e.value.code == code


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (8, 2), (5, 1), (64, 1)])
def test_workspace_grows_with_the_batch(nsv, dtype, heads, kv_heads):
    code = nsv.F32 if dtype == "f32" else nsv.BF16
    size = lambda rows, tokens: nsv.chunk_workspace_bytes(  # noqa: E731
        _shape(nsv, rows=rows, num_heads=heads, num_kv_heads=kv_heads, dtype=code), tokens, 152)
    sizes = [[size(r, t) for t in (1, 7, 64, 513, 4096, 100000)] for r in (1, 3, 100, 8192)]
    for row in sizes:
        assert row == sorted(row)
    for a, b in zip(sizes, sizes[1:]):
        assert all(x <= y for x, y in zip(a, b))
    # the partial states of a grid of CTAs at most, and the list
    assert size(8192, 100000) < 2 * 152 * 2 * 256 * (128 + 2) * 4 + \
        (8192 + 100000) * (48 + 4 * kv_heads)


def _call(nsv, shape, tokens=10, scores=None, step=False, **null):
    """A call with fake but aligned pointers: every refusal under test comes
    before any of them is used."""
    p = {k: 1 << 20 for k in ("q", "kn", "vn", "ws_", "k", "v", "bt", "starts", "ctx", "out",
                              "work")}
    p.update(null)
    lib = nsv._lib
    sc = ctypes.byref(scores) if scores is not None else None
    if step:
        return lib.nsv_chunk_step(ctypes.byref(shape), sc, tokens, p["q"], p["kn"], p["vn"],
                                  p["ws_"], p["k"], p["v"], p["bt"], p["starts"], p["ctx"], 1.0,
                                  p["out"], p["work"], 1 << 40, None)
    return lib.nsv_paged_chunk(ctypes.byref(shape), sc, tokens, p["q"], p["k"], p["v"], p["bt"],
                               p["starts"], p["ctx"], 1.0, p["out"], p["work"], 1 << 40, None)


@pytest.mark.parametrize("step", [False, True])
def test_null_and_misaligned_pointers(nsv, step):
    s = _shape(nsv)
    names = ["q", "k", "v", "bt", "starts", "ctx", "out"] + (["kn", "vn", "ws_"] if step else [])
    if not step:    # the step first asks for the device
        for name in names:
            assert _call(nsv, s, **{name: None}) == -1
            off = 2 if name in ("bt", "starts", "ctx") else 8
            assert _call(nsv, s, **{name: (1 << 20) + off}) == -4
    else:
        for name in ("kn", "vn", "ws_", "k", "v"):
            assert _call(nsv, s, step=True, **{name: None}) == -1
        for name, off in (("kn", 8), ("vn", 8), ("ws_", 4)):
            assert _call(nsv, s, step=True, **{name: (1 << 20) + off}) == -4


def test_bad_scores(nsv):
    s = _shape(nsv)
    for cap in (-1.0, math.nan, math.inf, 1e-7, 2e6):
        assert _call(nsv, s, scores=nsv.Scores(cap, None, None, None)) == -5
    for field in ("slopes", "see_begin", "see_end"):
        sc = nsv.Scores(0.0, None, None, None)
        setattr(sc, field, (1 << 20) + 2)
        assert _call(nsv, s, scores=sc) == -4


def test_nothing_to_do_is_no_error(nsv):
    for step in (False, True):
        assert _call(nsv, _shape(nsv, rows=0), step=step, q=None, k=None, v=None) == 0
        assert _call(nsv, _shape(nsv), tokens=0, step=step, q=None, k=None, v=None) == 0


def test_binding_checks_types_shapes_and_devices(nsv):
    import torch
    ok = torch.zeros(4, 3, dtype=torch.int32)
    cpu = ok.get_device()       # what a CPU tensor answers: no CUDA device's number
    assert nsv._arg(ok, "x", torch.int32, (4, 3), cpu) == ok.data_ptr()
    assert nsv._arg(None, "x", torch.int32, (4,), cpu) is None
    for t, dtype, shape, dev in (
            (ok, torch.int64, (4, 3), cpu), (ok, torch.int32, (4,), cpu),
            (ok, torch.int32, (5, 3), cpu), (ok.t(), torch.int32, (3, 4), cpu),
            (ok[:, :2], torch.int32, (4, 2), cpu), (ok, torch.int32, (4, 3), 0)):
        with pytest.raises(ValueError):
            nsv._arg(t, "x", dtype, shape, dev)
