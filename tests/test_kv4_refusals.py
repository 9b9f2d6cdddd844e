"""What the rotating appends and the 4-bit cache's operators refuse before they touch
a device (CPU), and the attention's workspace sizes."""

import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def nsv():
    from paged_kv_decode_nsv_gb300 import build
    build.build()
    from paged_kv_decode_nsv_gb300 import nsv as mod
    return mod


P = 1 << 20     # a fake but aligned pointer: every refusal comes before its use
TENSORS = ["q", "kn", "vn", "slots", "k", "v", "q_out"]


def _shape(nsv, **kw):
    d = dict(rows=4, num_heads=8, num_kv_heads=2, head_dim=128, max_blocks=64, num_blocks=200,
             dtype=nsv.BF16, query_len=0)
    d.update(kw)
    return nsv.make_shape(**d)


def _append(nsv, shape, four, tokens=5, rope=True, rope_kw=None, strides=(0, 0, 0), scales=(P, P),
            **given):
    p = dict.fromkeys(TENSORS, P)
    p.update(given)
    r = dict(table=P, positions=P, num_positions=100, rotary_dim=64, interleaved=0)
    r.update(rope_kw or {})
    rp = ctypes.byref(nsv.Rope(**r)) if rope else None
    args = (tokens, p["q"], p["kn"], p["vn"], *strides, p["slots"], p["k"], p["v"], p["q_out"], None)
    if four:
        return nsv._lib.nsv_kv4_write(ctypes.byref(shape), rp, *scales, *args)
    return nsv._lib.nsv_rope_write(ctypes.byref(shape), rp, *args)


@pytest.mark.parametrize("four", [False, True])
def test_append_pointers(nsv, four):
    s = _shape(nsv)
    for name in TENSORS:
        assert _append(nsv, s, four, **{name: None}) == -1     # q and q_out: one without the other
        assert _append(nsv, s, four, **{name: P + (4 if name == "slots" else 8)}) == -4
    for field in ("table", "positions"):
        assert _append(nsv, s, four, rope_kw={field: None}) == -1
        assert _append(nsv, s, four, rope_kw={field: P + 2}) == -4
    if four:
        assert _append(nsv, s, four, rope=False) == -5          # queries without a rotation
    else:
        assert _append(nsv, s, four, rope=False, q=None, q_out=None) == -1
    assert _append(nsv, s, four, tokens=0, k=None, q=None) == 0


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=8), dict(rotary_dim=40),
                                dict(rotary_dim=144), dict(rotary_dim=-16), dict(num_positions=0),
                                dict(interleaved=2)])
def test_append_rotations(nsv, four, kw):
    assert _append(nsv, _shape(nsv), four, rope_kw=kw) == -5


@pytest.mark.parametrize("four", [False, True])
def test_append_rotation_wider_than_the_head(nsv, four):
    assert _append(nsv, _shape(nsv, head_dim=64), four, rope_kw=dict(rotary_dim=80)) == -5


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("strides", [(1023, 0, 0), (8 * 128 - 8, 0, 0), (0, 248, 0), (0, 0, 260),
                                     (1 << 31, 0, 0), (0, -256, 0)])
def test_append_strides(nsv, four, strides):
    assert _append(nsv, _shape(nsv), four, strides=strides) == -3


SIZES = [(dict(head_dim=96), 10, -10), (dict(block_size=32), 10, -10), (dict(dtype=3), 10, -2),
         (dict(dtype=4), 10, -2), (dict(num_heads=7), 10, -3), (dict(rows=8193), 10, -3),
         (dict(), -1, -3), (dict(), 1 << 30, -3), (dict(num_heads=130), 10, -3),
         (dict(num_blocks=0), 10, -3)]


@pytest.mark.parametrize("kw,tokens,code", SIZES)
def test_sizes(nsv, kw, tokens, code):
    s = _shape(nsv, **kw)
    for four in (False, True):
        assert _append(nsv, s, four, tokens=tokens) == code
    assert _read(nsv, s, tokens=tokens) == code
    assert _chunk(nsv, s, tokens=tokens) == code
    with pytest.raises(nsv.NsvError) as e:
        nsv.kv4_workspace_bytes(s, tokens, num_sms=152)
    assert e.value.code == code


def test_append_of_more_heads_than_a_grid_holds(nsv):
    s = _shape(nsv, num_heads=1 << 20, num_kv_heads=1 << 20)
    for four in (False, True):
        assert _append(nsv, s, four, tokens=(1 << 14) // 3 + 1) == -3


def test_scales_are_aligned(nsv):
    s = _shape(nsv)
    # (the append asks for the device first, where there is one)
    assert _read(nsv, s, ks=P + 2) == -4 and _read(nsv, s, vs=P + 1) == -4
    assert _chunk(nsv, s, ks=P + 2) == -4 and _chunk(nsv, s, vs=P + 2) == -4


def _read(nsv, shape, tokens=5, ks=None, vs=None, **given):
    p = dict.fromkeys(["slots", "k", "v", "ko", "vo"], P)
    p.update(given)
    return nsv._lib.nsv_kv4_read(ctypes.byref(shape), ks, vs, tokens, p["slots"], p["k"], p["v"],
                                 p["ko"], p["vo"], None)


def test_read_pointers(nsv):
    s = _shape(nsv)
    for name in ("slots", "k", "v", "ko", "vo"):
        assert _read(nsv, s, **{name: None}) == -1
        assert _read(nsv, s, **{name: P + (4 if name == "slots" else 8)}) == -4
    assert _read(nsv, s, tokens=0, k=None) == 0
    wide = _shape(nsv, num_heads=1 << 10, num_kv_heads=1 << 10)
    assert _read(nsv, wide, tokens=1 << 25) == -3


def _chunk(nsv, shape, tokens=5, scores=None, ks=None, vs=None, ws=P, ws_bytes=1 << 40, **given):
    p = dict.fromkeys(["q", "k", "v", "bt", "starts", "ctx", "out"], P)
    p.update(given)
    sc = ctypes.byref(scores) if scores is not None else None
    return nsv._lib.nsv_kv4_chunk(ctypes.byref(shape), sc, ks, vs, tokens, p["q"], p["k"], p["v"],
                                  p["bt"], p["starts"], p["ctx"], 1.0, p["out"], ws, ws_bytes, None)


def test_chunk_pointers(nsv):
    s = _shape(nsv)
    for name in ("q", "k", "v", "bt", "starts", "ctx", "out"):
        assert _chunk(nsv, s, **{name: None}) == -1
        assert _chunk(nsv, s, **{name: P + (2 if name in ("bt", "starts", "ctx") else 8)}) == -4
    assert _chunk(nsv, s, tokens=0, q=None) == 0
    assert _chunk(nsv, _shape(nsv, rows=0), q=None) == 0


def test_chunk_scores(nsv):
    s = _shape(nsv)
    for cap in (-1.0, math.nan, math.inf, 1e-7, 2e6):
        assert _chunk(nsv, s, scores=nsv.Scores(cap, None, None, None)) == -5
    for field in ("slopes", "see_begin", "see_end"):
        sc = nsv.Scores(0.0, None, None, None)
        setattr(sc, field, P + 2)
        assert _chunk(nsv, s, scores=sc) == -4


@pytest.mark.parametrize("kw", [dict(query_len=65), dict(query_len=-1), dict(query_len=17)])
def test_chunk_query_len(nsv, kw):      # 4 heads per KV head: at most 16 tokens are named
    assert _chunk(nsv, _shape(nsv, **kw)) == -3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (8, 2), (5, 1), (64, 1), (21, 7), (40, 20)])
def test_workspace_grows_with_the_batch(nsv, dtype, heads, kv_heads):
    code = nsv.F32 if dtype == "f32" else nsv.BF16
    size = lambda rows, tokens, ql=0: nsv.kv4_workspace_bytes(  # noqa: E731
        _shape(nsv, rows=rows, num_heads=heads, num_kv_heads=kv_heads, dtype=code, query_len=ql),
        tokens, 152)
    sizes = [[size(r, t) for t in (1, 7, 64, 513, 4096, 100000)] for r in (1, 3, 100, 8192)]
    for row in sizes:
        assert row == sorted(row)
    for a, b in zip(sizes, sizes[1:]):
        assert all(x <= y for x, y in zip(a, b))
    assert all(size(100, 513, ql) == size(100, 513) for ql in range(1, 64 * kv_heads // heads + 1))


def test_binding_checks_layouts(nsv):
    import torch
    cpu = torch.zeros(1).get_device()       # what a CPU tensor answers: no CUDA device's number
    fused = torch.zeros(5, 12, 64)
    q = fused[:, 4:8]
    assert nsv._heads_arg(q, "q", torch.float32, (5, 4, 64), cpu) == (q.data_ptr(), 12 * 64)
    assert nsv._heads_arg(q[:1], "q", torch.float32, (1, 4, 64), cpu)[1] == 0
    for bad in (q.transpose(0, 1), fused[:, ::2][:, :4], fused.expand(5, 12, 64)[:, :4, ::1].double(),
                torch.zeros(1, 4, 64).expand(5, 4, 64), torch.zeros(5, 4, 128)[..., ::2]):
        with pytest.raises(ValueError):
            nsv._heads_arg(bad, "q", torch.float32, (5, 4, 64), cpu)
    with pytest.raises(ValueError):
        nsv._heads_arg(q, "q", torch.float32, (5, 4, 64), 0)
    assert nsv._kv4_sizes(torch.zeros((4, 2, 9 * 64), dtype=torch.uint8)) == (3, 2, 64)
    for bad in (torch.zeros((4, 2, 9 * 64)), torch.zeros((4, 2, 100), dtype=torch.uint8),
                torch.zeros((4, 2, 16, 72), dtype=torch.uint8)):
        with pytest.raises(ValueError):
            nsv._kv4_sizes(bad)


def test_page_operators_take_four_bit_pools_and_attention_does_not(nsv):
    s = _shape(nsv, dtype=nsv.KV4, num_heads=1 << 21, num_kv_heads=1 << 21)
    lib = nsv._lib
    # (a block beyond 256 MiB is refused, so the type was taken)
    assert lib.nsv_blocks_copy(ctypes.byref(s), 1, P, P, P, P, None) == -3
    assert lib.nsv_pages_workspace(ctypes.byref(s), ctypes.byref(ctypes.c_int64())) == 0
    assert lib.nsv_pages_workspace(ctypes.byref(_shape(nsv, dtype=nsv.KV4, head_dim=80)),
                                   ctypes.byref(ctypes.c_int64())) == -10
    with pytest.raises(nsv.NsvError) as e:
        nsv.chunk_workspace_bytes(_shape(nsv, dtype=nsv.KV4), 10, num_sms=152)
    assert e.value.code == -2


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("kv_heads,group,head_dim", [
    (1, 1, 64), (8, 4, 128), (5, 3, 64), (7, 1, 128), (1, 64, 128), (12, 5, 64), (3, 17, 128)])
def test_a_larger_batch_has_no_smaller_workspace(nsv, dtype, kv_heads, group, head_dim):
    """A workspace made for the largest batch serves all others."""
    def size(rows, tokens):
        shape = nsv.make_shape(rows, kv_heads * group, kv_heads, head_dim, 10, 100, dtype)
        return nsv.kv4_workspace_bytes(shape, tokens, 152)

    rows = [1, 2, 3, 31, 257, 3000]
    tokens = [0, 1, 2, 7, 8, 9, 33, 256, 300, 2049, 70000]
    for i, r in enumerate(rows):
        for j, t in enumerate(tokens):
            assert size(r, t) >= max(size(r, tokens[max(0, j - 1)]), size(rows[max(0, i - 1)], t))
