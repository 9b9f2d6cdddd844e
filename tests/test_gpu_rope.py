"""The appends that rotate on the way, and the way into and out of 4-bit pools (GPU),
against the definitions in 64 bits (kv4_common).

Tolerances: a rotated element is two fp32 products and their sum, each off by at
most half a step: 2^-24 (|a c| + |b s|) twice, at most 2^-22 of |a| + |b|.  bf16
results are off by another half step, 2^-8 of themselves.  What a 4-bit pool
holds is defined with its roundings, and has to be equal."""

import numpy as np
import pytest

import kv4_common as F

pytestmark = pytest.mark.gpu

HALF = {"f32": 0.0, "bf16": 2.0 ** -8}
SHAPES = [(4, 4, 64), (8, 2, 128), (5, 1, 128), (6, 3, 64), (40, 8, 128), (64, 1, 64), (9, 9, 128)]


def dtype_of(name):
    import torch
    return torch.float32 if name == "f32" else torch.bfloat16


def inputs(tokens, heads, kv_heads, head_dim, dtype, rotary_dim, four, seed=0, positions=300,
           fused=False):
    import torch
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = dtype_of(dtype)
    parts = torch.randn((tokens, heads + 2 * kv_heads, head_dim), generator=g).to(dt).cuda()
    q, k, v = parts.split([heads, kv_heads, kv_heads], 1)
    if not fused:
        q, k, v = (x.contiguous() for x in (q, k, v))
    blocks = -(-tokens // 16) + 3
    slots = rng.permutation(blocks * 16)[:tokens].astype(np.int64)
    if four:
        pools = [torch.from_numpy(rng.integers(0, 256, (blocks + 1, kv_heads, 9 * head_dim),
                                               dtype=np.uint8)).cuda() for _ in range(2)]
    else:
        pools = [torch.randn((blocks + 1, kv_heads, 16, head_dim), generator=g).to(dt).cuda()
                 for _ in range(2)]
    return {"q": q, "k": k, "v": v, "pools": pools, "slots": torch.from_numpy(slots).cuda(),
            "positions": torch.from_numpy(rng.integers(0, positions, tokens).astype(np.int32)).cuda(),
            "table": torch.from_numpy(F.table(positions, rotary_dim)).cuda()}


def host(t):
    return t.detach().double().cpu().numpy()


def turned(x, b, interleaved, rounded=False):
    return F.rotate(host(x), host(b["positions"]).astype(int), b["table"].cpu().numpy(), interleaved,
                    rounded)


def assert_turned(got, x, b, interleaved, dtype):
    ref = turned(x, b, interleaved)
    size = np.abs(host(x))
    half = b["table"].shape[1] // 2
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    both = size[..., ia] + size[..., ib]
    tol = np.zeros_like(size)
    tol[..., ia] = tol[..., ib] = 2.0 ** -22 * both
    tol += HALF[dtype] * (np.abs(ref) + tol)
    assert (np.abs(host(got) - ref) <= tol).all()
    rest = np.arange(2 * half, x.shape[-1])
    assert np.array_equal(host(got)[..., rest], host(x)[..., rest])


def by_slot(pool, slots):
    """A pool's rows [len(slots), kv_heads, head_dim]."""
    return pool.transpose(1, 2).reshape(-1, pool.shape[1], pool.shape[3])[slots]


def rope_and_check(b, dtype, interleaved=False, q_out=None, status=0):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    before = [p.clone() for p in b["pools"]]
    q = b["q"].clone()
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda") if q_out is None else q_out
    nsv.device_status(clear=True)
    nsv.rope_write(b["q"], b["k"], b["v"], b["positions"], b["table"], b["slots"], *b["pools"],
                   out, interleaved=interleaved)
    assert nsv.device_status(clear=True)[0] == status
    assert_turned(out, q, b, interleaved, dtype)
    assert_turned(by_slot(b["pools"][0], b["slots"]), b["k"], b, interleaved, dtype)
    assert torch.equal(by_slot(b["pools"][1], b["slots"]), b["v"])
    for pool, old in zip(b["pools"], before):      # every other slot is as it was
        rest = torch.ones(pool.shape[0] * 16, dtype=torch.bool, device="cuda")
        rest[b["slots"]] = False
        assert torch.equal(by_slot(pool, rest), by_slot(old, rest))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,head_dim", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_write(dtype, heads, kv_heads, head_dim, interleaved):
    for i, (tokens, rotary) in enumerate([(1, head_dim), (37, 16), (130, 48), (15, head_dim // 2)]):
        b = inputs(tokens, heads, kv_heads, head_dim, dtype, rotary, False, seed=i, fused=i % 2 == 1)
        rope_and_check(b, dtype, interleaved)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_write_in_place_and_without_queries(dtype):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = inputs(50, 8, 2, 128, dtype, 128, False)
    nsv.rope_write(None, b["k"], b["v"], b["positions"], b["table"], b["slots"], *b["pools"])
    alone = [p.clone() for p in b["pools"]]
    q = b["q"].clone()
    nsv.rope_write(b["q"], b["k"], b["v"], b["positions"], b["table"], b["slots"], *b["pools"], b["q"])
    assert_turned(b["q"], q, b, False, dtype)
    assert all(torch.equal(x, y) for x, y in zip(alone, b["pools"]))


def test_layouts_that_would_overlap_or_misalign_are_refused():
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = inputs(6, 8, 2, 128, "bf16", 128, False)
    args = lambda **kw: [kw.get(n, b[n]) for n in ("q", "k", "v", "positions", "table", "slots")]  # noqa: E731
    out = torch.empty_like(b["q"])
    one = b["k"][:1].expand(6, 2, 128)
    wide = torch.zeros((6, 2 * 128 + 4), dtype=torch.bfloat16, device="cuda")
    for bad, error in ((dict(k=one), ValueError), (dict(v=wide[:, 4:].unflatten(1, (2, 128))), nsv.NsvError),
                       (dict(v=wide[:, :256].unflatten(1, (2, 128))), nsv.NsvError),
                       (dict(positions=b["positions"].long()), ValueError),
                       (dict(table=b["table"][:, :24].contiguous()), nsv.NsvError),
                       (dict(q=b["q"].float()), ValueError)):
        with pytest.raises(error):
            nsv.rope_write(*args(**bad), *b["pools"], out)
    with pytest.raises(nsv.NsvError):
        nsv.rope_write(*args(), *b["pools"], None)


def test_rope_write_of_no_tokens():
    from paged_kv_decode_nsv_gb300 import nsv
    b = inputs(0, 8, 2, 128, "bf16", 128, False)
    nsv.rope_write(b["q"], b["k"], b["v"], b["positions"], b["table"], b["slots"], *b["pools"],
                   b["q"].clone())


@pytest.mark.parametrize("four", [False, True])
def test_bad_positions_and_slots_are_skipped_and_flagged(four):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = inputs(40, 8, 2, 128, "bf16", 64, four, positions=100)
    sink = (b["pools"][0].shape[0] - 1) * 16
    b["positions"][3], b["positions"][7] = -1, 100
    b["slots"][11], b["slots"][12], b["slots"][20], b["slots"][21] = -1, sink + 16, sink, sink
    before = [p.clone() for p in b["pools"]]
    out = torch.full(b["q"].shape, 7.5, dtype=b["q"].dtype, device="cuda")
    nsv.device_status(clear=True)
    if four:
        nsv.kv4_write(b["k"], b["v"], b["slots"], *b["pools"], q=b["q"], positions=b["positions"],
                      rotary=b["table"], q_out=out)
    else:
        nsv.rope_write(b["q"], b["k"], b["v"], b["positions"], b["table"], b["slots"], *b["pools"], out)
    assert nsv.device_status(clear=True)[0] == nsv.DEV_BAD_POS | nsv.DEV_BAD_SLOT
    gone = torch.tensor([3, 7], device="cuda")
    assert (out[gone] == 7.5).all()
    good = torch.tensor([i for i in range(40) if i not in (3, 7)], device="cuda")
    sub = {**b, "positions": b["positions"][good]}
    assert_turned(out[good], b["q"][good], sub, False, "bf16")
    written = torch.zeros((sink + 16,), dtype=torch.bool, device="cuda")
    real = torch.tensor([i for i in range(40) if i not in (3, 7, 11, 12)], device="cuda")
    written[b["slots"][real]] = True
    written[sink:] = True                    # unspecified
    for pool, old in zip(b["pools"], before):
        if four:
            data, scale = F.split_pool(pool.cpu().numpy(), 128)
            data0, scale0 = F.split_pool(old.cpu().numpy(), 128)
            keep = ~written.cpu().numpy().reshape(-1, 16)
            for x, y in ((data, data0), (scale, scale0)):
                assert np.array_equal(np.moveaxis(x, 1, 2)[keep], np.moveaxis(y, 1, 2)[keep])
        else:
            assert torch.equal(by_slot(pool, ~written), by_slot(old, ~written))


def write4_and_check(b, dtype, interleaved=False, scales=(None, None), rotate=True):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    kv_heads, dim = b["k"].shape[1:]
    before = [p.cpu().numpy() for p in b["pools"]]
    kw = {}
    if rotate:
        out = torch.empty(b["q"].shape, dtype=b["q"].dtype, device="cuda")
        kw = dict(q=b["q"], positions=b["positions"], rotary=b["table"], q_out=out,
                  interleaved=interleaved)
    nsv.device_status(clear=True)
    nsv.kv4_write(b["k"], b["v"], b["slots"], *b["pools"], k_scales=scales[0], v_scales=scales[1], **kw)
    k = torch.empty(b["k"].shape, dtype=b["k"].dtype, device="cuda")
    v = torch.empty_like(k)
    nsv.kv4_read(b["slots"], *b["pools"], k, v, k_scales=scales[0], v_scales=scales[1])
    assert nsv.device_status(clear=True)[0] == 0
    if rotate:
        assert_turned(out, b["q"], b, interleaved, dtype)
    slots = b["slots"].cpu().numpy()
    for pool, old, x, unit, back in (
            (b["pools"][0], before[0], turned(b["k"], b, interleaved, True) if rotate else host(b["k"]),
             scales[0], k),
            (b["pools"][1], before[1], host(b["v"]), scales[1], v)):
        u = np.ones(kv_heads) if unit is None else unit.cpu().numpy()
        code, sb = F.quantise(x, u)
        want = old.copy()
        data, sc = (np.moveaxis(y, 1, 2) for y in F.split_pool(want, dim))
        data = data.reshape(-1, kv_heads, dim // 2).copy()
        sc = sc.reshape(-1, kv_heads, dim // 16).copy()
        data[slots], sc[slots] = code[..., 0::2] | (code[..., 1::2] << 4), sb
        got_data, got_sc = (np.moveaxis(y, 1, 2) for y in F.split_pool(pool.cpu().numpy(), dim))
        assert np.array_equal(got_sc.reshape(sc.shape), sc)
        # (a zero keeps its sign in the pool: compared as numbers)
        got = got_data.reshape(data.shape)
        for shift in (0, 4):
            a, c = (got >> shift) & 15, (data >> shift) & 15
            assert ((a == c) | ((a & 7 == 0) & (c & 7 == 0))).all()
        ref = F.f32(F.dequantise(code, sb, np.ones(kv_heads)) * u.astype(np.float64)[:, None])
        ref = torch.from_numpy(ref.astype(np.float32)).to(back.dtype)
        assert torch.equal(back.cpu() + 0.0, ref + 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,head_dim", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_kv4_write_and_read(dtype, heads, kv_heads, head_dim, interleaved):
    import torch
    for i, (tokens, rotary) in enumerate([(1, head_dim), (37, 16), (130, 48), (15, head_dim // 2)]):
        b = inputs(tokens, heads, kv_heads, head_dim, dtype, rotary, True, seed=i, fused=i % 2 == 1)
        scales = [(torch.rand(kv_heads) * 4 + 0.05).cuda() for _ in range(2)] if i % 2 else (None, None)
        write4_and_check(b, dtype, interleaved, scales)
        write4_and_check(b, dtype, scales=scales, rotate=False)


def test_kv4_write_at_every_edge_of_the_format():
    """Zeros, scales that underflow or have few digits, saturation, halfway cases of
    both types."""
    import torch
    rows = []
    for top in (0.0, 1e-30, 2.0 ** -11 * 6, 2.0 ** -10 * 6, 2.0 ** -10 * 6.001, 2.0 ** -9 * 6, 0.01, 0.0933,
                6.0, 6.0 * 17 / 16, 6.0 * 19 / 16, 2688.0, 2688.0 * 1.04, 1e6, 3e38):
        grid = np.array([1.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2499, 0.2501, 3.0, 4.9, 5.1, 0.0,
                         0.1, 0.5]) / 6.0
        grid[0] = 1.0
        rows.append(grid * top * np.where(np.arange(16) % 3 == 1, -1, 1))
    x = torch.tensor(np.concatenate([np.array(rows)] * 4, 1), dtype=torch.float32)[:, None].cuda()
    b = inputs(len(rows), 1, 1, 64, "f32", 64, True)
    b["k"], b["v"] = x.contiguous(), x.flip(0).contiguous()
    write4_and_check(b, "f32", rotate=False)
    # head scales at both ends of their range, and ones that have no short reciprocal
    for units in ((2.0 ** -60, 2.0 ** 60), (3.0, 1.0 / 3.0), (1.1e-5, 9.7e4), (0.7, 7.0)):
        write4_and_check(b, "f32", rotate=False,
                         scales=[torch.tensor([u], dtype=torch.float32).cuda() for u in units])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_kv4_write_of_many_random_values(dtype):
    """Every rounding of two million values, of sizes over eight powers of two, is the
    definition's, quotients next to a border among them."""
    import torch
    b = inputs(4096, 4, 2, 128, dtype, 128, True)
    g = torch.Generator().manual_seed(9)
    for name in ("k", "v"):
        size = torch.exp2(torch.rand((4096, 2, 8), generator=g) * 8 - 6).repeat_interleave(16, -1)
        b[name] = (b[name].float().cpu() * size).to(b[name].dtype).cuda()
    units = [torch.tensor(u, dtype=torch.float32).cuda() for u in ((0.731, 1.0), (3.3, 0.0517))]
    write4_and_check(b, dtype, scales=units)
    write4_and_check(b, dtype, rotate=False)


def test_kv4_read_leaves_bad_slots_and_takes_repeated_ones():
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = inputs(40, 8, 2, 64, "f32", 64, True)
    nsv.kv4_write(b["k"], b["v"], b["slots"], *b["pools"])
    top = b["pools"][0].shape[0] * 16
    slots = torch.cat([b["slots"][:5], b["slots"][:5], torch.tensor([-1, top, top - 1]).cuda()])
    k = torch.full((13, 2, 64), 7.5, device="cuda")
    v = k.clone()
    nsv.device_status(clear=True)
    nsv.kv4_read(slots, *b["pools"], k, v)
    assert nsv.device_status(clear=True)[0] == nsv.DEV_BAD_SLOT
    assert (k[10:12] == 7.5).all() and (v[10:12] == 7.5).all()
    assert torch.equal(k[:5], k[5:10]) and torch.equal(v[:5], v[5:10])


@pytest.mark.parametrize("four", [False, True])
def test_many_tokens_and_a_pool_past_four_gigabytes(four):
    """The same results at slots whose bytes lie past 2^32 as at low ones."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    heads, dim, n = 8, 128, 5000
    tile = 9 * dim if four else 16 * dim * 2
    blocks = (1 << 32) // (heads * tile) + 400
    b = inputs(n, 32, heads, dim, "bf16", 128, four)
    shape = (blocks + 1, heads, 9 * dim) if four else (blocks + 1, heads, 16, dim)
    pools = [torch.zeros(shape, dtype=torch.uint8 if four else torch.bfloat16, device="cuda")
             for _ in range(2)]
    low = torch.arange(n, device="cuda")
    high = low + (blocks - 350) * 16
    outs = []
    for slots in (low, high):
        q = torch.empty_like(b["q"])
        if four:
            nsv.kv4_write(b["k"], b["v"], slots, *pools, q=b["q"], positions=b["positions"],
                          rotary=b["table"], q_out=q)
        else:
            nsv.rope_write(b["q"], b["k"], b["v"], b["positions"], b["table"], slots, *pools, q)
        outs.append(q)
    assert torch.equal(outs[0], outs[1])
    nb = -(-n // 16)
    for p in pools:
        assert torch.equal(p[:nb], p[blocks - 350:blocks - 350 + nb])
        assert p[:nb].any()


@pytest.mark.parametrize("four", [False, True])
def test_captured_and_replayed_with_new_inputs_on_another_stream(four):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = inputs(33, 8, 2, 128, "bf16", 128, four, fused=True)
    out = torch.empty((33, 8, 128), dtype=torch.bfloat16, device="cuda")

    def call():
        if four:
            nsv.kv4_write(b["k"], b["v"], b["slots"], *b["pools"], q=b["q"], positions=b["positions"],
                          rotary=b["table"], q_out=out)
        else:
            nsv.rope_write(b["q"], b["k"], b["v"], b["positions"], b["table"], b["slots"], *b["pools"], out)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    b["positions"].copy_(b["positions"].flip(0))
    b["q"].copy_(b["q"].flip(0).clone())
    graph.replay()
    replayed = [out.clone(), *(p.clone() for p in b["pools"])]
    out.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(replayed, [out, *b["pools"]]))
