"""Attention over a 4-bit paged cache (GPU), against the definition in 64 bits row
by row, and the serving loop around it.

Tolerances, per (token, head), against `big`, the largest over the dims of
|out| + sum p |v| (p: the softmax's weights):

  fp32  Queries and weights are the sum of two fp16 or tf32 numbers, off by at most 2^-21
        of themselves; products of 128 terms, the exponential, the running rescales
        and the sum each cost a few 2^-24 relative to the scores' size.  Scores here
        are below 16 in log2 units, so a weight is off by at most about
        16 * 128 * 2^-24 = 1.2e-4 in the worst case and by sqrt(128) in place of
        128, 1.1e-5, as the terms' signs fall: 4e-5 of sum p |v|.
  bf16  The weights are rounded by half a step of fp16 at most, 2^-11 of each (those
        below 2^-29 of the largest by 2^-40 of it), and their sum is taken before.  The
        output is rounded by at most 2^-8 of itself.  What is left of 2^-8 + 2^-12
        of |out| + sum p |v| is for the scores' fp32 arithmetic and the exponential unit.
"""

import numpy as np
import pytest

import kv4_common as F

pytestmark = pytest.mark.gpu

F32_TOL = 4e-5
BF16_TOL = 2.0 ** -8 + 2.0 ** -12


def random_pool(rng, blocks, kv_heads, head_dim):
    """Normally distributed values' bytes (a number of distinct tiles, repeated)."""
    tiles = min((blocks + 1) * kv_heads, 256)
    x = rng.standard_normal((tiles * 16, 1, head_dim)).astype(np.float32)
    code, sb = F.quantise(x, np.ones(1))
    data = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(tiles, -1)
    each = np.concatenate([data, sb.reshape(tiles, -1)], 1)
    pick = rng.integers(0, tiles, (blocks + 1) * kv_heads)
    return each[pick].reshape(blocks + 1, kv_heads, 9 * head_dim)


def spoil(pool, blocks, offs, head_dim):
    """Scales of the given slots become NaN, their numbers the largest."""
    data, sb = (pool[..., :8 * head_dim].reshape(*pool.shape[:2], 16, -1),
                pool[..., 8 * head_dim:].reshape(*pool.shape[:2], 16, -1))
    data[blocks, :, offs] = 0xff
    sb[blocks, :, offs] = 0x7f
    pool[..., :8 * head_dim] = data.reshape(*pool.shape[:2], -1)
    pool[..., 8 * head_dim:] = sb.reshape(*pool.shape[:2], -1)


def batch(ctx, new, heads, kv_heads, head_dim, dtype, seed=0, pad=0, scaled=False):
    """Inputs on the GPU: scattered blocks, NaN in every pool position that holds no
    token (the sink and free blocks too), `pad` tokens of no row."""
    import torch
    rng = np.random.default_rng(seed)
    nb = [-(-c // 16) for c in ctx]
    blocks = sum(nb) + 3
    perm = rng.permutation(blocks).astype(np.int32)
    width = max(nb + [1]) + 1
    tables = np.full((len(ctx), width), -1, np.int32)
    written = np.zeros((blocks + 1, 16), bool)
    at = 0
    for r, n in enumerate(nb):
        tables[r, :n] = perm[at:at + n]
        at += n
        t = np.arange(ctx[r])
        written[tables[r, t // 16], t % 16] = True
    pools = [random_pool(rng, blocks, kv_heads, head_dim) for _ in range(2)]
    dead = np.nonzero(~written)
    for p in pools:
        spoil(p, *dead, head_dim)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    tdt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(seed)
    units = [(torch.rand(kv_heads, generator=g) + 0.5).cuda() if scaled else None for _ in range(2)]
    return {"q": torch.randn((int(starts[-1]) + pad, heads, head_dim), generator=g).to(tdt).cuda(),
            "k": torch.from_numpy(pools[0]).cuda(), "v": torch.from_numpy(pools[1]).cuda(),
            "units": units, "bt": torch.from_numpy(tables).cuda(),
            "starts": torch.from_numpy(starts).cuda(),
            "ctx": torch.tensor(ctx, dtype=torch.int32).cuda(), "scale": head_dim ** -0.5,
            "lens": (list(ctx), list(new)), "group": heads // kv_heads}


def values(pool, unit):
    """A pool's 64-bit values on the GPU."""
    import torch
    n, h, d = pool.shape[0], pool.shape[1], pool.shape[2] // 9
    raw = pool.long()
    data, sb = raw[..., :8 * d].reshape(n, h, 16, d // 2), raw[..., 8 * d:].reshape(n, h, 16, d // 16)
    number = torch.tensor(np.concatenate([F.E2M1, -F.E2M1])).cuda()
    width = torch.tensor(np.concatenate([F.E4M3, np.full(129, np.nan)])).cuda()
    v = torch.stack([number[data & 15], number[data >> 4]], -1).flatten(-2)
    v = v * width[sb].repeat_interleave(16, -1)
    return v if unit is None else v * unit.double()[:, None, None]


def reference(b, softcap=0.0, slopes=None, see_begin=None, see_end=None):
    """The definition in 64 bits, and what its tolerance goes by (see above)."""
    import torch
    q = b["q"].double()
    out = torch.zeros_like(q)
    big = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    kp, vp = values(b["k"], b["units"][0]), values(b["v"], b["units"][1])
    D, at = q.shape[2], 0
    for r, (c, n) in enumerate(zip(*b["lens"])):
        if not n:
            continue
        ids = b["bt"][r, :-(-c // 16)].long()
        k = kp[ids].transpose(1, 2).reshape(-1, kp.shape[1], D)[:c].repeat_interleave(b["group"], 1)
        v = vp[ids].transpose(1, 2).reshape(-1, kp.shape[1], D)[:c].repeat_interleave(b["group"], 1)
        t = torch.arange(c, device="cuda")
        pos = torch.arange(c - n, c, device="cuda")
        lo = torch.zeros(n, device="cuda") if see_begin is None else see_begin[at:at + n].clamp(min=0)
        hi = (pos + 1 if see_end is None else see_end[at:at + n]).clamp(max=c)
        seen = (t >= lo[:, None]) & (t < hi[:, None])
        s = torch.einsum("ihd,thd->iht", q[at:at + n], k) * b["scale"]
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        if slopes is not None:
            s = s - slopes.double()[None, :, None] * (pos[:, None] - t).abs()[:, None]
        s = torch.where(seen[:, None], s, -np.inf)      # NaN keys that are not seen too
        s = s - s.amax(-1, keepdim=True).clamp(min=-1e300)
        p = torch.exp(s)
        p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
        out[at:at + n] = torch.einsum("iht,thd->ihd", p, v)
        big[at:at + n] = (out[at:at + n].abs() + torch.einsum("iht,thd->ihd", p, v.abs())).amax(-1)
        at += n
    return out, big


def call(b, out, **kw):
    from paged_kv_decode_nsv_gb300 import nsv
    return nsv.kv4_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], out,
                         k_scales=b["units"][0], v_scales=b["units"][1], **kw)


def check(b, dtype, garbage_out=7.5, status=0, max_new=0, tol=None, **scores):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    nsv.device_status(clear=True)
    out = torch.full_like(b["q"], garbage_out)
    call(b, out, max_new=max_new, **scores)
    st, _ = nsv.device_status(clear=True)
    assert st == status, "device status %#x" % st
    ref, big = reference(b, **scores)
    T = int(sum(b["lens"][1]))
    assert torch.isfinite(out.float()).all()
    err = (out[:T].double() - ref[:T]).abs().amax(-1)
    tol = tol or (F32_TOL if dtype == "f32" else BF16_TOL)
    worst = (err - tol * big[:T]).max().item() if T else 0.0
    assert worst <= 0.0, "off by %.3g above the tolerance (largest error %.3g)" % (worst, err.max())
    assert (out[T:] == garbage_out).all(), "tokens of no row were written"
    return out


SHAPES = [(4, 4, 64), (8, 2, 64), (4, 4, 128), (8, 2, 128), (6, 2, 128), (5, 1, 64), (16, 1, 128),
          (64, 1, 128), (12, 12, 128), (24, 8, 64), (17, 1, 64), (21, 7, 128)]
MIXES = [
    ([1], [1]),
    ([16, 40, 100, 257, 0], [1, 1, 1, 1, 0]),
    ([15, 17, 32, 33, 31, 48, 700], [1, 1, 1, 1, 1, 1, 1]),
    ([5, 64, 129, 300], [5, 7, 100, 33]),
    ([700, 33, 2, 1, 0, 90], [300, 1, 0, 1, 0, 20]),
    ([2049], [513]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,head_dim", SHAPES)
@pytest.mark.parametrize("mix", range(len(MIXES)))
def test_shapes_and_mixes(dtype, heads, kv_heads, head_dim, mix):
    ctx, new = MIXES[mix]
    b = batch(ctx, new, heads, kv_heads, head_dim, dtype, seed=mix, pad=3, scaled=mix % 2 == 1)
    check(b, dtype)
    if max(new) * (heads // kv_heads) <= 64:
        check(b, dtype, max_new=max(new))


def bounds(kind, ctx, new, rng):
    """Masks by their bounds (int32 tensors), among them tokens that see nothing."""
    import torch
    begin, end = [], []
    for c, n in zip(ctx, new):
        for i in range(n):
            pos = c - n + i
            if kind == "window":
                begin.append(pos + 1 - int(rng.integers(1, 70)))
            elif kind == "documents":
                begin.append(pos // 37 * 37)
            elif kind == "prefix":
                end.append(max(pos + 1, c // 2))
            elif kind == "all":
                end.append(2 ** 31 - 1)
            elif kind == "nothing":
                begin.append(int(rng.choice([0, pos + 1, 2 ** 31 - 1, -2 ** 31])))
                end.append(int(rng.choice([pos + 1, -2 ** 31, 0, 2 ** 31 - 1])))
    as_t = lambda x: torch.tensor(x, dtype=torch.int32).cuda() if x else None  # noqa: E731
    return {"see_begin": as_t(begin), "see_end": as_t(end)}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["window", "documents", "prefix", "all", "nothing"])
@pytest.mark.parametrize("form", ["plain", "cap", "slopes", "both"])
def test_masks_caps_and_biases(dtype, kind, form):
    import torch
    for i, (heads, kv_heads, dim, ctx, new) in enumerate([
            (8, 2, 128, [300, 5, 0, 77, 600], [1, 1, 0, 1, 1]),
            (6, 2, 64, [300, 64, 129, 1000], [3, 2, 5, 1]),
            (12, 4, 64, [300, 64, 129, 2000], [150, 64, 20, 1]),
            (16, 1, 128, [40, 700], [17, 200])]):
        b = batch(ctx, new, heads, kv_heads, dim, dtype, seed=i, scaled=i == 1)
        scores = bounds(kind, ctx, new, np.random.default_rng(i))
        if form in ("cap", "both"):
            scores["softcap"] = [20.0, 5.0, 50.0, 300.0][i]
        if form in ("slopes", "both"):
            scores["slopes"] = torch.exp2(-torch.arange(1.0, heads + 1) * 8 / heads).cuda()
        check(b, dtype, **scores)
        if max(new) <= 5:
            check(b, dtype, max_new=max(new), **scores)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
def test_unseen_keys_may_be_anything(dtype, new):
    """NaN keys at positions that no token sees; table entries before the first position
    seen are not looked at."""
    import torch
    ctx = [500, 200]
    b = batch(ctx, [new, new], 8, 2, 128, dtype)
    begin = torch.cat([torch.full((new,), 321), torch.full((new,), 100)]).int().cuda()
    kp = b["k"].cpu().numpy().copy()
    for r, lo in ((0, 321), (1, 100)):
        t = np.arange(lo)
        spoil(kp, b["bt"].cpu().numpy()[r, t // 16], t % 16, 128)
    b["k"] = torch.from_numpy(kp).cuda()
    saved = b["bt"].clone()
    ref_b = {**b, "bt": saved}
    bad = saved.clone()
    bad[0, :321 // 16], bad[1, :100 // 16] = 2 ** 30, -5
    b["bt"] = bad
    from paged_kv_decode_nsv_gb300 import nsv
    nsv.device_status(clear=True)
    out = call(b, torch.empty_like(b["q"]), see_begin=begin)
    assert nsv.device_status(clear=True)[0] == 0
    ref, big = reference(ref_b, see_begin=begin)
    tol = F32_TOL if dtype == "f32" else BF16_TOL
    assert ((out.double() - ref).abs().amax(-1) <= tol * big).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("most", [0, 1])     # with a list of tiles, and without
def test_bad_lengths_starts_blocks_and_counts(dtype, most):
    import functools

    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    call = functools.partial(globals()["call"], max_new=most)
    ctx, new = [300, 90, 33, 64], [1, 1, 1, 1]
    b = batch(ctx, new, 8, 2, 128, dtype)
    good = check(b, dtype, max_new=most)
    b["ctx"][1] = -3
    out = call(b, torch.full_like(b["q"], 7.5))
    assert nsv.device_status()[0] == nsv.DEV_BAD_CTX
    assert (out[1] == 0).all() and torch.equal(out[[0, 2, 3]], good[[0, 2, 3]])
    b["ctx"][1] = b["bt"].shape[1] * 16 + 1
    call(b, out)
    assert nsv.device_status()[0] == nsv.DEV_BAD_CTX
    b["ctx"][1] = 90
    b["bt"][2, 1], b["bt"][3, 0] = b["k"].shape[0], -1
    call(b, out)
    assert nsv.device_status()[0] == nsv.DEV_BAD_BLOCK
    assert torch.isfinite(out.float()).all() and torch.equal(out[:2], good[:2])
    b = batch(ctx, new, 8, 2, 128, dtype)
    b["starts"] = torch.tensor([0, 1, 0, 3, 4], dtype=torch.int32).cuda()
    out = call(b, torch.full_like(b["q"], 7.5))
    assert nsv.device_status()[0] == nsv.DEV_BAD_CHUNK
    assert torch.equal(out[3], good[3])
    # more new tokens than the caller said
    b = batch(ctx, [1, 3, 1, 1], 8, 2, 128, dtype)
    full = check(b, dtype)
    out = globals()["call"](b, torch.full_like(b["q"], 7.5), max_new=1)
    assert nsv.device_status()[0] == nsv.DEV_BAD_CHUNK
    assert (out[1:4] == 7.5).all()
    assert torch.allclose(out[[0, 4, 5]].float(), full[[0, 4, 5]].float(), atol=0.03)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,rows,ctx,new", [
    (8, 2, 1, 70001, 1), (4, 1, 3, 40000, 1), (8, 8, 2, 9000, 3), (8, 2, 1, 20000, 300)])
def test_rows_cut_into_many_pieces(dtype, heads, kv_heads, rows, ctx, new):
    b = batch([ctx - 7 * i for i in range(rows)], [new] * rows, heads, kv_heads, 128, dtype)
    check(b, dtype, max_new=new if new == 1 else 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
def test_long_sums_of_equal_weights(dtype, new):
    """Equal scores over 65536 positions: the mean of the values.  Weights of 2^k add up
    exactly, so that fp32 is off by the sums' rounding alone: within 2^-19."""
    import torch
    n = 65536
    b = batch([n], [new], 4, 2, 128, dtype)
    b["q"].zero_()
    check(b, dtype, max_new=1 if new == 1 else 0, tol=2.0 ** -19 if dtype == "f32" else None)
    b["v"][..., :8 * 128] = 0x55            # 3
    b["v"][..., 8 * 128:] = 0x38            # 1
    out = call(b, torch.empty_like(b["q"]), max_new=1 if new == 1 else 0)
    assert (out.double() - 3.0).abs().max() <= (3 * 2.0 ** -19 if dtype == "f32" else 3 * 2.0 ** -8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 300.0, 1e4])
def test_queries_of_any_size(dtype, size):
    """Large scores (one position takes all the weight) and vanishing ones, and vectors
    whose elements differ by many powers of two."""
    import torch
    ctx = [400, 33, 1000]
    b = batch(ctx, [1, 1, 1], 8, 2, 128, dtype)
    b["q"] = (b["q"].float() * size).to(b["q"].dtype)
    b["q"][1] *= torch.exp2(-torch.arange(128.0) / 4).cuda().to(b["q"].dtype)
    # a score of size * 128 terms is off by 2^-22 of itself or so: bounded by what that
    # does to a weight
    scores = float(size) * 12 * 1.45
    check(b, dtype, max_new=1, tol=(F32_TOL if dtype == "f32" else BF16_TOL) + scores * 128 ** 0.5 * 2.0 ** -22)


@pytest.mark.parametrize("rows,most,heads,kv_heads", [
    (8192, 1, 4, 1), (2048, 1, 4, 1), (600, 3, 4, 1), (257, 8, 4, 1),
    (2048, 1, 5, 5), (2048, 1, 6, 3), (1024, 2, 7, 7), (2047, 1, 12, 6), (2049, 1, 5, 5)])
def test_many_rows(rows, most, heads, kv_heads):
    """Around the number of tiles up to which no list is planned, with CTAs of 8 warps and
    of fewer, and the largest."""
    rng = np.random.default_rng(rows)
    ctx = rng.integers(0, 60, rows).tolist()
    new = [min(c, int(rng.integers(0, most + 1))) for c in ctx]
    b = batch(ctx, new, heads, kv_heads, 64, "bf16")
    check(b, "bf16", max_new=most)
    check(b, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30])
def test_scales_of_either_sign_and_none(dtype, scale):
    for ctx, new, most in (([300, 33, 5], [1, 1, 1], 1), ([300, 33, 150], [90, 1, 20], 0)):
        b = batch(ctx, new, 8, 2, 128, dtype)
        b["scale"] = scale
        check(b, dtype, max_new=most)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (20, 4), (40, 1)])
def test_either_side_of_the_forms(dtype, heads, kv_heads):
    """Rows of the most query vectors that the form for few takes, and of one token more."""
    at = (64 if dtype == "f32" else 24) // (heads // kv_heads)
    new = [at, at + 1, 1, 2 * at + 1, 0, max(1, at - 1)]
    check(batch([300, 77, 129, 200, 0, 50], new, heads, kv_heads, 128, dtype, pad=2), dtype)
    for most in (at, at + 1):
        check(batch([300, 77, 129], [most, 1, 0], heads, kv_heads, 64, dtype), dtype, max_new=most)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,most", [([1, 1, 1], 1), ([60, 40, 33], 0), ([20, 9, 70], 0)])
def test_neighbours_do_not_matter(dtype, new, most):
    """Query rows of other rows and of no row, whatever they hold, change no bit: query
    vectors are scaled together with those they share a tile with."""
    import torch
    b = batch([400, 300, 70], new, 8, 2, 128, dtype, pad=5)
    want = check(b, dtype, max_new=most)
    for garbage in (float("nan"), float("inf"), 1e38):
        for r in range(3):
            at = int(sum(new[:r]))
            q = b["q"].clone()
            b["q"].fill_(garbage)
            b["q"][at:at + new[r]] = q[at:at + new[r]]
            out = call(b, torch.full_like(b["q"], 7.5), max_new=most)
            b["q"].copy_(q)
            assert torch.equal(out[at:at + new[r]], want[at:at + new[r]])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_pool_past_four_gigabytes(dtype):
    """The same bits from blocks whose bytes lie past 2^32 as from low ones."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    heads, kv_heads, dim = 32, 8, 128
    b = batch([900, 333, 40], [1, 1, 1], heads, kv_heads, dim, dtype, scaled=True)
    c = batch([900, 333], [200, 40], heads, kv_heads, dim, dtype, scaled=True)
    blocks = (1 << 32) // (kv_heads * 9 * dim) + 500
    pools = [torch.zeros((blocks + 1, kv_heads, 9 * dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for x, most in ((b, 1), (c, 0)):
        want = check(x, dtype, max_new=most)
        n = x["k"].shape[0]
        for p, name in zip(pools, ("k", "v")):
            p[blocks - n:blocks] = x[name]
        moved = {**x, "k": pools[0], "v": pools[1], "bt": x["bt"] + (blocks - n)}
        assert torch.equal(call(moved, torch.empty_like(x["q"]), max_new=most), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_random_batches(dtype):
    rng = np.random.default_rng(11)
    for i in range(12):
        heads, kv_heads, dim = SHAPES[int(rng.integers(len(SHAPES)))]
        rows = int(rng.integers(1, 40))
        ctx = [int(x) for x in np.exp(rng.uniform(0, 7.5, rows))]
        new = [min(c, int(np.exp(rng.uniform(0, 5.0)))) if rng.random() < 0.4 else 1 for c in ctx]
        check(batch(ctx, new, heads, kv_heads, dim, dtype, seed=i, pad=int(rng.integers(0, 4))), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_and_shared_workspaces(dtype):
    """A second call gives the same bits; two captured graphs share one workspace and
    replay with new lengths."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    a = batch([3000, 700, 50], [1, 1, 1], 8, 2, 128, dtype, seed=1)
    c = batch([900, 333], [40, 300], 8, 2, 128, dtype, seed=2)
    sizes = []
    for b in (a, c):
        H, Hkv, D = b["q"].shape[1], b["k"].shape[1], 128
        sh = nsv.make_shape(b["bt"].shape[0], H, Hkv, D, b["bt"].shape[1], b["k"].shape[0] - 1,
                            nsv.F32 if dtype == "f32" else nsv.BF16, query_len=0)
        sizes.append(nsv.kv4_workspace_bytes(sh, b["q"].shape[0]))
    ws = torch.full((max(sizes),), 255, dtype=torch.uint8, device="cuda")
    outs = [call(b, torch.empty_like(b["q"])) for b in (a, c)]
    again = [call(b, torch.empty_like(b["q"]), workspace=ws) for b in (a, c)]
    assert all(torch.equal(x, y) for x, y in zip(outs, again))
    graphs, results = [], []
    for b in (a, c):
        out = torch.empty_like(b["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(b, out, workspace=ws)
        graphs.append(g)
        results.append(out)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, results))
    a["ctx"].copy_(torch.tensor([160, 700, 0], dtype=torch.int32))
    graphs[0].replay()
    graphs[1].replay()
    fresh = call(a, torch.empty_like(a["q"]))
    assert torch.equal(results[0], fresh) and torch.equal(results[1], outs[1])
    assert (results[0][2] == 0).all()


def test_two_streams_at_once():
    import torch
    b = [batch([5000 + 100 * i, 800], [1, 200], 8, 2, 128, "bf16", seed=i) for i in range(2)]
    want = [call(x, torch.empty_like(x["q"])) for x in b]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in b]
    outs = [torch.empty_like(x["q"]) for x in b]
    for _ in range(5):
        for x, s, o in zip(b, streams, outs):
            with torch.cuda.stream(s):
                call(x, o)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, outs))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rotate", [False, True])
def test_a_serving_loop_on_a_four_bit_cache(dtype, rotate):
    """Prompts, chunks beside single tokens, a fork, ends and a compaction: every
    attention against the cache's values in 64 bits, which follow from the definition."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    heads, kv_heads, dim, blocks, width, rows = 8, 2, 64, 90, 24, 4
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(5)
    pools = [nsv.kv4_pool(blocks, kv_heads, dim) for _ in range(2)]
    tables = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(rows, dtype=torch.int32, device="cuda")
    refs = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    table = torch.from_numpy(F.table(width * 16, dim)).cuda()
    units = [torch.tensor([0.7, 1.3]).cuda(), torch.tensor([2.0, 0.4]).cuda()]
    held = [[np.zeros((0, kv_heads, dim))] * 2 for _ in range(rows)]
    nsv.device_status(clear=True)
    for step, grow in enumerate([[140, 33, 16, 0], [20, 1, 1, 0], [1, 1, 1, 1], [1, 0, 60, 1], [1, 5, 1, 1]]):
        if step == 2:       # row 3 continues row 0
            nsv.rows_fork(torch.tensor([0], dtype=torch.int32).cuda(),
                          torch.tensor([3], dtype=torch.int32).cuda(), tables, ctx, refs, *pools)
            held[3] = list(held[0])
        if step == 3:       # row 1 ends
            nsv.rows_free(torch.tensor([1], dtype=torch.int32).cuda(), tables, ctx, refs)
            held[1] = [np.zeros((0, kv_heads, dim))] * 2
            nsv.blocks_compact(tables, ctx, refs, *pools)
        n = sum(grow)
        starts = torch.tensor([0] + grow).cumsum(0).int().cuda()
        fused = torch.randn((n, heads + 2 * kv_heads, dim), generator=g).to(dt).cuda()
        q, k, v = fused.split([heads, kv_heads, kv_heads], 1)
        slots, out = torch.empty(n, dtype=torch.int64, device="cuda"), torch.empty((n, heads, dim), dtype=dt, device="cuda")
        turned = torch.empty_like(out)
        before = ctx.clone()
        nsv.rows_extend(starts, tables, ctx, refs, slots)
        pos = torch.cat([torch.arange(int(c), int(c) + m) for c, m in zip(before, grow)]).int().cuda()
        kw = dict(q=q, positions=pos, rotary=table, q_out=turned) if rotate else {}
        nsv.kv4_write(k, v, slots, *pools, k_scales=units[0], v_scales=units[1], **kw)
        if not rotate:
            turned = q.contiguous()
        nsv.kv4_chunk(turned, *pools, tables, starts, ctx, dim ** -0.5, out, k_scales=units[0],
                      v_scales=units[1], max_new=max(grow))
        at = 0
        for r, m in enumerate(grow):
            kr = k[at:at + m].double().cpu().numpy()
            if rotate:
                kr = F.rotate(kr, pos[at:at + m].cpu().numpy(), table.cpu().numpy(), False, True)
            new = [F.dequantise(*F.quantise(x, u.cpu().numpy()), u.cpu().numpy())
                   for x, u in ((kr, units[0]), (v[at:at + m].double().cpu().numpy(), units[1]))]
            held[r] = [np.concatenate([old, x]) for old, x in zip(held[r], new)]
            c = len(held[r][0])
            assert c == int(ctx[r])
            for i in range(m):
                see = c - m + i + 1
                kk, vv = (np.repeat(x[:see], heads // kv_heads, 1) for x in held[r])
                s = np.einsum("hd,thd->ht", turned[at + i].double().cpu().numpy(), kk) * dim ** -0.5
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                ref = np.einsum("ht,thd->hd", p, vv)
                big = (np.abs(ref) + np.einsum("ht,thd->hd", p, np.abs(vv))).max(-1)
                err = np.abs(out[at + i].double().cpu().numpy() - ref).max(-1)
                assert (err <= (F32_TOL if dtype == "f32" else BF16_TOL) * big).all()
            at += m
    assert nsv.device_status(clear=True)[0] == 0
    assert int((refs > 0).sum()) == len(set(t for r in range(rows) for t in tables[r, :-(-int(ctx[r]) // 16)].tolist()))


def test_page_operators_move_four_bit_blocks():
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    for kv_heads, dim in ((1, 64), (3, 64), (8, 128), (1, 128)):
        rng = np.random.default_rng(dim + kv_heads)
        pools = [torch.from_numpy(rng.integers(0, 256, (41, kv_heads, 9 * dim), dtype=np.uint8)).cuda()
                 for _ in range(2)]
        before = [p.clone() for p in pools]
        perm = rng.permutation(40).astype(np.int32)
        src, dst = (torch.from_numpy(x.copy()).cuda() for x in (perm[:15], perm[20:35]))
        nsv.blocks_copy(src, dst, *pools)
        for p, old in zip(pools, before):
            old[dst.long()] = old[src.long()]
            assert torch.equal(p, old)
