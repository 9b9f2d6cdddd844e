"""Attention of a chunk of new tokens over the paged cache (GPU), against the
definition in 64 bits row by row.

Tolerances, per (token, head), against `big`, the largest over the dims of
|out| + sum p |v| (p: the softmax's weights; at most twice the largest |v|):

  fp32  Products of 128 terms with fp32 accumulation, the exponential, the
        running rescales and the sum each cost a few 2^-24 relative to the
        scores' size; scores here are below 16 in log2 units, so a weight is off
        by at most about 16 * 128 * 2^-24 = 1.2e-4 in the worst case and by
        sqrt(128) in place of 128, 1.1e-5, as the terms' signs fall: 4e-5 of
        sum p |v|.
  bf16  The probabilities are rounded to bf16 by half a step, at most 2^-8 of
        each, and their sum is taken before: together at most 2^-8 sum p |v|.
        So is the output, at most 2^-8 of itself.  2^-12 is left for the scores'
        fp32 arithmetic, the exponential unit and the products of these errors.
"""

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

F32_TOL = 4e-5
BF16_TOL = 2.0 ** -8 + 2.0 ** -12
NAN = float("nan")


def batch(ctx, new, heads, kv_heads, head_dim, dtype, seed=0, pad=0, garbage=NAN):
    """Inputs on the GPU: scattered blocks, `garbage` in every pool position
    that holds no token (the sink and free blocks too), `pad` tokens of no row."""
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
        for t in range(ctx[r]):
            written[tables[r, t // 16], t % 16] = True
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    tdt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(seed)

    def draw(*shape):
        return torch.randn(shape, generator=g).to(tdt).cuda()

    T = int(starts[-1]) + pad
    hold = torch.from_numpy(written).cuda()[:, None, :, None]
    pools = [torch.where(hold, draw(blocks + 1, kv_heads, 16, head_dim), garbage) for _ in range(2)]
    return {"q": draw(T, heads, head_dim), "k": pools[0], "v": pools[1],
            "bt": torch.from_numpy(tables).cuda(), "starts": torch.from_numpy(starts).cuda(),
            "ctx": torch.tensor(ctx, dtype=torch.int32).cuda(), "scale": head_dim ** -0.5,
            "lens": (list(ctx), list(new)), "group": heads // kv_heads}


def reference(b, softcap=0.0, slopes=None, see_begin=None, see_end=None):
    """The definition in 64 bits, and what its tolerance goes by (see above)."""
    import torch
    q = b["q"].double()
    out = torch.zeros_like(q)
    big = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for r, (c, n) in enumerate(zip(*b["lens"])):
        ids = b["bt"][r, :-(-c // 16)].long()
        for i in range(n):
            pos = c - n + i
            lo = 0 if see_begin is None else max(0, int(see_begin[at + i]))
            hi = min(c, pos + 1 if see_end is None else int(see_end[at + i]))
            if lo >= hi:
                continue
            k = b["k"][ids].transpose(1, 2).reshape(-1, b["k"].shape[1], q.shape[2])[lo:hi].double()
            v = b["v"][ids].transpose(1, 2).reshape(-1, b["k"].shape[1], q.shape[2])[lo:hi].double()
            k = k.repeat_interleave(b["group"], 1)
            v = v.repeat_interleave(b["group"], 1)
            s = torch.einsum("hd,thd->ht", q[at + i], k) * b["scale"]
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            if slopes is not None:
                t = torch.arange(lo, hi, device="cuda", dtype=torch.float64)
                s = s - slopes.double()[:, None] * (pos - t).abs()
            p = torch.softmax(s, -1)
            out[at + i] = torch.einsum("ht,thd->hd", p, v)
            big[at + i] = (out[at + i].abs() + torch.einsum("ht,thd->hd", p, v.abs())).amax(-1)
        at += n
    return out, big


def check(b, dtype, garbage_out=7.5, status=0, **scores):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    nsv.device_status(clear=True)
    out = torch.full_like(b["q"], garbage_out)
    nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], out,
                    **scores)
    st, _ = nsv.device_status(clear=True)
    assert st == status, "device status %#x" % st
    ref, big = reference(b, **scores)
    T = int(sum(b["lens"][1]))
    assert torch.isfinite(out.float()).all()
    err = (out[:T].double() - ref[:T]).abs().amax(-1)
    tol = F32_TOL if dtype == "f32" else BF16_TOL
    worst = (err - tol * big[:T]).max().item() if T else 0.0
    assert worst <= 0.0, "off by %.3g above the tolerance (largest error %.3g)" % (worst, err.max())
    assert (out[T:] == garbage_out).all(), "tokens of no row were written"
    return out


SHAPES = [(4, 4, 64), (8, 2, 64), (4, 4, 128), (8, 2, 128), (6, 2, 128), (5, 1, 64), (16, 1, 128),
          (64, 1, 128)]
MIXES = [
    ([1], [1]),
    ([16, 40, 100, 257, 0], [1, 1, 1, 1, 0]),
    ([17], [17]),
    ([128, 129, 127], [128, 129, 127]),
    ([300], [300]),
    ([700, 5, 1, 333], [65, 5, 0, 1]),
    ([2000], [3]),
    ([1025, 640], [64, 200]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,head_dim", SHAPES)
@pytest.mark.parametrize("mix", range(len(MIXES)))
def test_causal(dtype, heads, kv_heads, head_dim, mix):
    ctx, new = MIXES[mix]
    check(batch(ctx, new, heads, kv_heads, head_dim, dtype, seed=mix, pad=mix % 3), dtype)


def _bounds(b, kind, rng):
    """see_begin / see_end of a document mask, a window or a prefix, and a
    general pair that leaves some tokens with nothing to see."""
    import torch
    begin, end = [], []
    for c, n in zip(*b["lens"]):
        pos = np.arange(c - n, c)
        e = pos + 1
        if kind == "documents":
            cuts = np.unique(np.concatenate([[0], rng.integers(0, max(c, 1), 4)]))
            s = cuts[np.searchsorted(cuts, pos, side="right") - 1]
        elif kind == "window":
            s = pos + 1 - 50
        elif kind == "prefix":
            s, e = np.zeros(n), np.maximum(e, c // 2)
        else:
            s = rng.integers(-5, c + 3, n)
            e = s + rng.integers(-3, 200, n)
        begin.append(s)
        end.append(e)
    as_gpu = lambda a: torch.from_numpy(  # noqa: E731
        np.concatenate(a + [np.zeros(len(b["q"]) - sum(b["lens"][1]))]).astype(np.int32)).cuda()
    got = {"see_begin": as_gpu(begin), "see_end": as_gpu(end)}
    if kind in ("documents", "window"):
        del got["see_end"]
    elif kind == "prefix":
        del got["see_begin"]
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["documents", "window", "prefix", "any"])
@pytest.mark.parametrize("heads,kv_heads,head_dim", [(8, 2, 64), (4, 4, 128), (5, 1, 128)])
@pytest.mark.parametrize("ctx,new", [([400, 33, 260], [300, 33, 1]), ([900], [40])])
def test_masks(dtype, kind, heads, kv_heads, head_dim, ctx, new):
    b = batch(ctx, new, heads, kv_heads, head_dim, dtype, seed=5, pad=2)
    check(b, dtype, **_bounds(b, kind, np.random.default_rng(3)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("softcap,slopes", [(20.0, False), (0.5, False), (5e4, False), (0.0, True),
                                            (30.0, True)])
@pytest.mark.parametrize("heads,kv_heads,head_dim", [(8, 2, 64), (12, 4, 128)])
@pytest.mark.parametrize("ctx,new,kind", [([400, 33, 1], [300, 33, 1], None),
                                          ([513, 77], [1, 1], None), ([300, 40], [130, 9], "any")])
def test_scores(dtype, softcap, slopes, heads, kv_heads, head_dim, ctx, new, kind):
    import torch
    b = batch(ctx, new, heads, kv_heads, head_dim, dtype, seed=6)
    kw = _bounds(b, kind, np.random.default_rng(4)) if kind else {}
    if slopes:
        kw["slopes"] = torch.exp2(-torch.arange(heads, device="cuda", dtype=torch.float32) / 2)
    check(b, dtype, softcap=softcap, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scale_of_any_sign(dtype):
    for scale in (-0.1, 0.0, 0.3):
        b = batch([200, 130], [129, 1], 4, 2, 64, dtype, seed=7)
        b["scale"] = scale
        check(b, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_chunk_longer_than_its_context(dtype):
    """The first tokens sit before position 0: they see nothing and give 0."""
    b = batch([40], [40], 4, 2, 64, dtype, seed=8)
    b["ctx"][0] = 25
    b["lens"] = ([25], [40])
    b["k"][:] = b["k"].nan_to_num(0.0)
    b["v"][:] = b["v"].nan_to_num(0.0)
    out = check(b, dtype)
    assert (out[:15] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_scores_need_the_running_maximum(dtype):
    """Scores that grow along the context raise the maximum run after run."""
    import torch
    b = batch([1500], [130], 4, 2, 64, dtype, seed=9)
    b["q"].fill_(1.0)
    for t in range(1500):
        b["k"][b["bt"][0, t // 16].item(), :, t % 16] = t / 256.0 / 8 * 4
    torch.cuda.synchronize()
    check(b, dtype)


def test_same_call_same_bits():
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = batch([3000, 700, 64], [40, 300, 1], 8, 2, 128, "bf16", seed=10)
    outs = [torch.empty_like(b["q"]) for _ in range(3)]
    for o in outs:
        nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], o)
    assert all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_single_tokens_agree_with_the_decode_read(dtype):
    """One token per row: the same read as paged_decode, by another kernel."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    ctx = [1, 16, 700, 2049, 300]
    b = batch(ctx, [1] * 5, 8, 2, 128, dtype, seed=11)
    out = check(b, dtype)
    want = nsv.paged_decode(b["q"], b["k"], b["v"], b["bt"], b["ctx"], b["scale"],
                            torch.empty_like(out))
    _, big = reference(b)
    tol = 2 * (F32_TOL if dtype == "f32" else BF16_TOL)   # each within one of the definition
    assert ((out.double() - want.double()).abs().amax(-1) <= tol * big).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_values_are_skipped_and_flagged(dtype):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = batch([200, 100, 60], [50, 30, 20], 4, 2, 64, dtype, seed=12)

    def call():
        out = torch.full_like(b["q"], 3.0)
        nsv.device_status(clear=True)
        nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], out)
        return out, nsv.device_status(clear=True)[0]

    good, st = call()
    assert st == 0
    # a block id outside the pool: its positions are left out, other rows stay
    keep = b["bt"].clone()
    b["bt"][1, 2] = 10 ** 6
    b["bt"][2, 0] = -7
    out, st = call()
    assert st == nsv.DEV_BAD_BLOCK
    assert torch.equal(out[:50], good[:50]) and torch.isfinite(out.float()).all()
    b["bt"] = keep
    # a context beyond the table: the row reads as empty
    b["ctx"][1] = 16 * b["bt"].shape[1] + 1
    out, st = call()
    assert st == nsv.DEV_BAD_CTX
    assert (out[50:80] == 0).all() and torch.equal(out[:50], good[:50])
    b["ctx"][1] = 100
    # starts that do not ascend, or leave [0, tokens]: no tokens of that row
    for starts, untouched in (([0, 50, 40, 100], (50, 50)), ([0, 50, 80, 101], (80, 100)),
                              ([-5, 50, 80, 100], (0, 50))):
        b["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        out, st = call()
        assert st & nsv.DEV_BAD_CHUNK
        assert (out[untouched[0]:untouched[1]] == 3.0).all()
    # rows that all claim every token: more tiles than there is room for
    R = 64
    wide = dict(b, bt=b["bt"][:1].repeat(R, 1), ctx=b["ctx"][:1].repeat(R),
                starts=torch.tensor([0, 100] * (R // 2) + [0], dtype=torch.int32, device="cuda"))
    out = torch.zeros_like(b["q"])
    nsv.paged_chunk(wide["q"], b["k"], b["v"], wide["bt"], wide["starts"], wide["ctx"], 0.1, out)
    assert nsv.device_status(clear=True)[0] & nsv.DEV_BAD_CHUNK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_appends_then_reads(dtype):
    """The step's new tokens are in the pool before the read, bit for bit."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = batch([300, 40, 1], [130, 40, 1], 8, 2, 128, dtype, seed=13, pad=4)
    T, live = len(b["q"]), sum(b["lens"][1])
    sink = (b["k"].shape[0] - 1) * 16
    slots = np.full(T, sink, np.int64)
    at = 0
    for r, (c, n) in enumerate(zip(*b["lens"])):
        for i in range(n):
            pos = c - n + i
            slots[at] = int(b["bt"][r, pos // 16]) * 16 + pos % 16
            at += 1
    slots = torch.from_numpy(slots).cuda()
    blk, off = slots[:live] // 16, slots[:live] % 16
    new = [torch.zeros(T, 2, 128, dtype=b["q"].dtype, device="cuda") for _ in range(2)]
    want_k, want_v = b["k"].clone(), b["v"].clone()
    for pool, x in ((b["k"], new[0]), (b["v"], new[1])):
        x[:live] = pool[blk, :, off]
        pool[blk, :, off] = NAN     # nothing there before the step
    out = torch.full_like(b["q"], 7.5)
    nsv.device_status(clear=True)
    nsv.chunk_step(b["q"], new[0], new[1], slots, b["k"], b["v"], b["bt"], b["starts"], b["ctx"],
                   b["scale"], out)
    assert nsv.device_status(clear=True)[0] == 0
    assert torch.equal(b["k"][:-1].nan_to_num(9.0), want_k[:-1].nan_to_num(9.0))
    assert torch.equal(b["v"][:-1].nan_to_num(9.0), want_v[:-1].nan_to_num(9.0))
    ref, big = reference(b)
    tol = F32_TOL if dtype == "f32" else BF16_TOL
    assert ((out[:live].double() - ref[:live]).abs().amax(-1) <= tol * big[:live]).all()
    assert (out[live:] == 7.5).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_call_replays_with_new_lengths(dtype):
    """Captured on one batch, replayed on others of the same sizes: lengths,
    chunk starts and tables are read by the kernels alone."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    a = batch([500, 90, 33], [70, 20, 6], 8, 2, 128, dtype, seed=14, garbage=0.0)
    c = batch([64, 411, 148], [1, 90, 3], 8, 2, 128, dtype, seed=15, garbage=0.0, pad=2)
    assert len(a["q"]) == len(c["q"])
    # one pool for both: c's blocks behind a's
    na = a["k"].shape[0]
    k, v = torch.cat([a["k"], c["k"]]), torch.cat([a["v"], c["v"]])
    width = max(a["bt"].shape[1], c["bt"].shape[1])
    tables = [torch.full((3, width), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    tables[0][:, :a["bt"].shape[1]] = a["bt"]
    tables[1][:, :c["bt"].shape[1]] = torch.where(c["bt"] >= 0, c["bt"] + na, -1)
    q, bt, starts, ctx = (x.clone() for x in (a["q"], tables[0], a["starts"], a["ctx"]))
    out = torch.zeros_like(q)
    shape = nsv.make_shape(3, 8, 2, 128, width, k.shape[0] - 1,
                           nsv.F32 if dtype == "f32" else nsv.BF16)
    ws = torch.empty(nsv.chunk_workspace_bytes(shape, len(q)), dtype=torch.uint8, device="cuda")
    run = lambda: nsv.paged_chunk(q, k, v, bt, starts, ctx, a["scale"], out,  # noqa: E731
                                  workspace=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for b, t in ((c, tables[1]), (a, tables[0]), (c, tables[1])):
        q.copy_(b["q"]), bt.copy_(t), starts.copy_(b["starts"]), ctx.copy_(b["ctx"])
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        ref, big = reference(b)
        live = sum(b["lens"][1])
        tol = F32_TOL if dtype == "f32" else BF16_TOL
        assert ((out[:live].double() - ref[:live]).abs().amax(-1) <= tol * big[:live]).all()


def test_two_streams_with_a_workspace_each():
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    bs = [batch([2000, 64], [64, 3], 8, 2, 128, "bf16", seed=s) for s in (16, 17)]
    outs = [torch.empty_like(b["q"]) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, o, st in zip(bs, outs, streams):
            nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], o,
                            stream=st)
    torch.cuda.synchronize()
    for b, o in zip(bs, outs):
        ref, big = reference(b)
        assert ((o.double() - ref).abs().amax(-1) <= BF16_TOL * big).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,head_dim", [(8, 2, 128), (3, 3, 64)])
def test_long_rows_are_cut_into_many_pieces(dtype, heads, kv_heads, head_dim):
    check(batch([20011, 9000], [2, 70], heads, kv_heads, head_dim, dtype, seed=18), dtype)


def _sample(b, rows):
    """The batch cut down to some of its rows, and their tokens' indexes."""
    import torch
    ctx, new = b["lens"]
    starts = np.concatenate([[0], np.cumsum(new)])
    at = np.concatenate([np.arange(starts[r], starts[r + 1]) for r in rows])
    idx = torch.from_numpy(at).cuda()
    cut = dict(b, q=b["q"][idx], bt=b["bt"][torch.tensor(rows).cuda()],
               lens=([ctx[r] for r in rows], [new[r] for r in rows]))
    return cut, idx


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", [None, "window"])
def test_thousands_of_rows(dtype, kind):
    """More rows and tiles than one pass of the planning kernel covers, up to the
    largest batch; a few rows are checked."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    rng = np.random.default_rng(19)
    ctx = [int(x) for x in rng.integers(0, 60, 8192)]
    new = [min(c, int(x)) for c, x in zip(ctx, rng.integers(0, 4, 8192))]
    b = batch(ctx, new, 4, 2, 64, dtype, seed=19, pad=3)
    kw = _bounds(b, kind, rng) if kind else {}
    nsv.device_status(clear=True)
    out = torch.full_like(b["q"], 7.5)
    nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], out, **kw)
    assert nsv.device_status(clear=True)[0] == 0
    assert (out[-3:] == 7.5).all() and torch.isfinite(out.float()).all()
    cut, idx = _sample(b, [0, 1, 1023, 1024, 1025, 4000, 8190, 8191] + list(range(5000, 5040)))
    ref, big = reference(cut, **{k: v[idx] for k, v in kw.items()})
    tol = F32_TOL if dtype == "f32" else BF16_TOL
    assert ((out[idx].double() - ref).abs().amax(-1) <= tol * big).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pool_offsets_beyond_32_bits(dtype):
    """Blocks whose element offsets (and byte offsets) pass 2^31 and 2^32."""
    import torch
    b = batch([300, 40], [130, 1], 16, 8, 128, dtype, seed=20)
    blocks = 140000 if dtype == "bf16" else 280000 // 2 + 1000
    base = blocks - b["k"].shape[0]         # the batch's blocks at the pool's end
    for name in ("k", "v"):
        pool = torch.empty((blocks + 1,) + tuple(b[name].shape[1:]), dtype=b[name].dtype,
                           device="cuda")
        assert pool.numel() > 2 ** 31
        pool[:64] = 3.0                     # what a wrapped offset would read
        pool[base:base + b[name].shape[0]] = b[name]
        b[name] = pool
    b["bt"] = torch.where(b["bt"] >= 0, b["bt"] + base, -1).int()
    check(b, dtype)


def test_two_graphs_share_a_workspace():
    """Captured with one workspace and replayed in turn on one stream."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    bs = [batch([2100, 64], [64, 3], 8, 2, 128, "bf16", seed=s) for s in (21, 22)]
    outs = [torch.zeros_like(b["q"]) for b in bs]
    shape = nsv.make_shape(2, 8, 2, 128, bs[0]["bt"].shape[1], bs[0]["k"].shape[0] - 1, nsv.BF16)
    ws = torch.empty(nsv.chunk_workspace_bytes(shape, 67), dtype=torch.uint8, device="cuda")

    def run(b, o):
        nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], o,
                        workspace=ws)

    run(bs[0], outs[0])
    torch.cuda.synchronize()
    graphs = []
    for b, o in zip(bs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run(b, o)
    for o in outs:
        o.zero_()
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for b, o in zip(bs, outs):
        ref, big = reference(b)
        assert ((o.double() - ref).abs().amax(-1) <= BF16_TOL * big).all()


def test_calls_back_to_back_with_one_workspace():
    """Each call's planning overlaps the call before it; the workspace does not."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    cases = [batch(c, n, 8, 2, 128, "bf16", seed=30 + i) for i, (c, n) in enumerate(
        [([3000, 64], [40, 3]), ([17], [17]), ([900, 800, 700], [1, 1, 1]), ([2500], [260])])]
    shape = nsv.make_shape(3, 8, 2, 128, 400, 1000, nsv.BF16)
    ws = torch.empty(nsv.chunk_workspace_bytes(shape, 300), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(b["q"]) for b in cases]
    for _ in range(10):
        for b, o in zip(cases, outs):
            nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], o,
                            workspace=ws)
    torch.cuda.synchronize()
    for b, o in zip(cases, outs):
        ref, big = reference(b)
        assert ((o.double() - ref).abs().amax(-1) <= BF16_TOL * big).all()


def test_binding_refuses_what_does_not_fit():
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = batch([40], [8], 4, 2, 64, "bf16", seed=23)
    args = dict(q=b["q"], k_pool=b["k"], v_pool=b["v"], block_tables=b["bt"],
                chunk_starts=b["starts"], context_lens=b["ctx"], scale=0.1,
                out=torch.empty_like(b["q"]))
    for name, bad in (("q", b["q"].float()), ("q", b["q"].transpose(0, 1)), ("v_pool", b["v"][1:]),
                      ("block_tables", b["bt"].long()), ("chunk_starts", b["starts"][:1]),
                      ("context_lens", b["ctx"].cpu()), ("out", args["out"][:4]),
                      ("out", args["out"].expand(8, 4, 64)[:, :, ::2])):
        with pytest.raises(ValueError):
            nsv.paged_chunk(**dict(args, **{name: bad}))
    for name, bad in (("slopes", torch.zeros(3, device="cuda")), ("see_end", b["ctx"])):
        with pytest.raises(ValueError):
            nsv.paged_chunk(**args, **{name: bad})
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(nsv.NsvError) as e:
        nsv.paged_chunk(**args, workspace=small)
    assert e.value.code == -8


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_keys_that_a_token_does_not_see_hold_anything(dtype, value):
    """A key at position 150 of a row, inside the same run of positions as those
    that earlier tokens and other documents see."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = batch([200, 30], [100, 30], 8, 2, 128, dtype, seed=24)
    blk = int(b["bt"][0, 150 // 16])
    begin = torch.zeros(130, dtype=torch.int32, device="cuda")
    begin[60:100] = 151          # the row's last 40 tokens: another document
    kw = dict(see_begin=begin)
    b["k"][blk, :, 150 % 16] = 0.5
    ref, big = reference(b, **kw)
    b["k"][blk, :, 150 % 16] = value
    out = torch.empty_like(b["q"])
    nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], out, **kw)
    rest = [i for i in range(130) if not 50 <= i < 60]      # those ten see it
    tol = F32_TOL if dtype == "f32" else BF16_TOL
    assert ((out[rest].double() - ref[rest]).abs().amax(-1) <= tol * big[rest]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_blocks_that_a_window_has_left_need_not_be_there(dtype):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = batch([1000, 500], [40, 1], 8, 2, 64, dtype, seed=25)
    begin = torch.tensor([960 + i + 1 - 130 for i in range(40)] + [400], dtype=torch.int32,
                         device="cuda")
    end = torch.full((41,), 490, dtype=torch.int32, device="cuda")
    end[:40] = 990
    kw = dict(see_begin=begin, see_end=end)
    ref, big = reference(b, **kw)
    b["bt"][0, :831 // 16] = -1
    b["bt"][1, :25] = 1 << 29
    b["bt"][1, 31:] = 1 << 29
    nsv.device_status(clear=True)
    out = torch.empty_like(b["q"])
    nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], out, **kw)
    assert nsv.device_status(clear=True)[0] == 0
    tol = F32_TOL if dtype == "f32" else BF16_TOL
    assert ((out.double() - ref).abs().amax(-1) <= tol * big).all()


def test_more_work_than_a_share_counts_is_not_run():
    """65536 tokens that each see 2^31 - 16 positions, a run of 64 at a time."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    tokens, width = 1 << 16, (1 << 27) - 1
    q = torch.zeros((tokens, 64, 64), device="cuda")
    out = torch.full_like(q, 7.5)
    pools = [torch.zeros((2, 1, 16, 64), device="cuda") for _ in range(2)]
    bt = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([width * 16], dtype=torch.int32, device="cuda")
    nsv.device_status(clear=True)
    nsv.paged_chunk(q, *pools, bt, starts, ctx, 0.1, out)
    assert nsv.device_status(clear=True)[0] == nsv.DEV_BAD_CHUNK
    assert (out == 7.5).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_few_rows_then_many_on_one_cta(dtype, head_dim):
    """A tile of one token right before tiles of sixteen: its rows' exchange may
    still be under way when theirs are loaded."""
    check(batch([1294, 91, 361, 895], [1019, 81, 197, 766], 64, 4, head_dim, dtype, seed=26), dtype)


@pytest.mark.parametrize("seed", range(40))
def test_random_batches(seed):
    """Mixes of chunks of all lengths, so that tiles of all kinds follow each other."""
    rng = np.random.default_rng(100 + seed)
    rows = int(rng.integers(1, 40))
    new = [int(x) for x in np.exp(rng.uniform(0, math.log(rng.choice([2, 40, 400])), rows))]
    while sum(new) > 1500:
        new.pop()
    ctx = [n + int(rng.choice([0, 3, 150, 900]) * rng.random()) for n in new]
    kv_heads = int(rng.choice([1, 2, 4, 8]))
    group = int(rng.choice([1, 2, 4, 5, 16, 33, 64]))
    dtype = "f32" if seed % 4 == 3 else "bf16"
    b = batch(ctx, new, group * kv_heads, kv_heads, int(rng.choice([64, 128, 128])), dtype,
              seed=seed, pad=int(rng.integers(0, 3)))
    kind = rng.choice(["causal", "documents", "window", "prefix"])
    kw = {} if kind == "causal" else _bounds(b, kind, rng)
    if rng.random() < 0.3:
        kw["softcap"] = 20.0
    check(b, dtype, **kw)


@pytest.mark.parametrize("head_dim", [64, 128])
def test_long_sums_keep_their_precision(head_dim):
    """fp32 with equal weights: the mean of 8192 values near 3.  A run of 64 goes
    through 24 accumulating MMAs, which drop up to 2^-23 of the partial sum each, 2.9e-6
    in all; the sum over runs is rounded to nearest, and 2^-20 is left for it."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = batch([8192, 8000], [1, 2], 4, 4, head_dim, "f32", seed=27)
    b["q"].zero_()
    b["v"] += 3.0
    out = torch.empty_like(b["q"])
    nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], out)
    ref, _ = reference(b)
    assert ((out.double() - ref) / ref).abs().max() <= 24 * 2.0 ** -23 + 2.0 ** -20


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lent_workspaces(dtype):
    """Without a workspace of the caller's: on another stream, and captured, where
    eager calls and allocations between the replays must not meet the graph's."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    bs = [batch([2100, 64], [64, 3], 8, 2, 128, dtype, seed=s) for s in (28, 29)]
    tol = F32_TOL if dtype == "f32" else BF16_TOL
    outs = [torch.zeros_like(b["q"]) for b in bs]

    def run(b, o, **kw):
        nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], o, **kw)

    def right(b, o):
        ref, big = reference(b)
        return bool(((o.double() - ref).abs().amax(-1) <= tol * big).all())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for b, o in zip(bs, outs):
        run(b, o, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(right(b, o) for b, o in zip(bs, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(bs[0], outs[0])
        run(bs[1], outs[1])
    junk = []
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        junk.append(torch.full((1 << 20,), float("nan"), device="cuda"))
        extra = torch.zeros_like(outs[0])
        run(bs[0], extra)
        torch.cuda.synchronize()
        assert right(bs[0], extra) and all(right(b, o) for b, o in zip(bs, outs))


INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["both", "see_begin", "see_end"])
@pytest.mark.parametrize("heads,kv_heads,head_dim", [(4, 2, 64), (6, 2, 128)])
@pytest.mark.parametrize("ctx,new", [([700, 300, 40], [200, 1, 40]), ([1500], [3])])
def test_extreme_bounds(dtype, which, heads, kv_heads, head_dim, ctx, new):
    """Bounds at both ends of int32 ("sees nothing", "no bound"), in tiles whose other
    tokens see several runs."""
    import torch
    b = batch(ctx, new, heads, kv_heads, head_dim, dtype, seed=31)
    T = sum(new)
    end = np.concatenate([np.arange(c - n, c) + 1 for c, n in zip(ctx, new)])
    begin = np.maximum(end - 400, 0)
    at = np.arange(T)
    for step, lows, highs in ((3, end, begin), (7, begin, end)):
        lows[at % step == 1] = INT_MIN + (at[at % step == 1] * 37) % 600
        highs[at % (2 * step) == 2] = INT_MAX - at[at % (2 * step) == 2] % 5
    kw = {"see_begin": begin, "see_end": end}
    kw = {k: torch.from_numpy(v.astype(np.int32)).cuda() for k, v in kw.items()
          if which in ("both", k)}
    check(b, dtype, **kw)


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("ctx", [8192, 32768])
def test_sums_of_weights_keep_their_precision(head_dim, ctx):
    """fp32, rows that one CTA holds whole, one key above equal others: the row's sum
    adds the same weight over and over, and only the top key has a value, 1, so that
    the output is 1 / sum.  Relative errors: a weight is 2^x with x (at most 6 in size)
    rounded once and log2(e) as it is in fp32, 6 ln 2 (2^-24 + 1.4e-8) = 3.1e-7, and the
    exponential unit 2^-22; up to 16 additions in a row within a run, 2^-20; the runs'
    compensated sum, both threads', the quotient and the product, 6 x 2^-24.  Together
    1.9e-6, below 2^-19."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    heads, rows = 8, torch.cuda.get_device_properties(0).multi_processor_count
    steps = np.array([0.05, 0.3, 0.7, 1.15, 1.9, 2.6, 3.4, 5.3])
    c = np.round(steps * math.log(2) * 4096) / 4096     # short enough for exact products
    pools = [torch.zeros((ctx // 16 + 1, 1, 16, head_dim), device="cuda") for _ in range(2)]
    pools[0][:, :, :, 0] = -1.0
    pools[0][0, 0, 0, 0] = 0.0
    pools[1][0, 0, 0] = 1.0
    bt = torch.arange(ctx // 16, dtype=torch.int32, device="cuda").repeat(rows, 1)
    q = torch.zeros((rows, heads, head_dim), device="cuda")
    q[:, :, 0] = torch.from_numpy(c).float().cuda()
    starts = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    lens = torch.full((rows,), ctx, dtype=torch.int32, device="cuda")
    out = nsv.paged_chunk(q, *pools, bt, starts, lens, 1.0, torch.empty_like(q))
    want = torch.from_numpy(1 / (1 + (ctx - 1) * np.exp(-c))).cuda()
    err = (out.double() / want[None, :, None] - 1).abs().amax((0, 2))
    assert (err <= 2.0 ** -19).all(), err


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("softcap", [30.0, 200.0, 256.0, 257.0, 1000.0, 4096.0, 4097.0])
def test_caps_on_both_sides_of_the_short_tanh(head_dim, softcap):
    """bf16, 31 positions, of which the one with the highest score has the only values:
    the output is v / sum, v all significands of bf16.  Its own rounding is all that may
    be seen of bf16: everything else stays within 2^-12 of it."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    tokens, heads, ctx = 16, 8, 31
    pools = [torch.zeros((3, 1, 16, head_dim), dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    pools[0][:2, :, :, 0] = 0.5
    pools[0][0, 0, 7, 0] = 1.0
    outs, wants = [], []
    a = torch.from_numpy(np.linspace(0.25, 8.0, tokens * heads)).to(torch.bfloat16).cuda()
    q = torch.zeros((tokens, heads, head_dim), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = a.view(tokens, heads)
    i32 = dict(dtype=torch.int32, device="cuda")
    for first in range(0, 128, head_dim):
        v = 1 + torch.arange(first, first + head_dim, device="cuda").double() / 128
        pools[1][0, 0, 7] = v.to(torch.bfloat16)
        out = torch.empty_like(q)
        nsv.paged_chunk(q, *pools, torch.tensor([[0, 1]], **i32), torch.tensor([0, tokens], **i32),
                        torch.tensor([ctx], **i32), 1.0, out, softcap=softcap,
                        see_end=torch.full((tokens,), ctx, **i32))
        s = q[:, :, 0].double()
        top, rest = (softcap * torch.tanh(x / softcap) for x in (s, s * 0.5))
        outs.append(out)
        wants.append(v / (1 + (ctx - 1) * torch.exp(rest - top))[..., None])
    out, want = torch.cat(outs, -1), torch.cat(wants, -1)
    low, high = ((want * (1 + x)).to(torch.bfloat16) for x in (-2.0 ** -12, 2.0 ** -12))
    bad = (out < low) | (out > high)
    assert not bad.any(), "%d of %d outside" % (int(bad.sum()), bad.numel())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bounds_that_leave_a_gap(dtype):
    """Tokens that see positions far apart, some of them from the middle of a block: what
    lies before the first of them and past the last need not be there, nor be finite."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = batch([1000, 900], [9, 30], 8, 2, 128, dtype, seed=32)
    i = torch.arange(39, device="cuda", dtype=torch.int32)
    kw = dict(see_begin=torch.where(i % 2 == 0, 165 + i, 700), see_end=torch.where(
        i % 2 == 0, 181 + i, 733 + i))
    ref, big = reference(b, **kw)
    for r, c in enumerate((1000, 900)):
        for blk in list(range(10)) + list(range(772 // 16 + 1, c // 16)):
            for pool in (b["k"], b["v"]):
                pool[int(b["bt"][r, blk])] = NAN
            if blk % 2:
                b["bt"][r, blk] = -5 - blk
    nsv.device_status(clear=True)
    out = torch.empty_like(b["q"])
    nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], out, **kw)
    assert nsv.device_status(clear=True)[0] == 0
    tol = F32_TOL if dtype == "f32" else BF16_TOL
    assert ((out.double() - ref).abs().amax(-1) <= tol * big).all()


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("kv_heads,group", [(1, 8), (2, 1)])
def test_long_rows_of_one_cta_keep_their_precision(head_dim, kv_heads, group):
    """fp32, equal weights and values near 3 over 65536 positions, rows that one CTA holds
    whole: 1024 runs, whose sums are rounded to nearest, 2^-24 of the growing sum each,
    2^-15 in all; within a run 24 accumulating MMAs may drop 2^-23 of it each; the sum of
    the weights, the quotient and the product are off by a few 2^-24.  (Left to the tensor
    core's accumulator, sums over 8192 positions lost 6e-6 to 2e-5.)"""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    ctx, rows = 65536, torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device="cuda").manual_seed(33)
    pools = [torch.randn((ctx // 16 + 1, kv_heads, 16, head_dim), device="cuda", generator=g)
             for _ in range(2)]
    pools[1] += 3.0
    i32 = dict(dtype=torch.int32, device="cuda")
    bt = torch.arange(ctx // 16, **i32).repeat(rows, 1)
    q = torch.zeros((rows, kv_heads * group, head_dim), device="cuda")
    starts, lens = torch.arange(rows + 1, **i32), torch.full((rows,), ctx, **i32)
    out = nsv.paged_chunk(q, *pools, bt, starts, lens, 1.0, torch.empty_like(q))
    v = pools[1][:-1].double()
    ref = v.mean((0, 2)).repeat_interleave(group, 0)
    big = v.abs().mean((0, 2)).repeat_interleave(group, 0)
    assert ((out.double() - ref).abs() <= big * (2.0 ** -15 + 24 * 2.0 ** -23 + 2.0 ** -21)).all()


def test_same_call_same_bits_fp32():
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    b = batch([3000, 700, 64], [40, 300, 1], 8, 2, 128, "f32", seed=10)
    outs = [torch.empty_like(b["q"]) for _ in range(3)]
    for o in outs:
        nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], o)
    assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_two_streams_and_two_graphs_fp32():
    """Calls on two streams with a workspace each, then two graphs that share one."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    bs = [batch([2000, 64], [64, 3], 8, 2, 128, "f32", seed=s) for s in (34, 35)]
    outs = [torch.empty_like(b["q"]) for b in bs]
    shape = nsv.make_shape(2, 8, 2, 128, bs[0]["bt"].shape[1], bs[0]["k"].shape[0] - 1, nsv.F32)
    ws = torch.empty(nsv.chunk_workspace_bytes(shape, 67), dtype=torch.uint8, device="cuda")

    def run(b, o, **kw):
        nsv.paged_chunk(b["q"], b["k"], b["v"], b["bt"], b["starts"], b["ctx"], b["scale"], o, **kw)

    def right():
        torch.cuda.synchronize()
        for b, o in zip(bs, outs):
            ref, big = reference(b)
            assert ((o.double() - ref).abs().amax(-1) <= F32_TOL * big).all()

    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, o, st in zip(bs, outs, streams):
            run(b, o, stream=st)
    right()
    graphs = []
    for b, o in zip(bs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run(b, o, workspace=ws)
        o.zero_()
    for _ in range(5):
        for g in graphs:
            g.replay()
    right()


@pytest.mark.parametrize("seed", range(12))
def test_exchanges_of_few_rows_before_full_tiles(seed):
    """Tiles of one or a few tokens, whose rows lie two or four times over the MMA's, right
    before tiles that fill both halves, over and over on each CTA."""
    rng = np.random.default_rng(400 + seed)
    group = [4, 16, 32, 5][seed % 4]
    tile = 2 * (128 // group)
    new, ctx = [], []
    for _ in range(14):
        for n in (int(rng.integers(1, max(2, tile // 4))), int(rng.integers(1, 3)),
                  tile * int(rng.integers(1, 4)) + int(rng.integers(0, 2))):
            new.append(n)
            ctx.append(n + int(rng.integers(0, 300)))
    check(batch(ctx, new, 4 * group, 4, [64, 128][seed // 4 % 2], "bf16", seed=seed, pad=1), "bf16")
