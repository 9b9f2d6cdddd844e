"""Page operators of the paged cache (GPU) against a plain model of each, whole
numbers equal and blocks bit for bit; and a run of a cache's life, where every
read is checked against the tokens themselves."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

DTYPES = ["f32", "bf16"]


class Cache:
    """A cache on the host: tables, lengths, references and pools (one random
    int32 per 16-byte vector stands for a block's contents)."""

    def __init__(self, ctx, blocks, kv_heads=2, head_dim=64, dtype="bf16", extra=4, seed=0):
        rng = np.random.default_rng(seed)
        self.rng = rng
        rows, nb = len(ctx), [-(-c // 16) for c in ctx]
        self.bt = np.full((rows, max(nb + [0]) + extra), -1, np.int32)
        self.ctx = np.array(ctx, np.int32)
        self.refs = np.zeros(blocks, np.int32)
        perm, at = rng.permutation(blocks), 0
        for r, n in enumerate(nb):
            share = min(nb[r - 1], n, int(ctx[r] // 16), int(ctx[r - 1] // 16)) // 2 \
                if r % 3 == 2 else 0
            self.bt[r, :share] = self.bt[r - 1, :share]
            self.bt[r, share:n] = perm[at:at + n - share]
            at += n - share
            for b in self.bt[r, :n]:
                self.refs[b] += 1
        vecs = kv_heads * 16 * head_dim * (4 if dtype == "f32" else 2) // 4
        self.k, self.v = (rng.integers(0, 1 << 14, (blocks + 1, vecs)).astype(np.int32)
                          for _ in range(2))
        self.pool = (blocks + 1, kv_heads, 16, head_dim)
        self.dtype = dtype

    def gpu(self):
        import torch
        tdt = torch.float32 if self.dtype == "f32" else torch.bfloat16
        pools = [torch.from_numpy(p.copy()).cuda().view(tdt).view(self.pool)
                 for p in (self.k, self.v)]
        return [torch.from_numpy(x.copy()).cuda() for x in (self.bt, self.ctx, self.refs)] + pools

    def same(self, got, free_too=True):
        import torch
        bt, ctx, refs, k, v = got
        assert np.array_equal(bt.cpu().numpy(), self.bt)
        assert np.array_equal(ctx.cpu().numpy(), self.ctx)
        assert np.array_equal(refs.cpu().numpy(), self.refs)
        live = np.ones(len(self.refs), bool) if free_too else self.refs > 0
        for have, want in ((k, self.k), (v, self.v)):
            have = have.contiguous().view(len(have), -1).view(torch.int32).cpu().numpy()
            assert np.array_equal(have[:-1][live], want[:-1][live])

    # the operators, one item after the other
    def free_ids(self):
        return [int(b) for b in np.nonzero(self.refs == 0)[0]]

    def fork(self, parents, children):
        before, free, taken, seen = self.ctx.copy(), self.free_ids(), 0, set()
        for p, c in zip(parents, children):
            if p == -1 and c == -1:
                continue
            if not (0 <= p < len(before) and 0 <= c < len(before)) or before[c]:
                continue
            if c in seen:
                continue
            seen.add(c)
            n = int(before[p])
            taken += n % 16 != 0
            if taken > len(free):
                continue
            full = n // 16
            self.bt[c, :full] = self.bt[p, :full]
            for b in self.bt[c, :full]:
                self.refs[b] += 1
            if n % 16:
                b, src = free[taken - 1], self.bt[p, full]
                self.bt[c, full], self.refs[b] = b, 1
                self.k[b], self.v[b] = self.k[src], self.v[src]
            self.ctx[c] = n

    def extend(self, starts, tokens):
        free, taken = self.free_ids(), 0
        slots = np.full(tokens, len(self.refs) * 16, np.int64)
        for r in range(len(self.ctx)):
            n, old = int(starts[r + 1] - starts[r]), int(self.ctx[r])
            if n <= 0 or old + n > self.bt.shape[1] * 16:
                continue
            had, will = -(-old // 16), -(-(old + n) // 16)
            taken += will - had
            if taken > len(free):
                continue
            ids = free[taken - (will - had):taken]
            self.bt[r, had:will] = ids
            self.refs[ids] = 1
            for i in range(n):
                pos = old + i
                slots[starts[r] + i] = int(self.bt[r, pos // 16]) * 16 + pos % 16
            self.ctx[r] = old + n
        return slots

    def free(self, rows):
        for r in rows:
            if 0 <= r < len(self.ctx):
                n = -(-int(self.ctx[r]) // 16)
                for b in self.bt[r, :n]:
                    self.refs[b] -= 1
                self.bt[r, :n] = -1
                self.ctx[r] = 0

    def compact(self):
        live = np.nonzero(self.refs > 0)[0]
        n = len(live)
        src = live[live >= n]
        dst = np.array([b for b in self.free_ids() if b < n], np.int64)
        to = np.arange(len(self.refs))
        to[src] = dst
        for a, b in zip(src, dst):
            self.k[b], self.v[b] = self.k[a], self.v[a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for r, c in enumerate(self.ctx):
            m = -(-int(c) // 16)
            self.bt[r, :m] = to[self.bt[r, :m]]


def ids(*x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    from paged_kv_decode_nsv_gb300 import nsv
    return nsv.device_status(clear=True)[0]


@pytest.fixture(autouse=True)
def clean_status():
    status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kv_heads,head_dim", [(1, 64), (3, 64), (8, 128)])
@pytest.mark.parametrize("pairs", [0, 1, 7, 60])
def test_copy(dtype, kv_heads, head_dim, pairs):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    c = Cache([], 130, kv_heads, head_dim, dtype, seed=pairs)
    got = c.gpu()
    perm = c.rng.permutation(131)
    src, dst = perm[:pairs], perm[65:65 + pairs]
    if pairs > 2:
        src[2] = src[1]     # one source for two destinations
    c.k[dst], c.v[dst] = c.k[src], c.v[src]
    t = lambda a: torch.from_numpy(a.astype(np.int32)).cuda()  # noqa: E731
    nsv.blocks_copy(t(src), t(dst), got[3], got[4])
    c.same(got)
    assert status() == 0


def test_copy_skips_fillers_and_bad_ids():
    from paged_kv_decode_nsv_gb300 import nsv
    c = Cache([], 20)
    got = c.gpu()
    nsv.blocks_copy(ids(-1, 3), ids(-1, 3), got[3], got[4])
    assert status() == 0
    for s, d in ((-1, 4), (4, -1), (21, 4), (4, 21), (1 << 30, 2)):
        nsv.blocks_copy(ids(s), ids(d), got[3], got[4])
        assert status() == nsv.DEV_BAD_BLOCK
    c.same(got)


CTX = [100, 16, 33, 64, 0, 1, 257, 0, 0, 48, 0, 15]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("parents,children", [
    ([0], [4]), ([0, 0, 0], [4, 7, 8]), ([1, 3, 9], [10, 4, 7]), ([4], [7]), ([6, 11, 5], [8, 4, 10]),
    ([0, -1, 6], [7, -1, 8]),
    ([7, 0], [4, 7]),       # an empty parent that is itself a child of another fork
])
def test_fork(dtype, parents, children):
    from paged_kv_decode_nsv_gb300 import nsv
    c = Cache(CTX, 60, dtype=dtype, seed=1)
    got = c.gpu()
    c.fork(parents, children)
    nsv.rows_fork(ids(*parents), ids(*children), *got)
    c.same(got)
    assert status() == 0


def test_fork_refusals():
    from paged_kv_decode_nsv_gb300 import nsv
    for parents, children in (([0], [1]), ([0], [12]), ([12], [4]), ([-1], [4]), ([0], [-1]),
                              ([0], [0]), ([0, 6], [4, 4])):
        c = Cache(CTX, 60, seed=2)
        got = c.gpu()
        c.fork(parents, children)
        nsv.rows_fork(ids(*parents), ids(*children), *got)
        c.same(got)
        assert status() == nsv.DEV_BAD_ROW
    # two free blocks for three forks that need one each
    used = int((Cache(CTX, 60, seed=3).refs > 0).sum())
    c = Cache(CTX, used + 2, seed=3)
    got = c.gpu()
    c.fork([0, 3, 6, 2, 1], [4, 7, 8, 10, 10])
    nsv.rows_fork(ids(0, 3, 6, 2), ids(4, 7, 8, 10), *got)
    c.same(got)
    assert status() == nsv.DEV_NO_BLOCKS and c.ctx[10] == 0


@pytest.mark.parametrize("grow", [
    [0] * 12, [1] * 12, [5, 0, 31, 16, 40, 15, 0, 1, 0, 64, 17, 2], [0, 0, 0, 0, 64] + [0] * 7])
@pytest.mark.parametrize("pad", [0, 3])
def test_extend(grow, pad):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    c = Cache(CTX, 90, seed=4)
    got = c.gpu()
    starts = np.concatenate([[0], np.cumsum(grow)])
    want = c.extend(starts, int(starts[-1]) + pad)
    slots = torch.full((len(want),), -9, dtype=torch.int64, device="cuda")
    nsv.rows_extend(ids(*starts), *got[:3], slots)
    c.same(got)
    assert np.array_equal(slots.cpu().numpy(), want)
    assert status() == 0


def test_extend_refusals():
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    used = int((Cache(CTX, 90, seed=5).refs > 0).sum())

    def run(c, starts, bits, tokens=None):
        got = c.gpu()
        tokens = starts[-1] if tokens is None else tokens
        want = c.extend(starts, tokens)
        slots = torch.zeros(tokens, dtype=torch.int64, device="cuda")
        nsv.rows_extend(ids(*starts), *got[:3], slots)
        c.same(got)
        assert status() == bits
        return want, slots.cpu().numpy()

    # the rows need 1, 2, 1 and 0 blocks (100 to 120 tokens, 33 to 66, 64 to 80,
    # 15 to 16): four free ones are just enough, with three the third of them is
    # refused, with two the second, the third and the last, which needs none
    grow = [20, 0, 33, 16, 0, 0, 0, 0, 0, 0, 0, 1]
    for free, bits in ((4, 0), (3, nsv.DEV_NO_BLOCKS), (2, nsv.DEV_NO_BLOCKS)):
        want, got = run(Cache(CTX, used + free, seed=5), [0] + list(np.cumsum(grow)), bits)
        assert np.array_equal(want, got)
    # beyond the table
    c = Cache(CTX, 90, seed=5)
    grow = [c.bt.shape[1] * 16 - 100 + 1, 3] + [0] * 10
    want, got = run(c, [0] + list(np.cumsum(grow)), nsv.DEV_BAD_CTX)
    assert np.array_equal(want, got)
    # starts that are not ascending pairs within the tokens
    starts = [0, 3, 2, 2, 2, 2, 2, 2, 2, 2, 2, 2, 9]
    want, got = run(Cache(CTX, 90, seed=5), starts[:12] + [2], nsv.DEV_BAD_CHUNK, tokens=4)
    assert np.array_equal(want, got)
    # a last block that another row names too is not written into
    c = Cache(CTX, 90, seed=5)
    c.refs[c.bt[0, 6]] += 1
    dev = c.gpu()
    slots = torch.zeros(5, dtype=torch.int64, device="cuda")
    nsv.rows_extend(ids(0, *[5] * 12), *dev[:3], slots)
    c.same(dev)
    assert status() == nsv.DEV_BAD_ROW and (slots == 90 * 16).all()


@pytest.mark.parametrize("rows", [[0], [6, 2, 0, 9], [4], [0, 0, 3], [-1, 5], list(range(12))])
def test_free(rows):
    from paged_kv_decode_nsv_gb300 import nsv
    c = Cache(CTX, 60, seed=6)
    got = c.gpu()
    c.free(rows)
    nsv.rows_free(ids(*rows), *got[:3])
    c.same(got)
    assert status() == 0


def test_free_refusals():
    from paged_kv_decode_nsv_gb300 import nsv
    c = Cache(CTX, 60, seed=7)
    got = c.gpu()
    nsv.rows_free(ids(12, -2), *got[:3])
    assert status() == nsv.DEV_BAD_ROW
    c.same(got)
    got[0][3, 1] = 60           # outside the pool
    got[0][3, 2] = int(c.free_ids()[0])  # free already
    nsv.rows_free(ids(3), *got[:3])
    assert status() == nsv.DEV_BAD_BLOCK
    assert (got[2] >= 0).all() and (got[0][3, :4] == -1).all()
    got[1][0] = 1 << 20
    nsv.rows_free(ids(0), *got[:3])
    assert status() == nsv.DEV_BAD_CTX


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("blocks,freed", [(60, []), (60, [0, 2, 9]), (61, list(range(12))),
                                          (1500, [6]), (33000, [0])])
def test_compact(dtype, blocks, freed):
    from paged_kv_decode_nsv_gb300 import nsv
    c = Cache(CTX, blocks, dtype=dtype, seed=8)
    c.free(freed)
    got = c.gpu()
    c.compact()
    nsv.blocks_compact(*got)
    c.same(got, free_too=False)
    assert status() == 0
    n = int((c.refs > 0).sum())
    assert (c.refs[:n] > 0).all()


def test_many_rows_and_blocks():
    """Every operator past one warp's, one CTA's and one cluster's share."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    rng = np.random.default_rng(9)
    ctx = [int(x) for x in rng.integers(1, 120, 2500)] + [0] * 1500
    c = Cache(ctx, 40000, kv_heads=1, seed=9)
    got = c.gpu()
    parents, children = rng.integers(0, 2500, 1400), 2500 + rng.permutation(1500)[:1400]
    c.fork(parents, children)
    nsv.rows_fork(ids(*parents), ids(*children), *got)
    c.same(got)
    starts = np.concatenate([[0], np.cumsum(rng.integers(0, 30, 4000))])
    want = c.extend(starts, int(starts[-1]))
    slots = torch.zeros(len(want), dtype=torch.int64, device="cuda")
    nsv.rows_extend(ids(*starts), *got[:3], slots)
    c.same(got)
    assert np.array_equal(slots.cpu().numpy(), want)
    rows = rng.permutation(4000)[:3000]
    c.free(rows)
    nsv.rows_free(ids(*rows), *got[:3])
    c.same(got)
    c.compact()
    nsv.blocks_compact(*got)
    c.same(got, free_too=False)
    assert status() == 0


def test_captured_operators_replay():
    """One graph of extend, fork, free and compact, replayed on a restored state."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    c = Cache(CTX, 80, seed=10)
    got, keep = c.gpu(), c.gpu()
    grow = [5, 0, 31, 16, 0, 15, 0, 0, 0, 64, 0, 2]
    starts = np.concatenate([[0], np.cumsum(grow)])
    args = ids(*starts), ids(0, 6), ids(4, 7), ids(2, 9)
    slots = torch.zeros(int(starts[-1]), dtype=torch.int64, device="cuda")
    ws = torch.empty(nsv.pages_workspace_bytes(12, 80), dtype=torch.uint8, device="cuda")

    def run():
        nsv.rows_extend(args[0], *got[:3], slots, workspace=ws)
        nsv.rows_fork(args[1], args[2], *got, workspace=ws)
        nsv.rows_free(args[3], *got[:3])
        nsv.blocks_compact(*got, workspace=ws)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    c.extend(starts, int(starts[-1]))
    c.fork([0, 6], [4, 7])
    c.free([2, 9])
    c.compact()
    for _ in range(3):
        for x, y in zip(got, keep):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        c.same(got, free_too=False)
    assert status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_cache_from_prompts_to_compaction(dtype):
    """The operators together, as a server uses them: prompts are prefilled in
    chunks, rows are forked and decode on, some end, the pool is compacted and
    the rest decode on.  Every read is checked, in 64 bits, against the row's own
    tokens, which the test keeps itself."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    H, KV, D, R, NB, W = 8, 2, 64, 6, 64, 20
    tdt = torch.float32 if dtype == "f32" else torch.bfloat16
    # the tolerances of the chunk attention's tests, of the largest |v| seen
    tol = 4e-5 if dtype == "f32" else 2.0 ** -8 + 2.0 ** -12
    gen = torch.Generator().manual_seed(21)
    k_pool, v_pool = (torch.full((NB + 1, KV, 16, D), float("nan"), dtype=tdt, device="cuda")
                      for _ in range(2))
    bt = torch.full((R, W), -1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(R, dtype=torch.int32, device="cuda")
    refs = torch.zeros(NB, dtype=torch.int32, device="cuda")
    tokens = [[] for _ in range(R)]     # (k, v) of each row, on the host

    def draw(*shape):
        return torch.randn(shape, generator=gen).to(tdt)

    def step(new):
        T = sum(new)
        q, k, v = draw(T, H, D), draw(T, KV, D), draw(T, KV, D)
        starts = ids(0, *np.cumsum(new))
        slots = torch.empty(T, dtype=torch.int64, device="cuda")
        out = torch.empty(T, H, D, dtype=tdt, device="cuda")
        nsv.rows_extend(starts, bt, ctx, refs, slots)
        nsv.chunk_step(q.cuda(), k.cuda(), v.cuda(), slots, k_pool, v_pool, bt, starts, ctx,
                       D ** -0.5, out)
        out = out.double().cpu()
        at = 0
        for r, n in enumerate(new):
            for i in range(n):
                tokens[r].append((k[at + i], v[at + i]))
                ks = torch.stack([t[0] for t in tokens[r]]).double().repeat_interleave(H // KV, 1)
                vs = torch.stack([t[1] for t in tokens[r]]).double().repeat_interleave(H // KV, 1)
                s = torch.einsum("hd,thd->ht", q[at + i].double(), ks) * D ** -0.5
                want = torch.einsum("ht,thd->hd", torch.softmax(s, -1), vs)
                err = (out[at + i] - want).abs().amax(-1)
                assert (err <= tol * vs.abs().amax((0, 2))).all(), (r, i, err)
            at += n

    step([40, 0, 17, 0, 0, 130])
    step([33, 0, 1, 0, 0, 1])
    nsv.rows_fork(ids(0, 0, 5), ids(1, 3, 4), bt, ctx, refs, k_pool, v_pool)
    for p, c in ((0, 1), (0, 3), (5, 4)):
        tokens[c] = list(tokens[p])
    for _ in range(3):
        step([1, 1, 1, 1, 1, 1])
    nsv.rows_free(ids(0, 5), bt, ctx, refs)
    tokens[0], tokens[5] = [], []
    nsv.blocks_compact(bt, ctx, refs, k_pool, v_pool)
    live = int((refs > 0).sum())
    assert (refs[:live] > 0).all() and (refs[live:] == 0).all()
    k_pool[live:], v_pool[live:] = float("nan"), float("nan")   # the pool's tail is given back
    step([20, 1, 0, 5, 1, 0])
    step([1, 1, 1, 1, 1, 0])
    nsv.rows_free(ids(0, 1, 2, 3, 4, 5), bt, ctx, refs)
    assert (refs == 0).all() and (ctx == 0).all()
    assert status() == 0


def test_block_offsets_beyond_32_bits():
    """Copies and moves of blocks whose offsets pass 2^31 elements."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    blocks, shape = 140000, (8, 16, 128)
    pools = [torch.empty((blocks + 1,) + shape, dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    assert pools[0].numel() > 2 ** 31
    for i, p in enumerate(pools):
        p[0], p[-2], p[-3] = 1.0 + i, 3.0 + i, 5.0 + i
    nsv.blocks_copy(ids(blocks - 1, 0), ids(7, blocks - 9), *pools)
    for i, p in enumerate(pools):
        assert (p[7] == 3.0 + i).all() and (p[blocks - 9] == 1.0 + i).all()
    bt, ctx = ids(blocks - 2, blocks - 1).view(1, 2), ids(20)
    refs = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    refs[bt[0].long()] = 1
    nsv.blocks_compact(bt, ctx, refs, *pools)
    assert bt.tolist() == [[0, 1]] and int(refs.sum()) == 2 and refs[:2].tolist() == [1, 1]
    for i, p in enumerate(pools):
        assert (p[0] == 5.0 + i).all() and (p[1] == 3.0 + i).all()
    assert status() == 0


@pytest.mark.parametrize("grow", [[20000], [0, 700, 0, 0, 1300, 128, 129, 0, 1, 4097, 0, 257],
                                  [1] * 11 + [600], [1] * 11 + [0]])
def test_extend_by_long_prompts(grow):
    """Rows whose new tokens are dealt out in parts, beside rows of a few."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    c = Cache(CTX[:len(grow)], 2000, extra=1300, seed=10)
    got = c.gpu()
    starts = np.concatenate([[0], np.cumsum(grow)])
    want = c.extend(starts, int(starts[-1]) + 2)
    slots = torch.full((len(want),), -9, dtype=torch.int64, device="cuda")
    nsv.rows_extend(ids(*starts), *got[:3], slots)
    c.same(got)
    assert np.array_equal(slots.cpu().numpy(), want)
    assert status() == 0


@pytest.mark.parametrize("seed", range(12))
def test_random_lives(seed):
    """Random sequences of all operators on one cache, its pool nearly full."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    rng = np.random.default_rng(200 + seed)
    rows = int(rng.choice([5, 40, 300]))
    ctx = [int(x) if rng.random() < 0.6 else 0 for x in np.exp(rng.uniform(0, 6, rows))]
    need = sum(-(-c // 16) for c in ctx)
    c = Cache(ctx, need + int(rng.integers(1, rows + 4)), extra=int(rng.integers(0, 20)),
              seed=seed, dtype=DTYPES[seed % 2])
    got = c.gpu()
    for _ in range(14):
        kind = rng.choice(["extend", "extend", "fork", "free", "compact"])
        if kind == "extend":
            grow = np.where(rng.random(rows) < 0.5, 0, np.exp(rng.uniform(0, 5, rows)).astype(int))
            starts = np.concatenate([[0], np.cumsum(grow)])
            want = c.extend(starts, int(starts[-1]))
            slots = torch.zeros(len(want), dtype=torch.int64, device="cuda")
            nsv.rows_extend(ids(*starts), *got[:3], slots)
            assert np.array_equal(slots.cpu().numpy(), want)
        elif kind == "fork":
            n = int(rng.integers(1, rows + 1))
            parents, children = rng.integers(-1, rows, n), rng.integers(-1, rows, n)
            c.fork(parents, children)
            nsv.rows_fork(ids(*parents), ids(*children), *got)
        elif kind == "free":
            out = rng.integers(0, rows, int(rng.integers(1, rows // 3 + 2)))
            c.free(out)
            nsv.rows_free(ids(*out), *got[:3])
        else:
            c.compact()
            nsv.blocks_compact(*got)
            # what is free now may hold anything: the model takes it over
            for mine, dev in ((c.k, got[3]), (c.v, got[4])):
                mine[:-1][c.refs == 0] = dev.contiguous().view(len(dev), -1).view(
                    torch.int32).cpu().numpy()[:-1][c.refs == 0]
        c.same(got)


@pytest.mark.parametrize("freed", [[0, 2, 9], []])      # blocks move; none does
@pytest.mark.parametrize("bad", [-1, -7, -2 ** 31, 60, 61, 2 ** 31 - 1])
def test_compact_flags_entries_outside_the_pool(freed, bad):
    from paged_kv_decode_nsv_gb300 import nsv
    c = Cache(CTX, 60, seed=12)
    if not freed:       # the used blocks are the pool's first ones already
        c.compact()
    c.free(freed)
    got = c.gpu()
    c.compact()
    got[0][6, 3] = bad
    c.bt[6, 3] = bad
    nsv.blocks_compact(*got)
    c.same(got, free_too=False)
    assert status() == nsv.DEV_BAD_BLOCK


def test_extend_refuses_rows_that_overlap_without_end():
    """Starts that go back and forth: every other row claims all tokens.  The first is
    extended; the others' parts would add up beyond what any batch of these tokens has."""
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    R, T = 64, 20000
    c = Cache([5] * R, 100000, extra=1300, seed=13)
    got = c.gpu()
    want = c.extend([0] + [T] * R, T)
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    nsv.rows_extend(ids(*([0, T] * (R // 2) + [0])), *got[:3], slots)
    c.same(got)
    assert np.array_equal(slots.cpu().numpy(), want)
    assert status() == nsv.DEV_BAD_CHUNK
