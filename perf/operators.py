"""Cases that measure the chunk attention and the page operators of the paged KV cache.

Each case is one call of one operator, in two forms: a plain one made of elementary torch operations, and the
library's own call (``own``).  Kinds of case:

  chunk    attention of new tokens (whole prompts, chunks of long ones, single tokens, mixed in one batch) over a
           paged cache, causal; with ``cap``, ``slopes``, ``mask`` its scores are capped by a tanh, get a bias that
           falls with distance, or see a document, a sliding window or a shared prefix only
  copy     blocks copied to other blocks of the pool
  fork     rows that start as copies of others: full blocks shared, the last partial block copied
  extend   rows that grow: free blocks are dealt out, and every new token gets its write slot
  free     rows that end: their blocks lose a reference
  compact  live blocks moved to the front of the pool, tables renumbered

Layouts: q, out [tokens, heads, head_dim]; pools [blocks + 1, kv_heads, 16, head_dim], the last block being the sink;
block_tables [rows, max_blocks] int32; context_lens [rows] int32 (the new tokens counted); chunk_starts [rows + 1]
int32 (row r's new tokens are chunk_starts[r] .. chunk_starts[r + 1]); block_refs [blocks] int32, the number of table
entries that name each block (0: free).
"""

import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELEM = {"bf16": 2, "f32": 4}


def cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------------------------------ the cases


def chunk_case(name, rows, fresh, ctx_lo, ctx_hi, heads, kv_heads, head_dim, dtype="bf16", chunk_rows=None, cap=0.0,
               slopes=False, mask="causal", mix=0):
    """`rows` rows with contexts from [ctx_lo, ctx_hi]; the first `chunk_rows` of them (None: all) bring up to `fresh`
    new tokens each, the others one."""
    return {"name": name, "kind": "chunk", "rows": rows, "fresh": fresh, "chunk_rows": rows if chunk_rows is None else chunk_rows,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "dtype": dtype,
            "cap": cap, "slopes": slopes, "mask": mask, "mix": mix}


def page_case(name, kind, rows, count, ctx_lo, ctx_hi, kv_heads, head_dim, dtype="bf16", blocks=0, mix=0):
    """`rows` rows with contexts from [ctx_lo, ctx_hi] in a pool of `blocks` blocks (0: what they need and a quarter
    more); `count`: the pairs copied, forks made, rows freed, or the most tokens that a row grows by."""
    return {"name": name, "kind": kind, "rows": rows, "count": count, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "kv_heads": kv_heads,
            "head_dim": head_dim, "dtype": dtype, "blocks": blocks, "mix": mix}


def listed():
    return [
        # A few interactive users, one token each over short contexts: the smallest call, where latency counts.
        chunk_case("few_single_tokens", 4, 1, 30, 700, 32, 8, 128, mix=1),
        # A fresh prompt of 2048 tokens, prefilled in one call.
        chunk_case("whole_prompt", 1, 2048, 2048, 2048, 32, 8, 128, mix=2),
        # A serving step that mixes one row's 509-token chunk with 32 rows that decode single tokens.
        chunk_case("chunk_among_decodes", 33, 509, 200, 8192, 32, 8, 128, chunk_rows=1, mix=3),
        # A 4096-token chunk at the end of a long document: the largest work.
        chunk_case("long_context_chunk", 1, 4096, 32768, 32768, 32, 8, 128, mix=4),
        # The headline decode batch (256 rows, contexts 512 to 8192) with capped scores and a distance bias.
        chunk_case("capped_biased_decode", 256, 1, 512, 8192, 32, 8, 128, cap=50.0, slopes=True, mix=5),
        # Documents packed into two rows of one batch; a token sees its own document only.
        chunk_case("packed_documents", 2, 4099, 4099, 6000, 32, 32, 64, mask="documents", mix=6),
        # fp32 with a shared prefix that all tokens see in full, and a distance bias; odd sizes.
        chunk_case("shared_prefix_f32", 3, 257, 300, 2048, 12, 4, 128, dtype="f32", slopes=True, mask="prefix", mix=7),
        # Swapping rows in: 2048 block pairs of a grouped-query pool.
        page_case("copy_blocks", "copy", 0, 2048, 0, 0, 8, 128, blocks=8192, mix=8),
        # Beam search: 64 children of 64 rows with contexts up to 8192.
        page_case("fork_beams", "fork", 128, 64, 512, 8192, 8, 128, mix=9),
        # The blocks and write slots of a serving step: 256 rows that grow by up to 64 tokens.
        page_case("extend_batch", "extend", 256, 64, 512, 8192, 8, 128, mix=10),
        # Half of a batch of 256 rows has ended.
        page_case("free_half", "free", 256, 128, 512, 8192, 8, 128, mix=11),
        # A half-empty pool is packed before it is shrunk: about a quarter of its blocks move.
        page_case("compact_half_empty", "compact", 256, 0, 512, 8192, 8, 128, blocks=80000, mix=12),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["chunk"] * 8 + ["copy", "fork", "extend", "free", "compact"])
    mix = rng.randrange(1 << 30)
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    head_dim = rng.choice([64, 128])
    if kind != "chunk":
        kv = rng.choice([1, 2, 4, 8])
        rows = 0 if kind == "copy" else log_int(rng, 2, 300)
        lo = log_int(rng, 1, 500)
        hi = log_int(rng, lo, 8192)
        blocks = log_int(rng, 64, 20000) if kind == "copy" else 0
        count = {"copy": log_int(rng, 1, max(1, blocks // 2)), "fork": log_int(rng, 1, max(1, rows // 2)), "extend": log_int(rng, 1, 512),
                 "free": log_int(rng, 1, max(1, rows // 2)), "compact": 0}[kind]
        if kind == "compact":
            blocks = int(rows * cdiv(hi, BLOCK) * rng.uniform(1.1, 2.0)) + 1
        c = page_case("", kind, rows, count, lo, hi, kv, head_dim, dtype, blocks, mix)
        del c["name"]
        return c
    group = rng.choice([1, 1, 2, 3, 4, 4, 5, 8, 16])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = group * kv
    form = rng.choice(["single", "chunk", "mixed", "prompt"])
    rows = {"single": log_int(rng, 1, 256), "chunk": log_int(rng, 1, 12), "mixed": log_int(rng, 4, 48), "prompt": log_int(rng, 1, 4)}[form]
    fresh = 1 if form == "single" else log_int(rng, 2, 2048)
    hi = log_int(rng, max(fresh, 16), 16384)
    lo = hi if form == "prompt" else log_int(rng, 1, hi)
    if form == "prompt":
        fresh = hi = lo = min(hi, 4096)
    # the plain form's padded scores and gathered keys stay below those of the largest listed cases
    most = 1.0e9 if dtype == "f32" else 2.0e9
    while rows > 1 and (rows * fresh * heads * hi > most or rows * hi * kv * head_dim > 1e9):
        rows = max(1, rows // 2)
    while rows * fresh * heads * hi > most:
        fresh = max(1, fresh // 2)
        if form == "prompt":
            hi = lo = fresh
    c = chunk_case("", rows, fresh, lo, hi, heads, kv, head_dim, dtype, 1 if form == "mixed" else rows,
                   rng.choice([0.0, 0.0, 20.0, 50.0]), rng.random() < 0.4, rng.choice(["causal", "causal", "documents", "window", "prefix"]), mix)
    del c["name"]
    return c


# ----------------------------------------------------------------------------- sizes that follow from a case alone


def chunk_lengths(case):
    """Each row's context and new tokens, and each new token's first and last + 1 visible position."""
    rng = random.Random(case["mix"])
    ctx, new, begin, end = [], [], [], []
    for r in range(case["rows"]):
        c = case["ctx_hi"] if r == 0 else log_int(rng, case["ctx_lo"], case["ctx_hi"])
        n = min(c, case["fresh"] if r < case["chunk_rows"] else 1)
        if r and n > 1 and case["ctx_lo"] < case["ctx_hi"]:
            n = rng.randint(max(1, n // 2), n)  # ragged chunks
        ctx.append(c)
        new.append(n)
        pos = np.arange(c - n, c)
        b, e = np.zeros(n, np.int64), pos + 1
        if case["mask"] == "documents":
            cuts, at = [0], 0
            while at < c:
                at += log_int(rng, 40, 2000)
                cuts.append(at)
            cuts = np.array(cuts)
            b = cuts[np.searchsorted(cuts, pos, side="right") - 1]
        elif case["mask"] == "window":
            b = np.maximum(0, pos + 1 - log_int(rng, 16, 4096))
        elif case["mask"] == "prefix":
            e = np.maximum(e, rng.randint(1, c))
        begin.append(b)
        end.append(e)
    return ctx, new, np.concatenate(begin), np.concatenate(end)


def page_rows(case):
    """Contexts of the rows and how many leading blocks each shares with the row before it."""
    rng = random.Random(case["mix"])
    ctx, shared = [], []
    for r in range(case["rows"]):
        c = log_int(rng, case["ctx_lo"], case["ctx_hi"])
        if case["kind"] == "fork" and r >= case["rows"] - case["count"]:
            c = 0  # the children to be
        full = min(c, ctx[-1]) // BLOCK if r else 0
        shared.append(rng.randint(0, full) if r % 4 == 3 else 0)
        ctx.append(c)
    return ctx, shared


def page_blocks(case):
    if case["blocks"]:
        return case["blocks"]
    ctx, shared = page_rows(case)
    used = sum(cdiv(c, BLOCK) - s for c, s in zip(ctx, shared))
    more = case["rows"] * cdiv(case["count"], BLOCK) + case["rows"] if case["kind"] == "extend" else case["count"]
    return used + max(used // 4, more) + 1


def block_bytes(case):
    return 2 * case["kv_heads"] * BLOCK * case["head_dim"] * ELEM[case["dtype"]]


def work(case):
    """What one pass cannot do without: every input read once, every output written once."""
    if case["kind"] == "chunk":
        ctx, new, begin, end = chunk_lengths(case)
        seen, at = 0, 0
        for c, n in zip(ctx, new):  # positions that any of the row's new tokens sees
            edge = np.zeros(c + 1, np.int64)
            np.add.at(edge, begin[at:at + n], 1)
            np.add.at(edge, np.minimum(end[at:at + n], c), -1)
            seen += int((np.cumsum(edge)[:c] > 0).sum())
            at += n
        pairs = int((end - begin).sum())
        elem = ELEM[case["dtype"]]
        return {"bytes": 2 * at * case["heads"] * case["head_dim"] * elem + 2 * seen * case["kv_heads"] * case["head_dim"] * elem,
                "flops": 4 * pairs * case["heads"] * case["head_dim"]}
    ctx, shared = page_rows(case)
    refs = 4 * page_blocks(case)
    if case["kind"] == "copy":
        return {"bytes": 2 * case["count"] * block_bytes(case) + 8 * case["count"], "flops": 0}
    if case["kind"] == "fork":
        parents = fork_list(case, ctx)
        moved = sum(1 for p in parents if ctx[p] % BLOCK)
        return {"bytes": refs + 2 * moved * block_bytes(case) + 8 * sum(cdiv(ctx[p], BLOCK) for p in parents), "flops": 0}
    if case["kind"] == "extend":
        grow = extend_list(case)
        return {"bytes": refs + 8 * sum(grow) + 8 * case["rows"], "flops": 0}
    if case["kind"] == "free":
        return {"bytes": sum(16 * cdiv(ctx[r], BLOCK) + 8 for r in free_list(case)), "flops": 0}
    live = page_state(case)[1] > 0
    moved = int(live[int(live.sum()):].sum())
    return {"bytes": 2 * moved * block_bytes(case) + refs + 8 * sum(cdiv(c, BLOCK) for c in ctx), "flops": 0}


def fork_list(case, ctx):
    """The parent of each fork; the children are the last `count` rows, which are empty."""
    rng = random.Random(case["mix"] + 1)
    alive = [r for r, c in enumerate(ctx) if c]
    return [rng.choice(alive) for _ in range(case["count"])]


def extend_list(case):
    rng = random.Random(case["mix"] + 1)
    return [rng.randint(0, case["count"]) for _ in range(case["rows"])]


def free_list(case):
    return random.Random(case["mix"] + 1).sample(range(case["rows"]), case["count"])


# --------------------------------------------------------------------------------------------------- the inputs


def deal(ctx, shared, blocks, width, rng):
    """Block tables over a shuffled pool, and the references to each block."""
    perm, at = rng.permutation(blocks).astype(np.int32), 0
    tables = np.full((len(ctx), width), -1, np.int32)
    for r, c in enumerate(ctx):
        nb, sh = cdiv(c, BLOCK), shared[r]
        tables[r, :sh] = tables[r - 1, :sh]
        tables[r, sh:nb] = perm[at:at + nb - sh]
        at += nb - sh
    named = np.concatenate([tables[r, :cdiv(c, BLOCK)] for r, c in enumerate(ctx)]) if len(ctx) else np.zeros(0, np.int32)
    return tables, np.bincount(named, minlength=blocks).astype(np.int32)


def page_state(case, seed=0):
    ctx, shared = page_rows(case)
    more = case["count"] if case["kind"] == "extend" else 0
    width = max([cdiv(c + more, BLOCK) for c in ctx] + [1])
    # what compact has to move is part of its case; elsewhere the seed deals the blocks
    return deal(ctx, shared, page_blocks(case), width, np.random.default_rng([case["mix"], 0 if case["kind"] == "compact" else seed]))


def normal(shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16)


def on_gpu(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a)).to(dtype).cuda()


def prepare(case, seed):
    dtype = DTYPES[case["dtype"]]
    if case["kind"] == "chunk":
        ctx, new, begin, end = chunk_lengths(case)
        need = sum(cdiv(c, BLOCK) for c in ctx)
        blocks = need + need // 10 + 1
        width = cdiv(max(ctx), BLOCK)
        tables, _ = deal(ctx, [0] * len(ctx), blocks, width, np.random.default_rng([case["mix"], seed]))
        starts = np.concatenate([[0], np.cumsum(new)])
        pool = (blocks + 1, case["kv_heads"], BLOCK, case["head_dim"])
        heads = torch.arange(1, case["heads"] + 1, device="cuda", dtype=torch.float32)
        return {"kind": "chunk", "q": normal((int(starts[-1]), case["heads"], case["head_dim"]), dtype, 3 * seed),
                "k_pool": normal(pool, dtype, 3 * seed + 1), "v_pool": normal(pool, dtype, 3 * seed + 2),
                "tables": on_gpu(tables), "starts": on_gpu(starts), "ctx": on_gpu(ctx), "scale": case["head_dim"] ** -0.5,
                "cap": case["cap"], "slopes": torch.exp2(-8.0 * heads / case["heads"]) if case["slopes"] else None,
                "begin": on_gpu(begin) if case["mask"] in ("documents", "window") else None,
                "end": on_gpu(end) if case["mask"] == "prefix" else None, "n_max": max(new), "l_max": max(ctx)}
    ctx, _ = page_rows(case)
    tables, refs = page_state(case, seed)
    blocks = len(refs)
    state = {"kind": case["kind"], "tables": on_gpu(tables), "ctx": on_gpu(ctx), "refs": on_gpu(refs)}
    rng = np.random.default_rng([case["mix"], seed, 1])
    if case["kind"] in ("copy", "fork", "compact"):
        pool = (blocks + 1, case["kv_heads"], BLOCK, case["head_dim"])
        state.update(k_pool=normal(pool, dtype, 2 * seed), v_pool=normal(pool, dtype, 2 * seed + 1))
    if case["kind"] == "copy":
        perm = rng.permutation(blocks)
        state.update(src=on_gpu(perm[:case["count"]]), dst=on_gpu(perm[blocks - case["count"]:]))
    elif case["kind"] == "fork":
        parents, n = fork_list(case, ctx), case["count"]
        order = rng.permutation(n)
        state.update(parents=on_gpu(np.array(parents)[order]), children=on_gpu(case["rows"] - n + rng.permutation(n)))
    elif case["kind"] == "extend":
        grow = np.array(extend_list(case))[rng.permutation(case["rows"])]
        state.update(starts=on_gpu(np.concatenate([[0], np.cumsum(grow)])), tokens=int(grow.sum()))
    elif case["kind"] == "free":
        state.update(rows=on_gpu(np.array(free_list(case))[rng.permutation(case["count"])]))
    return state


# ---------------------------------------------------------------------------------------------- the plain forms


def plain_chunk(s):
    q, n_max, l_max = s["q"], s["n_max"], s["l_max"]
    tokens, heads, dim = q.shape
    kv_heads, rows = s["k_pool"].shape[1], s["tables"].shape[0]
    group = heads // kv_heads
    start, ctx = s["starts"].long(), s["ctx"].long()
    n = start[1:] - start[:-1]
    j = torch.arange(n_max, device=q.device)
    t = torch.arange(l_max, device=q.device)
    have = j < n[:, None]
    tok = (start[:-1, None] + j).clamp(max=tokens - 1)
    pos = (ctx - n)[:, None] + j
    end = torch.minimum(s["end"][tok].long() if s["end"] is not None else pos + 1, ctx[:, None])
    seen = (t < end[..., None]) & have[..., None]
    if s["begin"] is not None:
        seen &= t >= s["begin"][tok].long()[..., None]
    blocks = s["tables"][:, :cdiv(l_max, BLOCK)].clamp(min=0).long()
    k = s["k_pool"][blocks].transpose(1, 2).reshape(rows, kv_heads, -1, dim)[:, :, :l_max].float()
    v = s["v_pool"][blocks].transpose(1, 2).reshape(rows, kv_heads, -1, dim)[:, :, :l_max].float()
    x = q[tok].float().view(rows, n_max, kv_heads, group, dim).permute(0, 2, 3, 1, 4).reshape(rows, kv_heads, group * n_max, dim)
    p = torch.matmul(x, k.transpose(2, 3)).mul_(s["scale"]).view(rows, kv_heads, group, n_max, l_max)
    if s["cap"]:
        p.div_(s["cap"]).tanh_().mul_(s["cap"])
    if s["slopes"] is not None:
        p.sub_(s["slopes"].view(1, kv_heads, group, 1, 1) * (pos[..., None] - t).abs().float()[:, None, None])
    p.masked_fill_(~seen[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(top.masked_fill_(top == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(rows, kv_heads, group * n_max, l_max), v).view(rows, kv_heads, group, n_max, dim)
    o = (o / total.masked_fill_(total == 0, 1.0)).permute(0, 3, 1, 2, 4).reshape(rows, n_max, heads, dim)
    at = torch.arange(tokens, device=q.device)
    row = torch.searchsorted(start, at, right=True) - 1
    return o[row, at - start[row]].to(q.dtype)


def walked(tables, ctx):
    """Which table entries are in use."""
    return torch.arange(tables.shape[1], device=tables.device) < ((ctx + BLOCK - 1) // BLOCK)[:, None]


def plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    s["k_pool"][dst] = s["k_pool"][src]
    s["v_pool"][dst] = s["v_pool"][src]
    return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def plain_fork(s):
    tables, ctx, refs = s["tables"].clone(), s["ctx"].clone(), s["refs"].clone()
    parents, children = s["parents"].long(), s["children"].long()
    length = ctx[parents].long()
    need = (length % BLOCK != 0).long()
    taken = torch.cumsum(need, 0)
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)
    ok = taken <= (refs == 0).sum()
    fresh = free[(taken - need).clamp(max=refs.numel() - 1)]
    last = length // BLOCK
    col = torch.arange(tables.shape[1], device=tables.device)
    from_parent = tables[parents].long()
    line = torch.where((col == last[:, None]) & (need == 1)[:, None], fresh[:, None], from_parent)
    used = (col < ((length + BLOCK - 1) // BLOCK)[:, None]) & ok[:, None]
    refs.index_add_(0, torch.where(used, line, 0).reshape(-1), used.reshape(-1).to(refs.dtype))
    tables[children] = torch.where(used, line, tables[children].long()).to(tables.dtype)
    ctx[children] = torch.where(ok, length, ctx[children].long()).to(ctx.dtype)
    moves = (need == 1) & ok
    sink = s["k_pool"].shape[0] - 1
    src = torch.where(moves, from_parent.gather(1, last[:, None].clamp(max=tables.shape[1] - 1))[:, 0], sink)
    dst = torch.where(moves, fresh, sink)
    s["k_pool"][dst] = s["k_pool"][src]
    s["v_pool"][dst] = s["v_pool"][src]
    return {"tables": tables, "ctx": ctx, "refs": refs, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def plain_extend(s):
    tables, refs, old = s["tables"], s["refs"], s["ctx"].long()
    start, blocks = s["starts"].long(), s["refs"].numel()
    n = start[1:] - start[:-1]
    had, will = (old + BLOCK - 1) // BLOCK, (old + n + BLOCK - 1) // BLOCK
    taken = torch.cumsum(will - had, 0)
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)
    ok = taken <= (refs == 0).sum()
    col = torch.arange(tables.shape[1], device=tables.device)
    new = (col >= had[:, None]) & (col < will[:, None]) & ok[:, None]
    rank = (taken - (will - had))[:, None] + col - had[:, None]
    fresh = free[rank.clamp(0, blocks - 1)]
    tables = torch.where(new, fresh, tables.long())
    refs = refs.index_add(0, torch.where(new, fresh, 0).reshape(-1), new.reshape(-1).to(refs.dtype))
    at = torch.arange(s["tokens"], device=tables.device)
    row = torch.searchsorted(start, at, right=True) - 1
    pos = old[row] + at - start[row]
    slots = torch.where(ok[row], tables[row, (pos // BLOCK).clamp(max=tables.shape[1] - 1)] * BLOCK + pos % BLOCK, blocks * BLOCK)
    return {"tables": tables.to(torch.int32), "ctx": torch.where(ok, old + n, old).to(torch.int32), "refs": refs, "slots": slots}


def plain_free(s):
    tables, ctx, refs = s["tables"], s["ctx"], s["refs"]
    gone = torch.zeros_like(ctx, dtype=torch.bool)
    gone[s["rows"].long()] = True
    used = walked(tables, ctx) & gone[:, None]
    refs = refs.index_add(0, torch.where(used, tables, 0).reshape(-1), -used.reshape(-1).to(refs.dtype))
    return {"tables": tables.masked_fill(used, -1), "ctx": ctx.masked_fill(gone, 0), "refs": refs}


def plain_compact(s):
    tables, ctx, refs = s["tables"], s["ctx"], s["refs"].clone()
    ids = torch.arange(refs.numel(), device=refs.device)
    live = refs > 0
    front = ids < live.sum()
    src, dst = (live & ~front).nonzero()[:, 0], (~live & front).nonzero()[:, 0]
    s["k_pool"][dst] = s["k_pool"][src]
    s["v_pool"][dst] = s["v_pool"][src]
    to = ids.index_copy(0, src, dst)
    tables = torch.where(walked(tables, ctx), to[tables.clamp(min=0).long()].to(tables.dtype), tables)
    refs[dst] = refs[src]
    refs[src] = 0
    return {"tables": tables, "refs": refs, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


PLAIN = {"chunk": plain_chunk, "copy": plain_copy, "fork": plain_fork, "extend": plain_extend, "free": plain_free, "compact": plain_compact}


def run(state):
    s = state
    if not own:
        return PLAIN[s["kind"]](s)
    from paged_kv_decode_nsv_gb300 import nsv
    if s["kind"] == "chunk":
        return nsv.paged_chunk(s["q"], s["k_pool"], s["v_pool"], s["tables"], s["starts"], s["ctx"], s["scale"], torch.empty_like(s["q"]),
                               softcap=s["cap"], slopes=s["slopes"], see_begin=s["begin"], see_end=s["end"])
    if s["kind"] == "copy":
        nsv.blocks_copy(s["src"], s["dst"], s["k_pool"], s["v_pool"])
        return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    # these change the tables, lengths and references in place: the state's own stay as they are for the next pass
    tables, ctx, refs = s["tables"].clone(), s["ctx"].clone(), s["refs"].clone()
    if s["kind"] == "fork":
        nsv.rows_fork(s["parents"], s["children"], tables, ctx, refs, s["k_pool"], s["v_pool"])
        return {"tables": tables, "ctx": ctx, "refs": refs, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if s["kind"] == "extend":
        slots = torch.empty(s["tokens"], dtype=torch.int64, device=tables.device)
        nsv.rows_extend(s["starts"], tables, ctx, refs, slots)
        return {"tables": tables, "ctx": ctx, "refs": refs, "slots": slots}
    if s["kind"] == "free":
        nsv.rows_free(s["rows"], tables, ctx, refs)
        return {"tables": tables, "ctx": ctx, "refs": refs}
    nsv.blocks_compact(tables, ctx, refs, s["k_pool"], s["v_pool"])
    return {"tables": tables, "refs": refs, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


# --------------------------------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    """Row by row and KV head by KV head: softmax over the visible positions, in 64 bits.  The page operators return
    whole numbers and copied values, which have none to compute."""
    if case["kind"] != "chunk":
        return None
    s = prepare(case, seed)
    ctx, new, begin, end = chunk_lengths(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv_heads"]
    first, last = on_gpu(begin, torch.int64), on_gpu(end, torch.int64)
    at = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        ids = s["tables"][r, :cdiv(c, BLOCK)].long()
        t = torch.arange(c, device="cuda")
        for h in range(case["kv_heads"]):
            keys = s["k_pool"][ids, h].reshape(-1, case["head_dim"])[:c].double()
            values = s["v_pool"][ids, h].reshape(-1, case["head_dim"])[:c].double()
            for a in range(0, n, 1024):  # slices of the new tokens, to bound the scores' memory
                b = min(n, a + 1024)
                pos = torch.arange(c - n + a, c - n + b, device="cuda")
                hidden = (t < first[at + a:at + b, None]) | (t >= last[at + a:at + b, None])
                for g in range(h * group, (h + 1) * group):
                    x = s["q"][at + a:at + b, g].double() @ keys.T * s["scale"]
                    if case["cap"]:
                        x = case["cap"] * torch.tanh(x / case["cap"])
                    if case["slopes"]:
                        x = x - s["slopes"][g].double() * (pos[:, None] - t).abs()
                    x = x.masked_fill(hidden, -math.inf)
                    out[at + a:at + b, g] = torch.softmax(x, -1) @ values
        at += n
    return out
