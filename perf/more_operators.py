"""Cases that measure the rotating appends and the attention over a cache held in 4 bits.

Each case is one pass through one operator, in two forms: a plain one made of elementary torch operations, and the
library's own calls (``own``).  Kinds of case:

  rope   rotate a step's queries and keys by their positions; keys and values go to their slots of fp32 or bf16 pools
  write  the same into 4-bit pools; the values that the written slots then stand for are read back
  read   values of slots of 4-bit pools, widened to bf16 or fp32 (rows that leave the 4-bit cache)
  attend attention of new tokens (single ones, chunks, whole prompts, mixed) over a 4-bit paged cache

Layouts: q, out [tokens, heads, head_dim]; k, v [tokens, kv_heads, head_dim]; pools [blocks + 1, kv_heads, 16, head_dim],
the last block being the sink.  A 4-bit pool is uint8 [blocks + 1, kv_heads, 9 * head_dim]: 16 tokens of head_dim / 2
bytes, two e2m1 numbers each (the even dimension in the low half), then 16 tokens of head_dim / 16 e4m3 scales, one for
16 dimensions.  An element is its number times its scale times its KV head's fp32 scale (1 where there are none).  The
rotation's table is fp32 [positions, rotary_dim]: the cosines of the rotary_dim / 2 angles, then their sines.
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


def token_case(name, kind, tokens, heads, kv_heads, head_dim, dtype="bf16", rotary=0, interleaved=False, positions=8192, scaled=False,
               fused=False, mix=0):
    """`tokens` new tokens.  rotary: dimensions that the rotation takes (0: none, then `heads` is 0 too); positions: rows of
    its table; scaled: each KV head has an fp32 scale; fused: q, k and v are slices of one projection's output."""
    return {"name": name, "kind": kind, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "dtype": dtype,
            "rotary": rotary, "interleaved": interleaved, "positions": positions, "scaled": scaled, "fused": fused, "mix": mix}


def attend_case(name, rows, fresh, ctx_lo, ctx_hi, heads, kv_heads, head_dim, dtype="bf16", chunk_rows=None, cap=0.0, slopes=False,
                mask="causal", scaled=False, mix=0):
    """`rows` rows with contexts from [ctx_lo, ctx_hi]; the first `chunk_rows` of them (None: all) bring up to `fresh`
    new tokens each, the others one."""
    return {"name": name, "kind": "attend", "rows": rows, "fresh": fresh, "chunk_rows": rows if chunk_rows is None else chunk_rows,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "dtype": dtype,
            "cap": cap, "slopes": slopes, "mask": mask, "scaled": scaled, "mix": mix}


def listed():
    return [
        # The append of a decode step of 32 rows, from a fused projection: the smallest call, where latency counts.
        token_case("rope_single_tokens", "rope", 32, 32, 8, 128, rotary=128, fused=True, mix=1),
        # Prompts of 8192 tokens in all, appended in one call.
        token_case("rope_prompts", "rope", 8192, 32, 8, 128, rotary=128, fused=True, positions=32768, mix=2),
        # fp32, half of the dimensions rotated in adjacent pairs, odd sizes.
        token_case("rope_partial_f32", "rope", 1021, 12, 4, 64, dtype="f32", rotary=32, interleaved=True, mix=3),
        # The headline batch's decode step into a 4-bit cache.
        token_case("write_single_tokens", "write", 256, 32, 8, 128, rotary=128, fused=True, mix=4),
        # Long prompts into a 4-bit cache whose heads have calibrated scales.
        token_case("write_prompts", "write", 16381, 32, 8, 128, rotary=128, scaled=True, positions=32768, mix=5),
        # One short row leaves the 4-bit cache; fp32, odd number of heads.
        token_case("read_short_row", "read", 301, 0, 3, 64, dtype="f32", mix=6),
        # Rows of 65536 tokens in all leave the 4-bit cache (to be moved, or to go on in bf16).
        token_case("read_rows", "read", 65536, 0, 8, 128, scaled=True, mix=7),
        # A few interactive users, one token each over short contexts.
        attend_case("attend_few_single_tokens", 4, 1, 30, 700, 32, 8, 128, mix=8),
        # The headline decode batch: 256 rows, contexts 512 to 8192.
        attend_case("attend_decode", 256, 1, 512, 8192, 32, 8, 128, scaled=True, mix=9),
        # A 2048-token chunk at the end of a document: the largest work.
        attend_case("attend_long_chunk", 1, 2048, 32768, 32768, 32, 8, 128, mix=10),
        # A serving step that mixes one row's 509-token chunk with 32 rows that decode single tokens.
        attend_case("attend_chunk_among_decodes", 33, 509, 200, 8192, 32, 8, 128, chunk_rows=1, mix=11),
        # fp32 queries of a sliding-window model that verifies a few guessed tokens a row, capped scores; odd sizes.
        attend_case("attend_window_f32", 29, 3, 100, 6000, 20, 4, 64, dtype="f32", cap=50.0, mask="window", mix=12),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "write", "read"] + ["attend"] * 4)
    mix = rng.randrange(1 << 30)
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    head_dim = rng.choice([64, 128])
    group = rng.choice([1, 1, 2, 3, 4, 4, 5, 8, 16])
    kv = rng.choice([1, 2, 3, 4, 8])
    scaled = rng.random() < 0.5
    if kind != "attend":
        rotary = 0 if kind == "read" else rng.choice([head_dim, head_dim, head_dim, head_dim // 2, 16, 48])
        c = token_case("", kind, log_int(rng, 1, 16384 if kind == "read" else 8192), 0 if kind == "read" else group * kv, kv, head_dim, dtype,
                       rotary, rng.random() < 0.4, log_int(rng, 16, 100000), scaled and kind != "rope", rng.random() < 0.5, mix)
        del c["name"]
        return c
    heads = group * kv
    form = rng.choice(["single", "single", "few", "chunk", "mixed", "prompt"])
    rows = {"single": log_int(rng, 1, 256), "few": log_int(rng, 1, 64), "chunk": log_int(rng, 1, 12), "mixed": log_int(rng, 4, 48),
            "prompt": log_int(rng, 1, 4)}[form]
    fresh = 1 if form == "single" else rng.randint(2, 8) if form == "few" else log_int(rng, 2, 2048)
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
    c = attend_case("", rows, fresh, lo, hi, heads, kv, head_dim, dtype, 1 if form == "mixed" else rows, rng.choice([0.0, 0.0, 20.0, 50.0]),
                    rng.random() < 0.4, rng.choice(["causal", "causal", "documents", "window", "prefix"]), scaled, mix)
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


def work(case):
    """What one pass cannot do without: every input read once, every output written once."""
    elem, dim = ELEM[case["dtype"]], case["head_dim"]
    four = 9 * dim // 16  # bytes of one token and KV head of one 4-bit pool
    if case["kind"] == "attend":
        ctx, new, begin, end = chunk_lengths(case)
        seen, at = 0, 0
        for c, n in zip(ctx, new):  # positions that any of the row's new tokens sees
            edge = np.zeros(c + 1, np.int64)
            np.add.at(edge, begin[at:at + n], 1)
            np.add.at(edge, np.minimum(end[at:at + n], c), -1)
            seen += int((np.cumsum(edge)[:c] > 0).sum())
            at += n
        pairs = int((end - begin).sum())
        return {"bytes": 2 * at * case["heads"] * dim * elem + 2 * seen * case["kv_heads"] * four, "flops": 4 * pairs * case["heads"] * dim}
    n, heads, kv = case["tokens"], case["heads"], case["kv_heads"]
    if case["kind"] == "read":
        return {"bytes": n * (2 * kv * (four + dim * elem) + 8), "flops": 4 * n * kv * dim}
    rotated = n * (2 * heads * dim * elem + 2 * kv * dim * elem + 4 * case["rotary"] + 12)  # q, its result, k and v, table, positions, slots
    if case["kind"] == "rope":
        return {"bytes": rotated + n * 2 * kv * dim * elem, "flops": 3 * n * (heads + kv) * case["rotary"]}
    # stored in 4 bits, and the stored values once more as numbers
    return {"bytes": rotated + n * 2 * kv * (2 * four + dim * elem), "flops": n * (3 * (heads + kv) * case["rotary"] + 8 * kv * dim)}


# --------------------------------------------------------------------------------- 4-bit numbers, in the plain form


def codes_of(x, scales):
    """Codes (0 to 15) and e4m3 scales of x [..., head_dim] in fp32; scales broadcasts over x."""
    y = x / scales
    groups = y.view(*y.shape[:-1], -1, 16)
    s = (groups.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    w = s.float().unsqueeze(-1)
    a = groups.abs() / torch.where(w > 0, w, torch.ones_like(w))
    a = torch.where(w > 0, a, torch.zeros_like(a))
    # halfway cases go to the even code
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = code | (torch.signbit(groups).to(torch.uint8) << 3)
    return code.view(x.shape), s


def pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def unpack(data, s):
    """fp32 values of packed codes [..., head_dim / 2] and e4m3 scales [..., head_dim / 16]."""
    code = torch.stack([data & 15, data >> 4], -1).flatten(-2)
    mag = code & 7
    low = 0.5 * mag.float()  # 0, 0.5, 1, 1.5; above: 2, 3, 4, 6
    high = torch.where(mag < 6, (mag.float() - 2.0).clamp(min=0.0), 2.0 * mag.float() - 8.0)
    value = torch.where(mag < 4, low, high)
    value = torch.where(code >= 8, -value, value)
    return (value.view(*value.shape[:-1], -1, 16) * s.float().unsqueeze(-1)).flatten(-2)


def tiles(pool, dim):
    """A 4-bit pool's codes [blocks + 1, kv_heads, 16, dim / 2] and scales [blocks + 1, kv_heads, 16, dim / 16] (views)."""
    data = pool[..., :8 * dim].unflatten(-1, (BLOCK, dim // 2))
    return data, pool[..., 8 * dim:].unflatten(-1, (BLOCK, dim // 16)).view(torch.float8_e4m3fn)


# --------------------------------------------------------------------------------------------------- the inputs


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(shape, dtype, seed):
    return torch.randn(shape, generator=generator(seed), device="cuda", dtype=dtype)


def on_gpu(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a)).to(dtype).cuda()


def filled_pool(blocks, kv_heads, dim, seed):
    """A 4-bit pool of normally distributed numbers."""
    pool = torch.empty((blocks + 1, kv_heads, 9 * dim), dtype=torch.uint8, device="cuda")
    data, scale = tiles(pool, dim)
    g = generator(seed)
    step = max(1, (1 << 25) // (kv_heads * BLOCK * dim))
    for a in range(0, blocks + 1, step):
        b = min(blocks + 1, a + step)
        x = torch.randn((b - a, kv_heads, BLOCK, dim), generator=g, device="cuda")
        code, s = codes_of(x, torch.ones((), device="cuda"))
        data[a:b] = pack(code)
        scale.view(torch.uint8)[a:b] = s.view(torch.uint8)
    return pool


def head_scales(case, seed):
    if not case["scaled"]:
        return None, None
    g = generator(7 * seed + 3)
    k, v = (torch.rand(case["kv_heads"], generator=g, device="cuda") + 0.5 for _ in range(2))
    return k, 0.25 * v


def prepare(case, seed):
    dtype, dim, kv = DTYPES[case["dtype"]], case["head_dim"], case["kv_heads"]
    ks, vs = head_scales(case, seed)
    rng = np.random.default_rng([case["mix"], seed])
    if case["kind"] == "attend":
        ctx, new, begin, end = chunk_lengths(case)
        need = [cdiv(c, BLOCK) for c in ctx]
        blocks = sum(need) + sum(need) // 10 + 1
        tables, perm, at = np.full((len(ctx), max(need)), -1, np.int32), rng.permutation(blocks), 0
        for r, nb in enumerate(need):
            tables[r, :nb] = perm[at:at + nb]
            at += nb
        starts = np.concatenate([[0], np.cumsum(new)])
        heads = torch.arange(1, case["heads"] + 1, device="cuda", dtype=torch.float32)
        return {"kind": "attend", "q": normal((int(starts[-1]), case["heads"], dim), dtype, 3 * seed),
                "k_pool": filled_pool(blocks, kv, dim, 3 * seed + 1), "v_pool": filled_pool(blocks, kv, dim, 3 * seed + 2),
                "k_scales": ks, "v_scales": vs, "tables": on_gpu(tables), "starts": on_gpu(starts), "ctx": on_gpu(ctx), "scale": dim ** -0.5,
                "cap": case["cap"], "slopes": torch.exp2(-8.0 * heads / case["heads"]) if case["slopes"] else None,
                "begin": on_gpu(begin) if case["mask"] in ("documents", "window") else None,
                "end": on_gpu(end) if case["mask"] == "prefix" else None, "n_max": max(new), "l_max": max(ctx)}
    n, heads = case["tokens"], case["heads"]
    blocks = cdiv(n, BLOCK) + cdiv(n, 8 * BLOCK) + 1
    # the slots of rows: runs of a block's tokens, the blocks in any order; single tokens sit anywhere in theirs
    slots = (rng.permutation(blocks)[:cdiv(n, BLOCK), None] * BLOCK + np.arange(BLOCK)).reshape(-1)[:n]
    state = {"kind": case["kind"], "slots": on_gpu(slots, torch.int64), "k_scales": ks, "v_scales": vs, "interleaved": case["interleaved"]}
    if case["kind"] == "read":
        state.update(k_pool=filled_pool(blocks, kv, dim, 2 * seed), v_pool=filled_pool(blocks, kv, dim, 2 * seed + 1), dtype=dtype)
        return state
    if case["fused"]:
        parts = normal((n, heads + 2 * kv, dim), dtype, 5 * seed).split([heads, kv, kv], 1)
    else:
        parts = [normal((n, h, dim), dtype, 5 * seed + i) for i, h in enumerate((heads, kv, kv))]
    half, width = case["rotary"] // 2, case["positions"]
    angle = torch.arange(width, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    state.update(q=parts[0], k=parts[1], v=parts[2], positions=on_gpu(rng.integers(0, width, n)),
                 rotary=torch.cat([angle.cos(), angle.sin()], 1).float())
    if case["kind"] == "rope":
        pool = (blocks + 1, kv, BLOCK, dim)
        state.update(k_pool=normal(pool, dtype, 5 * seed + 3), v_pool=normal(pool, dtype, 5 * seed + 4))
    else:
        state.update(k_pool=filled_pool(blocks, kv, dim, 5 * seed + 3), v_pool=filled_pool(blocks, kv, dim, 5 * seed + 4))
    return state


# ---------------------------------------------------------------------------------------------- the plain forms


def rotated(x, s):
    """x [tokens, heads, head_dim] in fp32 with its first dimensions rotated; every product and sum is rounded."""
    x = x.float()
    row = s["rotary"][s["positions"].long()][:, None]
    half = row.shape[-1] // 2
    c, sn = row[..., :half], row[..., half:]
    if s["interleaved"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
    else:
        a, b = x[..., :half], x[..., half:2 * half]
    y0, y1 = a * c - b * sn, b * c + a * sn
    y = torch.stack([y0, y1], -1).flatten(-2) if s["interleaved"] else torch.cat([y0, y1], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def head_scale(t, like):
    return torch.ones((1, 1, 1), device=like.device) if t is None else t[None, :, None]


def plain_rope(s):
    blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
    s["k_pool"][blk, :, off] = rotated(s["k"], s).to(s["k"].dtype)
    s["v_pool"][blk, :, off] = s["v"]
    return {"q": rotated(s["q"], s).to(s["q"].dtype), "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def plain_read(s, dtype):
    blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
    out = {}
    for name in ("k", "v"):
        pool, scales = s[name + "_pool"], s[name + "_scales"]
        data, e4m3 = tiles(pool, pool.shape[-1] // 9)
        values = unpack(data[blk, :, off], e4m3.view(torch.uint8)[blk, :, off].view(torch.float8_e4m3fn))
        out[name] = (values * head_scale(scales, values)).to(dtype)
    return out


def plain_write(s):
    blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
    for name, x in (("k", rotated(s["k"], s)), ("v", s["v"].float())):
        code, e4m3 = codes_of(x.contiguous(), head_scale(s[name + "_scales"], x))
        data, scale = tiles(s[name + "_pool"], x.shape[-1])
        data[blk, :, off] = pack(code)
        scale.view(torch.uint8)[blk, :, off] = e4m3.view(torch.uint8)
    return {"q": rotated(s["q"], s).to(s["q"].dtype), **plain_read(s, s["q"].dtype)}


def plain_attend(s):
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
    out = torch.empty((rows, n_max, heads, dim), device=q.device)
    for h in range(kv_heads):
        k, v = (unpack(data[blocks, h], scale.view(torch.uint8)[blocks, h].view(torch.float8_e4m3fn)).reshape(rows, -1, dim)[:, :l_max]
                for data, scale in (tiles(s["k_pool"], dim), tiles(s["v_pool"], dim)))
        if s["k_scales"] is not None:
            k, v = k * s["k_scales"][h], v * s["v_scales"][h]
        x = q[tok, h * group:(h + 1) * group].float().transpose(1, 2).reshape(rows, group * n_max, dim)
        p = torch.matmul(x, k.transpose(1, 2)).mul_(s["scale"]).view(rows, group, n_max, l_max)
        if s["cap"]:
            p.div_(s["cap"]).tanh_().mul_(s["cap"])
        if s["slopes"] is not None:
            p.sub_(s["slopes"][h * group:(h + 1) * group].view(1, group, 1, 1) * (pos[..., None] - t).abs().float()[:, None])
        p.masked_fill_(~seen[:, None], -math.inf)
        top = p.amax(-1, keepdim=True)
        p.sub_(top.masked_fill_(top == -math.inf, 0.0)).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(rows, group * n_max, l_max), v).view(rows, group, n_max, dim)
        out[:, :, h * group:(h + 1) * group] = (o / total.masked_fill_(total == 0, 1.0)).transpose(1, 2)
    at = torch.arange(tokens, device=q.device)
    row = torch.searchsorted(start, at, right=True) - 1
    return out[row, at - start[row]].to(q.dtype)


def run(state):
    s = state
    if not own:
        if s["kind"] == "read":
            return plain_read(s, s["dtype"])
        return {"rope": plain_rope, "write": plain_write, "attend": plain_attend}[s["kind"]](s)
    from paged_kv_decode_nsv_gb300 import nsv
    if s["kind"] == "attend":
        return nsv.kv4_chunk(s["q"], s["k_pool"], s["v_pool"], s["tables"], s["starts"], s["ctx"], s["scale"], torch.empty_like(s["q"]),
                             k_scales=s["k_scales"], v_scales=s["v_scales"], softcap=s["cap"], slopes=s["slopes"], see_begin=s["begin"],
                             see_end=s["end"], max_new=s["n_max"])
    if s["kind"] == "rope":
        q = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
        nsv.rope_write(s["q"], s["k"], s["v"], s["positions"], s["rotary"], s["slots"], s["k_pool"], s["v_pool"], q, interleaved=s["interleaved"])
        return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    tokens, kv_heads, dim = len(s["slots"]), s["k_pool"].shape[1], s["k_pool"].shape[2] // 9
    k, v = (torch.empty((tokens, kv_heads, dim), dtype=s["dtype"] if s["kind"] == "read" else s["k"].dtype, device="cuda") for _ in range(2))
    out = {"k": k, "v": v}
    if s["kind"] == "write":
        out["q"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
        nsv.kv4_write(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], k_scales=s["k_scales"], v_scales=s["v_scales"], q=s["q"],
                      positions=s["positions"], rotary=s["rotary"], q_out=out["q"], interleaved=s["interleaved"])
    nsv.kv4_read(s["slots"], s["k_pool"], s["v_pool"], k, v, k_scales=s["k_scales"], v_scales=s["v_scales"])
    return out


# --------------------------------------------------------------------------------------- the definition in 64 bits


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]


def nearest(x, values):
    """Index of the nearest of `values` (ascending) to each x >= 0, in 64 bits; halfway cases go to the even index."""
    v = torch.tensor(values, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(v, x.contiguous()).clamp(1, len(values) - 1)
    lo = hi - 1
    below, above = x - v[lo], v[hi] - x
    return torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def to_f32(x):
    return x.float().double()


def stored(x, scales):
    """What the 4-bit cache holds for x [tokens, kv_heads, head_dim] (64 bits, fp32 values): the definition rounds the
    quotients to fp32, and the number and its scale to nearest."""
    unit = torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if scales is None else scales.double()
    y = to_f32(x / unit[:, None]).unflatten(-1, (-1, 16))
    s = torch.tensor(E4M3, dtype=torch.float64, device=x.device)[nearest(to_f32(y.abs().amax(-1) / 6), E4M3)][..., None]
    a = torch.where(s > 0, to_f32(y.abs() / s.clamp(min=2.0 ** -9)), torch.zeros_like(y))
    number = torch.tensor(E2M1, dtype=torch.float64, device=x.device)[nearest(a, E2M1)]
    return (torch.sign(y) * number * s).flatten(-2) * unit[:, None]


def turned(x, s, rounded):
    """x with its pairs turned by their positions' angles, as complex numbers' products; rounded: each product and sum
    to fp32, as the 4-bit cache's definition has it."""
    keep = to_f32 if rounded else lambda y: y
    x, row = x.double(), s["rotary"].double()[s["positions"].long()]
    half = row.shape[1] // 2
    out = x.clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        c, sn = row[:, i, None], row[:, half + i, None]
        out[..., a] = keep(keep(x[..., a] * c) - keep(x[..., b] * sn))
        out[..., b] = keep(keep(x[..., b] * c) + keep(x[..., a] * sn))
    return out


def values_of(pool, ids, h, dim):
    """64-bit values of blocks `ids` of one KV head, [len(ids) * 16, dim], by tables."""
    raw = pool[ids, h].long()
    data, scale = raw[:, :8 * dim].reshape(-1, dim // 2), raw[:, 8 * dim:].reshape(-1, dim // 16)
    number = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device=pool.device)
    width = torch.tensor(E4M3 + [math.nan] * 129, dtype=torch.float64, device=pool.device)
    return torch.stack([number[data & 15], number[data >> 4]], -1).view(-1, dim) * width[scale].repeat_interleave(16, 1)


def exact_attend(case, s):
    """Row by row and KV head by KV head: softmax over the visible positions."""
    ctx, new, begin, end = chunk_lengths(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group, dim = case["heads"] // case["kv_heads"], case["head_dim"]
    first, last = on_gpu(begin, torch.int64), on_gpu(end, torch.int64)
    at = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        ids = s["tables"][r, :cdiv(c, BLOCK)].long()
        t = torch.arange(c, device="cuda")
        for h in range(case["kv_heads"]):
            keys, values = values_of(s["k_pool"], ids, h, dim)[:c], values_of(s["v_pool"], ids, h, dim)[:c]
            if s["k_scales"] is not None:
                keys, values = keys * s["k_scales"][h].double(), values * s["v_scales"][h].double()
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


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "attend":
        return exact_attend(case, s)
    dim = case["head_dim"]
    out = {}
    if case["kind"] == "read":
        for name in ("k", "v"):
            pool, unit = s[name + "_pool"], s[name + "_scales"]
            out[name] = torch.stack([values_of(pool, torch.arange(len(pool), device="cuda"), h, dim)[s["slots"]]
                                     for h in range(case["kv_heads"])], 1)
            if unit is not None:
                out[name] = out[name] * unit.double()[:, None]
        return out
    q = turned(s["q"], s, False)
    if case["kind"] == "rope":
        pools = {}
        for name, x in (("k_pool", turned(s["k"], s, False)), ("v_pool", s["v"].double())):
            pools[name] = s[name].double()
            flat = pools[name].transpose(1, 2).reshape(-1, case["kv_heads"], dim)  # by slot
            flat[s["slots"]] = x
            pools[name] = flat.unflatten(0, (-1, BLOCK)).transpose(1, 2).contiguous()
        return {"q": q, **pools}
    return {"q": q, "k": stored(turned(s["k"], s, True), s["k_scales"]), "v": stored(s["v"].double(), s["v_scales"])}
