"""The attention over a 4-bit cache at the ends of what its arguments may be (GPU): head scales
from 2^-60 to 2^60, for keys or values alone too, and queries of thousands."""

import pytest

import test_gpu_kv4 as T

pytestmark = pytest.mark.gpu

# whole and cut rows in the form for few query vectors and in the one for many
BATCHES = [([300, 33, 700], [1, 1, 1], 1), ([20000], [1], 1), ([300, 150], [90, 40], 0), ([9000], [300], 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["plain", "both"])
@pytest.mark.parametrize("powers", [(-60, 60), (60, -60), (-60, None), (None, 60), (None, -60)])
@pytest.mark.parametrize("mix", range(len(BATCHES)))
def test_head_scales_of_powers_of_two_change_no_digit(dtype, form, powers, mix):
    """Keys times 2^a under queries times 2^-a give the same weights, and values times 2^b the
    same outputs times 2^b, bit for bit: nothing on the way leaves fp32's range."""
    import torch
    ctx, new, most = BATCHES[mix]
    b = T.batch(ctx, new, 8, 2, 128, dtype, seed=mix)
    scores = {}
    if form == "both":
        scores = dict(softcap=20.0, slopes=torch.exp2(-torch.arange(1.0, 9.0)).cuda())
    want = T.check(b, dtype, max_new=most, **scores)
    k, v = powers
    # (heads of different scales: each its own)
    unit = lambda p: None if p is None else torch.tensor([2.0 ** p, 2.0 ** (p // 2)]).cuda()  # noqa: E731
    b["units"] = [unit(k), unit(v)]
    each = lambda u: (torch.ones(2).cuda() if u is None else u).repeat_interleave(4)[:, None]  # noqa: E731
    b["q"] = (b["q"].float() / each(b["units"][0])).to(b["q"].dtype)
    out = T.call(b, torch.empty_like(b["q"]), max_new=most, **scores)
    assert torch.equal(out.float(), want.float() * each(b["units"][1]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("units", [((1.1e-18, 3.0), None), (None, (9.7e17, 1.1e-5)), ((9.7e17, 0.7), (1.1e-18, 7.0))])
@pytest.mark.parametrize("mix", range(len(BATCHES)))
def test_head_scales_of_any_size(dtype, units, mix):
    import torch
    ctx, new, most = BATCHES[mix]
    b = T.batch(ctx, new, 8, 2, 128, dtype, seed=mix)
    b["units"] = [None if u is None else torch.tensor(u).cuda() for u in units]
    if units[0] is not None:
        each = b["units"][0].repeat_interleave(4)[:, None]
        b["q"] = (b["q"].float() / each).to(b["q"].dtype)
    T.check(b, dtype, max_new=most)


def scores_of(b):
    """Each token's and head's scores in 64 bits [heads, positions] with -inf where it does not
    see, and its sums of |q_i k_i|."""
    import torch
    kp, at = T.values(b["k"], None), 0
    for r, (c, n) in enumerate(zip(*b["lens"])):
        ids = b["bt"][r, :-(-c // 16)].long()
        k = kp[ids].transpose(1, 2).reshape(-1, kp.shape[1], kp.shape[3])[:c].repeat_interleave(b["group"], 1)
        for i in range(n):
            q, see = b["q"][at + i].double(), c - n + i + 1
            yield at + i, (torch.einsum("hd,thd->ht", q, k[:see]) * b["scale"],
                           torch.einsum("hd,thd->ht", q.abs(), k[:see].abs()) * b["scale"])
        at += n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [300.0, 1e4])
@pytest.mark.parametrize("new,most", [(1, 1), (40, 0)])
def test_one_position_takes_the_weight_of_large_queries(dtype, size, new, most):
    """A score is off by the rounding of its factors and of at most 32 partial sums, each 2^-22
    of sum |q_i k_i| at most: e = 2^-17 of that.  Where the best position is ahead of all others
    by 2 e + 30, their weights are below e^-30 each, and the output is its value, with the
    ordinary tolerance."""
    import torch
    b = T.batch([400, 90, 1000], [new] * 3, 8, 2, 128, dtype, seed=int(size))
    b["q"] = (b["q"].float() * size).to(b["q"].dtype)
    out = T.call(b, torch.empty_like(b["q"]), max_new=most)
    ref, big = T.reference(b)
    err = (out.double() - ref).abs().amax(-1)
    tol = (T.F32_TOL if dtype == "f32" else T.BF16_TOL) * big
    held = 0
    for i, (s, total) in scores_of(b):
        top = s.topk(2, -1).values
        clear = top[:, 0] - top[:, 1] > 2 * 2.0 ** -17 * total.amax(-1) + 30
        held += int(clear.sum())
        assert (err[i][clear] <= tol[i][clear]).all()
    assert held > 0.6 * err.numel()
