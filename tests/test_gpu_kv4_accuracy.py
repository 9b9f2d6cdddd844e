"""How much the attention over a 4-bit cache keeps of queries and weights that differ by
many powers of two (GPU), in the form for few query vectors and in the one for many.

Tolerances.  fp32: queries and weights are off by 2^-22 of themselves, or by 2^-51 of their
vector's largest.  Elements of 1 beside one of 2^28 are off by 2^-23 at most, 128 of them, times
keys of about 1 and the scale 2^-3.5, by less than 2^-19 together.  The scores' rounding (below
2^5 in log2 units, a few steps of 2^-24: 2^-17) is the larger, and the 4e-5 of sum p |v| that
test_gpu_kv4 derives holds both.  bf16: weights are off by 2^-11 of themselves, or by 2^-32 of
the largest; the output by 2^-8 of itself.
"""

import numpy as np
import pytest

import test_gpu_kv4 as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("new,most", [(1, 1), (3, 0), (40, 0)])
@pytest.mark.parametrize("power", [16, 22, 28])
def test_queries_beside_one_that_meets_zero_keys(head_dim, new, most, power):
    """One dimension of the queries is 2^power times the others, and 0 in every key: what the
    others say stays."""
    b = T.batch([40 + 7 * i for i in range(12)], [new] * 12, 8, 2, head_dim, "f32", seed=power)
    b["q"][..., 0] = 2.0 ** power
    b["k"][:, :, :8 * head_dim:head_dim // 2] &= 0xf0
    T.check(b, "f32", max_new=most)


def far_weights(dtype, new, positions, bits):
    """A batch of one row in which every 32nd position has a large weight and values of 2^-10,
    and the others have weights of about 2^-bits of it and values of 2688."""
    import torch
    heads, kv_heads, dim = 8, 2, 64
    b = T.batch([positions], [new], heads, kv_heads, dim, dtype)
    k, v = (np.zeros(b[n].shape, np.uint8) for n in ("k", "v"))
    tables = b["bt"].cpu().numpy()
    t = np.arange(positions)
    block, off = tables[0, t // 16], t % 16
    for i, o, large in zip(block, off, t % 32 == 0):
        numbers, scales = o * dim // 2, 8 * dim + o * dim // 16
        v[i, :, numbers:numbers + dim // 2] = 0x11 if large else 0x77       # 0.5 or 6
        v[i, :, scales:scales + dim // 16] = 0x01 if large else 0x7e        # 2^-9 or 448
        if large:
            k[i, :, numbers], k[i, :, scales] = 7, 0x38                     # the first dimension: 6
    q = torch.zeros(b["q"].shape)
    apart = bits + 0.11 * torch.arange(heads)     # log2
    q[..., 0] = apart * np.log(2.0) / (6 * b["scale"])
    b.update(q=q.to(b["q"].dtype).cuda(), k=torch.from_numpy(k).cuda(), v=torch.from_numpy(v).cuda())
    return b


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,most", [(1, 1), (3, 0), (40, 0)])
@pytest.mark.parametrize("bits", [18, 24, 27, 30])
def test_small_weights_of_large_values(dtype, new, most, bits):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    n = 1024
    b = far_weights(dtype, new, n, bits)
    see_end = torch.full((new,), n, dtype=torch.int32, device="cuda")
    ref, big = T.reference(b, see_end=see_end)
    nsv.device_status(clear=True)
    out = T.call(b, torch.empty_like(b["q"]), max_new=most, see_end=see_end)
    assert nsv.device_status(clear=True)[0] == 0
    tol = (T.F32_TOL if dtype == "f32" else T.BF16_TOL) * big
    if dtype == "bf16":
        # (32 large weights share the sum, each 1/32 of it at most)
        tol = tol + 2.0 ** -32 / 32 * n * 2688.0
    assert ((out.double() - ref).abs().amax(-1) <= tol).all()
