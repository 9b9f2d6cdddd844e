"""Rotated queries and keys are the definition's bit for bit (GPU): every product and sum of a
pair rounded to fp32 on its own, then once to the element type."""

import numpy as np
import pytest

import test_gpu_rope as T

pytestmark = pytest.mark.gpu


def rotated(x, b, interleaved):
    """x [tokens, heads, head_dim] in fp32 arithmetic without multiply-adds, as x's type."""
    import torch
    y = x.float().cpu().numpy().copy()
    row = b["table"].cpu().numpy()[b["positions"].cpu().numpy()][:, None]
    half = row.shape[-1] // 2
    c, s = row[..., :half], row[..., half:]
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    e, f = y[..., ia].copy(), y[..., ib].copy()
    assert c.dtype == e.dtype == np.float32
    y[..., ia] = e * c - f * s
    y[..., ib] = f * c + e * s
    return torch.from_numpy(y).to(x.dtype).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,kv_heads,head_dim", [(5, 1, 128), (6, 3, 64), (40, 8, 128)])
@pytest.mark.parametrize("four", [False, True])
def test_rotation_bit_for_bit(dtype, interleaved, heads, kv_heads, head_dim, four):
    import torch
    from paged_kv_decode_nsv_gb300 import nsv
    for i, rotary in enumerate([16, 48, head_dim // 2, head_dim]):
        b = T.inputs(301, heads, kv_heads, head_dim, dtype, rotary, four, seed=i, fused=i % 2 == 1)
        out = torch.empty(b["q"].shape, dtype=b["q"].dtype, device="cuda")
        if four:
            nsv.kv4_write(b["k"], b["v"], b["slots"], *b["pools"], q=b["q"], positions=b["positions"],
                          rotary=b["table"], q_out=out, interleaved=interleaved)
        else:
            nsv.rope_write(b["q"], b["k"], b["v"], b["positions"], b["table"], b["slots"], *b["pools"],
                           out, interleaved=interleaved)
            assert torch.equal(T.by_slot(b["pools"][0], b["slots"]), rotated(b["k"], b, interleaved))
        assert torch.equal(out, rotated(b["q"], b, interleaved))
