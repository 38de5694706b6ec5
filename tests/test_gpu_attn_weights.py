"""Decode attention at the ends of the softmax weights' range."""
import numpy as np
import pytest
import torch

import bit_linear_moe_b200 as nv
from attn_checks import FMT, HALF_STEP, assert_close, dev, host, scalar
from oracle import attention as oat

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("extra", [0, 1200])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("fmt", (oat.BF16, oat.E4M3))
def test_neighbouring_huge_scores(cuda_device, fmt, odd, extra, y_dtype):
    """Scores beyond 2^27 in log2 units, which fp32 holds in steps of 16: one token's weight is
    2^16 times the others', more than fp16 holds if the maximum lagged by that.  400 sequences share
    the rows, so that one warp meets both tokens, apart."""
    D, page, n, B = 128, 16, 1024, 400
    cache = nv.KVCache.empty(n // page, page, 1, D, FMT[fmt], scalar(1.0), scalar(1.0))
    k = np.full((n, 1, D), 448.0, np.float32)
    k[:, 0, 0] = 0.0
    k[:16, 0, 0] = 1.0 + odd
    k[40, 0, 0] = 2.0 + odd                                      # 1 more than in tile 0
    v = np.random.default_rng(3).integers(-8, 9, (n, 1, D)).astype(np.float32)
    nv.nvfp4_kv_write(cache, dev(k), dev(v), dev(np.arange(n)))
    q = torch.full((B, 2, D), 256.0, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0                                             # q . k = 14,565,376 + k_0: exact in fp32
    scale = float(np.float32(16.0 * np.log(2.0)))
    assert np.float32(np.float32(scale) * np.float32(1.4426950408889634)) == 16.0
    table = torch.cat((torch.arange(n // page), torch.zeros(extra))).int().cuda().expand(B, -1).contiguous()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    y, lse = nv.nvfp4_attn_decode(q, cache, table, lens, scale=scale, want_lse=True, y_dtype=y_dtype)
    s = 16.0 * (k[:, 0, 0] - k[40, 0, 0]).astype(np.float64)     # log2 of the weights, exact in the kernel too
    w = np.exp2(s)
    ref = (w[:, None] * v[:, 0].astype(np.float64)).sum(0) / w.sum()
    # the largest weight is a power of two, exact; the others (16 of 2^-16, the rest 2^-32 and less) are
    # off by 2^-11 of themselves and by 2^-25; the sums and the quotient by 2^-20
    by = 8 * (2.0 ** -11 * 17 * 2.0 ** -16 + n * 2.0 ** -25 + 2.0 ** -20) + HALF_STEP[y_dtype] * np.abs(ref)
    assert_close(y, np.broadcast_to(ref, (B, 2, D)), by, "y")
    top = 16.0 * np.log(2.0) * (14565376.0 + float(k[40, 0, 0]))
    assert np.abs(host(lse) / top - 1).max() <= 2.0 ** -21
