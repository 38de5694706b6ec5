"""Decode attention at the ends of the softmax weights' range: scores that fp32 holds in
coarse steps; one token that takes almost all weight and holds next to nothing (an attention
sink), and a long tail far below it whose values are the output."""
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


# The sink's score over the tail's, in nats (2^-17 to 2^-32 in weight).
DEPTHS = (12.0, 14.25, 15.75, 16.5, 17.25, 18.0, 19.5, 21.75)
KEY = 0.75                                                       # exact in every format at the scales below


def sink_bounds(fmt, D, y, lse, spread, mag, top, v_sum, y_dtype):
    """Bounds of |y - ref| and of |lse - ref| of one row.  Scores, exponentials and sums as in
    attn_checks.attn_bounds (D fp32 additions a tensor-core step 2^-23 each of `mag`; 4 * 2^-23 of it and
    2^-21; fp32 sums over two parts of n / 16 tiles and the joins, 700 at most here).  A weight
    is rounded: one fp16 part 2^-11 (quantized cache, bf16 output), two fp16 parts 2^-22 (fp32
    output), two bf16 parts 2^-16.  fp16 is also off by 2^-25 where a weight is small; the row's
    largest is at least 2^10, so that is 2^-35 of the largest weight `top` for every token."""
    err = mag * (D + 12) * 2.0 ** -23 + 2.0 ** -21
    part = 2.0 ** -16 if fmt == oat.BF16 else 2.0 ** -22 if y_dtype == torch.float32 else 2.0 ** -11
    step = 0.0 if fmt == oat.BF16 else 2.0 ** -35
    rel = 2 * np.expm1(err) + part + 700 * 2.0 ** -23
    by = spread * rel[:, None] + step * top[:, None] * v_sum + HALF_STEP[y_dtype] * np.abs(y) + 1e-30
    return by, 2 * err + 700 * 2.0 ** -23 + 2.0 ** -22 * np.abs(lse)


@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G", [2, 6, 16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", (oat.BF16, oat.E4M3, oat.NVFP4))
def test_tail_below_a_sink(cuda_device, fmt, D, G, y_dtype):
    """600 sequences over the same 3,500 rows, so that a warp walks through thousands of them
    behind the sink; every sequence has its own depth."""
    n, page, B, Hkv = 3500, 64, 600, 4
    pages = -(-n // page)
    rng = np.random.default_rng(5)
    gs = {oat.BF16: 1.0, oat.E4M3: 1.0 / 64, oat.NVFP4: 1.0 / 512}[fmt]
    cache = nv.KVCache.empty(pages, page, Hkv, D, FMT[fmt], scalar(gs), scalar(gs))
    k = np.zeros((n, Hkv, D), np.float32)
    k[0] = KEY
    v = (0.5 * rng.standard_normal((n, Hkv, D)) + 0.3).astype(np.float32)
    v[0] = 0.0
    slots = dev(np.arange(n))
    nv.nvfp4_kv_write(cache, dev(k), dev(v), slots)
    kr, vr = (host(x) for x in nv.nvfp4_kv_read(cache, slots, y_dtype=torch.float32))
    assert np.array_equal(kr, k) and not vr[0].any()
    # scale q . k_0 = depth at scale 1 / D (16 .. 29: exact in bf16)
    depth = np.array([DEPTHS[b % len(DEPTHS)] for b in range(B)], np.float32)
    q = torch.from_numpy(depth / np.float32(KEY)).to(torch.bfloat16)[:, None, None].expand(B, Hkv * G, D).contiguous().cuda()
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, pages).contiguous()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    y, lse = nv.nvfp4_attn_decode(q, cache, table, lens, scale=1.0 / D, want_lse=True, y_dtype=y_dtype)
    for i in range(len(DEPTHS)):
        ry, rl, spread, mag = oat.attend(host(q[i]), kr, vr, 1.0 / D)
        top = np.exp(DEPTHS[i] - rl)
        v_sum = np.abs(vr).sum(0).repeat(G, 0)
        by, bl = sink_bounds(fmt, D, ry, rl, spread, mag, top, v_sum, y_dtype)
        for b in range(i, B, len(DEPTHS)):
            assert_close(y[b], ry, by, f"y[{b}], {DEPTHS[i]} nats")
            assert_close(lse[b], rl, bl, f"lse[{b}], {DEPTHS[i]} nats")
    assert nv.nvfp4_read_device_status() == nv.OK


@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,extra", [(1, 0), (1, 2400), (400, 0), (400, 1200)])
@pytest.mark.parametrize("fmt,v_gs", [(oat.E4M3, 2.0 ** 70), (oat.E4M3, 2.0 ** -110), (oat.NVFP4, 2.0 ** 70),
                                      (oat.NVFP4, 2.0 ** -110)])
def test_large_and_small_value_scales(cuda_device, fmt, v_gs, B, extra, y_dtype):
    """The same values (powers of two from 1/16 to 256 before the scale) at scales that are powers of
    two: the outputs are those at scale 1 times the scale, to the bit."""
    D, page, n = 128, 16, 1024
    rng = np.random.default_rng(8)
    k = rng.standard_normal((n, 1, D)).astype(np.float32)
    v = np.exp2(rng.integers(-4, 9, (n, 1, D))).astype(np.float32)
    q = torch.from_numpy(rng.standard_normal((B, 3, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    table = torch.cat((torch.arange(n // page), torch.zeros(extra))).int().cuda().expand(B, -1).contiguous()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    slots = dev(np.arange(n))
    out = []
    for gs in (1.0, v_gs):
        cache = nv.KVCache.empty(n // page, page, 1, D, FMT[fmt], scalar(0.02), scalar(1.0))
        nv.nvfp4_kv_write(cache, dev(k), dev(v), slots)
        cache = nv.KVCache(cache.data, page, 1, D, FMT[fmt], cache.k_gs, scalar(gs))
        out.append(nv.nvfp4_attn_decode(q, cache, table, lens, y_dtype=y_dtype))
    # (outputs lie above 2^-4 of a scale, far from the ends of fp32, and so do the sums behind them)
    assert torch.equal(out[1], out[0] * v_gs)
