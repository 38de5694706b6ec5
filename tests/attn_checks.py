"""Bounds and helpers of the rotary / cache / decode-attention tests (test side only)."""
import numpy as np
import torch

import bit_linear_moe_b200 as nv
from oracle import attention as oat

FMT = {oat.BF16: nv.KV_BF16, oat.E4M3: nv.KV_E4M3, oat.NVFP4: nv.KV_NVFP4}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def host(t):
    return t.detach().double().cpu().numpy()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def scalar(x):
    return torch.tensor([float(x)], dtype=torch.float32, device="cuda")


def device_cache(oc: oat.Cache) -> nv.KVCache:
    """The oracle cache's bytes on the device."""
    return nv.KVCache(dev(oc.data), oc.page_size, oc.heads, oc.D, FMT[oc.fmt], scalar(oc.gs[0]), scalar(oc.gs[1]))


def rope_bound(x, ref, positions, freqs, interleaved, mscale, y_dtype):
    """|y - ref| of a rotation: cos and sin are rounded once (2^-24 of at most mscale; the
    angle's fp64 product adds 2 pi |turns| 2^-53), then a product and a sum round
    (2^-24 each), on |u| + |v|; then y's own rounding.  Four roundings are counted."""
    x = np.abs(np.asarray(x, np.float64))
    n = len(freqs)
    pair = np.zeros_like(x)
    if interleaved:
        s = x[..., 0:2 * n:2] + x[..., 1:2 * n:2]
        pair[..., 0:2 * n:2], pair[..., 1:2 * n:2] = s, s
    else:
        s = x[..., :n] + x[..., n:2 * n]
        pair[..., :n], pair[..., n:2 * n] = s, s
    turns = np.abs(np.asarray(positions, np.float64)).max() * np.abs(freqs).max()
    return pair * mscale * (4 * 2.0 ** -24 + 2 * np.pi * turns * 2.0 ** -52) + HALF_STEP[y_dtype] * np.abs(ref) + 1e-38


def attn_bounds(fmt, D, n, y, lse, spread, mag, vmax, y_dtype):
    """(bound of y, bound of lse) for one token over n cache rows.

    Score error (natural units): D fp32 additions of exact products, each within a
    tensor-core step (2^-23, truncation allowed) of the sum of magnitudes `mag`; the factor,
    the subtraction of the maximum and the exponential add 4 * 2^-23 |s| + 2^-21.
    A weight is then off by e^err - 1 and by its rounding: fp16 2^-11 (bf16 output), fp16
    in two parts 2^-21, bf16 in two parts 2^-15; fp16 parts below 2^-14 also by 2^-25 of
    a row whose largest weight is at least 1.  Numerator and denominator both carry
    the weights' error, and sum in fp32 over n / 16 tiles and at most 600 joins (2^-23 each)."""
    err = mag * (D + 8) * 2.0 ** -23 + 2.0 ** -21
    part = 2.0 ** -15 if fmt == oat.BF16 else 2.0 ** -21 if y_dtype == torch.float32 else 2.0 ** -11
    sums = (n / 8 + 600) * 2.0 ** -23
    rel = 2 * np.expm1(err) + part + sums
    tiny = 0.0 if fmt == oat.BF16 else n * 2.0 ** -25 * vmax
    by = spread * rel[:, None] + tiny + HALF_STEP[y_dtype] * np.abs(y) + 1e-30
    bl = 2 * err + sums + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return by, bl


def assert_close(got, ref, bound, what):
    got = host(got) if isinstance(got, torch.Tensor) else np.asarray(got, np.float64)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside the bound; first at {i}: "
                             f"got {got[i]!r}, ref {ref[i]!r}, bound {np.broadcast_to(bound, got.shape)[i]!r}")
