"""Oracle for rotary positions, the paged key-value cache and decode attention.

TEST INFRASTRUCTURE ONLY (see :mod:`oracle`).

Plain numpy, fp64 arithmetic; the quantizer and the code values are the C
oracle's.  The cache is modelled as one flat byte array addressed by the layout
as include/nvfp4.h states it, one row at a time.
"""
from __future__ import annotations

import numpy as np

import oracle
from oracle.stack import bf16_round

BF16, E4M3, NVFP4 = "bf16", "e4m3", "nvfp4"

_E4M3 = None


def e4m3_table() -> np.ndarray:
    global _E4M3
    if _E4M3 is None:
        _E4M3 = np.array([oracle.e4m3_value(i) for i in range(256)])
    return _E4M3


# ---------------------------------------------------------------- rotary ----

def rope_freqs(rot: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(turns per token of each pair, magnitude of cos and sin)."""
    i = np.arange(rot // 2)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot) / (2 * np.pi)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        w = np.clip((f * original_len - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
        return f * w + f / factor * (1 - w), 0.1 * np.log(factor) + 1
    return f, 1.0


def rope(x, positions, freqs, interleaved: bool, mscale: float = 1.0, inverse: bool = False) -> np.ndarray:
    """x [T, heads, D] turned, as complex products in fp64 (the angle from an
    extended-precision product)."""
    x = np.asarray(x, np.float64)
    n = len(freqs)
    turns = np.asarray(positions).astype(np.longdouble)[:, None] * np.asarray(freqs).astype(np.longdouble)
    a = (turns - np.round(turns)).astype(np.float64) * (2 * np.pi)
    z = mscale * np.exp((-1j if inverse else 1j) * a)[:, None, :]
    y = x.copy()
    if interleaved:
        w = (x[..., 0:2 * n:2] + 1j * x[..., 1:2 * n:2]) * z
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = w.real, w.imag
    else:
        w = (x[..., :n] + 1j * x[..., n:2 * n]) * z
        y[..., :n], y[..., n:2 * n] = w.real, w.imag
    return y


# ----------------------------------------------------------------- cache ----

class Cache:
    """The bytes of a paged cache (``data``) and its global scales."""

    def __init__(self, num_pages, page_size, heads, D, fmt, k_gs=1.0, v_gs=1.0, fill=0xFF):
        self.num_pages, self.page_size, self.heads, self.D, self.fmt = num_pages, page_size, heads, D, fmt
        self.gs = (np.float32(k_gs), np.float32(v_gs))
        self.code = {BF16: 2 * D, E4M3: D, NVFP4: D // 2}[fmt]
        self.scale = D // 16 if fmt == NVFP4 else 0
        self.tile = 32 * (self.code + self.scale)
        self.data = np.full(num_pages * heads * (page_size // 16) * self.tile, fill, np.uint8)

    def _tile(self, slot: int, head: int) -> int:
        page, o = divmod(int(slot), self.page_size)
        return ((page * self.heads + head) * (self.page_size // 16) + o // 16) * self.tile

    def code_at(self, slot: int, head: int, which: int) -> np.ndarray:
        """Byte addresses of a row's codes, in order."""
        r = int(slot) % 16
        b = np.arange(self.code)
        turn = ((r & 6) ^ ((r & 1) << 2)) & (self.code // 16 - 1)
        return self._tile(slot, head) + (which * 16 + r) * self.code + (((b // 16) ^ turn) * 16 + b % 16)

    def scale_at(self, slot: int, head: int, which: int) -> np.ndarray:
        r = int(slot) % 16
        return self._tile(slot, head) + 32 * self.code + (which * 16 + r) * self.scale + np.arange(self.scale)

    def encode(self, row: np.ndarray, which: int):
        """(code bytes, scale bytes) of one row of D fp32 values."""
        row = np.ascontiguousarray(row, np.float32)
        if self.fmt == BF16:
            return (bf16_round(row).view(np.uint32) >> 16).astype("<u2").view(np.uint8), np.empty(0, np.uint8)
        if self.fmt == E4M3:
            return oracle.e4m3_encode(row / self.gs[which]), np.empty(0, np.uint8)
        c, s, _ = oracle.quantize(row[None], gs=self.gs[which])
        return c[0], s[0]

    def write(self, k, v, slots):
        """k, v [T, heads, D] fp32; negative slots are skipped."""
        for t, slot in enumerate(np.asarray(slots)):
            if slot < 0:
                continue
            for h in range(self.heads):
                for which, x in ((0, k), (1, v)):
                    c, s = self.encode(x[t, h], which)
                    self.data[self.code_at(slot, h, which)] = c
                    self.data[self.scale_at(slot, h, which)] = s

    def row(self, slot: int, head: int, which: int) -> np.ndarray:
        """fp64 value of each element (before the rounding of the product with gs)."""
        c = self.data[self.code_at(slot, head, which)]
        if self.fmt == BF16:
            return (c.view("<u2").astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        gs = float(self.gs[which])
        if self.fmt == E4M3:
            return e4m3_table()[c] * gs
        s = self.data[self.scale_at(slot, head, which)]
        return oracle.dequantize(c[None], s[None], gs)[0]

    def read(self, slots):
        """(k, v) [T, heads, D] fp64; zeros for negative slots."""
        out = np.zeros((2, len(slots), self.heads, self.D))
        for t, slot in enumerate(np.asarray(slots)):
            if slot >= 0:
                for h in range(self.heads):
                    for which in (0, 1):
                        out[which, t, h] = self.row(slot, h, which)
        return out[0], out[1]


# ------------------------------------------------------------- attention ----

def attend(q, k, v, scale: float):
    """One token: q [heads_q, D], k and v [n, heads, D], fp64.  Returns ``(y, lse, spread,
    score_mag)`` with spread = sum_j p_j |v_j| (the scale of y's rounding errors) and
    score_mag = max_j scale * sum_d |q_d k_jd| per query head."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    G = q.shape[0] // k.shape[1]
    y, lse = np.zeros_like(q), np.full(q.shape[0], -np.inf)
    spread, mag = np.zeros_like(q), np.zeros(q.shape[0])
    for h in range(q.shape[0]):
        kh, vh = k[:, h // G], v[:, h // G]
        if len(kh) == 0:
            continue
        s = scale * (kh @ q[h])
        m = s.max()
        e = np.exp(s - m)
        p = e / e.sum()
        y[h], lse[h], spread[h] = p @ vh, m + np.log(e.sum()), p @ np.abs(vh)
        mag[h] = abs(scale) * (np.abs(kh) @ np.abs(q[h])).max()
    return y, lse, spread, mag
