"""GPU rotary positions and the paged key-value cache against the oracle: cache bytes
bit for bit, reads bit for bit, rotations within the bound of their roundings, the fused
call bit for bit like the separate ones."""
import numpy as np
import pytest
import torch

import bit_linear_moe_b200 as nv
from attn_checks import FMT, assert_close, dev, device_cache, host, rope_bound, scalar
from oracle import attention as oat
from oracle.stack import bf16_round

pytestmark = pytest.mark.gpu

FMTS = (oat.BF16, oat.E4M3, oat.NVFP4)


def rows(rng, T, heads, D, dtype, extra=0):
    """[T, heads, D] as a slice of wider rows, with a few strong channels, an all-zero
    block and values on the quantizers' boundaries."""
    x = rng.standard_normal((T, heads + extra, D)).astype(np.float32)
    x[:, :, rng.choice(D, 3, replace=False)] *= 9.0
    if T > 2:
        x[1, 0, 16:32] = 0.0
        x[2, 0, :16] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0]
    return dev(x).to(dtype)[:, :heads]


@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,D,heads,page,T", [
    (oat.BF16, 64, 1, 16, 1), (oat.BF16, 128, 3, 32, 19), (oat.BF16, 256, 2, 48, 40),
    (oat.E4M3, 64, 2, 16, 33), (oat.E4M3, 128, 5, 64, 7), (oat.E4M3, 256, 1, 32, 18),
    (oat.NVFP4, 64, 2, 16, 5), (oat.NVFP4, 128, 4, 64, 40), (oat.NVFP4, 256, 1, 128, 21), (oat.NVFP4, 128, 20, 16, 3)])
def test_kv_write_and_read(cuda_device, fmt, D, heads, page, T, x_dtype):
    rng = np.random.default_rng([T, D, heads])
    pages = -(-T // page) + 3
    oc = oat.Cache(pages, page, heads, D, fmt, 0.0123, 0.0071)
    c = device_cache(oc)
    k, v = rows(rng, T, heads, D, x_dtype, extra=2), rows(rng, T, heads, D, x_dtype)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 4:
        slots[3] = -1                                            # a padding row
    nv.nvfp4_kv_write(c, k, v, dev(slots))
    oc.write(k.float().cpu().numpy(), v.float().cpu().numpy(), slots)
    assert np.array_equal(c.data.cpu().numpy(), oc.data)         # the named rows and nothing else
    ask = np.concatenate([slots, slots[:1], [-1]])               # a slot twice, a negative one
    rk, rv = oc.read(ask)
    for dt in (torch.bfloat16, torch.float32):
        gk, gv = nv.nvfp4_kv_read(c, dev(ask), y_dtype=dt)
        for got, ref in ((gk, rk), (gv, rv)):
            want = ref.astype(np.float32)                        # one fp32 rounding of code * scale * gs
            if dt == torch.bfloat16:
                want = bf16_round(want)
            assert np.array_equal(got.float().cpu().numpy(), want)
    assert nv.nvfp4_read_device_status() == nv.OK


@pytest.mark.parametrize("fmt", FMTS)
def test_kv_write_large_chunk(cuda_device, fmt):
    """Many tokens (16 per CTA): the reads give back what a direct quantization gives."""
    T, heads, D, page = 4099, 3, 128, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn((T, heads, D), generator=g, device="cuda") for _ in range(2))
    gs = scalar(0.002), scalar(0.003)
    c = nv.KVCache.empty(70, page, heads, D, FMT[fmt], *gs)
    slots = torch.randperm(70 * page, device="cuda", generator=g)[:T]
    nv.nvfp4_kv_write(c, k, v, slots)
    got = nv.nvfp4_kv_read(c, slots, y_dtype=torch.float32)
    for x, y, s in zip((k, v), got, gs):
        if fmt == oat.BF16:
            ref = x.to(torch.bfloat16).float()
        elif fmt == oat.E4M3:
            ref = (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).float() * s
        else:
            codes, scales, _ = nv.nvfp4_quantize(x.reshape(-1, D), gs_in=s)
            lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
            q = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), -1).flatten(-2)
            sc = scales.view(torch.float8_e4m3fn).float().view(-1, D // 16).repeat_interleave(16, -1)
            ref = (q * sc * s).view(T, heads, D)
        assert torch.equal(y, ref)


@pytest.mark.parametrize("fmt", [oat.E4M3, oat.NVFP4])
@pytest.mark.parametrize("gs", [2.0 ** -140, 1.2e-38, 2.0 ** -20, 0.0123, 1.0, 1e30, 5e37])
def test_kv_write_on_the_borders(cuda_device, fmt, gs):
    """Quotients on and one step beside the borders between codes, of every block scale,
    with global scales to the ends of fp32: bytes equal to those of the divisions."""
    rng = np.random.default_rng(7)
    T, heads, D, page = 64, 2, 64, 16
    g = np.float32(gs)
    oc = oat.Cache(T // page, page, heads, D, fmt, g, g)
    c = device_cache(oc)
    border = np.float32([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, 2.0, 3.0, 4.0, 0.0, 17 / 16, 27 / 16])
    with np.errstate(all="ignore"):
        scale = np.float32(rng.integers(8, 16, (T, heads, D // 16, 1)) * 2.0 ** rng.integers(-4, 5, (T, heads, D // 16, 1)))
        k = (border[rng.integers(0, 16, (T, heads, D // 16, 16))] * scale * g).astype(np.float32)
        k[..., 0] = (np.float32(6.0) * scale * g)[..., 0]        # the block's largest names its scale
        step = rng.integers(-1, 2, k.shape)
        k = np.where(step < 0, np.nextafter(k, np.float32(0)), np.where(step > 0, np.nextafter(k, np.float32(np.inf)), k))
        k = np.where(rng.random(k.shape) < 0.5, -k, k).astype(np.float32).reshape(T, heads, D)
    k = np.clip(k, -3e38, 3e38)
    v = np.ascontiguousarray(k[::-1])
    nv.nvfp4_kv_write(c, dev(k), dev(v), torch.arange(T, device="cuda"))
    with np.errstate(all="ignore"):
        oc.write(k, v, np.arange(T))
    assert np.array_equal(c.data.cpu().numpy(), oc.data)


def test_bad_slots_are_reported_and_skipped(cuda_device):
    """Slots past the cache: skipped by the kernel's own check, named in the status word."""
    oc = oat.Cache(2, 16, 2, 64, oat.E4M3, 0.01, 0.01)
    c = device_cache(oc)
    k = torch.ones((4, 2, 64), device="cuda")
    slots = np.array([3, 32, 1 << 40, -5], np.int64)
    nv.nvfp4_kv_write(c, k, k, dev(slots))
    assert nv.nvfp4_read_device_status() == nv.ERR_PAGE
    assert nv.nvfp4_read_device_status() == nv.OK
    oc.write(k.cpu().numpy(), k.cpu().numpy(), [3, -1, -1, -1])
    assert np.array_equal(c.data.cpu().numpy(), oc.data)
    rk, rv = nv.nvfp4_kv_read(c, dev(slots))
    assert nv.nvfp4_read_device_status() == nv.ERR_PAGE
    assert not rk[1:].any() and not rv[1:].any() and rk[0].all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("xd,yd", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
                                   (torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("T,heads,D,rot,start", [(1, 1, 16, 16, 5), (1, 60, 128, 128, 100003), (7, 3, 64, 32, 0),
                                                 (33, 5, 80, 48, 1 << 20), (2, 2, 256, 96, 1 << 31),
                                                 (3, 2, 1024, 1024, 77), (700, 24, 128, 64, 4000),
                                                 (2500, 20, 48, 32, 9), (900, 40, 80, 80, 70000), (3000, 9, 16, 16, 1)])
def test_rope(cuda_device, T, heads, D, rot, start, xd, yd, interleaved):
    rng = np.random.default_rng([T, D, rot])
    x = rows(rng, T, heads, D, xd, extra=1) if D != 16 else dev(rng.standard_normal((T, heads, D))).to(xd)
    f, m = nv.nvfp4_rope_freqs(rot, 10000.0, nv.ROPE_SCALE_YARN, factor=4.0, original_len=4096.0)
    pos = start + np.arange(T, dtype=np.int64)
    pos[-1] = -pos[-1]
    lay = nv.ROPE_INTERLEAVED if interleaved else nv.ROPE_HALF
    xh = host(x)
    for inverse in (False, True):
        y = nv.nvfp4_rope(x, dev(pos), f.cuda(), layout=lay, mscale=m, inverse=inverse, y_dtype=yd)
        ref = oat.rope(xh, pos, f.numpy(), interleaved, m, inverse)
        assert_close(y, ref, rope_bound(xh, ref, pos, f.numpy(), interleaved, m, yd), f"rope inverse={inverse}")
    if rot < D:
        assert torch.equal(y[..., rot:], x[..., rot:].to(yd))
    # in place (y = x), and into a slice of wider rows
    if xd == yd:
        y = nv.nvfp4_rope(x, dev(pos), f.cuda(), layout=lay, mscale=m, y_dtype=yd)
        wide = torch.full((T, heads + 2, D), 7.0, dtype=yd, device="cuda")
        nv.nvfp4_rope(x, dev(pos), f.cuda(), layout=lay, mscale=m, y=wide[:, 1:heads + 1])
        assert torch.equal(wide[:, 1:heads + 1], y) and (wide[:, 0] == 7).all() and (wide[:, -1] == 7).all()
        z = x.clone()
        nv.nvfp4_rope(z, dev(pos), f.cuda(), layout=lay, mscale=m, y=z)
        assert torch.equal(z, y)


def test_rope_gradient_is_the_inverse_rotation(cuda_device):
    """<g, rope(x + h e) - rope(x - h e)> / 2h = <rope^-1(g), e>: the map is linear, so the
    differences are exact up to the fp32 roundings (2^-22 of the terms' magnitudes)."""
    rng = np.random.default_rng(8)
    x, g, e = (dev(rng.standard_normal((5, 2, 64)), torch.float32) for _ in range(3))
    f = nv.nvfp4_rope_freqs(64)[0].cuda()
    pos = dev(np.array([0, 3, 99, 5000, 70001], np.int64))

    def turn(t, inv=False):
        return nv.nvfp4_rope(t, pos, f, inverse=inv, y_dtype=torch.float32).double()
    h = 0.5
    diff = (g.double() * (turn(x + h * e) - turn(x - h * e))).sum() / (2 * h)
    grad = (turn(g, True) * e.double()).sum()
    mag = (g.abs().double() * (x.abs() + e.abs()).double()).sum()
    assert abs(diff - grad) <= 4 * 2.0 ** -22 * mag


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,interleaved", [(1, 40, 20, 128, 128, False), (32, 8, 1, 64, 64, True),
                                                        (5, 6, 2, 128, 48, False), (9, 2, 2, 256, 16, True),
                                                        (1203, 12, 3, 128, 96, False), (401, 32, 8, 64, 32, True),
                                                        (300, 16, 4, 256, 256, False)])
def test_rope_kv_write_equals_the_separate_calls(cuda_device, T, Hq, Hkv, D, rot, interleaved, xd, fmt):
    rng = np.random.default_rng([T, Hq, D])
    qkv = rows(rng, T, Hq + 2 * Hkv, D, xd)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    f, m = nv.nvfp4_rope_freqs(rot, 10000.0, nv.ROPE_SCALE_YARN, factor=4.0, original_len=2048.0)
    f = f.cuda()
    lay = nv.ROPE_INTERLEAVED if interleaved else nv.ROPE_HALF
    pages = -(-T // 32) + 2
    pos = dev(rng.integers(0, 200000, T))
    slots = rng.permutation(pages * 32)[:T].astype(np.int64)
    if T > 2:
        slots[::7] = -1
    slots = dev(slots)
    gs = scalar(0.011), scalar(0.004)
    one, two = (nv.KVCache(torch.full((nv.nvfp4_kv_cache_bytes(pages, 32, Hkv, D, FMT[fmt]),), 0xFF, dtype=torch.uint8,
                                      device="cuda"), 32, Hkv, D, FMT[fmt], *gs) for _ in range(2))
    got = nv.nvfp4_rope_kv_write(one, q, k, v, pos, slots, f, layout=lay, mscale=m)
    want = nv.nvfp4_rope(q, pos, f, layout=lay, mscale=m)
    kr = nv.nvfp4_rope(k, pos, f, layout=lay, mscale=m, y_dtype=torch.bfloat16)
    if xd == torch.float32:                                      # one dtype per write: the keys' bf16 values in fp32
        kr = kr.float()
    nv.nvfp4_kv_write(two, kr, v, slots)
    assert torch.equal(got, want)
    assert torch.equal(one.data, two.data)


def test_cache_past_4_gib(cuda_device):
    """Pages beyond 2^32 bytes are addressed as 64-bit offsets."""
    heads, D, page = 2, 256, 64
    per = nv.nvfp4_kv_cache_bytes(1, page, heads, D, nv.KV_BF16)
    pages = (1 << 32) // per + 40
    c = nv.KVCache.empty(pages, page, heads, D, nv.KV_BF16)
    x = torch.randn((48, heads, D), device="cuda").to(torch.bfloat16)
    slots = torch.arange(48, device="cuda") + (pages - 1) * page
    low = slots - ((1 << 32) // per) * page                      # where a 32-bit offset would land
    nv.nvfp4_kv_write(c, torch.zeros_like(x), torch.zeros_like(x), low)
    nv.nvfp4_kv_write(c, x, -x, slots)
    k, v = nv.nvfp4_kv_read(c, slots)
    assert torch.equal(k, x) and torch.equal(v, -x)
    k, v = nv.nvfp4_kv_read(c, low)
    assert not k.any() and not v.any()


def test_captured_write_and_read(cuda_device):
    """A captured step replays on new rows, slots and positions; it and an eager call agree."""
    g = torch.Generator(device="cuda").manual_seed(9)
    T, Hq, Hkv, D = 6, 8, 2, 128
    f = nv.nvfp4_rope_freqs(D)[0].cuda()
    gs = scalar(0.01), scalar(0.01)
    c, e = (nv.KVCache(torch.zeros(nv.nvfp4_kv_cache_bytes(4, 16, Hkv, D, nv.KV_NVFP4), dtype=torch.uint8,
                                   device="cuda"), 16, Hkv, D, nv.KV_NVFP4, *gs) for _ in range(2))
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda")
    pos, slots = torch.arange(T, device="cuda"), torch.arange(T, device="cuda")

    def step(cache):
        q = nv.nvfp4_rope_kv_write(cache, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, slots, f)
        return (q, *nv.nvfp4_kv_read(cache, slots))
    step(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(c)
    for i in range(3):
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        pos.add_(1000 * i)
        slots.add_(T)
        graph.replay()
        ref = step(e)
        for a, b in zip(out, ref):
            assert torch.equal(a, b)
    assert torch.equal(c.data[-100:], e.data[-100:])


def test_other_stream(cuda_device):
    """Calls are enqueued on the current stream: ordered after what made their inputs there."""
    s = torch.cuda.Stream()
    c = nv.KVCache.empty(300, 64, 4, 128, nv.KV_BF16)
    slots = torch.arange(300 * 64, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x = torch.randn((300 * 64, 4, 128), device="cuda")
        for _ in range(5):
            x = x * 0.5 + 1.0
        x = x.to(torch.bfloat16)
        nv.nvfp4_kv_write(c, x, x, slots)
        k, v = nv.nvfp4_kv_read(c, slots)
    s.synchronize()
    assert torch.equal(k, x) and torch.equal(v, x)
