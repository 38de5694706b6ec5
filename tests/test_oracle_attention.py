"""Pins of the rotary / cache / attention oracle, the host-side frequency helper and the
host-side checks of their entry points (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import bit_linear_moe_b200 as nv
import oracle
from oracle import attention as oat

FAKE, FAKE2, FAKE3 = (ctypes.c_void_p(0x10000 * i) for i in (1, 2, 3))
MISALIGNED = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    from bit_linear_moe_b200 import build
    build.build()
    return nv.lib()


# ---- oracle pins ---------------------------------------------------------------

@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_rotation(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 64))
    f, _ = oat.rope_freqs(32)
    pos = np.array([0, 1, 7, 1000, 123456])
    y = oat.rope(x, pos, f, interleaved)
    assert np.array_equal(y[..., 32:], x[..., 32:])              # elements past rot_dim pass through
    assert np.allclose(y[0], x[0], atol=1e-15)                   # position 0: identity
    assert np.allclose(np.sum(y ** 2, -1), np.sum(x ** 2, -1))   # pairs keep their length
    assert np.allclose(oat.rope(y, pos, f, interleaved, inverse=True), x, atol=1e-12)
    # scores depend on the distance alone
    a, b = oat.rope(x, pos + 10, f, interleaved), oat.rope(x[::-1], pos[::-1] + 10, f, interleaved)
    c, d = oat.rope(x, pos + 500, f, interleaved), oat.rope(x[::-1], pos[::-1] + 500, f, interleaved)
    assert np.allclose(np.sum(a * b, -1), np.sum(c * d, -1), atol=1e-9)


def test_rope_layouts_pair_what_they_say():
    x = np.zeros((1, 1, 16))
    x[0, 0, 1] = 1.0
    f = np.full(8, 0.25)                                         # a quarter turn per token
    assert np.argmax(np.abs(oat.rope(x, [1], f, False)[0, 0])) == 9
    x = np.zeros((1, 1, 16))
    x[0, 0, 2] = 1.0
    assert np.argmax(np.abs(oat.rope(x, [1], f, True)[0, 0])) == 3


@pytest.mark.parametrize("fmt", [oat.BF16, oat.E4M3, oat.NVFP4])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_cache_layout_is_a_bijection_and_round_trips(fmt, D):
    c = oat.Cache(2, 32, 2, D, fmt, 0.01, 0.02)
    seen = np.concatenate([np.concatenate([c.code_at(s, h, w), c.scale_at(s, h, w)])
                           for s in range(64) for h in range(2) for w in (0, 1)])
    assert len(np.unique(seen)) == len(seen) == len(c.data)      # every byte belongs to one row
    rng = np.random.default_rng(D)
    k, v = (rng.standard_normal((3, 2, D)).astype(np.float32) for _ in range(2))
    c.write(k, v, [5, 37, -1])
    rk, rv = c.read([5, 37, -1])
    step = {oat.BF16: 2.0 ** -8, oat.E4M3: 2.0 ** -4, oat.NVFP4: 0.25}[fmt]
    for x, r in ((k, rk), (v, rv)):
        amax = np.abs(x[:2]).reshape(2, 2, -1, 16).max(-1).repeat(16, -1).reshape(2, 2, D)
        assert (np.abs(r[:2] - x[:2]) <= step * (np.abs(x[:2]) if fmt != oat.NVFP4 else amax) + 1e-4).all()
        assert not r[2].any()
    assert (c.data[c.code_at(6, 0, 0)] == 0xFF).all()            # other rows untouched


def test_attend_against_brute_force():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    y, lse, _, _ = oat.attend(q, k, v, 0.5)
    for h in range(4):
        w = [np.exp(0.5 * sum(q[h, d] * k[j, h // 2, d] for d in range(8))) for j in range(5)]
        assert lse[h] == pytest.approx(np.log(sum(w)))
        for d in range(8):
            assert y[h, d] == pytest.approx(sum(w[j] * v[j, h // 2, d] for j in range(5)) / sum(w))
    y, lse, _, _ = oat.attend(q, k[:0], v[:0], 0.5)
    assert not y.any() and (lse == -np.inf).all()


# ---- nvfp4_rope_freqs (host) ----------------------------------------------------

@pytest.mark.parametrize("rot", [2, 32, 96, 128, 256])
@pytest.mark.parametrize("name,code,kw", [
    ("none", nv.ROPE_SCALE_NONE, {}), ("linear", nv.ROPE_SCALE_LINEAR, dict(factor=8.0)),
    ("ntk", nv.ROPE_SCALE_NTK, dict(factor=4.0)),
    ("yarn", nv.ROPE_SCALE_YARN, dict(factor=16.0, original_len=4096.0)),
    ("yarn", nv.ROPE_SCALE_YARN, dict(factor=2.0, original_len=8192.0, beta_fast=20.0, beta_slow=2.0))])
def test_rope_freqs(L, rot, name, code, kw):
    if name == "ntk" and rot == 2:
        with pytest.raises(nv.NVFP4Error):
            nv.nvfp4_rope_freqs(rot, 500000.0, code, **kw)
        return
    f, m = nv.nvfp4_rope_freqs(rot, 500000.0, code, **kw)
    rf, rm = oat.rope_freqs(rot, 500000.0, name, **kw)
    assert f.dtype == torch.float64 and f.shape == (rot // 2,)
    assert np.allclose(f.numpy(), rf, rtol=1e-13, atol=0) and m == pytest.approx(rm, rel=1e-15)


def test_rope_freqs_refusals(L):
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=2048), dict(rot_dim=32, theta=0.0),
               dict(rot_dim=32, theta=-1.0), dict(rot_dim=32, scaling=nv.ROPE_SCALE_LINEAR, factor=0.5),
               dict(rot_dim=32, scaling=nv.ROPE_SCALE_YARN, factor=2.0),
               dict(rot_dim=32, scaling=nv.ROPE_SCALE_YARN, factor=2.0, original_len=10.0, beta_fast=1.0),
               dict(rot_dim=32, theta=float("nan")), dict(rot_dim=32, theta=float("inf")),
               dict(rot_dim=32, scaling=nv.ROPE_SCALE_LINEAR, factor=float("inf"))):
        with pytest.raises(nv.NVFP4Error) as e:
            nv.nvfp4_rope_freqs(**kw)
        assert e.value.status == nv.ERR_SHAPE
    with pytest.raises(nv.NVFP4Error) as e:
        nv.nvfp4_rope_freqs(32, scaling=9)
    assert e.value.status == nv.ERR_MODE


# ---- host-side checks: nothing is launched ----------------------------------------

def desc(**kw):
    a = dict(data=0x10000, k_gs=0x20000, v_gs=0x20010, num_pages=4, page_size=16, heads=2, head_dim=64,
             format=nv.KV_NVFP4)
    a.update(kw)
    return nv.KvCacheDesc(a["data"], a["k_gs"], a["v_gs"], a["num_pages"], a["page_size"], a["heads"], a["head_dim"],
                          a["format"])


BAD_CACHES = [(dict(data=None), nv.ERR_NULL), (dict(k_gs=None), nv.ERR_NULL), (dict(v_gs=None), nv.ERR_NULL),
              (dict(format=3), nv.ERR_MODE), (dict(format=-1), nv.ERR_MODE), (dict(num_pages=0), nv.ERR_SHAPE),
              (dict(num_pages=1 << 31), nv.ERR_SHAPE), (dict(page_size=8), nv.ERR_SHAPE),
              (dict(page_size=24), nv.ERR_SHAPE), (dict(page_size=8192), nv.ERR_SHAPE),
              (dict(heads=0), nv.ERR_SHAPE), (dict(head_dim=96), nv.ERR_SHAPE), (dict(head_dim=512), nv.ERR_SHAPE),
              (dict(data=0x10008), nv.ERR_ALIGN), (dict(k_gs=0x20002), nv.ERR_ALIGN)]


def no_gpu(call, *a, **kw):
    """A valid call (with addresses that are not memory, so made only without a GPU) is
    refused for want of a B200 alone."""
    return torch.cuda.is_available() or call(*a, **kw) == nv.ERR_ARCH


def test_cache_bytes(L):
    assert nv.nvfp4_kv_cache_bytes(3, 32, 2, 128, nv.KV_BF16) == 3 * 2 * 32 * 2 * 256
    assert nv.nvfp4_kv_cache_bytes(3, 32, 2, 128, nv.KV_E4M3) == 3 * 2 * 32 * 2 * 128
    assert nv.nvfp4_kv_cache_bytes(3, 32, 2, 128, nv.KV_NVFP4) == 3 * 2 * 32 * 2 * 72
    assert nv.nvfp4_kv_cache_bytes(1 << 30, 4096, 8, 256, nv.KV_BF16) == (1 << 30) * 4096 * 8 * 1024   # past 2^32
    for a in ((0, 16, 1, 64, 0), (1, 17, 1, 64, 0), (1, 16, 0, 64, 0), (1, 16, 1, 80, 0), (1, 16, 1, 64, 3)):
        assert nv.nvfp4_kv_cache_bytes(*a) == 0


def test_rope_validation(L):
    def r(**kw):
        a = dict(x=FAKE, xd=nv.DTYPE_F32, T=2, heads=3, D=64, xl=256, pos=FAKE3, f=FAKE3, rot=64, lay=nv.ROPE_HALF, y=FAKE2,
                 yd=nv.DTYPE_BF16, yl=192)
        a.update(kw)
        return L.nvfp4_rope(a["x"], a["xd"], a["T"], a["heads"], a["D"], a["xl"], a["pos"], a["f"], a["rot"], a["lay"],
                            1.0, 0, a["y"], a["yd"], a["yl"], None)
    for n in ("x", "pos", "f", "y"):
        assert r(**{n: None}) == nv.ERR_NULL
    assert r(xd=2) == nv.ERR_DTYPE and r(yd=-1) == nv.ERR_DTYPE
    assert r(lay=2) == nv.ERR_LAYOUT
    for kw in (dict(T=0), dict(heads=0), dict(D=72), dict(D=2048, xl=6144, yl=6144), dict(rot=0), dict(rot=24),
               dict(rot=80), dict(xl=191), dict(yl=191), dict(y=FAKE), dict(y=FAKE, yd=nv.DTYPE_F32),
               dict(heads=70000, xl=1 << 23, yl=1 << 23), dict(T=1 << 31)):
        assert r(**kw) == nv.ERR_SHAPE, kw
    for kw in (dict(x=MISALIGNED), dict(y=MISALIGNED), dict(xl=194), dict(yl=196), dict(pos=ctypes.c_void_p(0x10004)),
               dict(f=ctypes.c_void_p(0x10004))):
        assert r(**kw) == nv.ERR_ALIGN, kw
    assert no_gpu(r)


def test_kv_validation(L):
    def w(c=None, **kw):
        a = dict(k=FAKE, v=FAKE2, xd=nv.DTYPE_BF16, T=4, kl=128, vl=256, s=FAKE3)
        a.update(kw)
        return L.nvfp4_kv_write(c if c is not None else ctypes.byref(desc()), a["k"], a["v"], a["xd"], a["T"], a["kl"],
                                a["vl"], a["s"], None)

    def rd(c=None, **kw):
        a = dict(k=FAKE, v=FAKE2, yd=nv.DTYPE_BF16, T=4, s=FAKE3)
        a.update(kw)
        return L.nvfp4_kv_read(c if c is not None else ctypes.byref(desc()), a["s"], a["T"], a["k"], a["v"], a["yd"],
                               None)

    def f(c=None, **kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE2, xd=nv.DTYPE_BF16, T=4, hq=4, ql=512, kl=512, vl=512, pos=FAKE3, s=FAKE3,
                 fr=FAKE3, rot=32, lay=0, qo=FAKE3)
        a.update(kw)
        return L.nvfp4_rope_kv_write(c if c is not None else ctypes.byref(desc()), a["q"], a["k"], a["v"], a["xd"],
                                     a["T"], a["hq"], a["ql"], a["kl"], a["vl"], a["pos"], a["s"], a["fr"], a["rot"],
                                     a["lay"], 1.0, a["qo"], None)
    for kw, status in BAD_CACHES:
        for call in (w, rd, f):
            assert call(ctypes.byref(desc(**kw))) == status, kw
    for call in (w, rd, f):
        assert no_gpu(call, ctypes.byref(desc(k_gs=None, v_gs=None, format=nv.KV_BF16)))
        assert call(s=None) == nv.ERR_NULL and call(k=None) == nv.ERR_NULL and call(v=None) == nv.ERR_NULL
        assert call(T=0) == nv.ERR_SHAPE
        assert call(k=MISALIGNED) == nv.ERR_ALIGN and call(s=ctypes.c_void_p(0x10004)) == nv.ERR_ALIGN
        assert no_gpu(call)
    assert L.nvfp4_kv_write(None, FAKE, FAKE, 1, 1, 128, 128, FAKE, None) == nv.ERR_NULL
    assert rd(v=FAKE) == nv.ERR_SHAPE                            # both outputs in one place
    assert w(xd=7) == nv.ERR_DTYPE and rd(yd=7) == nv.ERR_DTYPE and f(xd=7) == nv.ERR_DTYPE
    assert w(kl=127) == nv.ERR_SHAPE and w(vl=120) == nv.ERR_SHAPE and f(ql=248) == nv.ERR_SHAPE
    assert w(kl=132) == nv.ERR_ALIGN and no_gpu(w, kl=132, xd=nv.DTYPE_F32)
    assert f(q=None) == nv.ERR_NULL and f(qo=None) == nv.ERR_NULL and f(pos=None) == nv.ERR_NULL
    assert f(lay=5) == nv.ERR_LAYOUT and f(rot=72) == nv.ERR_SHAPE and f(rot=128) == nv.ERR_SHAPE
    assert f(hq=0) == nv.ERR_SHAPE and f(qo=FAKE) == nv.ERR_SHAPE


def test_attn_decode_validation(L):
    def a_(c=None, **kw):
        a = dict(q=FAKE, B=3, hq=8, ql=512, t=FAKE3, mp=5, tl=5, sl=FAKE3, sc=0.1, win=0, y=FAKE2, yd=nv.DTYPE_BF16,
                 lse=None, ws=FAKE2)
        a.update(kw)
        c = c if c is not None else ctypes.byref(desc())
        wsb = a.get("wsb", L.nvfp4_attn_decode_workspace(c, a["B"], a["hq"], a["mp"]))
        return L.nvfp4_attn_decode(a["q"], a["B"], a["hq"], a["ql"], c, a["t"], a["mp"], a["tl"], a["sl"], a["sc"],
                                   a["win"], a["y"], a["yd"], a["lse"], a["ws"], wsb, None)
    for kw, status in BAD_CACHES:
        assert a_(ctypes.byref(desc(**kw))) == status, kw
    assert L.nvfp4_attn_decode_workspace(None, 1, 1, 1) == 0
    for n in ("q", "t", "sl", "y"):
        assert a_(**{n: None}) == nv.ERR_NULL
    assert a_(yd=4) == nv.ERR_DTYPE
    for kw in (dict(B=0), dict(B=4097, tl=5), dict(hq=7), dict(hq=0), dict(mp=0), dict(tl=4), dict(win=-1), dict(ql=504),
               dict(sc=float("inf")), dict(sc=float("nan")), dict(mp=1 << 30, tl=1 << 30),
               dict(y=FAKE)):
        assert a_(**kw) == nv.ERR_SHAPE, kw
    for kw in (dict(q=MISALIGNED), dict(y=MISALIGNED), dict(ql=516), dict(t=ctypes.c_void_p(0x10002)),
               dict(sl=ctypes.c_void_p(0x10002)), dict(lse=ctypes.c_void_p(0x10002)), dict(ws=MISALIGNED)):
        assert a_(**kw) == nv.ERR_ALIGN, kw
    assert a_(ws=None) == nv.ERR_WORKSPACE and a_(wsb=64) == nv.ERR_WORKSPACE
    # the longest table: its tokens, and 32 behind them, are counted in 32 bits
    long = ctypes.byref(desc(page_size=16, heads=1))
    for pages, ok in (((1 << 27) - 1, False), ((1 << 27) - 4, False), ((1 << 27) - 5, True)):
        kw = dict(B=1, hq=1, mp=pages, tl=pages)
        assert no_gpu(a_, long, **kw) if ok else a_(long, **kw) == nv.ERR_SHAPE
    assert no_gpu(a_) and no_gpu(a_, lse=FAKE3) and no_gpu(a_, B=4096, mp=40_000, tl=40_000)


def test_python_refusals(L):
    cpu = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        nv.KVCache(cpu, 16, 2, 64, nv.KV_BF16)                   # not on a GPU
    with pytest.raises(ValueError):
        nv.KVCache(cpu, 20, 2, 64, nv.KV_BF16)
    with pytest.raises(ValueError):
        nv.KVCache.empty(0, 16, 2, 64, nv.KV_BF16)
    with pytest.raises(ValueError):
        nv.nvfp4_rope(torch.zeros(2, 3, 64), torch.zeros(2, dtype=torch.int64), torch.zeros(32, dtype=torch.float64))
