"""GPU decode attention over the paged cache against the fp64 oracle, within the bound
derived in attn_checks.attn_bounds; masked and unused rows hold NaN patterns throughout."""
import numpy as np
import pytest
import torch

import bit_linear_moe_b200 as nv
import oracle
from attn_checks import FMT, assert_close, attn_bounds, dev, device_cache, host
from bit_linear_moe_b200 import synth
from nvfp4_checks import assert_within_bound, rowmajor_to_tiled
from oracle import attention as oat
from oracle import stack as ost
from oracle.stack import bf16_round

pytestmark = pytest.mark.gpu

FMTS = (oat.BF16, oat.E4M3, oat.NVFP4)
# The host knows lengths only by the table's width: a narrow table is served by a cluster
# of CTAs per (sequence, key head), a wide one by an even split of all tiles.
WIDE = 600
WIDTHS = pytest.mark.parametrize("extra", [0, WIDE], ids=["narrow", "wide"])


class Batch:
    """Sequences of the given lengths in a shuffled paged cache filled with 0xFF (NaN in
    every format) outside their rows; queries as a slice of wider rows."""

    def __init__(self, fmt, D, Hkv, G, page, lens, seed=0, k_scale=1.0, extra_cols=0):
        rng = np.random.default_rng([seed, D, Hkv, G, len(lens)])
        self.fmt, self.D, self.Hkv, self.G, self.page, self.lens = fmt, D, Hkv, G, page, list(lens)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 2
        order = list(rng.permutation(pages)[:sum(need)])
        self.table = np.full((len(lens), max(1, max(need)) + extra_cols), -7, np.int32)   # unused entries: no page
        for b, n in enumerate(need):
            self.table[b, :n] = [order.pop() for _ in range(n)]
        gs = {oat.BF16: 1.0, oat.E4M3: 0.02, oat.NVFP4: 0.002}[fmt]
        self.oc = oat.Cache(pages, page, Hkv, D, fmt, gs * k_scale, gs)
        self.c = device_cache(self.oc)
        self.slots = []
        for b, n in enumerate(lens):
            t = np.arange(n)
            s = self.table[b, t // page].astype(np.int64) * page + t % page
            self.slots.append(s)
            if n:
                k = (k_scale * rng.standard_normal((n, Hkv, D))).astype(np.float32)
                v = (rng.standard_normal((n, Hkv, D)) + 0.3).astype(np.float32)
                nv.nvfp4_kv_write(self.c, dev(k), dev(v), dev(s))
        torch.cuda.synchronize()
        self.oc.data = self.c.data.cpu().numpy()                 # (the writes have a test of their own)
        q = rng.standard_normal((len(lens), Hkv * G + 3, D)).astype(np.float32)
        self.q = dev(q).to(torch.bfloat16)[:, 1:1 + Hkv * G]
        self.dtable, self.dlens = dev(self.table), dev(np.array(lens, np.int32))

    def run(self, **kw):
        return nv.nvfp4_attn_decode(self.q, self.c, self.dtable, self.dlens, want_lse=True, **kw)

    def rows(self, b, lo, n):
        """(k, v) [n - lo, Hkv, D] fp64 of tokens lo .. n - 1, vectorised from the bytes."""
        s = self.slots[b][lo:n]
        oc = self.oc
        out = np.zeros((2, len(s), self.Hkv, self.D))
        for r in range(16):
            at = s[s % 16 == r]
            if not len(at):
                continue
            pick = np.nonzero(s % 16 == r)[0]
            for h in range(self.Hkv):
                base = np.array([oc._tile(x, h) for x in at])
                for w in (0, 1):
                    code = oc.data[base[:, None] + (oc.code_at(r, 0, w) - oc._tile(r, 0))]
                    if self.fmt == oat.BF16:
                        val = (code.view("<u2").astype(np.uint32) << 16).view(np.float32).astype(np.float64)
                    elif self.fmt == oat.E4M3:
                        val = oat.e4m3_table()[code] * float(oc.gs[w])
                    else:
                        sc = oc.data[base[:, None] + (oc.scale_at(r, 0, w) - oc._tile(r, 0))]
                        val = oracle.dequantize(code, sc, oc.gs[w])
                    out[w, pick, h] = val
        return out

    def check(self, y, lse, window=0, scale=None, seqs=None, what=""):
        scale = self.D ** -0.5 if scale is None else scale
        for b in range(len(self.lens)) if seqs is None else seqs:
            n = self.lens[b]
            lo = max(0, n - window) if window else 0
            k, v = self.rows(b, lo, n)
            ry, rl, spread, mag = oat.attend(host(self.q[b]), k, v, scale)
            if n == 0:
                assert not y[b].float().any() and (lse[b] == -float("inf")).all()
                continue
            by, bl = attn_bounds(self.fmt, self.D, n - lo, ry, rl, spread, mag, np.abs(v).max(), y.dtype)
            assert_close(y[b], ry, by, f"{what} y[{b}] (len {n})")
            assert_close(lse[b], rl, bl, f"{what} lse[{b}] (len {n})")


LENS = (0, 1, 2, 15, 16, 17, 31, 48, 100, 129)


@WIDTHS
@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_lengths_around_tiles_and_pages(cuda_device, fmt, D, y_dtype, extra):
    b = Batch(fmt, D, 2, 4, 32, LENS, extra_cols=extra)
    y, lse = b.run(y_dtype=y_dtype)
    b.check(y, lse)
    assert nv.nvfp4_read_device_status() == nv.OK


@WIDTHS
@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("fmt,D", [(oat.NVFP4, 128), (oat.NVFP4, 256), (oat.E4M3, 64), (oat.BF16, 128)])
def test_query_heads_per_key_head(cuda_device, fmt, D, G, extra):
    b = Batch(fmt, D, 3, G, 16, (37, 200, 5), extra_cols=extra)
    b.check(*b.run())


@pytest.mark.parametrize("fmt,D,page", [(oat.NVFP4, 128, 48), (oat.NVFP4, 64, 256), (oat.E4M3, 128, 16),
                                        (oat.BF16, 256, 64)])
@pytest.mark.parametrize("window,extra", [(1, 0), (16, 0), (40, 0), (1000, 0), (5000, WIDE)])
def test_window(cuda_device, fmt, D, page, window, extra):
    b = Batch(fmt, D, 2, 2, page, (0, 1, 16, 41, 300, 513, 5300), extra_cols=extra)
    b.check(*b.run(window=window), window=window)


@pytest.mark.parametrize("y_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,Hkv,G,lens", [
    (128, 1, 8, (9001,)), (128, 2, 2, (4097, 33)), (64, 1, 16, (20000,)), (256, 1, 3, (6000, 0, 700)),
    (128, 4, 2, tuple(int(x) for x in np.random.default_rng(2).integers(0, 700, 60)))])
@WIDTHS
def test_work_split_over_ctas(cuda_device, fmt, D, Hkv, G, lens, extra, y_dtype):
    """Long sequences over many CTAs, and ragged batches whose segments end anywhere in a
    CTA's or a warp's range; fp32 output shows a join that lost or doubled a piece."""
    b = Batch(fmt, D, Hkv, G, 64, lens, extra_cols=extra)
    y, lse = b.run(y_dtype=y_dtype)
    b.check(y, lse)
    y2, lse2 = b.run(y_dtype=y_dtype)
    assert torch.equal(y, y2) and torch.equal(lse, lse2)         # the same bits


@WIDTHS
@pytest.mark.parametrize("fmt", FMTS)
def test_sharp_and_flat_scores(cuda_device, fmt, extra):
    """Large keys (one token takes almost all weight, the maximum rises often) and scale 0."""
    b = Batch(fmt, 128, 2, 4, 16, (700, 64), k_scale=30.0, extra_cols=extra)
    b.check(*b.run())
    b.check(*b.run(scale=0.0), scale=0.0)
    b.check(*b.run(scale=-0.05), scale=-0.05)


def test_queries_of_unequal_size(cuda_device):
    """The fp16 prescale of the queries: heads far apart in size, tiny and zero heads."""
    b = Batch(oat.NVFP4, 128, 2, 4, 16, (100, 30))
    f = torch.tensor([1e-30, 1.0, 0.0, 1e20, 1e-6, 300.0, 1e4, 1e-38], device="cuda")
    b.q = (b.q.float() * f[None, :, None]).to(torch.bfloat16)
    y, lse = b.run(scale=1e-3)
    b.q[:, 3] = 0                                                # (e^(1e17) has no finite bound; checked apart)
    keep = [h for h in range(8) if h != 3]
    for s in range(2):
        k, v = b.rows(s, 0, b.lens[s])
        ry, rl, spread, mag = oat.attend(host(b.q[s]), k, v, 1e-3)
        by, bl = attn_bounds(b.fmt, 128, b.lens[s], ry, rl, spread, mag, np.abs(v).max(), y.dtype)
        assert_close(y[s][keep], ry[keep], by[keep], "y")
        assert_close(lse[s][keep], rl[keep], bl[keep], "lse")
    assert torch.isfinite(y[:, 3]).all()                         # one token has all the weight


@WIDTHS
def test_nan_and_infinity_stay_where_they_are(cuda_device, extra):
    b = Batch(oat.BF16, 128, 2, 2, 16, (40, 40, 40), extra_cols=extra)
    base, base_lse = b.run()
    b.q = b.q.clone()
    b.q[1, 2] = float("nan")
    y, lse = b.run()
    assert torch.isnan(y[1, 2]).all() and torch.isnan(lse[1, 2])
    rest = torch.ones((3, 4), dtype=torch.bool, device="cuda")
    rest[1, 2] = False
    assert torch.equal(y[rest], base[rest]) and torch.equal(lse[rest], base_lse[rest])
    # every score -inf: nothing to weigh, zeros (keys of -inf against positive queries)
    b.q = torch.ones_like(b.q)
    k = torch.full((40, 2, 128), -float("inf"), device="cuda")
    nv.nvfp4_kv_write(b.c, k, torch.ones_like(k), dev(b.slots[2]))
    y, lse = b.run()
    assert not y[2].any() and (lse[2] == -float("inf")).all()
    # a value of +inf in a seen row: its element is not finite, the other key head's are
    v = torch.zeros((1, 2, 128), device="cuda")
    v[0, 1, 5] = float("inf")
    nv.nvfp4_kv_write(b.c, torch.zeros_like(v), v, dev(b.slots[0][3:4]))
    y, _ = b.run()
    assert not torch.isfinite(y[0, 2:, 5]).any() and torch.isfinite(y[0, :2]).all()


def test_shared_pages_and_table_views(cuda_device):
    """Two sequences share a prefix's pages; the table is a column slice of a wider one."""
    b = Batch(oat.NVFP4, 128, 2, 4, 16, (64, 80, 64), extra_cols=3)
    b.table[0, :2] = b.table[1, :2]
    b.slots[0][:32] = b.slots[1][:32]
    wide = torch.full((3, 20), -1, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + b.table.shape[1]] = dev(b.table)
    b.dtable = wide[:, 4:4 + b.table.shape[1]]
    b.check(*b.run())


@WIDTHS
def test_bad_pages_and_lengths_are_reported(cuda_device, extra):
    """Indexes out of range are caught by the kernel's own check (page 0 is read in their
    place, lengths are cut to the table) and named in the status word; other sequences
    are right."""
    b = Batch(oat.NVFP4, 128, 2, 4, 16, (64, 80, 64), extra_cols=extra)
    b.dtable[1, 2] = 1 << 20
    y, lse = b.run()
    assert nv.nvfp4_read_device_status() == nv.ERR_PAGE
    b.check(y, lse, seqs=(0, 2))
    b.dtable[1, 2] = -3
    y, lse = b.run()
    assert nv.nvfp4_read_device_status() == nv.ERR_PAGE
    b.check(y, lse, seqs=(0, 2))
    b.dtable.copy_(dev(b.table))
    b.dlens[1] = 1 << 30
    y, lse = b.run()
    assert nv.nvfp4_read_device_status() == nv.ERR_PAGE
    b.dlens[1] = -4                                              # like 0
    y, lse = b.run()
    assert nv.nvfp4_read_device_status() == nv.OK and not y[1].any() and (lse[1] == -float("inf")).all()
    b.check(y, lse, seqs=(0, 2))


@WIDTHS
def test_nothing_outside_the_outputs_is_written(cuda_device, extra):
    b = Batch(oat.E4M3, 64, 2, 3, 16, (0, 130, 7), extra_cols=extra)
    before = b.c.data.clone()
    need = nv.nvfp4_attn_decode_workspace(b.c, 3, 6, b.table.shape[1])
    room = torch.full((need + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    out = torch.full((5, 6, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    y, lse = b.run(y=out[1:4], ws=room[256:256 + need])
    b.check(y, lse)
    assert (out[0] == 9).all() and (out[4] == 9).all()
    assert (room[:256] == 0xAB).all() and (room[256 + need:] == 0xAB).all()
    assert torch.equal(b.c.data, before)


@WIDTHS
def test_large_batch(cuda_device, extra):
    """More sequences than threads in a CTA (the list is scanned in pieces)."""
    lens = [int(x) for x in np.random.default_rng(4).integers(0, 40, 1500)]
    b = Batch(oat.NVFP4, 64, 1, 2, 16, lens, extra_cols=extra)
    y, lse = b.run()
    b.check(y, lse, seqs=list(range(0, 1500, 37)) + [0, 255, 256, 511, 512, 1499])


@pytest.mark.parametrize("D,fmt", [(64, oat.NVFP4), (256, oat.BF16)])
@pytest.mark.parametrize("max_pages", [4, 1200])
def test_largest_batch(cuda_device, D, fmt, max_pages):
    """4,096 sequences that share their pages, 64 of each length 0 .. 63: every one is held to
    the oracle's bound (the work split, and with it the rounding, differs between them)."""
    one = Batch(fmt, D, 2, 2, 16, tuple(range(64)))
    B = 4096
    lens = torch.arange(B, device="cuda", dtype=torch.int32) % 64
    table = torch.zeros((B, max_pages), dtype=torch.int32, device="cuda")
    table[:, :4] = one.dtable[63, :4]
    q = one.q[:1].expand(B, -1, -1).contiguous()
    y, lse = nv.nvfp4_attn_decode(q, one.c, table, lens, want_lse=True)
    for n in range(64):
        k, v = one.rows(63, 0, n)
        ry, rl, spread, mag = oat.attend(host(q[0]), k, v, D ** -0.5)
        if n:
            by, bl = attn_bounds(fmt, D, n, ry, rl, spread, mag, np.abs(v).max(), y.dtype)
            for i in range(n, B, 64):
                assert_close(y[i], ry, by, f"y, sequence {i}")
                assert_close(lse[i], rl, bl, f"lse, sequence {i}")
        else:
            assert not y[::64].any() and (lse[::64] == -torch.inf).all()


@WIDTHS
def test_captured_graphs_share_a_workspace(cuda_device, extra):
    """Two captured calls with one workspace, replayed in turn on lengths that change on
    the device between replays."""
    a = Batch(oat.NVFP4, 128, 2, 4, 16, (600, 33), seed=1, extra_cols=extra)
    c = Batch(oat.BF16, 64, 1, 3, 32, (90, 1, 500), seed=2, extra_cols=extra)
    n = max(nv.nvfp4_attn_decode_workspace(x.c, len(x.lens), x.Hkv * x.G, x.table.shape[1]) for x in (a, c))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for x in (a, c):
        x.run(ws=ws)
    torch.cuda.synchronize()
    graphs = []
    for x in (a, c):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = x.run(ws=ws)
        graphs.append((g, out))
    full = [list(x.lens) for x in (a, c)]
    for cut in (0, 7, 20):
        for x, lens in zip((a, c), full):
            x.lens = [max(0, n - cut) for n in lens]
            x.dlens.copy_(dev(np.array(x.lens, np.int32)))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, (_, (y, lse)) in zip((a, c), graphs):
            x.check(y, lse)


@WIDTHS
def test_two_streams_at_once(cuda_device, extra):
    """Concurrent calls with workspaces of their own."""
    a = Batch(oat.NVFP4, 128, 4, 4, 16, (2000, 900), seed=1, extra_cols=extra)
    c = Batch(oat.E4M3, 128, 4, 2, 32, (1500, 3000), seed=2, extra_cols=extra)
    ref = [x.run() for x in (a, c)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(10):
        for st, x in zip(s, (a, c)):
            with torch.cuda.stream(st):
                got.append(x.run())
    torch.cuda.synchronize()
    for i, (y, lse) in enumerate(got):
        assert torch.equal(y, ref[i % 2][0]) and torch.equal(lse, ref[i % 2][1])


def test_cache_past_4_gib(cuda_device):
    """Pages beyond 2^32 bytes."""
    Hkv, D, page, n = 2, 256, 64, 150
    per = nv.nvfp4_kv_cache_bytes(1, page, Hkv, D, nv.KV_BF16)
    pages = (1 << 32) // per + 10
    c = nv.KVCache.empty(pages, page, Hkv, D, nv.KV_BF16)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((n, Hkv, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    t = torch.arange(n, device="cuda")
    nv.nvfp4_kv_write(c, k, v, table[0].long()[t // page] * page + t % page)
    q = torch.randn((1, 8, D), generator=g, device="cuda").to(torch.bfloat16)
    y, lse = nv.nvfp4_attn_decode(q, c, table, torch.tensor([n], dtype=torch.int32, device="cuda"), want_lse=True)
    ry, rl, spread, mag = oat.attend(host(q[0]), host(k), host(v), D ** -0.5)
    by, bl = attn_bounds(oat.BF16, D, n, ry, rl, spread, mag, np.abs(host(v)).max(), y.dtype)
    assert_close(y[0], ry, by, "y")
    assert_close(lse[0], rl, bl, "lse")


# ---- the run of them, as a decode step uses them ------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
def test_decode_steps_of_a_layer(cuda_device, fmt):
    """A prefill chunk and three decode steps of one layer on small shapes (hidden 512, 8
    query and 2 key heads of 64, fused QKV 768 wide): QKV linear -> rotation and cache
    write -> attention -> rms -> output linear, each stage against the oracle on the GPU's
    own input to it, the cache against a model kept beside it."""
    hid, Hq, Hkv, D, page, B = 512, 8, 2, 64, 16, 3
    N = (Hq + 2 * Hkv) * D
    rng = np.random.default_rng(77)
    wq, wo = oracle.quantize(synth.weight(rng, N, hid)), oracle.quantize(synth.weight(rng, hid, Hq * D))

    def weights(w, n, k):
        return (dev(w[0]), dev(rowmajor_to_tiled(w[1], n, k).ravel()), torch.tensor([w[2]], device="cuda"))
    dq, do = weights(wq, N, hid), weights(wo, hid, Hq * D)
    freqs = nv.nvfp4_rope_freqs(D)[0]
    df = freqs.cuda()
    oc = oat.Cache(12, page, Hkv, D, fmt, {oat.BF16: 1.0, oat.E4M3: 0.01, oat.NVFP4: 0.0015}[fmt],
                   {oat.BF16: 1.0, oat.E4M3: 0.008, oat.NVFP4: 0.001}[fmt])
    c = device_cache(oc)
    table = rng.permutation(12).reshape(B, 4).astype(np.int32)
    lens = np.array([20, 15, 1])

    def write(x, pos, seq):
        """QKV linear and the fused step for rows of sequences `seq` at positions `pos`."""
        qkv = nv.nvfp4_linear(x, *dq, w_sf_layout=nv.SF_TILED, mode=nv.MODE_W4A16)
        rows = qkv.view(-1, Hq + 2 * Hkv, D)
        slots = table[seq, pos // page].astype(np.int64) * page + pos % page
        q = nv.nvfp4_rope_kv_write(c, rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], dev(pos), dev(slots), df)
        ref, ad = oracle.linear_w4a16(x.float().cpu().numpy(), *wq)
        assert_within_bound(qkv, ref, ad, False, "qkv")
        # the cache model: the kernel's own rotated keys (bf16), tested apart
        kr = nv.nvfp4_rope(rows[:, Hq:Hq + Hkv], dev(pos), df)
        oc.write(kr.float().cpu().numpy(), rows[:, Hq + Hkv:].cpu().numpy(), slots)
        return q

    for b in range(B):                                           # prefill, sequence by sequence
        x = dev(bf16_round(rng.standard_normal((lens[b], hid)))).to(torch.bfloat16)
        write(x, np.arange(lens[b]), np.full(lens[b], b))
    assert np.array_equal(c.data.cpu().numpy(), oc.data)
    x = dev(bf16_round(rng.standard_normal((B, hid)))).to(torch.bfloat16)
    for step in range(3):
        q = write(x, lens, np.arange(B))
        lens = lens + 1
        assert np.array_equal(c.data.cpu().numpy(), oc.data)
        y = nv.nvfp4_attn_decode(q, c, dev(table), dev(lens.astype(np.int32)), y_dtype=torch.float32)
        for b in range(B):
            t = np.arange(lens[b])
            k, v = oc.read(table[b, t // page].astype(np.int64) * page + t % page)
            ry, rl, spread, mag = oat.attend(host(q[b]), k, v, D ** -0.5)
            by, _ = attn_bounds(fmt, D, lens[b], ry, rl, spread, mag, np.abs(v).max(), y.dtype)
            assert_close(y[b], ry, by, f"step {step} y[{b}]")
        o_in = nv.nvfp4_rms_norm(y.view(B, Hq * D))
        o = nv.nvfp4_linear(o_in, *do, w_sf_layout=nv.SF_TILED, mode=nv.MODE_W4A16)
        ref, ad = oracle.linear_w4a16(host(o_in).astype(np.float32), *wo)
        assert_within_bound(o, ref, ad, False, "o")
        x = nv.nvfp4_rms_norm(o)
        assert np.abs(host(x) - ost.rms_norm_exact(host(o))).max() <= 2.0 ** -7 * 8
    assert nv.nvfp4_read_device_status() == nv.OK
