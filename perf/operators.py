"""The attention side of a decode step, as measured: rotary positions, the paged key-value cache (written with
quantization, read back) and attention of one new token per sequence over it.

``run`` makes one pass through one operator.  With ``own`` false it computes the operator's plain form from elementary
torch operations in fp32 (angles in fp64); with ``own`` true it calls the library.  ``exact`` computes the same outputs
from the definitions in fp64, without either.

A case's ``kind``:

* ``rope``   rotary positions of the query and key heads of fused QKV rows;
* ``cache``  a chunk's keys and values quantized into cache pages, then a context read back as dense bf16;
* ``step``   both at once: queries rotated, rotated keys and values written to the cache, the chunk's rows read back;
* ``attn``   attention of one new token per sequence over the paged cache.

The cache (one byte tensor) is ``[pages, heads, page_size / 16]`` tiles of 16 tokens.  A tile holds the 16 key rows, the
16 value rows, and (NVFP4) the 16 + 16 rows of E4M3 block scales.  A row's 16-byte pieces are stored permuted: piece c of
the tile's token r lies at c ^ (((r & 6) ^ ((r & 1) << 2)) & (pieces - 1)).
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
HALF, INTERLEAVED = 0, 1


def device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ------------------------------------------------------------------ cases ----

def listed():
    wide = {"Hq": 40, "Hkv": 20, "D": 128}     # the 27B-shaped decoder's fused QKV: 10240 = (40 + 2 * 20) * 128
    gqa = {"Hq": 32, "Hkv": 8, "D": 128}
    return [
        # one token's queries and keys deep in a context, straight from the fp32 QKV output: latency
        {"name": "rope-decode-1", "kind": "rope", "T": 1, **wide, "rot": 128, "layout": "half", "x": "f32",
         "scaling": "none", "start": 100003},
        # a prefill chunk of odd length, half of each head rotated in interleaved pairs, frequencies stretched
        {"name": "rope-prefill-8191", "kind": "rope", "T": 8191, **gqa, "rot": 64, "layout": "interleaved",
         "x": "bf16", "scaling": "yarn", "start": 65536},
        # a few tokens of a small model into an E4M3 cache, its short context read back: latency
        {"name": "cache-small-e4m3", "kind": "cache", "T": 5, "R": 133, "Hkv": 2, "D": 64, "fmt": "e4m3", "x": "bf16",
         "page": 16},
        # a 2,048-token prefill chunk into the NVFP4 cache and the 10,240 tokens so far read back for its attention
        {"name": "cache-prefill-nvfp4", "kind": "cache", "T": 2048, "R": 10240, "Hkv": 20, "D": 128, "fmt": "nvfp4",
         "x": "bf16", "page": 64},
        # the step between the QKV linear and attention for 32 decoding sequences, one of them a padding row
        {"name": "step-decode-32-nvfp4", "kind": "step", "T": 32, **wide, "rot": 128, "layout": "half", "x": "f32",
         "scaling": "none", "fmt": "nvfp4", "page": 16, "pad": True, "start": 4096},
        # the same for a prefill chunk with an unquantized cache
        {"name": "step-prefill-2048-bf16", "kind": "step", "T": 2048, **gqa, "rot": 128, "layout": "half", "x": "bf16",
         "scaling": "linear", "fmt": "bf16", "page": 64, "pad": False, "start": 8192},
        # a single user early in a conversation: latency
        {"name": "attn-1x97-nvfp4", "kind": "attn", "B": 1, "ctx": 97, **wide, "fmt": "nvfp4", "page": 16,
         "ragged": False, "window": 0},
        # a single user, 8K context
        {"name": "attn-1x8192-nvfp4", "kind": "attn", "B": 1, "ctx": 8192, **wide, "fmt": "nvfp4", "page": 64,
         "ragged": False, "window": 0},
        # a full decode batch of unequal contexts, an empty one among them: the largest case
        {"name": "attn-32x16384-nvfp4", "kind": "attn", "B": 32, "ctx": 16384, **wide, "fmt": "nvfp4", "page": 64,
         "ragged": True, "window": 0},
        # one long document
        {"name": "attn-1x131071-e4m3", "kind": "attn", "B": 1, "ctx": 131071, **gqa, "fmt": "e4m3", "page": 128,
         "ragged": False, "window": 0},
        # many short contexts, sixteen query heads on each key head, unquantized cache
        {"name": "attn-64x2048-bf16", "kind": "attn", "B": 64, "ctx": 2048, "Hq": 32, "Hkv": 2, "D": 64, "fmt": "bf16",
         "page": 32, "ragged": True, "window": 0},
        # wide heads that see the last 1,000 tokens only
        {"name": "attn-16x4000-window", "kind": "attn", "B": 16, "ctx": 4000, "Hq": 16, "Hkv": 8, "D": 256,
         "fmt": "nvfp4", "page": 16, "ragged": True, "window": 1000},
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(("rope", "cache", "step", "attn", "attn", "attn"))
    hkv = rng.choice((1, 2, 4, 5, 8, 20))
    d = rng.choice((64, 128, 128, 256))
    heads = {"Hq": hkv * rng.choice((1, 2, 3, 4, 5, 8, 16)), "Hkv": hkv, "D": d}
    if heads["Hq"] > 64:
        heads["Hq"] = hkv * 2
    fmt = rng.choice(("bf16", "e4m3", "nvfp4", "nvfp4"))
    page = rng.choice((16, 32, 64, 128))
    turn = {"rot": rng.choice([r for r in (32, 64, 96, 128, 256) if r <= d]), "layout": rng.choice(("half", "interleaved")),
            "scaling": rng.choice(("none", "linear", "yarn")), "start": log_int(1, 1 << 20)}
    x = rng.choice(("bf16", "f32"))
    width = (heads["Hq"] + 2 * hkv) * d
    most = max(4, min(8192, 20_000_000 // width))
    if kind == "rope":
        return {"kind": kind, "T": log_int(1, most), **heads, **turn, "x": x}
    if kind == "cache":
        t = log_int(1, max(2, min(4096, 4_000_000 // (hkv * d))))
        return {"kind": kind, "T": t, "R": t + log_int(1, max(2, min(16384, 20_000_000 // (hkv * d)))), "Hkv": hkv,
                "D": d, "fmt": fmt, "x": x, "page": page}
    if kind == "step":
        return {"kind": kind, "T": log_int(1, most), **heads, **turn, "x": x, "fmt": fmt, "page": page,
                "pad": rng.random() < 0.3}
    b = log_int(1, 128)
    per_token = 2 * hkv * row_bytes(fmt, d) * b
    ctx = log_int(1, max(16, min(131072, 600_000_000 // per_token, 600_000_000 // (hkv * d * b))))
    return {"kind": kind, "B": b, "ctx": ctx, **heads, "fmt": fmt, "page": page, "ragged": rng.random() < 0.6,
            "window": log_int(1, ctx) if rng.random() < 0.25 else 0}


# ------------------------------------------------------- layout of the cache ----

def code_bytes(fmt, d):
    return {"bf16": 2 * d, "e4m3": d, "nvfp4": d // 2}[fmt]


def scale_bytes(fmt, d):
    return d // 16 if fmt == "nvfp4" else 0


def row_bytes(fmt, d):
    return code_bytes(fmt, d) + scale_bytes(fmt, d)


def pieces(cache, fmt, d, which):
    """The key (0) or value (1) rows as [pages, heads, tiles, 16 tokens, pieces, 16 bytes], a view."""
    n = 16 * code_bytes(fmt, d)
    return cache[..., which * n:(which + 1) * n].unflatten(-1, (16, code_bytes(fmt, d) // 16, 16))


def block_scales(cache, fmt, d, which):
    """The block scales as [pages, heads, tiles, 16 tokens, d / 16], a view; None for the other formats."""
    if fmt != "nvfp4":
        return None
    n, first = 16 * scale_bytes(fmt, d), 32 * code_bytes(fmt, d)
    return cache[..., first + which * n:first + (which + 1) * n].unflatten(-1, (16, d // 16))


def placed(r, n, dev):
    """Where the n pieces of token r of a tile lie (its own inverse)."""
    f = ((r & 6) ^ ((r & 1) << 2)) & (n - 1)
    return torch.arange(n, device=dev) ^ f[..., None]


# ------------------------------------------------------------------ plain form ----

def values(raw, scales, fmt, gs):
    """fp32 values of code bytes [..., code_bytes] and block scales [..., d / 16]."""
    if fmt == "bf16":
        return raw.contiguous().view(torch.bfloat16).float()
    if fmt == "e4m3":
        return raw.contiguous().view(torch.float8_e4m3fn).float() * gs
    v = torch.tensor(E2M1 + tuple(-a for a in E2M1), device=raw.device)
    both = torch.stack((v.repeat(16), v.repeat_interleave(16)), -1)      # the two values of every byte
    v = both.index_select(0, raw.reshape(-1).int()).view(*scales.shape, 16)
    return (v * scales.contiguous().view(torch.float8_e4m3fn).float()[..., None] * gs).flatten(-2)


def coded(x, fmt, gs):
    """Code bytes and block scales of fp32 values [..., d]."""
    if fmt == "bf16":
        return x.to(torch.bfloat16).view(torch.uint8), None
    if fmt == "e4m3":
        return (x / gs).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), None
    b = x.unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / (gs * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    r = (s.float() * gs)[..., None]
    a = torch.where(r > 0, b.abs() / r, torch.zeros_like(b))
    c = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() +
         (a >= 3.5).byte() + (a > 5.0).byte())
    c = (c + 8 * ((b < 0) & (r > 0)).byte()).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), s.view(torch.uint8)


def write_rows(cache, fmt, page, slots, which, raw, scales):
    """Rows [T, heads, ...] to their slots (page 0 is nobody's: rows without a slot leave it as it is)."""
    t, h, d = raw.shape[0], raw.shape[1], raw.shape[2] * 8 // {"bf16": 16, "e4m3": 8, "nvfp4": 4}[fmt]
    keep, at = (slots >= 0)[:, None, None], slots.clamp(min=0)
    i = (at // page)[:, None], torch.arange(h, device=raw.device)[None], (at % page // 16)[:, None], (at % 16)[:, None]
    p = pieces(cache, fmt, d, which)
    new = raw.unflatten(-1, (-1, 16))
    where = placed(at % 16, new.shape[2], raw.device)[:, None, :].expand(t, h, -1)
    new = new.gather(2, where[..., None].expand_as(new))
    p[i] = torch.where(keep[..., None], new, p[i])
    if scales is not None:
        s = block_scales(cache, fmt, d, which)
        s[i] = torch.where(keep, scales, s[i])


def read_rows(cache, fmt, d, page, slots, which, gs):
    """fp32 rows [R, heads, d] of the slots, zeros for the negative ones."""
    at = slots.clamp(min=0)
    h = torch.arange(cache.shape[1], device=cache.device)[None]
    i = (at // page)[:, None], h, (at % page // 16)[:, None], (at % 16)[:, None]
    raw = pieces(cache, fmt, d, which)[i]
    where = placed(at % 16, raw.shape[2], cache.device)[:, None, :, None].expand_as(raw)
    raw = raw.gather(2, where).flatten(-2)
    s = block_scales(cache, fmt, d, which)
    return torch.where((slots >= 0)[:, None, None], values(raw, None if s is None else s[i], fmt, gs), 0.0)


def rotated(x, positions, freqs, layout, mscale):
    """Rotary positions of x [T, heads, d] fp32; freqs in turns per token (fp64), rot = 2 * len(freqs)."""
    turns = positions.double()[:, None] * freqs
    angle = (turns - turns.round()) * (2 * math.pi)
    c, s = (torch.cos(angle) * mscale).float()[:, None], (torch.sin(angle) * mscale).float()[:, None]
    n = freqs.numel()
    y = x.clone()
    if layout == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        y[..., :n], y[..., n:2 * n] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a * c - b * s, b * c + a * s
    return y


def attended(s):
    q, fmt, d = s["q"].float(), s["fmt"], s["D"]
    b, hq = q.shape[0], q.shape[1]
    h = s["cache"].shape[1]
    table, lens = s["table"].long(), s["lens"].long()
    n = table.shape[1] * s["page"]
    r = torch.arange(16, device=q.device)
    pos = torch.arange(n, device=q.device)
    seen = (pos < lens[:, None]) & (pos >= (lens[:, None] - s["window"] if s["window"] else 0))     # [B, n]
    held = s["cache"][table]                                                  # [B, pages, heads, tiles, bytes]

    def dense(which, gs):
        p = pieces(held, fmt, d, which)
        raw = p[..., r[:, None], placed(r, p.shape[-2], q.device), :].flatten(-2)
        sc = block_scales(held, fmt, d, which)
        return values(raw, sc, fmt, gs).permute(0, 2, 1, 3, 4, 5).reshape(b, h, n, d)

    qs = q.view(b, h, hq // h, d) * s["scale"]
    score = torch.matmul(qs, dense(0, s["k_gs"]).transpose(2, 3)).masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    v = dense(1, s["v_gs"]).masked_fill(~seen[:, None, :, None], 0.0)
    y = torch.matmul(w, v) / w.sum(-1, keepdim=True)
    y = torch.where(seen.any(-1)[:, None, None, None], y, 0.0)
    return y.reshape(b, hq, d).to(torch.bfloat16)


def plain(s):
    kind = s["kind"]
    if kind == "attn":
        return attended(s)
    if kind == "rope":
        return rotated(s["x"].float(), s["positions"], s["freqs"], s["layout"], s["mscale"]).to(torch.bfloat16)
    k, v, q = s["k"].float(), s["v"].float(), None
    if kind == "step":
        q = rotated(s["q"].float(), s["positions"], s["freqs"], s["layout"], s["mscale"]).to(torch.bfloat16)
        k = rotated(k, s["positions"], s["freqs"], s["layout"], s["mscale"]).to(torch.bfloat16).float()
    a = s["cache"], s["fmt"], s["page"], s["slots"]
    write_rows(*a, 0, *coded(k, s["fmt"], s["k_gs"]))
    write_rows(*a, 1, *coded(v, s["fmt"], s["v_gs"]))
    a = s["cache"], s["fmt"], s["D"], s["page"], s["read"]
    k, v = (read_rows(*a, w, gs).to(torch.bfloat16) for w, gs in ((0, s["k_gs"]), (1, s["v_gs"])))
    return {"k": k, "v": v} if q is None else {"q": q, "k": k, "v": v}


# ------------------------------------------------------------------- the library ----

def library(s):
    import bit_linear_moe_b200 as nv
    layout = nv.ROPE_INTERLEAVED if s.get("layout") == "interleaved" else nv.ROPE_HALF
    if s["kind"] == "rope":
        return nv.nvfp4_rope(s["x"], s["positions"], s["freqs"], layout=layout, mscale=s["mscale"])
    if "handle" not in s:                       # a program's own cache object and workspace, kept beside the cache
        fmt = {"bf16": nv.KV_BF16, "e4m3": nv.KV_E4M3, "nvfp4": nv.KV_NVFP4}[s["fmt"]]
        s["handle"] = nv.KVCache(s["cache"], page_size=s["page"], heads=s["cache"].shape[1], head_dim=s["D"], format=fmt,
                                 k_gs=s["k_gs"], v_gs=s["v_gs"])
        if s["kind"] == "attn":
            n = nv.nvfp4_attn_decode_workspace(s["handle"], s["q"].shape[0], s["q"].shape[1], s["table"].shape[1])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=s["q"].device)
    if s["kind"] == "attn":
        return nv.nvfp4_attn_decode(s["q"], s["handle"], s["table"], s["lens"], scale=s["scale"], window=s["window"],
                                    ws=s["ws"])
    if s["kind"] == "step":
        q = nv.nvfp4_rope_kv_write(s["handle"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freqs"],
                                   layout=layout, mscale=s["mscale"])
        k, v = nv.nvfp4_kv_read(s["handle"], s["read"])
        return {"q": q, "k": k, "v": v}
    nv.nvfp4_kv_write(s["handle"], s["k"], s["v"], s["slots"])
    k, v = nv.nvfp4_kv_read(s["handle"], s["read"])
    return {"k": k, "v": v}


def run(state):
    return library(state) if own else plain(state)


# ------------------------------------------------------------------------ inputs ----

def frequencies(rot, scaling):
    """(turns per token of each pair, magnitude of cos and sin): base 10,000; contexts stretched eight times."""
    f = [10000.0 ** (-2.0 * i / rot) / (2 * math.pi) for i in range(rot // 2)]
    if scaling == "linear":
        return [a / 8 for a in f], 1.0
    if scaling == "yarn":   # fast pairs keep their frequency, slow ones are stretched, a ramp in between
        full = [max(0.0, min(1.0, (a * 8192 - 1.0) / (32.0 - 1.0))) for a in f]
        return [a * w + a / 8 * (1 - w) for a, w in zip(f, full)], 0.1 * math.log(8) + 1
    return f, 1.0


def lengths(case):
    """Contexts in a fixed spread (the seed decides which sequence has which); ragged batches of 8 and more have one
    empty sequence and one of a single token."""
    b, ctx = case["B"], case["ctx"]
    if not case["ragged"]:
        return [ctx] * b
    n = [max(1, ctx - (i * ctx) // b) for i in range(b)]
    if b >= 8:
        n[-1], n[-2] = 0, 1
    return n


def heads_like(gen, t, h, d, dev):
    """N(0, 1) values with a few strong channels, as keys have them."""
    x = torch.randn((t, h, d), generator=gen, device=dev)
    strong = torch.randint(0, d, (h, 4), generator=gen, device=dev)
    return x.scatter(2, strong[None].expand(t, -1, -1), 3.0 * x.gather(2, strong[None].expand(t, -1, -1)))


def global_scale(x, fmt):
    return (x.abs().amax() / {"bf16": 1.0, "e4m3": 448.0, "nvfp4": 2688.0}[fmt]).reshape(1)


def prepare(case, seed):
    dev = device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    d, hkv, kind = case["D"], case["Hkv"], case["kind"]
    s = {"kind": kind, "D": d}
    xt = torch.float32 if case.get("x") == "f32" else torch.bfloat16
    if kind in ("rope", "step"):
        f, s["mscale"] = frequencies(case["rot"], case["scaling"])
        s["freqs"] = torch.tensor(f, dtype=torch.float64, device=dev)
        s["layout"] = case["layout"]
        first = case["start"] + rng.randrange(1000)
        s["positions"] = torch.arange(first, first + case["T"], device=dev)
    if kind in ("rope", "step"):
        hq = case["Hq"]
        rows = torch.cat((torch.randn((case["T"], hq, d), generator=gen, device=dev),
                          heads_like(gen, case["T"], 2 * hkv, d, dev)), 1).to(xt)      # fused QKV output rows
        if kind == "rope":
            s["x"] = rows[:, :hq + hkv]
            return s
        s["q"], s["k"], s["v"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    if kind == "cache":
        rows = heads_like(gen, case["T"], 2 * hkv, d, dev).to(xt)
        s["k"], s["v"] = rows[:, :hkv], rows[:, hkv:]

    fmt, page = case["fmt"], case["page"]
    s["fmt"], s["page"] = fmt, page
    if kind == "attn":
        n = lengths(case)
        rng.shuffle(n)
    else:
        n = [case["R"] if kind == "cache" else case["T"] + rng.randrange(64)]
    need = [-(-a // page) for a in n]
    order = list(range(1, sum(need) + 1))       # page 0 belongs to nobody
    rng.shuffle(order)
    total = len(order) + 1
    # unused rows hold bytes 0xFF: NaN in every format
    cache = torch.full((total, hkv, page // 16, 32 * row_bytes(fmt, d)), 0xFF, dtype=torch.uint8, device=dev)
    s["cache"] = cache
    width = max(1, max(need))
    table = torch.zeros((len(n), width), dtype=torch.int32)
    at = 0
    for i, c in enumerate(need):
        table[i, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
        at += c
    table = table.to(dev)
    lens = torch.tensor(n, dtype=torch.int32, device=dev)
    pos = torch.arange(width * page, device=dev)
    slots = table.long()[:, pos // page] * page + pos % page                 # [sequences, width * page]
    if kind == "attn":
        held = slots[pos < lens[:, None].long()]
    else:
        held = slots[0, :n[0] - case["T"]]                                    # what came before
        s["slots"] = slots[0, n[0] - case["T"]:n[0]].contiguous()
        s["read"] = slots[0, :n[0]].contiguous() if kind == "cache" else s["slots"]
        if case.get("pad"):
            s["slots"] = s["slots"].clone()
            s["slots"][-1] = -1
            s["read"] = s["slots"]
    s["k_gs"] = s["v_gs"] = None
    for which in (0, 1):
        x = heads_like(gen, max(1, held.numel()), hkv, d, dev)
        if which == 0:
            x = x * 1.5
        gs = global_scale(x, fmt) if held.numel() else torch.ones(1, device=dev) * 0.01
        s["k_gs" if which == 0 else "v_gs"] = gs
        for a in range(0, held.numel(), 65536):
            part = slice(a, min(a + 65536, held.numel()))
            write_rows(cache, fmt, page, held[part], which, *coded(x[part].to(torch.bfloat16).float(), fmt, gs))
        del x
    if kind == "attn":
        s["table"], s["lens"], s["window"] = table, lens, case["window"]
        s["scale"] = 1.0 / math.sqrt(d)
        s["q"] = torch.randn((case["B"], case["Hq"] + 2 * hkv, d), generator=gen, device=dev).to(torch.bfloat16)[
            :, :case["Hq"]]                                                   # in place in the QKV rows
    return s


def work(case):
    d, hkv, kind = case["D"], case["Hkv"], case["kind"]
    xb = 4 if case.get("x") == "f32" else 2
    if kind == "rope":
        n = case["T"] * (case["Hq"] + hkv) * d
        return {"bytes": n * (xb + 2) + 8 * case["T"] + 4 * case["rot"],
                "flops": 3 * case["T"] * (case["Hq"] + hkv) * case["rot"]}
    row = 2 * hkv * row_bytes(case["fmt"], d)       # a token in the cache
    if kind == "attn":
        seen = sum(min(a, case["window"] or a) for a in lengths(case))
        return {"bytes": seen * row + 4 * case["B"] * case["Hq"] * d + 4 * case["B"] +
                4 * sum(-(-a // case["page"]) for a in lengths(case)), "flops": 4 * seen * case["Hq"] * d}
    wrote, read = case["T"], case["R"] if kind == "cache" else case["T"]
    n = wrote * (2 * hkv * d * xb + row + 8) + read * (row + 4 * hkv * d + 8)
    flops = 4 * (wrote + read) * hkv * d
    if kind == "step":
        n += wrote * (case["Hq"] * d * (xb + 2) + 8) + 4 * case["rot"]
        flops += 3 * wrote * (case["Hq"] + hkv) * case["rot"]
    return {"bytes": n, "flops": flops}


# ----------------------------------------------------------- definitions in 64 bits ----

def e2m1_64(code):
    m = code & 7
    e = (m >> 1).double()
    v = torch.where(m < 2, m.double() * 0.5, (1 + 0.5 * (m & 1).double()) * torch.exp2(e - 1))
    return torch.where(code >= 8, -v, v)


def e4m3_64(byte):
    e, m = ((byte >> 3) & 15).double(), (byte & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e - 7))
    return torch.where(byte >= 128, -v, v)


def nearest(a, bits, least, most):
    """|a| rounded to `bits` significant bits (ties to even), spacing at least `least`, at most `most`."""
    e = torch.floor(torch.log2(a.clamp(min=1e-300)))
    step = torch.exp2(e - (bits - 1)).clamp(min=least)
    return (torch.round(a / step) * step).clamp(max=most)


def f32(a):
    return a.float().double()       # a quotient or product of binary32 numbers, rounded once


def held_64(x, fmt, gs):
    """The values the cache holds for x [..., d] (fp64), from the rounding rules; gs a binary32 number."""
    if fmt == "bf16":
        return x.float().to(torch.bfloat16).double()
    if fmt == "e4m3":
        return torch.sign(x) * nearest(f32(x.abs() / gs), 4, 2.0 ** -9, 448.0) * gs
    b = x.unflatten(-1, (-1, 16))
    sc = nearest(f32(b.abs().amax(-1) / f32(gs * 6)), 4, 2.0 ** -9, 448.0)
    r = f32(sc * gs)[..., None]
    a = torch.where(r > 0, f32(b.abs() / r.clamp(min=1e-300)), 0.0)
    return (torch.sign(b) * nearest(a, 2, 0.5, 6.0) * sc[..., None] * gs).flatten(-2)


def stored_64(s, slots, which):
    """fp64 rows [n, heads, d] of nonnegative slots, byte by byte from the layout."""
    cache, fmt, d, page = s["cache"], s["fmt"], s["D"], s["page"]
    nb = code_bytes(fmt, d)
    r = slots % 16
    f = ((r & 6) ^ ((r & 1) << 2)) & (nb // 16 - 1)
    byte = torch.arange(nb, device=slots.device)
    offset = which * 16 * nb + r[:, None] * nb + (((byte >> 4)[None] ^ f[:, None]) << 4) + (byte & 15)
    tile = cache[slots // page, :, slots % page // 16]                        # [n, heads, bytes]
    b = tile.gather(2, offset[:, None].expand(-1, tile.shape[1], -1)).int()
    gs = (s["k_gs"] if which == 0 else s["v_gs"]).double()
    if fmt == "bf16":
        return (b[..., 0::2] | (b[..., 1::2] << 8)).to(torch.int16).view(torch.bfloat16).double()
    if fmt == "e4m3":
        return e4m3_64(b) * gs
    so = 32 * nb + which * d + r[:, None] * (d // 16) + torch.arange(d // 16, device=slots.device)
    sc = e4m3_64(tile.gather(2, so[:, None].expand(-1, tile.shape[1], -1)).int())
    v = torch.stack((e2m1_64(b & 15), e2m1_64(b >> 4)), -1).flatten(-2)
    return v * sc.repeat_interleave(16, -1) * gs


def turned_64(x, s):
    n = s["freqs"].numel()
    angle = torch.remainder(s["positions"].double()[:, None] * s["freqs"], 1.0) * (2 * math.pi)
    z = torch.polar(torch.full_like(angle, s["mscale"]), angle)[:, None]
    x = x.double()
    pair = x[..., :2 * n].unflatten(-1, (2, n)).transpose(-1, -2) if s["layout"] == "half" else \
        x[..., :2 * n].unflatten(-1, (n, 2))
    w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    w = (w.transpose(-1, -2) if s["layout"] == "half" else w).flatten(-2)
    return torch.cat((w, x[..., 2 * n:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "rope":
        return turned_64(s["x"], s)
    if kind == "attn":
        out = []
        for b, n in enumerate(s["lens"].tolist()):
            lo = max(0, n - s["window"]) if s["window"] else 0
            pos = torch.arange(lo, n, device=s["cache"].device)
            if n == 0:
                out.append(torch.zeros(s["q"].shape[1:], dtype=torch.float64, device=s["cache"].device))
                continue
            slots = s["table"][b].long()[pos // s["page"]] * s["page"] + pos % s["page"]
            k, v = stored_64(s, slots, 0), stored_64(s, slots, 1)
            q = s["q"][b].double().view(case["Hkv"], -1, s["D"])
            w = torch.softmax(q @ k.permute(1, 2, 0) * s["scale"], -1)
            out.append((w @ v.permute(1, 0, 2)).reshape(case["Hq"], s["D"]))
        return torch.stack(out)
    k, v = s["k"].double(), s["v"].double()
    got = {}
    if kind == "step":
        got["q"] = turned_64(s["q"], s)
        k = turned_64(k, s).float().to(torch.bfloat16).double()
    there = s["slots"] >= 0
    for name, x, gs, which in (("k", k, s["k_gs"], 0), ("v", v, s["v_gs"], 1)):
        new = held_64(x, s["fmt"], gs.double())
        old = s["read"][:-case["T"]]
        got[name] = torch.cat((stored_64(s, old, which), torch.where(there[:, None, None], new, 0.0)))
    return got
