// K10: rotary positions and the paged key-value cache of a decode stack (the
// steps between the QKV linear and attention; imp v0.20.0 release notes,
// "Highlights": a first-party quantizer; Ignis README, "The decode round").
//
//   rope_kernel      y = rotary(x) over the heads of each token
//   kv_write_kernel  keys and values -> cache tiles (bf16, E4M3 or NVFP4);
//                    with ROPE also the rotation: queries rotated to bf16,
//                    keys rotated, rounded to bf16 and quantized, in one pass
//   kv_read_kernel   cache rows -> dense bf16 / fp32
//
// Rotary mathematics.  Pair i of a head turns by a = 2 pi frac(pos * f_i)
// with f_i in turns per token: the product is taken in fp64 (a far position
// times an fp32 frequency would lose the angle: 2^20 * 2^-24 turns), its
// fraction is exact, and cos and sin of it are fp64, rounded once to fp32.
// B200 runs fp64 at half the fp32 rate and a CTA computes each angle once for
// all of its heads, so no table of the context's length is kept.  The
// rotation is fp32 with every product and sum rounded (no contraction), so
// the same inputs give the same bits in the separate and the fused kernel.
//
// All three kernels move each byte once and are bound by HBM for long chunks
// and by latency for decode steps.  A thread takes units of 16 elements (two
// runs of 8) of a row, a row being one head of one token.  A warp takes one
// head at a time, its lanes covering 2 to 8 whole rows, so that everything but
// a row's place is known per head; the loads of two rows per lane go out together
// (four, with the registers they take: 38.8 and 45.0 us for the first two cases
// below, against 29.7 and 35.0 of two then).  fp32 products go two to an
// instruction.  All are programmatic dependents.
//
// Measured (B200, replayed from a graph):
//   rotation of 8,191 tokens x 40 heads of 128, 64 rotated, bf16: 27.3 us, 6.1 TB/s
//     (94 % of a copy's rate); one token: 1.9 us, the launch
//   2,048 tokens of 20 heads written to NVFP4 pages and 10,240 read back: 33.1 us,
//     4.9 TB/s (74 %).  The write is what is slow (12.0 us alone, 4.1 of it bytes).  Half
//     is instructions (19 an element, 6.8 M of warps), half the grid: 768 CTAs are 1.3
//     waves of the 592 resident ones, the last of three groups of heads is half empty,
//     and each wave begins with the latency of its loads (56 % of the issue slots)
//   2,048 tokens, bf16 / fp32 rows, to BF16, E4M3 and NVFP4 pages: write of 2 x 20 heads 8.3
//     / 11.4, 9.8 / 10.6 and 12.0 / 11.1 us; rotation and write of 40 + 2 x 20 14.7 / 22.2,
//     18.2 / 24.3 and 22.8 / 26.7; the latter of 32 tokens, fp32 rows, 3.1, 3.5 and 4.0.
//     Read of 10,240 tokens of 20 heads 34.2, 26.8 and 24.1 us (94, 89 and 85 %).  The
//     global scales are those of the data's largest elements; where fewer quotients meet
//     a border between codes the NVFP4 write takes 9.1 us, with the rotation 19.4
//   rotation, write and read of 2,048 tokens, 32 / 8 heads, bf16: 14.8 us, 4.5 TB/s
//     (69 %): two short kernels, each with its ramp; 32 decoding tokens: 5.6 us
#include "internal.h"
#include "kv_layout.cuh"
#include "quotient.cuh"
#include "tma.cuh"

namespace nvfp4 {

// Eight consecutive elements with ordinary loads (x may be rotated in place).
NVFP4_DEV void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo_to_f32(w[i]);
        v[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
}
NVFP4_DEV void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
NVFP4_DEV uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
NVFP4_DEV uint4 pack8_bf16(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
NVFP4_DEV void store8(__nv_bfloat16* p, const float (&v)[8]) { *reinterpret_cast<uint4*>(p) = pack8_bf16(v); }
NVFP4_DEV void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Two fp32 operations in one instruction, each rounded (never contracted).
NVFP4_DEV uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
NVFP4_DEV void unpack2(uint64_t p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
NVFP4_DEV uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
NVFP4_DEV uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
NVFP4_DEV uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// v[i] * f
NVFP4_DEV void scale8(const float (&v)[8], float f, float (&y)[8]) {
    const uint64_t ff = pack2(f, f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) unpack2(mul2(pack2(v[i], v[i + 1]), ff), y[i], y[i + 1]);
}

// ---- rotary ------------------------------------------------------------------

struct RopeParams {
    const int64_t* positions;  // [T]
    const double* freqs;       // [pairs], turns per token
    int pairs;                 // rot_dim / 2, a multiple of 8 (0: no rotation)
    int layout;                // NVFP4_ROPE_HALF / INTERLEAVED
    double mscale;
    int inverse;
};

// sin and cos of 2 pi t, |t| <= 1/2, in fp64: t = q / 4 + r with |r| <= 1/8, the
// Taylor series of x = 2 pi r to x^13 and x^14 (the next terms are below 2^-45),
// and the quarter turns.  Rounded to fp32 this is the fp32 nearest the true
// value but about once in 2^21.
NVFP4_DEV void sincos_turns(double t, double& s, double& c) {
    const double q = rint(4.0 * t);
    const double x = (t - 0.25 * q) * 6.283185307179586476925, z = x * x;
    double ps = 1.0 / 6227020800.0, pc = -1.0 / 87178291200.0;
    ps = fma(ps, z, -1.0 / 39916800.0), pc = fma(pc, z, 1.0 / 479001600.0);
    ps = fma(ps, z, 1.0 / 362880.0), pc = fma(pc, z, -1.0 / 3628800.0);
    ps = fma(ps, z, -1.0 / 5040.0), pc = fma(pc, z, 1.0 / 40320.0);
    ps = fma(ps, z, 1.0 / 120.0), pc = fma(pc, z, -1.0 / 720.0);
    ps = fma(ps, z, -1.0 / 6.0), pc = fma(pc, z, 1.0 / 24.0);
    pc = fma(pc, z, -0.5);
    const double sn = fma(x * z, ps, x), cn = fma(pc, z, 1.0);
    const int k = (int)q & 3;
    s = (k & 1) ? cn : sn;
    c = (k & 1) ? sn : cn;
    if (k & 2) s = -s;
    if (k == 1 || k == 2) c = -c;
}

// cos and sin of the CTA's tokens, two pairs to a word (c, c', s, s') and ordered
// so that neighbouring lanes read neighbouring words: pairs 2 m and 2 m + 1 of token
// tl at [tl][m % w][m / w], w the words a run of 8 elements needs (4 where it
// holds one element of each pair, else 2).
NVFP4_DEV void rope_angles(const RopeParams& rp, int64_t t0, int nt, float4* cs) {
    const int lw = rp.layout == NVFP4_ROPE_HALF ? 2 : 1, runs = rp.pairs >> (lw + 1);
    float* out = reinterpret_cast<float*>(cs);
    for (int i = threadIdx.x; i < nt * rp.pairs; i += blockDim.x) {
        const int tl = i / rp.pairs, p = i - tl * rp.pairs, m = p >> 1;
        const double turns = (double)rp.positions[t0 + tl] * rp.freqs[p];
        double s, c;
        sincos_turns(turns - rint(turns), s, c);
        if (rp.inverse) s = -s;
        const int at = 4 * (tl * (rp.pairs >> 1) + (m & ((1 << lw) - 1)) * runs + (m >> lw)) + (p & 1);
        out[at] = (float)(c * rp.mscale);
        out[at + 2] = (float)(s * rp.mscale);
    }
}

// Unit j of a head: the element offsets of its two runs of 8.  Both runs of a
// region (the rotated elements, the rest) advance by 8 per unit, so that a
// warp's 16-byte accesses are contiguous in either layout.
NVFP4_DEV void rope_runs(const RopeParams& rp, int j, int D, int& lo, int& hi) {
    const int n8 = rp.pairs >> 3;
    if (j < n8) {
        lo = j * 8;
        hi = rp.pairs + j * 8;
    } else {
        lo = 2 * rp.pairs + (j - n8) * 8;
        hi = lo + (D >> 1) - rp.pairs;
    }
}

// Pairs (a0, b0) and (a1, b1).
NVFP4_DEV void rotate2(float& a0, float& a1, float& b0, float& b1, const float4& cs) {
    const uint64_t x = pack2(a0, a1), y = pack2(b0, b1), c = pack2(cs.x, cs.y), s = pack2(cs.z, cs.w);
    unpack2(sub2(mul2(x, c), mul2(y, s)), a0, a1);
    unpack2(add2(mul2(y, c), mul2(x, s)), b0, b1);
}

// Rotates the two runs of unit j of token tl.
NVFP4_DEV void rope_unit(const RopeParams& rp, int j, int tl, const float4* cs, float (&lo)[8], float (&hi)[8]) {
    const int n8 = rp.pairs >> 3;
    if (j >= n8) return;
    cs += tl * (rp.pairs >> 1) + j;
    if (rp.layout == NVFP4_ROPE_HALF) {
#pragma unroll
        for (int i = 0; i < 4; ++i) rotate2(lo[2 * i], lo[2 * i + 1], hi[2 * i], hi[2 * i + 1], cs[i * n8]);
    } else {
        const int runs = 2 * n8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            rotate2(lo[4 * i], lo[4 * i + 2], lo[4 * i + 1], lo[4 * i + 3], cs[i * runs]);
            rotate2(hi[4 * i], hi[4 * i + 2], hi[4 * i + 1], hi[4 * i + 3], cs[i * runs + n8]);
        }
    }
}

constexpr int kCtaThreads = 256, kWarps = kCtaThreads / 32;
constexpr int kBatch = 2;  // rows per lane whose loads go out together

// Units are as raw 16-byte words while they are on their way.
template <typename T>
struct Raw16 {
    uint4 w[sizeof(T)];  // 16 elements: 2 words of bf16, 4 of fp32
    // elements 0 .. 7 from lo, 8 .. 15 from hi
    NVFP4_DEV void load(const T* lo, const T* hi) {
        constexpr int h = sizeof(T) / 2;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            w[i] = reinterpret_cast<const uint4*>(lo)[i];
            w[h + i] = reinterpret_cast<const uint4*>(hi)[i];
        }
    }
    NVFP4_DEV void clear() {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    NVFP4_DEV void values(float (&lo)[8], float (&hi)[8]) const {
        constexpr int h = sizeof(T) / 2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = at(0, i);
            hi[i] = at(h, i);
        }
    }

   private:
    NVFP4_DEV float at(int base, int i) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t x = word(w[base], i >> 1);
            return (i & 1) ? bf16hi_to_f32(x) : bf16lo_to_f32(x);
        } else {
            return __uint_as_float(word(w[base + (i >> 2)], i & 3));
        }
    }
    static NVFP4_DEV uint32_t word(const uint4& v, int k) { return k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w; }
};

// A CTA takes `tt` tokens and `hc` heads.
template <typename XT, typename YT>
__global__ void __launch_bounds__(kCtaThreads, 4) rope_kernel(const XT* x, int64_t T, int heads, int units, int64_t x_ld,
                                                           RopeParams rp, YT* y, int64_t y_ld, int tt, int hc) {
    extern __shared__ __align__(16) uint8_t smem[];
    float4* cs = reinterpret_cast<float4*>(smem);
    griddep_launch_dependents();
    griddep_wait();
    const int64_t t0 = (int64_t)blockIdx.x * tt;
    const int nt = (int)(T - t0 < tt ? T - t0 : tt);
    const int h0 = blockIdx.y * hc, h1 = min(heads, h0 + hc);
    // lanes: `per` rows of `units` units (one row, 32 units at a time, for wide heads)
    const int lane = threadIdx.x & 31, per = units < 32 ? 32 / units : 1;
    const int row = units < 32 ? lane / units : 0, D = units * 16;
    const int first = row < per ? row : 0x40000000;  // lanes past the last row idle
    int j = lane - row * units, h = h0 + (threadIdx.x >> 5), tl0 = first, lo, hi;
    rope_runs(rp, j, D, lo, hi);
    Raw16<XT> raw[kBatch];
    auto load = [&]() {
        const XT* xp = x + (t0 + tl0) * x_ld + h * D;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (h < h1 && tl0 + k * per < nt) raw[k].load(xp + k * per * x_ld + lo, xp + k * per * x_ld + hi);
    };
    load();  // on their way while the angles are found
    rope_angles(rp, t0, nt, cs);
    __syncthreads();
    while (h < h1) {
        YT* yp = y + (t0 + tl0) * y_ld + h * D;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (tl0 + k * per < nt) {
                float a[8], b[8];
                raw[k].values(a, b);
                rope_unit(rp, j, tl0 + k * per, cs, a, b);
                store8(yp + k * per * y_ld + lo, a);
                store8(yp + k * per * y_ld + hi, b);
            }
        }
        tl0 += kBatch * per;
        if (tl0 >= nt) {
            tl0 = first;
            j += 32;
            if (j >= units) {
                j = lane - row * units;
                h += kWarps;
            }
            rope_runs(rp, j, D, lo, hi);
        }
        load();
    }
}

// ---- cache writes ------------------------------------------------------------

// Global scale of one of K / V with what its quotients need: reciprocals
// within 2^-22 (0: divide).
struct GsPar {
    float gs, denom, inv_denom, inv_gs;
};
NVFP4_DEV GsPar gs_par(float gs) {
    GsPar g;
    g.gs = gs;
    g.denom = __fmul_rn(g.gs, 6.0f);
    g.inv_denom = rcp_safe(g.denom) ? rcp_approx(g.denom) : 0.0f;
    g.inv_gs = rcp_safe(g.gs) ? rcp_approx(g.gs) : 0.0f;
    return g;
}

NVFP4_DEV uint32_t f32x2_to_e4m3(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
NVFP4_DEV uint2 f32x8_to_e4m3(const float (&v)[8]) {
    return make_uint2(f32x2_to_e4m3(v[0], v[1]) | (f32x2_to_e4m3(v[2], v[3]) << 16),
                      f32x2_to_e4m3(v[4], v[5]) | (f32x2_to_e4m3(v[6], v[7]) << 16));
}
NVFP4_DEV void divide8(const float (&v)[8], float r, float (&q)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(v[i], r);
}

// Codes of the quotients RN(v[i] / r), r > 0, of two runs x and y of a lane, without
// dividing where that is certain: inv is within 2^-22 of 1 / r, so
// v * RN(inv (1 - 2^-18)) and v * RN(inv (1 + 2^-18)), two roundings each, lie below
// and above RN(v / r) in magnitude; rounding to a code is monotone, so where both
// give one code it is that of RN(v / r).  (Products too small or too large
// for that bound round to 0 or to the largest code either way.)  All is decided
// first, without branches; one rare branch divides where that is needed.

NVFP4_DEV void e4m3_runs(const float (&x)[8], const float (&y)[8], const GsPar& g, uint2& cx, uint2& cy) {
    const float down = __fmul_rn(g.inv_gs, kBracketLo), up = __fmul_rn(g.inv_gs, kBracketHi);
    float t[8];
    scale8(x, down, t);
    cx = f32x8_to_e4m3(t);
    scale8(y, down, t);
    cy = f32x8_to_e4m3(t);
    scale8(x, up, t);
    const uint2 dx = f32x8_to_e4m3(t);
    scale8(y, up, t);
    const uint2 dy = f32x8_to_e4m3(t);
    if (((cx.x ^ dx.x) | (cx.y ^ dx.y) | (cy.x ^ dy.x) | (cy.y ^ dy.y)) != 0u || g.inv_gs == 0.0f) {
        divide8(x, g.gs, t);
        cx = f32x8_to_e4m3(t);
        divide8(y, g.gs, t);
        cy = f32x8_to_e4m3(t);
    }
}

// NVFP4: also the block scale's E4M3 byte, of the block's amax (as
// e4m3_of_quotient gives it).  diff: bits set in the codes that a division has to
// decide; redo: so has the scale.
struct Block {
    uint32_t sb, code, diff;
    float r;
    bool redo;
};
NVFP4_DEV Block quick_block(const float (&v)[8], float amax, const GsPar& g) {
    Block b;
    const float a = __fmul_rn(amax, g.inv_denom);
    const uint32_t pr = f32x2_to_e4m3(__fmul_rn(a, kBracketLo), __fmul_rn(a, kBracketHi));
    b.sb = pr & 0xFFu;
    b.r = __fmul_rn(e4m3_to_f32(b.sb), g.gs);
    const bool safe = rcp_safe(b.r);
    const float inv = safe ? rcp_approx(b.r) : 0.0f;
    float t[8];
    scale8(v, __fmul_rn(inv, kBracketLo), t);
    b.code = f32x8_to_e2m1(t);
    scale8(v, __fmul_rn(inv, kBracketHi), t);
    b.diff = f32x8_to_e2m1(t) ^ b.code;
    if (b.r == 0.0f) b.code = 0u;
    b.redo = b.sb != pr >> 8 || g.inv_denom == 0.0f || !(safe || b.r == 0.0f);
    return b;
}
NVFP4_DEV void mend_block(const float (&v)[8], float amax, const GsPar& g, Block& b) {
    if (b.redo) {
        b.sb = e4m3_of_quotient(amax, g.denom, 0.0f);
        b.r = __fmul_rn(e4m3_to_f32(b.sb), g.gs);
        b.code = 0u;
        b.diff = b.r != 0.0f ? 0xFFFFFFFFu : 0u;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (b.diff & (0xFu << (4 * j)))
            b.code = (b.code & ~(0xFu << (4 * j))) | (e2m1_of_division(v[j], b.r) << (4 * j));
}

// Where a token's rows lie, for head 0: the key row's codes `off` bytes from the
// cache's start (-1: not stored), its block scales `scale` bytes on; its 16-byte
// pieces are turned by `turn` bytes.  Values lie 16 rows further.
struct Slot {
    int64_t off;
    int scale, turn;
};
template <int FMT, int D>
NVFP4_DEV void find_slots(const KvView& c, const int64_t* slots, int64_t t0, int nt, int64_t head_bytes, int* status,
                          Slot* out) {
    constexpr int CB = kv_code_bytes(FMT, D);
    if ((int)threadIdx.x >= nt) return;
    const int64_t slot = slots[t0 + threadIdx.x];
    Slot s{-1, 0, 0};
    if (slot >= 0) {
        // (a 32-bit division where it does, which is nearly always)
        const int64_t page = slot >> 31 ? slot / c.page_size : (int64_t)((uint32_t)slot / (uint32_t)c.page_size);
        const int in = (int)(slot - page * c.page_size), r = in % kKvTile;
        s.scale = 2 * kKvTile * CB + r * (kv_scale_bytes(FMT, D) - CB);
        s.turn = kv_turn(r, CB / 16) << 4;
        if (page < c.num_pages)
            s.off = page * c.heads * head_bytes + (int64_t)(in / kKvTile) * kv_tile_bytes(FMT, D) + r * CB;
        else if (status)
            atomicExch(status, NVFP4_ERR_PAGE);
    }
    out[threadIdx.x] = s;
}
// Byte `o` of a row's codes (o: of element e, e * CB / D).
NVFP4_DEV int turned(const Slot& s, int o) { return o ^ s.turn; }
// From a key's code / scale bytes to its value's.
template <int FMT, int D>
NVFP4_DEV constexpr int64_t value_codes() {
    return kKvTile * kv_code_bytes(FMT, D);
}
template <int FMT, int D>
NVFP4_DEV constexpr int value_scales() {
    return kKvTile * (kv_scale_bytes(FMT, D) - kv_code_bytes(FMT, D));
}

struct KvWriteArgs {
    KvView c;
    const void* q;  // ROPE: [T] rows of q_heads heads
    const void* k;
    const void* v;
    int64_t q_ld, k_ld, v_ld;
    int64_t T;
    int q_heads;  // 0 without ROPE
    const int64_t* slots;
    RopeParams rp;         // without ROPE: head_dim / 2 pairs (the units' two runs)
    __nv_bfloat16* q_out;  // [T, q_heads, D]
    int tt, hc;            // tt <= kBatch rows of lanes
    int* status;
};

// Heads 0 .. q_heads - 1 are the queries, then the keys, then the values.  An
// NVFP4 block is two runs: those
// of lanes 2 i and 2 i + 1, or, where the rotated part is an odd number of
// units, of whichever lanes have runs 2 b and 2 b + 1 of the row.
template <typename XT, int FMT, int D, bool ROPE>
__global__ void __launch_bounds__(kCtaThreads, sizeof(XT) == 2 ? 4 : 3) kv_write_kernel(const KvWriteArgs a) {
    constexpr int units = D / 16, per = 32 / units, CB = kv_code_bytes(FMT, D);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Slot s_slot[kBatch * per];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t t0 = (int64_t)blockIdx.x * a.tt;
    const int nt = (int)(a.T - t0 < a.tt ? a.T - t0 : a.tt);
    const int k0 = a.q_heads, v0 = a.q_heads + a.c.heads, heads = v0 + a.c.heads;
    const int h0 = blockIdx.y * a.hc, h1 = min(heads, h0 + a.hc);
    const int64_t head_bytes = (int64_t)(a.c.page_size / kKvTile) * kv_tile_bytes(FMT, D);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % units, first = lane / units;
    int lo, hi;
    rope_runs(a.rp, j, D, lo, hi);
    Raw16<XT> raw[kBatch];
    auto load = [&](int h, int k) {  // the lane's row k of head h
        if (h >= h1 || first + k * per >= nt) return;
        const bool is_q = ROPE && h < k0, is_v = h >= v0;
        const int64_t ld = is_q ? a.q_ld : is_v ? a.v_ld : a.k_ld;
        const XT* src = (is_q ? (const XT*)a.q : is_v ? (const XT*)a.v : (const XT*)a.k) +
                        (t0 + first + k * per) * ld + (is_q ? h : is_v ? h - v0 : h - k0) * D;
        raw[k].load(src + lo, src + hi);
    };
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        raw[k].clear();
        load(h0 + warp, k);  // on their way while slots and angles are found
    }
    find_slots<FMT, D>(a.c, a.slots, t0, nt, head_bytes, a.status, s_slot);
    const float4* cs = reinterpret_cast<const float4*>(smem);
    if constexpr (ROPE) rope_angles(a.rp, t0, nt, reinterpret_cast<float4*>(smem));
    float gk = 1.0f, gv = 1.0f;
    if constexpr (FMT != NVFP4_KV_BF16) {
        gk = *a.c.k_gs;
        gv = *a.c.v_gs;
    }
    // the lane of the other half of each run's block, and whether it is that lane's hi
    const int n8 = a.rp.pairs >> 3;
    const bool paired = !ROPE || n8 % 2 == 0;
    int lane_lo = 0, lane_hi = 0;
    bool lo_hi = false, hi_hi = false;
    if (FMT == NVFP4_KV_NVFP4 && !paired) {
        auto find = [&](int run, int& ln, bool& in_hi) {
            if (run < 2 * n8) {
                in_hi = run >= n8;
                ln = run - (in_hi ? n8 : 0);
            } else {
                in_hi = run - 2 * n8 >= units - n8;
                ln = run - n8 - (in_hi ? units - n8 : 0);
            }
            ln += lane - j;
        };
        find((lo >> 3) ^ 1, lane_lo, lo_hi);
        find((hi >> 3) ^ 1, lane_hi, hi_hi);
    }
    __syncthreads();
    for (int h = h0 + warp; h < h1; h += kWarps) {
        const bool is_q = ROPE && h < k0, is_v = h >= v0;
        const int64_t at = (is_v ? h - v0 : h - k0) * head_bytes + (is_v ? value_codes<FMT, D>() : 0);
        const int to_scales = is_v ? value_scales<FMT, D>() : 0;
        const GsPar g = gs_par(is_v ? gv : gk);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int tl = first + k * per;
            float x[8], y[8];
            raw[k].values(x, y);
            if (ROPE) load(h + kWarps, k);  // on its way while this one is turned and quantized
            if (ROPE && !is_v) {
                if (tl < nt) rope_unit(a.rp, j, tl, cs, x, y);
                const uint4 xw = pack8_bf16(x), yw = pack8_bf16(y);
                if (is_q) {
                    if (tl < nt) {
                        __nv_bfloat16* yp = a.q_out + ((t0 + tl) * a.q_heads + h) * D;
                        *reinterpret_cast<uint4*>(yp + lo) = xw;
                        *reinterpret_cast<uint4*>(yp + hi) = yw;
                    }
                    continue;
                }
                load8(reinterpret_cast<const __nv_bfloat16*>(&xw), x);  // quantized from the bf16 values
                load8(reinterpret_cast<const __nv_bfloat16*>(&yw), y);
            }
            const Slot w = s_slot[tl < nt ? tl : 0];
            const bool live = tl < nt && w.off >= 0;
            uint8_t* codes = a.c.data + at + w.off;
            uint8_t *p = codes + turned(w, lo * CB / D), *p_hi = codes + turned(w, hi * CB / D);
            if constexpr (FMT == NVFP4_KV_BF16) {
                if (live) {
                    *reinterpret_cast<uint4*>(p) = pack8_bf16(x);
                    *reinterpret_cast<uint4*>(p_hi) = pack8_bf16(y);
                }
            } else if constexpr (FMT == NVFP4_KV_E4M3) {
                uint2 cx, cy;
                e4m3_runs(x, y, g, cx, cy);
                if (live) {
                    *reinterpret_cast<uint2*>(p) = cx;
                    *reinterpret_cast<uint2*>(p_hi) = cy;
                }
            } else {
                const float mx = amax8(x), my = amax8(y);
                float ox, oy;
                if (paired) {
                    ox = __shfl_xor_sync(0xffffffffu, mx, 1);
                    oy = __shfl_xor_sync(0xffffffffu, my, 1);
                } else {
                    const float b0 = __shfl_sync(0xffffffffu, mx, lane_lo), b1 = __shfl_sync(0xffffffffu, my, lane_lo);
                    const float b2 = __shfl_sync(0xffffffffu, mx, lane_hi), b3 = __shfl_sync(0xffffffffu, my, lane_hi);
                    ox = lo_hi ? b1 : b0;
                    oy = hi_hi ? b3 : b2;
                }
                const float ax = fmaxf(mx, ox), ay = fmaxf(my, oy);
                Block bx = quick_block(x, ax, g), by = quick_block(y, ay, g);
                if ((bx.diff | by.diff) != 0u || bx.redo || by.redo) {
                    mend_block(x, ax, g, bx);
                    mend_block(y, ay, g, by);
                }
                if (live) {
                    uint8_t* scale = codes + w.scale + to_scales;
                    *reinterpret_cast<uint32_t*>(p) = bx.code;
                    *reinterpret_cast<uint32_t*>(p_hi) = by.code;
                    if ((lo & 8) == 0) scale[lo / 16] = (uint8_t)bx.sb;
                    if ((hi & 8) == 0) scale[hi / 16] = (uint8_t)by.sb;
                }
            }
        }
        if (!ROPE) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) load(h + kWarps, k);
        }
    }
}

// ---- cache reads -------------------------------------------------------------

// Eight elements as stored, and their fp32 values.
template <int FMT>
struct RawRun {
    uint32_t c[FMT == NVFP4_KV_BF16 ? 4 : FMT == NVFP4_KV_E4M3 ? 2 : 1];
    uint32_t sb;
};
template <int FMT>
NVFP4_DEV void load_run(const uint8_t* codes, const uint8_t* scale, RawRun<FMT>& x) {
    if constexpr (FMT == NVFP4_KV_BF16) {
        const uint4 c = *reinterpret_cast<const uint4*>(codes);
        x.c[0] = c.x, x.c[1] = c.y, x.c[2] = c.z, x.c[3] = c.w;
    } else if constexpr (FMT == NVFP4_KV_E4M3) {
        const uint2 c = *reinterpret_cast<const uint2*>(codes);
        x.c[0] = c.x, x.c[1] = c.y;
    } else {
        x.c[0] = *reinterpret_cast<const uint32_t*>(codes);
        x.sb = *scale;
    }
}
template <int FMT>
NVFP4_DEV void run_values(const RawRun<FMT>& x, float gs, float (&v)[8]) {
    if constexpr (FMT == NVFP4_KV_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16lo_to_f32(x.c[i]);
            v[2 * i + 1] = bf16hi_to_f32(x.c[i]);
        }
    } else {
        uint32_t p[4];
        if constexpr (FMT == NVFP4_KV_E4M3) {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = e4m3x2_to_f16x2((uint16_t)(x.c[i >> 1] >> (16 * (i & 1))));
        } else {
            const __half2 s = __half2half2(__ushort_as_half((unsigned short)e4m3x2_to_f16x2((uint16_t)x.sb)));
            e2m1x8_to_f16x2(x.c[0], p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&p[i]), s);  // E2M1 * E4M3: exact
                p[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = f16x2_to_f32x2(p[i]);
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
        scale8(f, gs, v);
    }
}

struct KvReadArgs {
    KvView c;
    const int64_t* slots;
    int64_t T;
    void* k_out;  // [T, heads, D]
    void* v_out;
    int tt, hc;  // as in KvWriteArgs
    int* status;
};

// Heads 0 .. heads - 1 are the keys, then the values.
template <typename YT, int FMT, int D>
__global__ void __launch_bounds__(kCtaThreads, 6) kv_read_kernel(const KvReadArgs a) {
    constexpr int units = D / 16, per = 32 / units, CB = kv_code_bytes(FMT, D);
    __shared__ Slot s_slot[kBatch * per];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t t0 = (int64_t)blockIdx.x * a.tt;
    const int nt = (int)(a.T - t0 < a.tt ? a.T - t0 : a.tt);
    const int h0 = blockIdx.y * a.hc, h1 = min(2 * a.c.heads, h0 + a.hc);
    const int64_t head_bytes = (int64_t)(a.c.page_size / kKvTile) * kv_tile_bytes(FMT, D);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % units, first = lane / units;
    find_slots<FMT, D>(a.c, a.slots, t0, nt, head_bytes, a.status, s_slot);
    float gk = 1.0f, gv = 1.0f;
    if constexpr (FMT != NVFP4_KV_BF16) {
        gk = *a.c.k_gs;
        gv = *a.c.v_gs;
    }
    __syncthreads();
    const int64_t y_ld = (int64_t)a.c.heads * D, y_row = (t0 + first) * y_ld + 8 * j;
    for (int h = h0 + warp; h < h1; h += kWarps) {
        const bool is_v = h >= a.c.heads;
        const int hk = is_v ? h - a.c.heads : h;
        const int64_t at = hk * head_bytes + (is_v ? value_codes<FMT, D>() : 0);
        const int to_scales = is_v ? value_scales<FMT, D>() : 0;
        RawRun<FMT> x[kBatch][2] = {};
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int tl = first + k * per;
            const Slot w = s_slot[tl < nt ? tl : 0];
            if (tl < nt && w.off >= 0) {
                const uint8_t* codes = a.c.data + at + w.off;
                const uint8_t* scale = codes + w.scale + to_scales + j / 2;
                load_run<FMT>(codes + turned(w, j * CB / units / 2), scale, x[k][0]);
                load_run<FMT>(codes + turned(w, CB / 2 + j * CB / units / 2), scale + D / 32, x[k][1]);
            }
        }
        YT* out = (YT*)(is_v ? a.v_out : a.k_out) + y_row + hk * D;
        const float gs = is_v ? gv : gk;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (first + k * per < nt) {
                float v[8];
                run_values<FMT>(x[k][0], gs, v);
                store8(out + k * per * y_ld, v);
                run_values<FMT>(x[k][1], gs, v);
                store8(out + k * per * y_ld + D / 2, v);
            }
    }
}

// ---- launches ----------------------------------------------------------------

// Tokens and heads of a CTA.  Where a warp per head and one row per lane leave
// the GPU unfilled (decode steps), that: latency counts.  Else kBatch rows per lane,
// and as many heads as still leave `per_sm` CTAs per SM: more heads share the
// CTA's angles and slots, more CTAs even out better.  Measured (us): rotation of
// 8,191 x 40 heads with 4 / 8 / 16 per SM 28.2 / 27.5 / 28.3 (four rows per lane, 4:
// 28.8); rotation and write of 2,048 x (40 + 2 x 20) heads, NVFP4, with 4 / 8: 23.0 /
// 24.6 (four rows, 4: 32.9), 32 + 2 x 8 heads, bf16: 11.3 / 12.8; write of 2,048 x 2 x
// 20 heads, NVFP4, with 4 / 16: 11.7 / 12.5; read of them 6.1 / 5.5.  Doubling hc leaves
// uneven grids: 1.3 waves (1.7 of the three CTAs per SM of fp32 rows) for 2,048
// tokens and 40, 48 or 80 heads.
static void cta_shape(int64_t T, int heads, int units, int per_sm, int& tt, int& hc) {
    const int per = units < 32 ? 32 / units : 1;
    tt = per;
    hc = kWarps;
    if ((T + tt - 1) / tt * ((heads + hc - 1) / hc) > 148 * 4) {
        tt = per * kBatch;
        const int64_t groups = (T + tt - 1) / tt;
        while (hc < heads && groups * ((heads + 2 * hc - 1) / (2 * hc)) >= 148 * per_sm) hc *= 2;
    }
}

static cudaLaunchConfig_t pdl_config(cudaLaunchAttribute* attr, int64_t T, int heads, int tt, int hc, size_t smem,
                                     cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((T + tt - 1) / tt), (unsigned)((heads + hc - 1) / hc));
    cfg.blockDim = dim3(kCtaThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    set_pdl_attr(attr[0]);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

int launch_rope(const void* x, int x_dtype, int64_t T, int heads, int D, int64_t x_ld, const int64_t* positions,
                const double* freqs, int rot, int layout, double mscale, int inverse, void* y, int y_dtype,
                int64_t y_ld, cudaStream_t st) {
    const RopeParams rp{positions, freqs, rot / 2, layout, mscale, inverse};
    int tt, hc;
    cta_shape(T, heads, D / 16, 8, tt, hc);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, T, heads, tt, hc, (size_t)(tt * rp.pairs) * sizeof(float2), st);
    cudaError_t e;
#define NVFP4_R(XT, YT)                                                                                             \
    e = cudaLaunchKernelEx(&cfg, rope_kernel<XT, YT>, (const XT*)x, T, heads, D / 16, x_ld, rp, (YT*)y, y_ld, tt, hc)
    if (x_dtype == NVFP4_DTYPE_BF16) {
        if (y_dtype == NVFP4_DTYPE_BF16) NVFP4_R(__nv_bfloat16, __nv_bfloat16);
        else NVFP4_R(__nv_bfloat16, float);
    } else {
        if (y_dtype == NVFP4_DTYPE_BF16) NVFP4_R(float, __nv_bfloat16);
        else NVFP4_R(float, float);
    }
#undef NVFP4_R
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

template <typename XT, int FMT, bool ROPE>
static cudaError_t kv_write_dim(cudaLaunchConfig_t& cfg, const KvWriteArgs& a) {
    switch (a.c.head_dim) {
        case 64: return cudaLaunchKernelEx(&cfg, kv_write_kernel<XT, FMT, 64, ROPE>, a);
        case 128: return cudaLaunchKernelEx(&cfg, kv_write_kernel<XT, FMT, 128, ROPE>, a);
        default: return cudaLaunchKernelEx(&cfg, kv_write_kernel<XT, FMT, 256, ROPE>, a);
    }
}
template <typename XT, bool ROPE>
static cudaError_t kv_write_fmt(cudaLaunchConfig_t& cfg, const KvWriteArgs& a) {
    switch (a.c.format) {
        case NVFP4_KV_BF16: return kv_write_dim<XT, NVFP4_KV_BF16, ROPE>(cfg, a);
        case NVFP4_KV_E4M3: return kv_write_dim<XT, NVFP4_KV_E4M3, ROPE>(cfg, a);
        default: return kv_write_dim<XT, NVFP4_KV_NVFP4, ROPE>(cfg, a);
    }
}

int launch_kv_write(const KvView& c, const void* k, const void* v, int x_dtype, int64_t T, int64_t k_ld, int64_t v_ld,
                    const int64_t* slots, int* status, cudaStream_t st) {
    KvWriteArgs a{};
    a.c = c;
    a.k = k;
    a.v = v;
    a.k_ld = k_ld;
    a.v_ld = v_ld;
    a.T = T;
    a.slots = slots;
    a.rp.pairs = c.head_dim / 2;
    a.status = status;
    cta_shape(T, 2 * c.heads, c.head_dim / 16, 4, a.tt, a.hc);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, T, 2 * c.heads, a.tt, a.hc, 0, st);
    const cudaError_t e = x_dtype == NVFP4_DTYPE_BF16 ? kv_write_fmt<__nv_bfloat16, false>(cfg, a)
                                                      : kv_write_fmt<float, false>(cfg, a);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

int launch_rope_kv_write(const KvView& c, const void* q, const void* k, const void* v, int x_dtype, int64_t T,
                         int q_heads, int64_t q_ld, int64_t k_ld, int64_t v_ld, const int64_t* positions,
                         const int64_t* slots, const double* freqs, int rot, int layout, double mscale, void* q_out,
                         int* status, cudaStream_t st) {
    KvWriteArgs a{};
    a.c = c;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_ld = q_ld;
    a.k_ld = k_ld;
    a.v_ld = v_ld;
    a.T = T;
    a.q_heads = q_heads;
    a.slots = slots;
    a.rp = RopeParams{positions, freqs, rot / 2, layout, mscale, 0};
    a.q_out = (__nv_bfloat16*)q_out;
    a.status = status;
    const int heads = q_heads + 2 * c.heads;
    cta_shape(T, heads, c.head_dim / 16, 4, a.tt, a.hc);
    const size_t smem = (size_t)(a.tt * a.rp.pairs) * sizeof(float2);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, T, heads, a.tt, a.hc, smem, st);
    const cudaError_t e = x_dtype == NVFP4_DTYPE_BF16 ? kv_write_fmt<__nv_bfloat16, true>(cfg, a)
                                                      : kv_write_fmt<float, true>(cfg, a);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

template <typename YT, int FMT>
static cudaError_t kv_read_dim(cudaLaunchConfig_t& cfg, const KvReadArgs& a) {
    switch (a.c.head_dim) {
        case 64: return cudaLaunchKernelEx(&cfg, kv_read_kernel<YT, FMT, 64>, a);
        case 128: return cudaLaunchKernelEx(&cfg, kv_read_kernel<YT, FMT, 128>, a);
        default: return cudaLaunchKernelEx(&cfg, kv_read_kernel<YT, FMT, 256>, a);
    }
}
template <typename YT>
static cudaError_t kv_read_fmt(cudaLaunchConfig_t& cfg, const KvReadArgs& a) {
    switch (a.c.format) {
        case NVFP4_KV_BF16: return kv_read_dim<YT, NVFP4_KV_BF16>(cfg, a);
        case NVFP4_KV_E4M3: return kv_read_dim<YT, NVFP4_KV_E4M3>(cfg, a);
        default: return kv_read_dim<YT, NVFP4_KV_NVFP4>(cfg, a);
    }
}

int launch_kv_read(const KvView& c, const int64_t* slots, int64_t T, void* k_out, void* v_out, int y_dtype,
                   int* status, cudaStream_t st) {
    KvReadArgs a{};
    a.c = c;
    a.slots = slots;
    a.T = T;
    a.k_out = k_out;
    a.v_out = v_out;
    a.status = status;
    cta_shape(T, 2 * c.heads, c.head_dim / 16, 16, a.tt, a.hc);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, T, 2 * c.heads, a.tt, a.hc, 0, st);
    const cudaError_t e =
        y_dtype == NVFP4_DTYPE_BF16 ? kv_read_fmt<__nv_bfloat16>(cfg, a) : kv_read_fmt<float>(cfg, a);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

}  // namespace nvfp4
