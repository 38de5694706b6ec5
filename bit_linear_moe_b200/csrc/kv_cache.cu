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
// and by latency for decode steps.  A thread takes units of 16 elements (one
// NVFP4 block) of a row, a row being one head of one token.  A warp takes one
// head at a time and the CTA's tokens along it, its lanes covering 2 to 8 whole
// rows, so that everything but a row's place is known per head; the loads of
// two rows per lane go out together (four, with the registers they take: 38.8 and
// 45.0 us for the first two cases below).  All
// are programmatic dependents.
//
// Measured (B200, replayed from a graph):
//   rotation of 8,191 tokens x 40 heads of 128, 64 rotated, bf16: 29.8 us, 5.6 TB/s
//     (86 % of a copy's rate); one token: 2.0 us, the launch
//   2,048 tokens of 20 heads written to NVFP4 pages and 10,240 read back: 35.0 us,
//     4.6 TB/s (70 %): the quotients' brackets when writing (issue), byte and
//     4-byte accesses when reading
//   rotation, write and read of 2,048 tokens, 32 / 8 heads, bf16: 16.9 us, 4.0 TB/s
//     (60 %): two short kernels, each with its ramp; 32 decoding tokens: 5.5 us
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

// (cos, sin) of the CTA's tokens, ordered so that neighbouring lanes read
// neighbouring words: pair p of token tl at [tl][p % w][p / w], w the pairs of a
// run of 8 elements (8 where a run holds one element of each pair, else 4).
NVFP4_DEV void rope_angles(const RopeParams& rp, int64_t t0, int nt, float2* cs) {
    const int lw = rp.layout == NVFP4_ROPE_HALF ? 3 : 2, runs = rp.pairs >> lw;
    for (int i = threadIdx.x; i < nt * rp.pairs; i += blockDim.x) {
        const int tl = i / rp.pairs, p = i - tl * rp.pairs;
        const double turns = (double)rp.positions[t0 + tl] * rp.freqs[p];
        double s, c;
        sincos_turns(turns - rint(turns), s, c);
        if (rp.inverse) s = -s;
        cs[tl * rp.pairs + (p & ((1 << lw) - 1)) * runs + (p >> lw)] =
            make_float2((float)(c * rp.mscale), (float)(s * rp.mscale));
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

NVFP4_DEV void rotate(float& a, float& b, float2 cs) {
    const float x = a, y = b;
    a = __fsub_rn(__fmul_rn(x, cs.x), __fmul_rn(y, cs.y));
    b = __fadd_rn(__fmul_rn(y, cs.x), __fmul_rn(x, cs.y));
}

// Rotates the two runs of unit j of token tl.
NVFP4_DEV void rope_unit(const RopeParams& rp, int j, int tl, const float2* cs, float (&lo)[8], float (&hi)[8]) {
    const int n8 = rp.pairs >> 3;
    if (j >= n8) return;
    cs += tl * rp.pairs + j;
    if (rp.layout == NVFP4_ROPE_HALF) {
#pragma unroll
        for (int i = 0; i < 8; ++i) rotate(lo[i], hi[i], cs[i * n8]);
    } else {
        const int runs = 2 * n8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rotate(lo[2 * i], lo[2 * i + 1], cs[i * runs]);
            rotate(hi[2 * i], hi[2 * i + 1], cs[i * runs + n8]);
        }
    }
}

constexpr int kCtaThreads = 256, kWarps = kCtaThreads / 32;
constexpr int kBatch = 2;       // rows per lane whose loads go out together
constexpr int kMaxTokens = 32;  // tokens per CTA, at most

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
    float2* cs = reinterpret_cast<float2*>(smem);
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

// Global scale of one of K / V with what its quotients need.
struct GsPar {
    float gs, denom, inv_denom, inv_gs;
};
NVFP4_DEV GsPar gs_par(const float* p) {
    GsPar g;
    g.gs = *p;
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
// E4M3 codes of RN(a / gs), RN(b / gs): the reciprocal product's bracket
// decides (as e4m3_of_quotient, with a sign), the division where it does not.
NVFP4_DEV uint32_t e4m3x2_of_quotients(float a, float b, const GsPar& g) {
    if (g.inv_gs != 0.0f) {
        const float p = __fmul_rn(a, g.inv_gs), q = __fmul_rn(b, g.inv_gs);
        const uint32_t lo = f32x2_to_e4m3(__fmul_rn(p, kBracketLo), __fmul_rn(q, kBracketLo));
        if (lo == f32x2_to_e4m3(__fmul_rn(p, kBracketHi), __fmul_rn(q, kBracketHi))) return lo;
    }
    return f32x2_to_e4m3(__fdiv_rn(a, g.gs), __fdiv_rn(b, g.gs));
}

// Where a token's rows lie: bytes from a head's first tile to its tile's codes
// (key rows; -1: not stored), the tile row, and how its pieces are turned.
struct Slot {
    int64_t tile;
    int r, turn;
};
template <int FMT, int D>
NVFP4_DEV void find_slots(const KvView& c, const int64_t* slots, int64_t t0, int nt, int64_t head_bytes, int* status,
                          Slot* out) {
    if ((int)threadIdx.x >= nt) return;
    const int64_t slot = slots[t0 + threadIdx.x];
    Slot s{-1, 0, 0};
    if (slot >= 0) {
        // (a 32-bit division where it does, which is nearly always)
        const int64_t page = slot >> 31 ? slot / c.page_size : (int64_t)((uint32_t)slot / (uint32_t)c.page_size);
        const int in = (int)(slot - page * c.page_size);
        s.r = in % kKvTile;
        s.turn = kv_turn(s.r, kv_code_bytes(FMT, D) / 16);
        if (page < c.num_pages)
            s.tile = page * c.heads * head_bytes + (int64_t)(in / kKvTile) * kv_tile_bytes(FMT, D);
        else if (status)
            atomicExch(status, NVFP4_ERR_PAGE);
    }
    out[threadIdx.x] = s;
}

// Address of byte o of row s.r of the keys (which 0) or values (1) of a tile.
template <int FMT, int D>
NVFP4_DEV uint8_t* row_at(uint8_t* tile, int which, const Slot& s, int o) {
    return tile + (which * kKvTile + s.r) * kv_code_bytes(FMT, D) + ((((o >> 4) ^ s.turn) << 4) | (o & 15));
}
template <int D>
NVFP4_DEV uint8_t* scale_at(uint8_t* tile, int which, const Slot& s, int j) {
    return tile + 2 * kKvTile * kv_code_bytes(NVFP4_KV_NVFP4, D) + (which * kKvTile + s.r) * (D / 16) + j;
}

// E2M1 codes (a word) of v[j] / r, j < 8: e2m1x16_of_quotients' argument for
// half a block (amax: the block's).
NVFP4_DEV uint32_t e2m1x8_of_quotients(const float (&v)[8], float amax, float r) {
    const float inv = rcp_safe(r) ? rcp_approx(r) : 0.0f;
    uint32_t code = 0u, diff = 0xFFFFFFFFu;
    if (inv != 0.0f && __fmul_rn(amax, inv) < 15.0f) {
        float lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float p = __fmul_rn(v[j], inv);
            lo[j] = __fmul_rn(p, kBracketLo);
            hi[j] = __fmul_rn(p, kBracketHi);
        }
        code = f32x8_to_e2m1(hi);
        diff = f32x8_to_e2m1(lo) ^ code;
    }
    if (diff) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (diff & (0xFu << (4 * j))) code = (code & ~(0xFu << (4 * j))) | (e2m1_of_division(v[j], r) << (4 * j));
    }
    return code;
}

// Eight elements e .. e + 7 of a row.  NVFP4: lanes 2 i and 2 i + 1 hold the
// halves of a block; every lane of the warp calls (live: something is stored).
template <int FMT, int D>
NVFP4_DEV void store_run(bool live, uint8_t* tile, int which, const Slot& s, int e, const float (&v)[8],
                         const GsPar& g) {
    if constexpr (FMT == NVFP4_KV_BF16) {
        if (live) *reinterpret_cast<uint4*>(row_at<FMT, D>(tile, which, s, 2 * e)) = pack8_bf16(v);
    } else if constexpr (FMT == NVFP4_KV_E4M3) {
        if (live) {
            const uint32_t w0 = e4m3x2_of_quotients(v[0], v[1], g) | (e4m3x2_of_quotients(v[2], v[3], g) << 16);
            const uint32_t w1 = e4m3x2_of_quotients(v[4], v[5], g) | (e4m3x2_of_quotients(v[6], v[7], g) << 16);
            *reinterpret_cast<uint2*>(row_at<FMT, D>(tile, which, s, e)) = make_uint2(w0, w1);
        }
    } else {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        if (live) {
            const uint32_t sb = e4m3_of_quotient(amax, g.denom, g.inv_denom);
            const float rsc = __fmul_rn(e4m3_to_f32(sb), g.gs);
            *reinterpret_cast<uint32_t*>(row_at<FMT, D>(tile, which, s, e / 2)) =
                rsc != 0.0f ? e2m1x8_of_quotients(v, amax, rsc) : 0u;
            if ((e & 8) == 0) *scale_at<D>(tile, which, s, e / 16) = (uint8_t)sb;
        }
    }
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
    RopeParams rp;
    __nv_bfloat16* q_out;  // [T, q_heads, D]
    int tt, hc;
    int* status;
};

// Heads 0 .. q_heads - 1 are the queries, then the keys, then the values.
// Rotated keys of the NVFP4 cache pass through the warp's own piece of shared
// memory (bf16): a unit's two runs of 8 lie in two blocks.
template <typename XT, int FMT, int D, bool ROPE>
__global__ void __launch_bounds__(kCtaThreads, sizeof(XT) == 2 ? 4 : 3) kv_write_kernel(const KvWriteArgs a) {
    constexpr int units = D / 16, per = 32 / units;
    constexpr int batch = kBatch;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Slot s_slot[kMaxTokens];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t t0 = (int64_t)blockIdx.x * a.tt;
    const int nt = (int)(a.T - t0 < a.tt ? a.T - t0 : a.tt);
    const int k0 = a.q_heads, v0 = a.q_heads + a.c.heads, heads = v0 + a.c.heads;
    const int h0 = blockIdx.y * a.hc, h1 = min(heads, h0 + a.hc);
    const int64_t head_bytes = (int64_t)(a.c.page_size / kKvTile) * kv_tile_bytes(FMT, D);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % units, first = lane / units;
    int h = h0 + warp, tb = 0;
    Raw16<XT> raw[batch];
    auto head_of = [&](int hh) { return hh < k0 ? hh : hh >= v0 ? hh - v0 : hh - k0; };
    auto load = [&]() {  // the lane's rows of head h from token tb on
        if (h >= h1) return;
        const bool is_q = h < k0, is_v = h >= v0;  // without ROPE there are no queries
        const int64_t ld = is_q ? a.q_ld : is_v ? a.v_ld : a.k_ld;
        const XT* src = (is_q ? (const XT*)a.q : is_v ? (const XT*)a.v : (const XT*)a.k) + (t0 + tb + first) * ld +
                        head_of(h) * D;
        int lo = 8 * j, hi = D / 2 + 8 * j;
        if (ROPE && !is_v) rope_runs(a.rp, j, D, lo, hi);
#pragma unroll
        for (int k = 0; k < batch; ++k)
            if (tb + first + k * per < nt) raw[k].load(src + k * per * ld + lo, src + k * per * ld + hi);
    };
#pragma unroll
    for (int k = 0; k < batch; ++k) raw[k].clear();
    load();  // on their way while slots and angles are found
    find_slots<FMT, D>(a.c, a.slots, t0, nt, head_bytes, a.status, s_slot);
    float2* cs = reinterpret_cast<float2*>(smem);
    if constexpr (ROPE) rope_angles(a.rp, t0, nt, cs);
    GsPar gk{}, gv{};
    if constexpr (FMT != NVFP4_KV_BF16) {
        gk = gs_par(a.c.k_gs);
        gv = gs_par(a.c.v_gs);
    }
    __nv_bfloat16* staged =
        reinterpret_cast<__nv_bfloat16*>(smem + (ROPE ? a.tt * a.rp.pairs * (int)sizeof(float2) : 0)) +
        warp * batch * per * D;
    __syncthreads();
    while (h < h1) {
        uint8_t* base = a.c.data + head_of(h) * head_bytes;
        const bool is_q = h < k0, is_v = h >= v0, turned = ROPE && !is_v;
#pragma unroll
        for (int k = 0; k < batch; ++k) {
            const int tl = tb + first + k * per;
            const bool in = tl < nt;
            const Slot s = s_slot[in ? tl : 0];
            const bool live = in && s.tile >= 0;
            float x[8], y[8];
            raw[k].values(x, y);
            if (ROPE && turned) {
                int lo, hi;
                rope_runs(a.rp, j, D, lo, hi);
                if (in) rope_unit(a.rp, j, tl, cs, x, y);
                if (is_q) {
                    if (in) {
                        __nv_bfloat16* yp = a.q_out + ((t0 + tl) * a.q_heads + h) * D;
                        store8(yp + lo, x);
                        store8(yp + hi, y);
                    }
                } else if constexpr (FMT == NVFP4_KV_NVFP4) {
                    store8(staged + (first + k * per) * D + lo, x);
                    store8(staged + (first + k * per) * D + hi, y);
                } else {  // quantized from the bf16 values
                    const uint4 xw = pack8_bf16(x), yw = pack8_bf16(y);
                    load8(reinterpret_cast<const __nv_bfloat16*>(&xw), x);
                    load8(reinterpret_cast<const __nv_bfloat16*>(&yw), y);
                    store_run<FMT, D>(live, base + s.tile, 0, s, lo, x, gk);
                    store_run<FMT, D>(live, base + s.tile, 0, s, hi, y, gk);
                }
            } else {
                store_run<FMT, D>(live, base + s.tile, is_v, s, 8 * j, x, is_v ? gv : gk);
                store_run<FMT, D>(live, base + s.tile, is_v, s, D / 2 + 8 * j, y, is_v ? gv : gk);
            }
        }
        if constexpr (ROPE && FMT == NVFP4_KV_NVFP4) {
            if (!is_q && !is_v) {
                __syncwarp();
#pragma unroll
                for (int k = 0; k < batch; ++k) {
                    const int tl = tb + first + k * per;
                    const Slot s = s_slot[tl < nt ? tl : 0];
                    const bool live = tl < nt && s.tile >= 0;
                    float x[8], y[8];
                    load8(staged + (first + k * per) * D + 8 * j, x);
                    load8(staged + (first + k * per) * D + D / 2 + 8 * j, y);
                    store_run<FMT, D>(live, base + s.tile, 0, s, 8 * j, x, gk);
                    store_run<FMT, D>(live, base + s.tile, 0, s, D / 2 + 8 * j, y, gk);
                }
                __syncwarp();
            }
        }
        tb += batch * per;
        if (tb >= nt) {
            tb = 0;
            h += kWarps;
        }
        load();
    }
}

// ---- cache reads -------------------------------------------------------------

// Eight elements e .. e + 7 of a tile row as stored, and their fp32 values.
template <int FMT>
struct RawRun {
    uint32_t c[FMT == NVFP4_KV_BF16 ? 4 : FMT == NVFP4_KV_E4M3 ? 2 : 1];
    uint32_t sb;
};
template <int FMT, int D>
NVFP4_DEV void load_run(const uint8_t* tile_, int which, const Slot& s, int e, RawRun<FMT>& x) {
    uint8_t* tile = const_cast<uint8_t*>(tile_);
    if constexpr (FMT == NVFP4_KV_BF16) {
        const uint4 c = *reinterpret_cast<const uint4*>(row_at<FMT, D>(tile, which, s, 2 * e));
        x.c[0] = c.x, x.c[1] = c.y, x.c[2] = c.z, x.c[3] = c.w;
    } else if constexpr (FMT == NVFP4_KV_E4M3) {
        const uint2 c = *reinterpret_cast<const uint2*>(row_at<FMT, D>(tile, which, s, e));
        x.c[0] = c.x, x.c[1] = c.y;
    } else {
        x.c[0] = *reinterpret_cast<const uint32_t*>(row_at<FMT, D>(tile, which, s, e / 2));
        x.sb = *scale_at<D>(tile, which, s, e / 16);
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
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = f16x2_to_f32x2(p[i]);
            v[2 * i] = __fmul_rn(f.x, gs);
            v[2 * i + 1] = __fmul_rn(f.y, gs);
        }
    }
}

struct KvReadArgs {
    KvView c;
    const int64_t* slots;
    int64_t T;
    void* k_out;  // [T, heads, D]
    void* v_out;
    int tt, hc;
    int* status;
};

// Heads 0 .. heads - 1 are the keys, then the values.
template <typename YT, int FMT, int D>
__global__ void __launch_bounds__(kCtaThreads, FMT == NVFP4_KV_BF16 ? 6 : 8) kv_read_kernel(const KvReadArgs a) {
    constexpr int units = D / 16, per = 32 / units;
    __shared__ Slot s_slot[kMaxTokens];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t t0 = (int64_t)blockIdx.x * a.tt;
    const int nt = (int)(a.T - t0 < a.tt ? a.T - t0 : a.tt);
    const int h0 = blockIdx.y * a.hc, h1 = min(2 * a.c.heads, h0 + a.hc);
    const int64_t head_bytes = (int64_t)(a.c.page_size / kKvTile) * kv_tile_bytes(FMT, D);
    find_slots<FMT, D>(a.c, a.slots, t0, nt, head_bytes, a.status, s_slot);
    float gk = 1.0f, gv = 1.0f;
    if constexpr (FMT != NVFP4_KV_BF16) {
        gk = *a.c.k_gs;
        gv = *a.c.v_gs;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % units, first = lane / units;
    const int64_t y_ld = (int64_t)a.c.heads * D;
    __syncthreads();
    for (int h = h0 + warp; h < h1; h += kWarps) {
        const bool is_v = h >= a.c.heads;
        const int hk = is_v ? h - a.c.heads : h;
        const uint8_t* base = a.c.data + hk * head_bytes;
        YT* out = (YT*)(is_v ? a.v_out : a.k_out) + t0 * y_ld + hk * D + j * 8;
        const float gs = is_v ? gv : gk;
        constexpr int batch = kBatch;
        for (int tl0 = first; tl0 < nt; tl0 += batch * per) {
            RawRun<FMT> x[batch][2] = {};
#pragma unroll
            for (int k = 0; k < batch; ++k) {
                const int tl = tl0 + k * per;
                const Slot s = s_slot[tl < nt ? tl : 0];
                if (tl < nt && s.tile >= 0) {
                    load_run<FMT, D>(base + s.tile, is_v, s, 8 * j, x[k][0]);
                    load_run<FMT, D>(base + s.tile, is_v, s, D / 2 + 8 * j, x[k][1]);
                }
            }
#pragma unroll
            for (int k = 0; k < batch; ++k) {
                const int tl = tl0 + k * per;
                if (tl < nt) {
                    float v[8];
                    run_values<FMT>(x[k][0], gs, v);
                    store8(out + tl * y_ld, v);
                    run_values<FMT>(x[k][1], gs, v);
                    store8(out + tl * y_ld + D / 2, v);
                }
            }
        }
    }
}

// ---- launches ----------------------------------------------------------------

// Tokens and heads of a CTA.  Where a warp per head and one pass of its lanes
// leave the GPU unfilled (decode steps), that: latency counts.  Else `passes`
// passes, and as many heads as still leave `per_sm` CTAs per SM.  Rotations
// take 4 and 4: angles are found once for more heads (8,191 x 40 heads, 64 of
// 128 rotated: 29.9 us, against 32.1 with 16 per SM).  Plain writes and reads
// take 2 and 16: nothing is shared but the slots, and short CTAs even out
// better (10,240 tokens of 20 heads read after 2,048 are written, NVFP4: 35.0
// us for both, against 37.4 with 4 passes).
static void cta_shape(int64_t T, int heads, int units, int passes, int per_sm, int& tt, int& hc) {
    const int per = units < 32 ? 32 / units : 1;
    tt = per;
    hc = kWarps;
    if ((T + tt - 1) / tt * ((heads + hc - 1) / hc) > 148 * 4) {
        tt = per * passes;
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
    cta_shape(T, heads, D / 16, 4, 4, tt, hc);
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
    a.status = status;
    cta_shape(T, 2 * c.heads, c.head_dim / 16, 2, 16, a.tt, a.hc);
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
    cta_shape(T, heads, c.head_dim / 16, 4, 4, a.tt, a.hc);
    // angles; for NVFP4 a batch of bf16 key rows per warp
    const size_t rows = (size_t)kWarps * kBatch * (32 / (c.head_dim / 16)) * c.head_dim * 2;
    const size_t smem = (size_t)(a.tt * a.rp.pairs) * sizeof(float2) + (c.format == NVFP4_KV_NVFP4 ? rows : 0);
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
    cta_shape(T, 2 * c.heads, c.head_dim / 16, 2, 16, a.tt, a.hc);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, T, 2 * c.heads, a.tt, a.hc, 0, st);
    const cudaError_t e =
        y_dtype == NVFP4_DTYPE_BF16 ? kv_read_fmt<__nv_bfloat16>(cfg, a) : kv_read_fmt<float>(cfg, a);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

}  // namespace nvfp4
