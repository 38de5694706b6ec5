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
// all of its heads, so this costs less than a table would cost in reads.  The
// rotation is fp32 with every product and sum rounded (no contraction), so
// the same inputs give the same bits in the separate and the fused kernel.
//
// All three kernels move each byte once and are bound by HBM for long chunks
// and by latency for decode steps; a thread owns a unit of 16 elements (one
// NVFP4 block).  All are programmatic dependents.
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

// (cos, sin) of the CTA's tokens into cs[token][pair].
NVFP4_DEV void rope_angles(const RopeParams& rp, int64_t t0, int nt, float2* cs) {
    for (int i = threadIdx.x; i < nt * rp.pairs; i += blockDim.x) {
        const int tl = i / rp.pairs, p = i - tl * rp.pairs;
        const double turns = (double)rp.positions[t0 + tl] * rp.freqs[p];
        double s, c;
        sincospi(2.0 * (turns - rint(turns)), &s, &c);
        if (rp.inverse) s = -s;
        cs[i] = make_float2((float)(c * rp.mscale), (float)(s * rp.mscale));
    }
}

// Unit j of a head: the element offsets of its two runs of 8.
NVFP4_DEV void rope_runs(const RopeParams& rp, int j, int& lo, int& hi) {
    if (j * 8 < rp.pairs && rp.layout == NVFP4_ROPE_HALF) {
        lo = j * 8;
        hi = rp.pairs + j * 8;
    } else {
        lo = j * 16;
        hi = lo + 8;
    }
}

NVFP4_DEV void rotate(float& a, float& b, float2 cs) {
    const float x = a, y = b;
    a = __fsub_rn(__fmul_rn(x, cs.x), __fmul_rn(y, cs.y));
    b = __fadd_rn(__fmul_rn(y, cs.x), __fmul_rn(x, cs.y));
}

// Rotates the two runs of unit j (cs: the token's angles).
NVFP4_DEV void rope_unit(const RopeParams& rp, int j, const float2* cs, float (&lo)[8], float (&hi)[8]) {
    if (j * 8 >= rp.pairs) return;
    cs += j * 8;
    if (rp.layout == NVFP4_ROPE_HALF) {
#pragma unroll
        for (int i = 0; i < 8; ++i) rotate(lo[i], hi[i], cs[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rotate(lo[2 * i], lo[2 * i + 1], cs[i]);
            rotate(hi[2 * i], hi[2 * i + 1], cs[4 + i]);
        }
    }
}

constexpr int kCtaThreads = 256;

// A CTA takes `tt` tokens and `hc` heads; consecutive threads take
// consecutive units of a head, so a warp's loads are contiguous.
template <typename XT, typename YT>
__global__ void __launch_bounds__(kCtaThreads) rope_kernel(const XT* x, int64_t T, int heads, int units, int64_t x_ld,
                                                           RopeParams rp, YT* y, int64_t y_ld, int tt, int hc) {
    extern __shared__ __align__(16) uint8_t smem[];
    float2* cs = reinterpret_cast<float2*>(smem);
    griddep_launch_dependents();
    griddep_wait();
    const int64_t t0 = (int64_t)blockIdx.x * tt;
    const int nt = (int)(T - t0 < tt ? T - t0 : tt);
    const int h0 = blockIdx.y * hc, nh = min(heads - h0, hc);
    rope_angles(rp, t0, nt, cs);
    __syncthreads();
    const int per = nh * units;
    for (int u = threadIdx.x; u < nt * per; u += kCtaThreads) {
        const int tl = u / per, hj = u - tl * per;
        const int h = h0 + hj / units, j = hj % units;
        int lo, hi;
        rope_runs(rp, j, lo, hi);
        const int64_t col = (int64_t)h * units * 16;
        const XT* xp = x + (t0 + tl) * x_ld + col;
        float a[8], b[8];
        load8(xp + lo, a);
        load8(xp + hi, b);
        rope_unit(rp, j, cs + tl * rp.pairs, a, b);
        YT* yp = y + (t0 + tl) * y_ld + col;
        store8(yp + lo, a);
        store8(yp + hi, b);
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

// Block j (16 elements) of tile row r, into the keys (which 0) or values (1)
// of the tile.
template <int FMT>
NVFP4_DEV void store_block(uint8_t* tile, int which, int r, int j, int D, const float (&v)[16], const GsPar& g) {
    const int db = kv_code_bytes(FMT, D), pieces = db >> 4;
    uint8_t* row = tile + (which * kKvTile + r) * db;
    if constexpr (FMT == NVFP4_KV_BF16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = v[8 * h + i];
            *reinterpret_cast<uint4*>(row + kv_place(r, (2 * j + h) * 16, pieces)) = pack8_bf16(w);
        }
    } else if constexpr (FMT == NVFP4_KV_E4M3) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = e4m3x2_of_quotients(v[4 * i], v[4 * i + 1], g) |
                   (e4m3x2_of_quotients(v[4 * i + 2], v[4 * i + 3], g) << 16);
        *reinterpret_cast<uint4*>(row + kv_place(r, j * 16, pieces)) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
        const uint32_t sb = e4m3_of_quotient(amax, g.denom, g.inv_denom);
        const float rsc = __fmul_rn(e4m3_to_f32(sb), g.gs);
        uint2 packed = make_uint2(0u, 0u);
        if (rsc != 0.0f) packed = e2m1x16_of_quotients(v, amax, rsc, rcp_safe(rsc) ? rcp_approx(rsc) : 0.0f);
        *reinterpret_cast<uint2*>(row + kv_place(r, j * 8, pieces)) = packed;
        tile[2 * kKvTile * db + (which * kKvTile + r) * (D >> 4) + j] = (uint8_t)sb;
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

constexpr int kMaxTokens = 16;  // tokens per CTA, at most

// Heads 0 .. q_heads - 1 are the queries, then the keys, then the values.
// Rotated keys pass through shared memory (bf16): a unit's two runs of 8 lie
// in two blocks when pairs are half a head apart.
template <typename XT, int FMT, bool ROPE>
__global__ void __launch_bounds__(kCtaThreads) kv_write_kernel(const KvWriteArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int64_t s_tile[kMaxTokens];  // byte offset of the token's tile, head 0; -1: not stored
    __shared__ int s_row[kMaxTokens];
    griddep_launch_dependents();
    griddep_wait();
    const int D = a.c.head_dim, units = D >> 4;
    const int64_t t0 = (int64_t)blockIdx.x * a.tt;
    const int nt = (int)(a.T - t0 < a.tt ? a.T - t0 : a.tt);
    const int heads = a.q_heads + 2 * a.c.heads;
    const int h0 = blockIdx.y * a.hc, nh = min(heads - h0, a.hc);
    const int tiles = a.c.page_size / kKvTile;
    const int64_t head_bytes = (int64_t)tiles * kv_tile_bytes(FMT, D);
    if ((int)threadIdx.x < nt) {
        const int64_t slot = a.slots[t0 + threadIdx.x];
        int64_t off = -1;
        int r = 0;
        if (slot >= 0) {
            const int64_t page = slot / a.c.page_size;
            const int in = (int)(slot - page * a.c.page_size);
            r = in % kKvTile;
            if (page < a.c.num_pages)
                off = page * a.c.heads * head_bytes + (int64_t)(in / kKvTile) * kv_tile_bytes(FMT, D);
            else if (a.status)
                atomicExch(a.status, NVFP4_ERR_PAGE);
        }
        s_tile[threadIdx.x] = off;
        s_row[threadIdx.x] = r;
    }
    float2* cs = reinterpret_cast<float2*>(smem);
    __nv_bfloat16* staged = reinterpret_cast<__nv_bfloat16*>(smem + (ROPE ? a.tt * a.rp.pairs * (int)sizeof(float2) : 0));
    if constexpr (ROPE) rope_angles(a.rp, t0, nt, cs);
    GsPar gk{}, gv{};
    if constexpr (FMT != NVFP4_KV_BF16) {
        gk = gs_par(a.c.k_gs);
        gv = gs_par(a.c.v_gs);
    }
    __syncthreads();
    const int k0 = a.q_heads, v0 = a.q_heads + a.c.heads;
    const int kfirst = max(h0, k0), nk = max(0, min(h0 + nh, v0) - kfirst);  // key heads of this CTA
    const int per = nh * units;
    for (int u = threadIdx.x; u < nt * per; u += kCtaThreads) {
        const int tl = u / per, hj = u - tl * per;
        const int h = h0 + hj / units, j = hj % units;
        const int64_t t = t0 + tl;
        if (ROPE && h < v0) {
            const bool is_q = h < k0;
            if (!is_q && s_tile[tl] < 0) continue;
            const XT* xp = is_q ? (const XT*)a.q + t * a.q_ld + (int64_t)h * D
                                : (const XT*)a.k + t * a.k_ld + (int64_t)(h - k0) * D;
            int lo, hi;
            rope_runs(a.rp, j, lo, hi);
            float x[8], y[8];
            load8(xp + lo, x);
            load8(xp + hi, y);
            rope_unit(a.rp, j, cs + tl * a.rp.pairs, x, y);
            __nv_bfloat16* yp =
                is_q ? a.q_out + (t * a.q_heads + h) * D : staged + (tl * nk + (h - kfirst)) * D;
            store8(yp + lo, x);
            store8(yp + hi, y);
        } else {
            if (s_tile[tl] < 0) continue;
            const bool is_v = h >= v0;
            const int hk = is_v ? h - v0 : h - k0;
            const XT* xp = is_v ? (const XT*)a.v + t * a.v_ld : (const XT*)a.k + t * a.k_ld;
            xp += (int64_t)hk * D + j * 16;
            float x[8], y[8], w[16];
            load8(xp, x);
            load8(xp + 8, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = x[i];
                w[8 + i] = y[i];
            }
            store_block<FMT>(a.c.data + s_tile[tl] + hk * head_bytes, is_v, s_row[tl], j, D, w, is_v ? gv : gk);
        }
    }
    if constexpr (ROPE) {
        __syncthreads();
        const int kper = nk * units;
        for (int u = threadIdx.x; u < nt * kper; u += kCtaThreads) {
            const int tl = u / kper, hj = u - tl * kper;
            const int hl = hj / units, j = hj % units;
            if (s_tile[tl] < 0) continue;
            const __nv_bfloat16* xp = staged + (tl * nk + hl) * D + j * 16;
            float x[8], y[8], w[16];
            load8(xp, x);
            load8(xp + 8, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = x[i];
                w[8 + i] = y[i];
            }
            store_block<FMT>(a.c.data + s_tile[tl] + (kfirst - k0 + hl) * head_bytes, 0, s_row[tl], j, D, w, gk);
        }
    }
}

// ---- cache reads -------------------------------------------------------------

// Block j of tile row r as fp32 values.
template <int FMT>
NVFP4_DEV void load_block(const uint8_t* tile, int which, int r, int j, int D, float gs, float (&v)[16]) {
    const int db = kv_code_bytes(FMT, D), pieces = db >> 4;
    const uint8_t* row = tile + (which * kKvTile + r) * db;
    if constexpr (FMT == NVFP4_KV_BF16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float w[8];
            load8(reinterpret_cast<const __nv_bfloat16*>(row + kv_place(r, (2 * j + h) * 16, pieces)), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[8 * h + i] = w[i];
        }
    } else if constexpr (FMT == NVFP4_KV_E4M3) {
        const uint4 c = *reinterpret_cast<const uint4*>(row + kv_place(r, j * 16, pieces));
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
            v[2 * i] = __fmul_rn(f.x, gs);
            v[2 * i + 1] = __fmul_rn(f.y, gs);
        }
    } else {
        const uint2 c = *reinterpret_cast<const uint2*>(row + kv_place(r, j * 8, pieces));
        const float s = e4m3_to_f32(tile[2 * kKvTile * db + (which * kKvTile + r) * (D >> 4) + j]);
        const uint32_t w[2] = {c.x, c.y};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t p[4];
            e2m1x8_to_f16x2(w[h], p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = f16x2_to_f32x2(p[i]);
                v[8 * h + 2 * i] = __fmul_rn(__fmul_rn(f.x, s), gs);  // E2M1 * E4M3 is exact
                v[8 * h + 2 * i + 1] = __fmul_rn(__fmul_rn(f.y, s), gs);
            }
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
template <typename YT, int FMT>
__global__ void __launch_bounds__(kCtaThreads) kv_read_kernel(const KvReadArgs a) {
    __shared__ int64_t s_tile[kMaxTokens];
    __shared__ int s_row[kMaxTokens];
    griddep_launch_dependents();
    griddep_wait();
    const int D = a.c.head_dim, units = D >> 4;
    const int64_t t0 = (int64_t)blockIdx.x * a.tt;
    const int nt = (int)(a.T - t0 < a.tt ? a.T - t0 : a.tt);
    const int h0 = blockIdx.y * a.hc, nh = min(2 * a.c.heads - h0, a.hc);
    const int tiles = a.c.page_size / kKvTile;
    const int64_t head_bytes = (int64_t)tiles * kv_tile_bytes(FMT, D);
    if ((int)threadIdx.x < nt) {
        const int64_t slot = a.slots[t0 + threadIdx.x];
        int64_t off = -1;
        int r = 0;
        if (slot >= 0) {
            const int64_t page = slot / a.c.page_size;
            const int in = (int)(slot - page * a.c.page_size);
            r = in % kKvTile;
            if (page < a.c.num_pages)
                off = page * a.c.heads * head_bytes + (int64_t)(in / kKvTile) * kv_tile_bytes(FMT, D);
            else if (a.status)
                atomicExch(a.status, NVFP4_ERR_PAGE);
        }
        s_tile[threadIdx.x] = off;
        s_row[threadIdx.x] = r;
    }
    float gk = 1.0f, gv = 1.0f;
    if constexpr (FMT != NVFP4_KV_BF16) {
        gk = *a.c.k_gs;
        gv = *a.c.v_gs;
    }
    __syncthreads();
    const int per = nh * units;
    for (int u = threadIdx.x; u < nt * per; u += kCtaThreads) {
        const int tl = u / per, hj = u - tl * per;
        const int h = h0 + hj / units, j = hj % units;
        const bool is_v = h >= a.c.heads;
        const int hk = is_v ? h - a.c.heads : h;
        float v[16];
        if (s_tile[tl] >= 0) {
            load_block<FMT>(a.c.data + s_tile[tl] + hk * head_bytes, is_v, s_row[tl], j, D, is_v ? gv : gk, v);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0.0f;
        }
        YT* yp = (YT*)(is_v ? a.v_out : a.k_out) + ((t0 + tl) * a.c.heads + hk) * D + j * 16;
        float x[8], y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = v[i];
            y[i] = v[8 + i];
        }
        store8(yp, x);
        store8(yp + 8, y);
    }
}

// ---- launches ----------------------------------------------------------------

// Tokens and heads of a CTA.  Few units in all: one per thread, one token per
// CTA (latency).  Many: about four per thread and up to 16 tokens, so that
// angles and addresses are shared.
static void cta_shape(int64_t T, int heads, int units, int pairs, int& tt, int& hc) {
    int per_thread = 1;
    tt = 1;
    if (T * heads * units > (int64_t)148 * 8 * kCtaThreads) {
        per_thread = 4;
        tt = pairs ? kCtaThreads / pairs : kMaxTokens;
        tt = tt < 1 ? 1 : tt > kMaxTokens ? kMaxTokens : tt;
    }
    hc = (kCtaThreads * per_thread + tt * units - 1) / (tt * units);
    if (hc < 1) hc = 1;
    if (hc > heads) hc = heads;
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
    cta_shape(T, heads, D / 16, rp.pairs, tt, hc);
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

template <typename XT, bool ROPE>
static cudaError_t kv_write_fmt(cudaLaunchConfig_t& cfg, const KvWriteArgs& a) {
    switch (a.c.format) {
        case NVFP4_KV_BF16: return cudaLaunchKernelEx(&cfg, kv_write_kernel<XT, NVFP4_KV_BF16, ROPE>, a);
        case NVFP4_KV_E4M3: return cudaLaunchKernelEx(&cfg, kv_write_kernel<XT, NVFP4_KV_E4M3, ROPE>, a);
        default: return cudaLaunchKernelEx(&cfg, kv_write_kernel<XT, NVFP4_KV_NVFP4, ROPE>, a);
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
    cta_shape(T, 2 * c.heads, c.head_dim / 16, 0, a.tt, a.hc);
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
    cta_shape(T, heads, c.head_dim / 16, a.rp.pairs, a.tt, a.hc);
    const int staged_heads = a.hc < c.heads ? a.hc : c.heads;
    const size_t smem = (size_t)(a.tt * a.rp.pairs) * sizeof(float2) + (size_t)a.tt * staged_heads * c.head_dim * 2;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, T, heads, a.tt, a.hc, smem, st);
    const cudaError_t e = x_dtype == NVFP4_DTYPE_BF16 ? kv_write_fmt<__nv_bfloat16, true>(cfg, a)
                                                      : kv_write_fmt<float, true>(cfg, a);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

template <typename YT>
static cudaError_t kv_read_fmt(cudaLaunchConfig_t& cfg, const KvReadArgs& a) {
    switch (a.c.format) {
        case NVFP4_KV_BF16: return cudaLaunchKernelEx(&cfg, kv_read_kernel<YT, NVFP4_KV_BF16>, a);
        case NVFP4_KV_E4M3: return cudaLaunchKernelEx(&cfg, kv_read_kernel<YT, NVFP4_KV_E4M3>, a);
        default: return cudaLaunchKernelEx(&cfg, kv_read_kernel<YT, NVFP4_KV_NVFP4>, a);
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
    cta_shape(T, 2 * c.heads, c.head_dim / 16, 0, a.tt, a.hc);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, T, 2 * c.heads, a.tt, a.hc, 0, st);
    const cudaError_t e =
        y_dtype == NVFP4_DTYPE_BF16 ? kv_read_fmt<__nv_bfloat16>(cfg, a) : kv_read_fmt<float>(cfg, a);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

}  // namespace nvfp4
