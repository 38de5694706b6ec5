// K11: attention of one new token per sequence over the paged key-value cache
// (the step the dense decode stack leaves out; Ignis README, "The decode
// round": a decode step reads what it needs once, at the card's bandwidth).
//
//   s_j = scale * q . k_j   over  max(0, len - window) <= j < len
//   y   = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),   lse = ln sum_j e^(s_j)
//
// Bound: HBM.  Each seen cache row is read once for all query heads of its
// key head.  At G query heads per key head a cached byte (NVFP4, D = 128)
// carries 4 * G / 0.5625 / 2 flop, so the tensor cores are far from busy; what
// has to be watched is the number of instructions per tile (355 a warp for an
// NVFP4 tile at D = 128).  That is why the products use warp-level mma (m16n8k16): the fragments come straight from the
// 4-bit codes in registers (no round trip of dequantized tiles through shared
// or tensor memory), and N = 8 is the width that one token's query heads have.
// Both products are taken transposed:
//   S^T = K Q^T    A = 16 tokens x D (codes converted in registers), B = Q^T
//   O^T = V^T P^T  A = D x 16 tokens, B = P^T, from S^T's accumulators by
//                  movmatrix; token pairs of V are formed by byte permutes
// The inner dimension of the first product may be permuted at will, so a
// thread takes 16 contiguous bytes of a key row for its fragments; the rows
// of the second are the head's columns, so a thread takes contiguous bytes of
// value rows.
//
// Work split.  All tiles of all (sequence, key head, block of query columns)
// segments form one list; every CTA takes an equal contiguous range of it and
// every warp an equal range of that, whatever the lengths in the batch.  (Equal
// in cost: a segment counts kSegmentCost tiles more than it has, so that a
// warp does not get a dozen one-tile segments.)  A
// warp streams its tiles through a ring of its own (one bulk copy per tile,
// a ring's worth in flight) with its running maximum, sum and O^T in registers,
// and never meets another warp until the end.  Segments that lie inside a warp
// are written at once; the rest are joined per CTA through shared memory, and
// segments that span CTAs by attn_join_kernel from the workspace, in list
// order (the same inputs give the same bits).  Few tiles per warp go to
// attn_segment_kernel instead (kSegmentTiles).
//
// Measured (B200, replayed from a graph; floor: the bytes at 6,566 GB/s):
//   32 ragged sequences of up to 16,384 tokens, 40 query / 20 key heads, NVFP4:
//     170 us, 4.6 TB/s, 69 % of the floor.  Copies alone (no products) take 129;
//     without the values' half 144, without the scores' 150 (of 190, then).  Both
//     products' conversions and fragments count, but the issue slots are 62 % used (8 x
//     8,192 tokens) and DRAM less than half: a warp's scores, softmax and values follow
//     one another, and four warps per scheduler do not cover their latencies.
//   1 x 131,071, 32 / 8 heads, E4M3: 53 us, 5.1 TB/s, 78 %; copies alone 50
//     (about 9 us of it before the first bytes and in the join).  fp32 output: 53 us;
//     of the batch above 189.
//   1 x 8,192, 40 / 20 heads, NVFP4: 12.8 us (segment kernel), latency: 8 tiles
//     one after the other per warp, launch, page table and two joins.
//   64 ragged x 2,048, 32 / 2 heads of 64, BF16: 14.1 us; 16 x 4,000 with a
//     window of 1,000, 16 / 8 heads of 256, NVFP4: 13.2 us; 1 x 97: 4.0 us.
//   The same with a page table of 131,072 tokens (even split and join): 1 x 8,192
//     16.3 us, 64 x 2,048 21.8, 1 x 97 8.4; the others as above.
// Slower, measured on the first of these: the scores on the block-scaled
// tcgen05 MMA, queries as six NVFP4 terms (344 us; 382 with separate roles: a
// tile's 16 rows fill an eighth of an MMA), codes unpacked by bit operations (217
// against 191: a conversion takes a pair and names its byte), 10 warps per CTA
// (210 against 191: the registers no longer hold a step of two tiles).
#pragma once

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "kv_layout.cuh"
#include "tma.cuh"

namespace nvfp4 {
namespace attn {

constexpr int kCtasPerSm = 2;
constexpr int kMaxGrid = 148 * kCtasPerSm;

struct Args {
    KvView c;
    const __nv_bfloat16* q;  // [B] rows of q_heads * D at stride q_ld
    int64_t q_ld;
    int B, q_heads, G, chunks;  // chunks: blocks of `cols` query heads per key head
    const int32_t* table;       // [B, max_pages] at stride table_ld
    int64_t table_ld;
    int max_pages;
    const int32_t* lens;
    float scale_log2;  // scale * log2(e)
    int window;        // 0: all
    void* y;           // [B, q_heads, D]
    float* lse;        // [B, q_heads] or null
    uint32_t* header;  // workspace: [0] cost per CTA, then the list (see List)
    float* partial;    // workspace: [grid][2] pieces
    int* status;
    uint32_t zero;     // always 0 (see refill)
};

// What the host knows of a call: the grid of the even split, and the most
// tiles a segment can have.
struct Shape {
    int64_t grid, seg_tiles;
};
// Up to this many tiles per warp a cluster per segment is used.  Measured (us,
// cluster per segment / even split, and the cluster's tiles per warp): NVFP4, 20 key
// heads of 128: 1 x 8,192 tokens (8) 13.2 / 16.4, 16 x 1,024 (8) 12.1 / 19.1, 1 x 16,384
// (16) 21.8 / 21.9, 16 x 4,096 (32) 36.0 / 35.3, 1 x 32,768 (32) 38.4 / 32.5; 8 heads of
// 256: 1 x 4,096 (8) 10.9 / 12.7, 1 x 8,192 (16) 16.1 / 15.0; E4M3, 8 heads of 128: 4 x
// 16,384 (16) 19.9 / 24.4, 1 x 32,768 (32) 23.6 / 23.2; BF16, 8 heads of 128: 4 x 4,096
// (8) 10.9 / 14.2, 1 x 16,384 (32) 24.5 / 22.5.  At 16 tiles neither is always the faster.
// Segments beyond the resident CTAs run in waves: 8 heads of 128, NVFP4, 512 x 1,024 tokens (8)
// 148 / 143, 900 x 1,024 (8) 255 / 238, 4,096 x 256 (2) 525 / 407.
constexpr int64_t kSegmentTiles = 16;
// What beginning and ending a segment costs a warp, in tiles (measured: 2 x
// the 2,000 cycles of an NVFP4 tile at D = 128).
constexpr uint32_t kSegmentCost = 2;

// A piece: O [cols] rows of D (kLd apart: the fragments' stores, 16 elements
// apart from lane group to lane group and two columns from lane to lane, would
// meet in two banks without the two floats of padding), then m [cols] (log2
// units), then l [cols].
template <int D, int NT>
struct Piece {
    static constexpr int kCols = 8 * NT, kLd = D + 2;
    static constexpr int kMax = kCols * kLd, kSum = kMax + kCols;
    static constexpr int kFloats = (kSum + kCols + 3) / 4 * 4;
};

template <int FMT, int D, int NT>
struct Cfg {
    static constexpr int kDb = kv_code_bytes(FMT, D), kSb = kv_scale_bytes(FMT, D);
    static constexpr int kTile = kv_tile_bytes(FMT, D);
    static constexpr int kPieces = kDb / 16;
    static constexpr int kWarps = (D == 256 || kTile >= 8192 || (D == 128 && NT == 2)) ? 4 : 8;
    // ring: about 72 KB per CTA, so that two CTAs fit an SM (with the list of up to some
    // 940 sequences) and some 140 KB are on their way per SM (44 bytes per ns times
    // ~1 us of loaded latency asks for at least 44 KB)
    static constexpr int kRing = kTile >= 16384 ? 2 : (72 * 1024) / (kWarps * kTile) > 8 ? 8 : (72 * 1024) / (kWarps * kTile);
    static constexpr int kRingBytes = kWarps * kRing * kTile;
    static constexpr int kPieceBytes = Piece<D, NT>::kFloats * 4;
    static constexpr int kFixed = kRingBytes + kWarps * kPieceBytes;  // then the prefix
    static constexpr int kMt = D / 16;                                 // 16-row tiles of O^T
    // Tiles a warp works on at a time.  Two where the codes are converted: their
    // chains interleave and share the softmax's exchange and the loop (355
    // instructions a tile, 450 one at a time).
    static constexpr int kStep = FMT == NVFP4_KV_NVFP4 && kRing >= 4 ? 2 : 1;
    static_assert(kRing >= 2, "one tile in flight while one is used");
    static_assert(kRing * kTile >= kPieceBytes, "a warp's last piece goes into its ring");
};

NVFP4_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
NVFP4_DEV uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }
NVFP4_DEV uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
NVFP4_DEV uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
NVFP4_DEV uint32_t pack_b16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
NVFP4_DEV uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
template <bool BF16>
NVFP4_DEV void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shared memory by its 32-bit address (volatile: stays behind the barrier wait).
// N bytes (4, 8 or 16) as words.
template <int N>
NVFP4_DEV void lds(uint32_t p, uint32_t (&w)[N / 4]) {
    if constexpr (N == 16)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(p));
    else if constexpr (N == 8)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(p));
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(p));
}
NVFP4_DEV uint32_t lds_u16(uint32_t p) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p));
    return v;
}
NVFP4_DEV uint32_t lds_u8(uint32_t p) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(p));
    return v;
}

// Where a tile of the list lies.
struct Place {
    uint32_t b, s, j, tiles;  // sequence, segment of it (key head, chunk), tile of the seen ones, their number
};

// The list of all tiles: sequence b's hc segments begin at tile hc * first[b];
// rank[b] non-empty sequences come before it.  The list's cost positions count
// kSegmentCost more for every segment.
struct List {
    const uint32_t *first, *rank;  // [B + 1] each
    uint32_t B, hc;
    // sequence with at(b) <= u < at(b + 1)
    template <typename F>
    NVFP4_DEV uint32_t find(uint32_t u, F at) const {
        uint32_t lo = 0, hi = B;
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) >> 1;
            if (at(mid) <= u) lo = mid;
            else hi = mid;
        }
        return lo;
    }
    NVFP4_DEV uint32_t cost_at(uint32_t b) const { return hc * (first[b] + kSegmentCost * rank[b]); }
    // Where tile t of the list is.
    NVFP4_DEV Place place_of(uint32_t t) const {
        Place p;
        p.b = find(t / hc, [&](uint32_t b) { return first[b]; });
        p.tiles = first[p.b + 1] - first[p.b];
        const uint32_t rem = t - first[p.b] * hc;
        p.s = rem / p.tiles;
        p.j = rem - p.s * p.tiles;
        return p;
    }
    // The tiles before cost position u.
    NVFP4_DEV uint32_t tiles_before(uint32_t u) const {
        if (u >= cost_at(B)) return hc * first[B];
        const uint32_t b = find(u, [&](uint32_t k) { return cost_at(k); });
        const uint32_t tiles = first[b + 1] - first[b], rem = u - cost_at(b), s = rem / (tiles + kSegmentCost);
        return hc * first[b] + s * tiles + min(rem - s * (tiles + kSegmentCost), tiles);
    }
};

// Seen tokens of a sequence: [lo, len).
NVFP4_DEV void seen_range(const Args& a, int b, int& lo, int& len) {
    const int cap = a.max_pages * a.c.page_size;
    len = min(max(a.lens[b], 0), cap);
    lo = (a.window > 0 && len > a.window) ? len - a.window : 0;
}

// The page-table entry of tile jt of sequence b, and where that tile lies for
// key head hk.  A page out of range is reported and page 0 read in its place.
NVFP4_DEV uint32_t page_of(const Args& a, uint32_t jt) {
    const uint32_t per = (uint32_t)(a.c.page_size / kKvTile);
    return (per & (per - 1)) == 0 ? jt >> (31 - __clz(per)) : jt / per;
}
NVFP4_DEV int32_t table_entry(const Args& a, uint32_t b, uint32_t jt) {
    return a.table[(int64_t)b * a.table_ld + page_of(a, jt)];
}
template <int TILE>
NVFP4_DEV const uint8_t* tile_in_page(const Args& a, int64_t page, uint32_t hk, uint32_t jt) {
    const uint32_t per = (uint32_t)(a.c.page_size / kKvTile);
    if (page < 0 || page >= a.c.num_pages) {
        if (a.status) atomicExch(a.status, NVFP4_ERR_PAGE);
        page = 0;
    }
    return a.c.data + ((page * a.c.heads + hk) * per + (jt - page_of(a, jt) * per)) * TILE;
}

// Writes out[v] (eight consecutive columns) of one query head.
NVFP4_DEV void store_y8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_b16(v[0], v[1]), pack_b16(v[2], v[3]), pack_b16(v[4], v[5]), pack_b16(v[6], v[7]));
}
NVFP4_DEV void store_y8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

NVFP4_DEV void store_y2(__nv_bfloat16* p, float a, float b) { *reinterpret_cast<uint32_t*>(p) = pack_b16(a, b); }
NVFP4_DEV void store_y2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }

// 1 / l, or 0 where nothing was seen (or every score is -inf).  A NaN stays.
NVFP4_DEV float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
NVFP4_DEV float lse_of(float m, float l) {
    return l == 0.0f ? __int_as_float(0xff800000) : (m + log2f(l)) * 0.693147180559945309f;
}

// The weights of two pieces' running maxima.
NVFP4_DEV float weight(float m, float M) { return m == __int_as_float(0xff800000) ? 0.0f : ex2(m - M); }

// One tile's work for a warp.  The weights are p = 2^(x - m) with m the running maximum
// of a piece's scores (log2 units) less kLift, and l adds them in fp32.  For the
// product they are rounded:
//   quantized cache, bf16 output  one fp16 part, off by 2^-11 of each weight, where the
//                                 output's own rounding is 2^-8.  Two parts: 189 us against
//                                 170 for 32 x 16,384 tokens of NVFP4 (177 with the low
//                                 part in the columns that pad G <= 4 to 8), 9.7 against
//                                 8.7 for 1 x 8,192 of E4M3
//   quantized cache, fp32 output  two fp16 parts multiplied in turn, 2^-22
//   BF16 cache                    two bf16 parts, 2^-16
// fp16 parts also have an absolute step: a weight is off by up to 2^-25 however
// small it is.  So weights use fp16's range: the row's largest lies between
// 2^10 and 2^15, and that error is at most 2^-35 of it (with m the maximum
// itself, all tokens below 2^-25 of a dominant one would be lost, however many).  A
// lift of 12 would raise m for every rise by 2^3, not 2^5: 16 x 8,192 tokens of E4M3, 64 /
// 4 heads of 64, 20.4 us against 19.9 (19.7 with 2^8 and none).  bf16 parts have no
// such step and need no lift.
template <int FMT, int D, int NT, typename YT>
struct Warp {
    using C = Cfg<FMT, D, NT>;
    static constexpr bool kBf16 = FMT == NVFP4_KV_BF16;
    static constexpr bool kSplit = kBf16 || std::is_same<YT, float>::value;
    static constexpr float kLift = kBf16 ? 0.0f : 10.0f, kTop = kBf16 ? 8.0f : 15.0f;
    static constexpr int kUk = C::kDb / 4 < 16 ? C::kDb / 4 : 16;  // bytes of a key row a thread takes at a time
    static constexpr int kNk = C::kDb / (4 * kUk);
    static constexpr int kUv = C::kDb / 8 < 16 ? C::kDb / 8 : 16;  // bytes of a value row
    static constexpr int kNv = C::kDb / (8 * kUv);
    static constexpr int kPerByteX2 = FMT == NVFP4_KV_BF16 ? 1 : FMT == NVFP4_KV_E4M3 ? 2 : 4;  // elements per 2 bytes
    static constexpr int kEk = kUk * kPerByteX2 / 2, kEv = kUv * kPerByteX2 / 2;                // elements per unit
    static constexpr int kQw = D / 8;  // query words of a thread per column block

    uint32_t q[NT][kQw];
    float o[NT][C::kMt][4];
    float m[NT][2], l[NT][2], f[NT][2];  // columns 2t, 2t + 1: maximum, sum (this thread's tokens), factor of the scores

    // Queries of segment (b, hk, chunk): column n = lane / 4 of each block.
    NVFP4_DEV void fetch_q(const Args& a, int b, int hk, int chunk) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int col = (chunk * NT + n) * 8 + g;
            const bool live = col < a.G;
            const __nv_bfloat16* qp = a.q + (int64_t)b * a.q_ld + (int64_t)(hk * a.G + col) * D;
#pragma unroll
            for (int i = 0; i < kNk; ++i)
#pragma unroll
                for (int e = 0; e < kEk / 8; ++e) {
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (live) w = *reinterpret_cast<const uint4*>(qp + kEk * (t + 4 * i) + 8 * e);
                    const int at = i * (kEk / 2) + 4 * e;
                    q[n][at] = w.x, q[n][at + 1] = w.y, q[n][at + 2] = w.z, q[n][at + 3] = w.w;
                }
        }
    }

    // Turns fetched queries into operands and starts a piece.  Quantized caches
    // multiply in fp16: a column is prescaled by a power of two that brings its
    // largest element to [2^14, 2^15), exact for every element within 2^31 of
    // it; the factor of the scores undoes it.
    NVFP4_DEV void start(const Args& a, float gs) {
        const int t = threadIdx.x & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float back = 1.0f;
            if constexpr (!kBf16) {
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < kQw; ++i)
                    amax = fmaxf(amax, fmaxf(fabsf(bf16lo_to_f32(q[n][i])), fabsf(bf16hi_to_f32(q[n][i]))));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                int p = amax > 0.0f ? 14 - ((int)(__float_as_uint(amax) >> 23) - 127) : 0;
                p = min(max(p, -112), 112);
                const float up = __uint_as_float((uint32_t)(127 + p) << 23);
                back = __uint_as_float((uint32_t)(127 - p) << 23);
#pragma unroll
                for (int i = 0; i < kQw; ++i)
                    q[n][i] = pack_f16(bf16lo_to_f32(q[n][i]) * up, bf16hi_to_f32(q[n][i]) * up);
            }
            // the factors of this thread's two score columns
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float bk = __shfl_sync(0xffffffffu, back, (2 * t + c) * 4);
                f[n][c] = a.scale_log2 * gs * bk;
                m[n][c] = __int_as_float(0xff800000);
                l[n][c] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < C::kMt; ++k)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[n][k][c] = 0.0f;
        }
    }

    // Block scale bytes of a key row's unit -> fp16 pairs (s, s), one per block.
    static NVFP4_DEV void key_scale(uint32_t p, uint32_t (&sc)[2]) {
        uint32_t h;
        if constexpr (kUk == 16) h = e4m3x2_to_f16x2((uint16_t)lds_u16(p));
        else h = e4m3x2_to_f16x2((uint16_t)lds_u8(p));
        sc[0] = prmt(h, h, 0x1010);
        sc[1] = prmt(h, h, 0x3232);
    }

    // Would a score x weigh more than 2^kTop?  fp16 cannot hold 2^16, so the difference is
    // rounded as the weight's exponent is: scores from 2^26 on lie 8 and more apart.
    static NVFP4_DEV bool passes(float x, float m) { return kBf16 ? x > m + kTop : x - m > kTop; }
    // m for a maximum mx; mx itself where the difference rounds to more than kTop.
    static NVFP4_DEV float lifted(float mx) {
        const float m = mx - kLift;
        return mx - m > kTop ? mx : m;
    }

    // kStep tiles with tokens tok0 .. tok0 + 16 kStep - 1 at tp[0], tp[1]; tokens
    // outside [lo, hi) are masked (their bytes may be anything, NaN included).
    static constexpr int kStep = C::kStep;
    NVFP4_DEV void tiles(const uint32_t (&tp)[kStep], int tok0, int lo, int hi) {
        const bool edge = tok0 < lo || tok0 + kStep * kKvTile > hi;
        const int lane = threadIdx.x & 31, g = lane >> 2;
        float s[kStep][NT][4];
#pragma unroll
        for (int u = 0; u < kStep; ++u) scores(tp[u], s[u]);
        // ---- softmax: tokens tok0 + 16 u + g (c 0, 1) and + 8 (c 2, 3), columns 2t, 2t + 1
        uint32_t ph[kStep][NT][2], pl[kStep][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x[kStep][4];
#pragma unroll
            for (int u = 0; u < kStep; ++u)
#pragma unroll
                for (int c = 0; c < 4; ++c) x[u][c] = s[u][n][c] * f[n][c & 1];
            if (edge) {
#pragma unroll
                for (int u = 0; u < kStep; ++u)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int tok = tok0 + u * kKvTile + g + 8 * (c >> 1);
                        if (tok < lo || tok >= hi) x[u][c] = __int_as_float(0xff800000);
                    }
            }
            // m is raised only when a weight would pass 2^kTop: most tiles need no
            // exchange
            float up[2] = {fmaxf(x[0][0], x[0][2]), fmaxf(x[0][1], x[0][3])};
            if constexpr (kStep == 2) {
                up[0] = fmaxf(up[0], fmaxf(x[1][0], x[1][2]));
                up[1] = fmaxf(up[1], fmaxf(x[1][1], x[1][3]));
            }
            if (__any_sync(0xffffffffu, passes(up[0], m[n][0]) || passes(up[1], m[n][1]))) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = up[c];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                    mx = fmaxf(lifted(mx), m[n][c]);
                    const float al = weight(m[n][c], mx);
                    m[n][c] = mx;
                    l[n][c] *= al;
#pragma unroll
                    for (int k = 0; k < C::kMt; ++k) {
                        o[n][k][c] *= al;
                        o[n][k][2 + c] *= al;
                    }
                }
            }
            const float m0 = m[n][0] == __int_as_float(0xff800000) ? 0.0f : m[n][0];
            const float m1 = m[n][1] == __int_as_float(0xff800000) ? 0.0f : m[n][1];
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                const float p[4] = {ex2(x[u][0] - m0), ex2(x[u][1] - m1), ex2(x[u][2] - m0), ex2(x[u][3] - m1)};
                l[n][0] += p[0] + p[2];
                l[n][1] += p[1] + p[3];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float a = p[2 * h], b = p[2 * h + 1];
                    const uint32_t hi_part = kBf16 ? pack_b16(a, b) : pack_f16(a, b);
                    ph[u][n][h] = movmatrix_trans(hi_part);
                    if constexpr (kSplit) {
                        float ra, rb;
                        if constexpr (kBf16) {
                            ra = a - bf16lo_to_f32(hi_part);
                            rb = b - bf16hi_to_f32(hi_part);
                        } else {
                            const float2 r = f16x2_to_f32x2(hi_part);
                            ra = a - r.x;
                            rb = b - r.y;
                        }
                        pl[u][n][h] = movmatrix_trans(kBf16 ? pack_b16(ra, rb) : pack_f16(ra, rb));
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kStep; ++u) values(tp[u], edge, tok0 + u * kKvTile, lo, hi, ph[u], pl[u]);
    }

    // S^T = K Q^T of a tile (before the factor): this thread's rows g and g + 8.
    NVFP4_DEV void scores(uint32_t tp, float (&sum)[NT][4]) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const uint32_t ks = tp + 32 * C::kDb;  // key scales, then value scales
        float s[NT][2][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[n][p][c] = 0.0f;
        const int turn = kv_turn(g, C::kPieces);
#pragma unroll
        for (int i = 0; i < kNk; ++i) {
            const int off = kUk * (t + 4 * i);
            const int at = (((off >> 4) ^ turn) << 4) | (off & 15);
            uint32_t w0[kUk / 4], w1[kUk / 4];
            lds<kUk>(tp + g * C::kDb + at, w0);
            lds<kUk>(tp + (g + 8) * C::kDb + at, w1);
            if constexpr (FMT == NVFP4_KV_NVFP4) {
                const uint32_t sp = ks + g * C::kSb + (off >> 3);
                uint32_t sc0[2], sc1[2];
                key_scale(sp, sc0);
                key_scale(sp + 8 * C::kSb, sc1);
#pragma unroll
                for (int w = 0; w < kUk / 4; ++w) {
                    uint32_t a0[4], a1[4];
                    e2m1x8_to_f16x2(w0[w], a0);
                    e2m1x8_to_f16x2(w1[w], a1);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // E2M1 x E4M3: exact in fp16
                        a0[e] = mul_f16x2(a0[e], sc0[w >> 1]);
                        a1[e] = mul_f16x2(a1[e], sc1[w >> 1]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const int at_q = i * (kEk / 2) + 4 * w + 2 * h;
                            mma16816<false>(s[n][h], a0[2 * h], a1[2 * h], a0[2 * h + 1], a1[2 * h + 1], q[n][at_q],
                                            q[n][at_q + 1]);
                        }
                }
            } else if constexpr (FMT == NVFP4_KV_E4M3) {
#pragma unroll
                for (int w = 0; w < kUk / 4; ++w) {
                    const uint32_t a0 = e4m3x2_to_f16x2((uint16_t)w0[w]), a2 = e4m3x2_to_f16x2((uint16_t)(w0[w] >> 16));
                    const uint32_t a1 = e4m3x2_to_f16x2((uint16_t)w1[w]), a3 = e4m3x2_to_f16x2((uint16_t)(w1[w] >> 16));
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int at_q = i * (kEk / 2) + 2 * w;
                        mma16816<false>(s[n][w & 1], a0, a1, a2, a3, q[n][at_q], q[n][at_q + 1]);
                    }
                }
            } else {
#pragma unroll
                for (int w = 0; w < kUk / 8; ++w)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int at_q = i * (kEk / 2) + 2 * w;
                        mma16816<true>(s[n][w & 1], w0[2 * w], w1[2 * w], w0[2 * w + 1], w1[2 * w + 1], q[n][at_q],
                                       q[n][at_q + 1]);
                    }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[n][c] = s[n][0][c] + s[n][1][c];
    }

    // O^T += V^T P^T of a tile.
    NVFP4_DEV void values(uint32_t tp, bool edge, int tok0, int lo, int len, const uint32_t (&ph)[NT][2],
                          const uint32_t (&pl)[NT][2]) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const uint32_t ks = tp + 32 * C::kDb;
        // ---- O^T += V^T P^T: this thread's columns of tokens 2t, 2t + 1, 2t + 8, 2t + 9
        const uint32_t vp = tp + 16 * C::kDb, vs = ks + 16 * C::kSb;
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            const int off = kUv * (g + 8 * i);
            uint32_t w[4][kUv / 4];
            uint32_t sb[4];  // NVFP4: block scale byte(s) of each token
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = 2 * t + (k & 1) + 8 * (k >> 1);
                lds<kUv>(vp + r * C::kDb + kv_place(r, off, C::kPieces), w[k]);
                if constexpr (FMT == NVFP4_KV_NVFP4) {
                    const uint32_t sp = vs + r * C::kSb + (off >> 3);
                    if constexpr (kUv == 16) sb[k] = lds_u16(sp);
                    else sb[k] = lds_u8(sp);
                }
            }
            if (edge) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int tok = tok0 + 2 * t + (k & 1) + 8 * (k >> 1);
                    if (tok < lo || tok >= len) {
#pragma unroll
                        for (int e = 0; e < kUv / 4; ++e) w[k][e] = 0u;
                        sb[k] = 0u;
                    }
                }
            }
            // a word's codes of two tokens -> fp16 / bf16 pairs (token, next token)
            // of one column each: v[2 x + p][y], column 2 y + p, tokens of pair x
            constexpr int kPairs = FMT == NVFP4_KV_NVFP4 ? 4 : FMT == NVFP4_KV_E4M3 ? 2 : 1;  // columns / 2 per word
#pragma unroll
            for (int e = 0; e < kUv / 4; ++e) {
                uint32_t v[4][kPairs];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t p = w[2 * x][e], r = w[2 * x + 1][e];
                    if constexpr (FMT == NVFP4_KV_NVFP4) {
                        e2m1x8_to_f16x2((p & 0x0F0F0F0Fu) | ((r << 4) & 0xF0F0F0F0u), v[2 * x]);
                        e2m1x8_to_f16x2(((p >> 4) & 0x0F0F0F0Fu) | (r & 0xF0F0F0F0u), v[2 * x + 1]);
                        const uint32_t sc =
                            e4m3x2_to_f16x2((uint16_t)prmt(sb[2 * x], sb[2 * x + 1], (e >> 1) ? 0x0051 : 0x0040));
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            v[2 * x][y] = mul_f16x2(v[2 * x][y], sc);
                            v[2 * x + 1][y] = mul_f16x2(v[2 * x + 1][y], sc);
                        }
                    } else if constexpr (FMT == NVFP4_KV_E4M3) {
                        const uint32_t a = prmt(p, r, 0x5140), b = prmt(p, r, 0x7362);
                        v[2 * x][0] = e4m3x2_to_f16x2((uint16_t)a);
                        v[2 * x + 1][0] = e4m3x2_to_f16x2((uint16_t)(a >> 16));
                        v[2 * x][1] = e4m3x2_to_f16x2((uint16_t)b);
                        v[2 * x + 1][1] = e4m3x2_to_f16x2((uint16_t)(b >> 16));
                    } else {
                        v[2 * x][0] = prmt(p, r, 0x5410);
                        v[2 * x + 1][0] = prmt(p, r, 0x7632);
                    }
                }
#pragma unroll
                for (int y = 0; y < kPairs; ++y) {
                    const int mt = (i * (kUv / 4) + e) * kPairs + y;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16816<kBf16>(o[n][mt], v[0][y], v[1][y], v[2][y], v[3][y], ph[n][0], ph[n][1]);
                        if constexpr (kSplit)
                            mma16816<kBf16>(o[n][mt], v[0][y], v[1][y], v[2][y], v[3][y], pl[n][0], pl[n][1]);
                    }
                }
            }
        }
    }

    NVFP4_DEV void scale_values(float v_gs) {
        if constexpr (FMT != NVFP4_KV_BF16) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < C::kMt; ++k)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[n][k][c] *= v_gs;
        }
    }

    // A value that depends on everything the last tiles read from shared memory:
    // one accumulator of each value unit (the scores, hence all keys, feed them
    // all; a step's tiles add to the accumulators in turn).
    NVFP4_DEV uint32_t depend() const {
        uint32_t d = 0;
#pragma unroll
        for (int i = 0; i < kNv; ++i) d ^= __float_as_uint(o[0][i * (C::kMt / kNv)][0]);
        return d;
    }

    // First column (element of the head) of this thread's O^T rows of mt: rows
    // g and g + 8 of the tile are the head's elements d and d + 1.
    static NVFP4_DEV int column(int mt) {
        constexpr int per_unit = kEv / 2;
        const int g = (threadIdx.x & 31) >> 2;
        return kEv * (g + 8 * (mt / per_unit)) + 2 * (mt % per_unit);
    }

    NVFP4_DEV void finish_sums() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], d);
    }

    // This warp's piece to `dst`.
    NVFP4_DEV void store_piece(float* dst) {
        finish_sums();
        write_piece(dst);
    }
    NVFP4_DEV void write_piece(float* dst) const {
        const int lane = threadIdx.x & 31, t = lane & 3;
        using P = Piece<D, NT>;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = n * 8 + 2 * t + c;
#pragma unroll
                for (int mt = 0; mt < C::kMt; ++mt)
                    *reinterpret_cast<float2*>(dst + col * P::kLd + column(mt)) =
                        make_float2(o[n][mt][c], o[n][mt][2 + c]);
                if (lane < 4) {
                    dst[P::kMax + col] = m[n][c];
                    dst[P::kSum + col] = l[n][c];
                }
            }
    }

    // A whole segment, straight to the output.
    NVFP4_DEV void store_output(const Args& a, int b, int hk, int chunk) {
        finish_sums();
        write_output(a, b, hk, chunk);
    }
    NVFP4_DEV void write_output(const Args& a, int b, int hk, int chunk) const {
        const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = (chunk * NT + n) * 8 + 2 * t + c;
                if (col >= a.G) continue;
                const int64_t row = (int64_t)b * a.q_heads + hk * a.G + col;
                const float inv = inverse_sum(l[n][c]);
                YT* yp = (YT*)a.y + row * D;
#pragma unroll
                for (int mt = 0; mt < C::kMt; mt += 4) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[2 * e] = o[n][mt + e][c] * inv;
                        v[2 * e + 1] = o[n][mt + e][2 + c] * inv;
                    }
                    store_y8(yp + column(mt), v);
                }
                if (a.lse && lane < 4) a.lse[row] = lse_of(m[n][c], l[n][c]);
            }
    }
};

// Waits for the next `count` (<= kStep) tiles of a warp's ring.  Of a step of
// two with one tile left the second pointer names bytes that are masked.
template <int S>
struct Step {
    bool ok;
    uint32_t slot, second, phase;  // the slot after the step's, the step's second, the phase after it
};
template <int kStep, int S>
NVFP4_DEV Step<S> wait_tiles(const uint8_t* ring, int tile, uint64_t* full, uint32_t slot, uint32_t phase,
                             uint32_t count, int* status, uint32_t (&tp)[kStep]) {
    Step<S> r;
    bool ok = mbar_wait(&full[slot], phase, status);
    tp[0] = smem_u32(ring) + slot * tile;
    uint32_t next = slot + 1, ph = phase;
    if (next == (uint32_t)S) next = 0, ph ^= 1;
    r.second = next;
    if constexpr (kStep == 2) {
        tp[1] = smem_u32(ring) + next * tile;
        if (count == 2) {
            ok = mbar_wait(&full[next], ph, status) && ok;
            if (++next == (uint32_t)S) next = 0, ph ^= 1;
        }
    }
    r.slot = next;
    r.phase = ph;
    r.ok = __all_sync(0xffffffffu, ok);
    return r;
}
// After a copy that never arrived: waits (again bounded) for every copy that may
// still be in flight.
template <int S>
NVFP4_DEV void drain(uint64_t* full, uint32_t i, uint32_t n_warp, int* status) {
    for (uint32_t k = i; k < i + S && k < n_warp; ++k) mbar_wait(&full[k % S], (k / S) & 1, status);
}

// One column of several pieces joined by a warp; a lane holds D / 32
// consecutive elements of the head.
template <int D>
struct Joined {
    static constexpr int kV = D / 32;
    float v[kV], M, L;

    // Pieces p with bit p of `set` (p < P; kAll: every p), at piece(p) in shared memory.
    template <int NT, int P, bool kAll, typename F>
    NVFP4_DEV void join(F piece, uint32_t set, int col) {
        using Pc = Piece<D, NT>;
        const int lane = threadIdx.x & 31;
        const bool in = lane < P && (set >> lane & 1);
        const float* mine = piece(in ? lane : __ffs(set) - 1) + Pc::kMax + col;
        const float m = in ? mine[0] : __int_as_float(0xff800000);
        M = warp_max(m);
        const float w = in ? weight(m, M) : 0.0f;
        L = warp_sum(in ? w * mine[Pc::kCols] : 0.0f);
#pragma unroll
        for (int k = 0; k < kV; ++k) v[k] = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (!kAll && !(set >> p & 1)) continue;
            const float* src = piece(p) + col * Pc::kLd + lane * kV;
            const float wp = __shfl_sync(0xffffffffu, w, p);
#pragma unroll
            for (int k = 0; k < kV; k += 2) {
                const float2 x = *reinterpret_cast<const float2*>(src + k);
                v[k] += wp * x.x;
                v[k + 1] += wp * x.y;
            }
        }
    }

    // The pieces of a cluster's CTAs, each at the same place in its shared memory.
    template <int NT>
    NVFP4_DEV void join_cluster(const float* mine, int cluster, int col) {
        using Pc = Piece<D, NT>;
        const int lane = threadIdx.x & 31;
        float m = __int_as_float(0xff800000), l = 0.0f;
        if (lane < cluster) {
            m = ld_dsmem_f32(mine + Pc::kMax + col, (uint32_t)lane);
            l = ld_dsmem_f32(mine + Pc::kSum + col, (uint32_t)lane);
        }
        float2 x[8][kV / 2];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < cluster) {
#pragma unroll
                for (int k = 0; k < kV / 2; ++k)
                    x[c][k] = ld_dsmem_f32x2(mine + col * Pc::kLd + lane * kV + 2 * k, (uint32_t)c);
            }
        M = warp_max(m);
        const float w = weight(m, M);
        L = warp_sum(w * l);
#pragma unroll
        for (int k = 0; k < kV; ++k) v[k] = 0.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < cluster) {
                const float wc = __shfl_sync(0xffffffffu, w, c);
#pragma unroll
                for (int k = 0; k < kV / 2; ++k) {
                    v[2 * k] += wc * x[c][k].x;
                    v[2 * k + 1] += wc * x[c][k].y;
                }
            }
    }

    template <typename YT>
    NVFP4_DEV void store_output(const Args& a, uint32_t b, uint32_t hk, int qc) const {
        if (qc >= a.G) return;
        const int lane = threadIdx.x & 31;
        const int64_t row = (int64_t)b * a.q_heads + hk * a.G + qc;
        const float inv = inverse_sum(L);
        YT* yp = (YT*)a.y + row * D + lane * kV;
#pragma unroll
        for (int k = 0; k < kV; k += 2) store_y2(yp + k, v[k] * inv, v[k + 1] * inv);
        if (a.lse && lane == 0) a.lse[row] = lse_of(M, L);
    }

    template <int NT>
    NVFP4_DEV void store_piece(float* part, int col) const {
        using Pc = Piece<D, NT>;
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int k = 0; k < kV; k += 2)
            *reinterpret_cast<float2*>(part + col * Pc::kLd + lane * kV + k) = make_float2(v[k], v[k + 1]);
        if (lane == 0) {
            part[Pc::kMax + col] = M;
            part[Pc::kSum + col] = L;
        }
    }
};

template <int FMT, int D, int NT, typename YT>
__global__ void __launch_bounds__(Cfg<FMT, D, NT>::kWarps * 32, Cfg<FMT, D, NT>::kTile >= 16384 ? 1 : kCtasPerSm)
    attn_decode_kernel(const Args a) {
    using C = Cfg<FMT, D, NT>;
    constexpr int W = C::kWarps, S = C::kRing, kCols = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* ring_all = smem;
    float* pieces = reinterpret_cast<float*>(smem + C::kRingBytes);
    uint32_t* first = reinterpret_cast<uint32_t*>(smem + C::kFixed);  // [B + 1] (List), then rank
    uint32_t* rank_of = first + a.B + 1;
    __shared__ uint64_t s_full[W][S];
    __shared__ uint32_t s_seg[2 * W];
    __shared__ uint2 s_scan[W];
    __shared__ uint4 s_desc[2 * W];  // of a stored piece: tiles, sequence, key head, chunk
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    griddep_launch_dependents();
    if (lane == 0) {
        for (int i = 0; i < S; ++i) mbar_init(&s_full[warp][i], 1);
        fence_barrier_init();
    }
    if (lane < 2) s_seg[2 * warp + lane] = 0xffffffffu;
    griddep_wait();

    // ---- the list: first tile of each sequence (in tiles of one segment)
    const uint32_t B = (uint32_t)a.B;
    uint32_t tiles_so_far = 0, seqs_so_far = 0;
    for (uint32_t b0 = 0; b0 < B; b0 += W * 32) {
        const uint32_t b = b0 + threadIdx.x;
        uint32_t n = 0;
        if (b < B) {
            int lo, len;
            seen_range(a, (int)b, lo, len);
            if (a.lens[b] > len && a.lens[b] > 0 && a.status) atomicExch(a.status, NVFP4_ERR_PAGE);
            n = len > lo ? (uint32_t)((len + kKvTile - 1) / kKvTile - lo / kKvTile) : 0u;
        }
        uint32_t x = n;
        const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) s_scan[warp] = make_uint2(x, (uint32_t)__popc(some));
        __syncthreads();
        uint32_t before = tiles_so_far, rank = seqs_so_far + __popc(some & ((1u << lane) - 1));
        for (int w = 0; w < W; ++w) {
            const uint2 v = s_scan[w];
            if (w < warp) before += v.x, rank += v.y;
            tiles_so_far += v.x;
            seqs_so_far += v.y;
        }
        if (b < B) {
            first[b] = before + x - n;
            rank_of[b] = rank;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        first[B] = tiles_so_far;
        rank_of[B] = seqs_so_far;
    }
    __syncthreads();

    const uint32_t hc = (uint32_t)(a.c.heads * a.chunks);
    const List list{first, rank_of, B, hc};
    const uint32_t cost = list.cost_at(B);
    uint32_t per_cta = (cost + gridDim.x - 1) / gridDim.x;
    if (per_cta < (uint32_t)W) per_cta = W;
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) a.header[0] = per_cta;
        for (uint32_t b = threadIdx.x; b < 2 * (B + 1); b += W * 32) a.header[1 + b] = first[b];
    }
    // this CTA's and this warp's ranges of cost, then of tiles
    const uint32_t u0 = min(cost, per_cta * blockIdx.x), u1 = min(cost, u0 + per_cta), n_cta = u1 - u0;
    const uint32_t t0 = list.tiles_before(u0), t1 = list.tiles_before(u1);
    const uint32_t wu0 = u0 + (n_cta / W) * warp + min(n_cta % W, (uint32_t)warp);
    const uint32_t wu1 = wu0 + n_cta / W + ((uint32_t)warp < n_cta % W ? 1u : 0u);
    const uint32_t w0 = list.tiles_before(wu0), n_warp = list.tiles_before(wu1) - w0;

    // ---- this warp's tiles
    uint8_t* ring = ring_all + (size_t)warp * S * C::kTile;
    uint64_t* full = s_full[warp];
    float* my_first = pieces + warp * Piece<D, NT>::kFloats;
    float* my_last = reinterpret_cast<float*>(ring);
    if (n_warp > 0) {
        // addresses of tiles i0 .. i0 + 31 of this warp, one per lane; `pl` is
        // the place of a tile at or before them in the same segment
        const uint8_t* addr = nullptr;
        auto look_up = [&](uint32_t i0, const Place& pl, uint32_t pl_i) {
            const uint32_t i = i0 + lane;
            if (i < n_warp) {
                Place p = pl;
                p.j += i - pl_i;
                if (p.j >= p.tiles) p = list.place_of(w0 + i);
                int lo, len;
                seen_range(a, (int)p.b, lo, len);
                const uint32_t jt = (uint32_t)(lo / kKvTile) + p.j;
                addr = tile_in_page<C::kTile>(a, table_entry(a, p.b, jt), p.s / (uint32_t)a.chunks, jt);
            }
        };
        // `dep` is made of registers that hold the results of everything read
        // from the slot; adding dep & 0 to the byte count makes the copy wait
        // for those reads to have returned (a.zero is 0 at run time).
        auto refill = [&](uint32_t i, uint32_t slot, uint32_t dep) {
            if (i < n_warp && lane == (int)(i & 31)) {
                const uint32_t bytes = (uint32_t)C::kTile + (dep & a.zero);
                mbar_expect_tx(&full[slot], bytes);
                bulk_load(ring + slot * C::kTile, addr, bytes, &full[slot]);
            }
        };
        Place at = list.place_of(w0);
        uint32_t hk = at.s / (uint32_t)a.chunks, chunk = at.s - hk * (uint32_t)a.chunks;
        Warp<FMT, D, NT, YT> wk;
        wk.fetch_q(a, (int)at.b, (int)hk, (int)chunk);  // on their way while the page table is read
        look_up(0, at, 0);
        for (uint32_t i = 0; i < (uint32_t)S; ++i) refill(i, i, 0u);
        float k_gs = 1.0f;
        float v_gs = 1.0f;
        if constexpr (FMT != NVFP4_KV_BF16) {
            k_gs = *a.c.k_gs;
            v_gs = *a.c.v_gs;
        }
        int lo, len;
        seen_range(a, (int)at.b, lo, len);
        int tok0 = (lo / kKvTile + (int)at.j) * kKvTile;
        uint32_t begun = at.j;  // tile of the segment this piece starts with
        uint32_t slot = 0, phase = 0;
        wk.start(a, k_gs);
        for (uint32_t i = 0; i < n_warp;) {
            // this step's tiles: up to kStep, of one segment
            const uint32_t count = min((uint32_t)C::kStep, min(n_warp - i, at.tiles - at.j));
            uint32_t tp[C::kStep];
            const Step<S> step = wait_tiles<C::kStep, S>(ring, C::kTile, full, slot, phase, count, a.status, tp);
            if (!step.ok) {
                drain<S>(full, i, n_warp, a.status);
                break;
            }
            wk.tiles(tp, tok0, lo, min(len, tok0 + (int)count * kKvTile));
            const uint32_t dep = wk.depend();
#pragma unroll
            for (uint32_t u = 0; u < (uint32_t)C::kStep; ++u) {
                if (u < count) {
                    const uint32_t next = i + u + S;
                    if ((next & 31) == 0) look_up(next, at, i);
                    refill(next, u ? step.second : slot, dep);
                }
            }
            slot = step.slot, phase = step.phase;
            tok0 += (int)count * kKvTile;
            i += count;
            at.j += count;
            // ---- end of the segment or of the range
            const bool ends = at.j == at.tiles;
            if (ends || i == n_warp) {
                wk.scale_values(v_gs);
                if (ends && begun == 0) {
                    wk.store_output(a, (int)at.b, (int)hk, (int)chunk);
                } else {
                    const uint32_t id = first[at.b] * hc + at.s * at.tiles;  // the segment's first tile names it
                    wk.store_piece(ends ? my_first : my_last);
                    if (lane == 0) {
                        s_seg[2 * warp + (ends ? 0 : 1)] = id;
                        s_desc[2 * warp + (ends ? 0 : 1)] = make_uint4(at.tiles, at.b, hk, chunk);
                    }
                }
            }
            if (ends && i < n_warp) {  // the next segment
                at.j = begun = 0;
                if (++at.s == hc) {
                    at.s = 0;
                    do ++at.b;
                    while (first[at.b + 1] == first[at.b]);
                    at.tiles = first[at.b + 1] - first[at.b];
                }
                hk = at.s / (uint32_t)a.chunks;
                chunk = at.s - hk * (uint32_t)a.chunks;
                wk.fetch_q(a, (int)at.b, (int)hk, (int)chunk);
                seen_range(a, (int)at.b, lo, len);
                tok0 = lo / kKvTile * kKvTile;
                wk.start(a, k_gs);
            }
        }
    }
    __syncthreads();

    // ---- segments that several warps share: a warp per (segment, column)
    const uint32_t my_seg = lane < 2 * W ? s_seg[lane] : 0xffffffffu;
    const uint32_t same = __match_any_sync(0xffffffffu, my_seg);
    const bool leads = my_seg != 0xffffffffu && (same & ((1u << lane) - 1)) == 0;
    const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
    const int rank = __popc(leaders & ((1u << lane) - 1));
    const int tasks = __popc(leaders) * kCols;
    auto piece = [&](int p) -> const float* {  // the warp's first (even) or, in its ring, its last (odd)
        return (p & 1) ? reinterpret_cast<const float*>(ring_all + (size_t)(p >> 1) * S * C::kTile)
                       : pieces + (p >> 1) * Piece<D, NT>::kFloats;
    };
    for (int task = warp; task < tasks; task += W) {
        const int col = task % kCols, lead = __ffs(__ballot_sync(0xffffffffu, leads && rank == task / kCols)) - 1;
        const uint32_t id = __shfl_sync(0xffffffffu, my_seg, lead), set = __shfl_sync(0xffffffffu, same, lead);
        const uint4 ds = s_desc[lead];
        Joined<D> r;
        if ((int)ds.w * kCols + col >= a.G) continue;  // a column of padding
        r.template join<NT, 2 * W, false>(piece, set, col);
        if (id >= t0 && id + ds.x <= t1) r.template store_output<YT>(a, ds.y, ds.z, ds.w * kCols + col);
        else r.template store_piece<NT>(a.partial + ((int64_t)blockIdx.x * 2 + (id >= t0 ? 1 : 0)) * Piece<D, NT>::kFloats, col);
    }
}

// The same for few tiles per warp (short contexts, few sequences), where the
// latencies of the list, of shared segments and of a second kernel weigh more
// than an even split: a cluster of CTAs takes one segment, each an equal
// contiguous range of its tiles, and joins it through distributed shared
// memory.  No workspace.
template <int FMT, int D, int NT, typename YT>
__global__ void __launch_bounds__(Cfg<FMT, D, NT>::kWarps * 32, Cfg<FMT, D, NT>::kTile >= 16384 ? 1 : kCtasPerSm)
    attn_segment_kernel(const Args a, const int cluster) {
    using C = Cfg<FMT, D, NT>;
    constexpr int W = C::kWarps, S = C::kRing, kCols = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    float* joined = reinterpret_cast<float*>(smem + C::kRingBytes);  // this CTA's piece
    __shared__ uint64_t s_full[W][S];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t seg = blockIdx.x / (uint32_t)cluster, rank = blockIdx.x - seg * (uint32_t)cluster;
    const uint32_t hc = (uint32_t)(a.c.heads * a.chunks);
    const uint32_t b = seg / hc, s = seg - b * hc, hk = s / (uint32_t)a.chunks, chunk = s - hk * (uint32_t)a.chunks;
    uint8_t* ring = smem + (size_t)warp * S * C::kTile;
    uint64_t* full = s_full[warp];

    griddep_launch_dependents();
    if (lane == 0) {
        for (int i = 0; i < S; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
    }
    __syncwarp();
    griddep_wait();
    Warp<FMT, D, NT, YT> wk;
    wk.fetch_q(a, (int)b, (int)hk, (int)chunk);
    float k_gs = 1.0f, v_gs = 1.0f;
    if constexpr (FMT != NVFP4_KV_BF16) {
        k_gs = *a.c.k_gs;
        v_gs = *a.c.v_gs;
    }
    int lo, len;
    seen_range(a, (int)b, lo, len);
    if (a.lens[b] > len && a.lens[b] > 0 && a.status) atomicExch(a.status, NVFP4_ERR_PAGE);
    const uint32_t j_first = (uint32_t)(lo / kKvTile);
    const uint32_t tiles = len > lo ? (uint32_t)((len + kKvTile - 1) / kKvTile) - j_first : 0u;
    // warp `rank * W + warp` of cluster * W takes an equal range
    const uint32_t parts = (uint32_t)(cluster * W), part = rank * W + warp;
    const uint32_t each = tiles / parts, more = tiles - each * parts;
    const uint32_t n_warp = each + (part < more ? 1u : 0u);
    const uint32_t j0 = j_first + each * part + min(part, more);

    const uint8_t* addr = nullptr;
    auto look_up = [&](uint32_t i0) {
        const uint32_t jt = j0 + i0 + lane;
        if (i0 + lane < n_warp) addr = tile_in_page<C::kTile>(a, table_entry(a, b, jt), hk, jt);
    };
    auto refill = [&](uint32_t i, uint32_t slot, uint32_t dep) {  // as in attn_decode_kernel
        if (i < n_warp && lane == (int)(i & 31)) {
            const uint32_t bytes = (uint32_t)C::kTile + (dep & a.zero);
            mbar_expect_tx(&full[slot], bytes);
            bulk_load(ring + slot * C::kTile, addr, bytes, &full[slot]);
        }
    };
    look_up(0);
    for (uint32_t i = 0; i < (uint32_t)S; ++i) refill(i, i, 0u);
    wk.start(a, k_gs);
    uint32_t slot = 0, phase = 0;
    int tok0 = (int)j0 * kKvTile;
    for (uint32_t i = 0; i < n_warp;) {
        const uint32_t count = min((uint32_t)C::kStep, n_warp - i);
        uint32_t tp[C::kStep];
        const Step<S> step = wait_tiles<C::kStep, S>(ring, C::kTile, full, slot, phase, count, a.status, tp);
        if (!step.ok) {
            drain<S>(full, i, n_warp, a.status);
            break;
        }
        wk.tiles(tp, tok0, lo, min(len, tok0 + (int)count * kKvTile));
        const uint32_t dep = wk.depend();
#pragma unroll
        for (uint32_t u = 0; u < (uint32_t)C::kStep; ++u) {
            if (u < count) {
                const uint32_t next = i + u + S;
                if ((next & 31) == 0) look_up(next);
                refill(next, u ? step.second : slot, dep);
            }
        }
        slot = step.slot, phase = step.phase;
        tok0 += (int)count * kKvTile;
        i += count;
    }
    wk.scale_values(v_gs);
    wk.store_piece(reinterpret_cast<float*>(ring));
    __syncthreads();

    auto piece = [&](int p) -> const float* {
        return reinterpret_cast<const float*>(smem + (size_t)p * S * C::kTile);
    };
    const uint32_t set = (1u << W) - 1;
    const int live = min(kCols, a.G - (int)chunk * kCols);  // columns that are not padding
    if (cluster == 1) {
        for (int col = warp; col < live; col += W) {
            Joined<D> r;
            r.template join<NT, W, true>(piece, set, col);
            r.template store_output<YT>(a, b, hk, (int)chunk * kCols + col);
        }
        return;
    }
    for (int col = warp; col < live; col += W) {
        Joined<D> r;
        r.template join<NT, W, true>(piece, set, col);
        r.template store_piece<NT>(joined, col);
    }
    cluster_sync();
    // the cluster's CTAs share the columns
    for (int col = (int)rank + cluster * warp; col < live; col += cluster * W) {
        Joined<D> r;
        r.template join_cluster<NT>(joined, cluster, col);
        r.template store_output<YT>(a, b, hk, (int)chunk * kCols + col);
    }
    cluster_sync();  // pieces stay until every CTA has read them
}

// Joins the segments that several CTAs share and writes zeros for sequences
// without tokens: one block of lanes per output row, pieces in list order.
// kRows rows per CTA: 8 (a warp each) or 1 (eight warps, each every eighth
// piece; for few rows of many pieces).
template <int D, int NT, typename YT, int kRows>
__global__ void __launch_bounds__(256) attn_join_kernel(const Args a) {
    constexpr int kCols = 8 * NT, kV = D / 32;  // floats per lane
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = kRows == 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kRows + warp;
    if (row >= (int64_t)a.B * a.q_heads) return;
    const int b = (int)(row / a.q_heads), hq = (int)(row - (int64_t)b * a.q_heads);
    const int hk = hq / a.G, gq = hq - hk * a.G, chunk = gq / kCols, col = gq - chunk * kCols;
    const uint32_t per = a.header[0], f0 = a.header[1 + b], f1 = a.header[2 + b], rank = a.header[2 + a.B + b];
    const uint32_t tiles = f1 - f0, hc = (uint32_t)(a.c.heads * a.chunks);
    YT* yp = (YT*)a.y + row * D;
    if (tiles == 0) {
        if (kRows == 1 && warp) return;
        for (int k = 0; k < kV; ++k) store_out<YT>(yp + lane + 32 * k, 0.0f);
        if (a.lse && lane == 0) a.lse[row] = __int_as_float(0xff800000);
        return;
    }
    const uint32_t ts = hc * (f0 + kSegmentCost * rank) + (uint32_t)(hk * a.chunks + chunk) * (tiles + kSegmentCost);
    const uint32_t c0 = ts / per, c1 = (ts + tiles - 1) / per;
    if (c0 == c1) return;
    const int step = kRows == 1 ? 8 : 1, off = kRows == 1 ? warp : 0;
    using Pc = Piece<D, NT>;
    auto part = [&](uint32_t c) { return a.partial + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * Pc::kFloats; };
    // one pass with a running maximum, so that a piece's maximum, sum and values are
    // on their way together
    float M = __int_as_float(0xff800000), L = 0.0f, v[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) v[k] = 0.0f;
    auto add = [&](float m, float l, const float(&x)[kV]) {
        const float top = fmaxf(M, m), wo = weight(M, top), wn = weight(m, top);
        L = L * wo + wn * l;
#pragma unroll
        for (int k = 0; k < kV; ++k) v[k] = v[k] * wo + wn * x[k];
        M = top;
    };
#pragma unroll 4
    for (uint32_t c = c0 + off; c <= c1; c += step) {
        const float* src = part(c);
        float x[kV];
#pragma unroll
        for (int k = 0; k < kV; ++k) x[k] = src[col * Pc::kLd + lane + 32 * k];
        add(src[Pc::kMax + col], src[Pc::kSum + col], x);
    }
    if constexpr (kRows == 1) {
        __shared__ float s_v[8][D + 2];
#pragma unroll
        for (int k = 0; k < kV; ++k) s_v[warp][lane + 32 * k] = v[k];
        if (lane == 0) {
            s_v[warp][D] = M;
            s_v[warp][D + 1] = L;
        }
        __syncthreads();
        if (warp) return;
        for (int w = 1; w < 8; ++w) {
            float x[kV];
#pragma unroll
            for (int k = 0; k < kV; ++k) x[k] = s_v[w][lane + 32 * k];
            add(s_v[w][D], s_v[w][D + 1], x);
        }
    }
    const float inv = inverse_sum(L);
#pragma unroll
    for (int k = 0; k < kV; ++k) store_out<YT>(yp + lane + 32 * k, v[k] * inv);
    if (a.lse && lane == 0) a.lse[row] = lse_of(M, L);
}

// Dynamic shared memory above 48 KB is allowed once per kernel and device.
template <typename K>
static bool allow_smem(K kern, std::atomic<uint64_t>& done, int bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (done.load(std::memory_order_relaxed) >> dev & 1) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(1ull << dev, std::memory_order_relaxed);
    return true;
}

// The join: a warp per row, or a CTA per row where rows may have many pieces.
template <int D, int NT, typename YT>
static int run_join(const Args& a, int64_t grid, cudaStream_t st) {
    cudaLaunchAttribute attr[1];
    set_pdl_attr(attr[0]);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int64_t rows = (int64_t)a.B * a.q_heads;
    cudaError_t e;
    if ((int64_t)a.B * a.c.heads * a.chunks * 8 > grid) {
        cfg.gridDim = dim3((unsigned)((rows + 7) / 8));
        e = cudaLaunchKernelEx(&cfg, attn_join_kernel<D, NT, YT, 8>, a);
    } else {
        cfg.gridDim = dim3((unsigned)rows);
        e = cudaLaunchKernelEx(&cfg, attn_join_kernel<D, NT, YT, 1>, a);
    }
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

template <int FMT, int D, int NT, typename YT>
static int run(const Args& a, const Shape& sh, cudaStream_t st) {
    using C = Cfg<FMT, D, NT>;
    cudaLaunchAttribute attr[2];
    set_pdl_attr(attr[0]);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(C::kWarps * 32);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // One cluster per segment: as many CTAs as leave every segment its own
    // (8 at most, the portable size), no more than give a warp one tile.
    const int64_t segments = (int64_t)a.B * a.c.heads * a.chunks;
    const int64_t slots = C::kTile >= 16384 ? kMaxGrid / kCtasPerSm : kMaxGrid;
    int64_t cluster = slots / segments, most = (sh.seg_tiles + C::kWarps - 1) / C::kWarps;
    cluster = cluster < 1 ? 1 : cluster > 8 ? 8 : cluster;
    if (cluster > most) cluster = most;
    if (sh.seg_tiles <= cluster * C::kWarps * kSegmentTiles) {
        static std::atomic<uint64_t> done{0};
        constexpr int bytes = C::kRingBytes + C::kPieceBytes;
        if (!allow_smem(attn_segment_kernel<FMT, D, NT, YT>, done, bytes)) return NVFP4_ERR_LAUNCH;
        cfg.gridDim = dim3((unsigned)(segments * cluster));
        cfg.dynamicSmemBytes = bytes;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, attn_segment_kernel<FMT, D, NT, YT>, a, (int)cluster) == cudaSuccess
                   ? NVFP4_OK
                   : NVFP4_ERR_LAUNCH;
    }
    static std::atomic<uint64_t> done{0};
    constexpr int kMostB = 4096;
    if (!allow_smem(attn_decode_kernel<FMT, D, NT, YT>, done, C::kFixed + (kMostB + 2) * 8)) return NVFP4_ERR_LAUNCH;
    cfg.gridDim = dim3((unsigned)sh.grid);
    cfg.dynamicSmemBytes = (size_t)C::kFixed + (size_t)(a.B + 2) * 8;
    if (cudaLaunchKernelEx(&cfg, attn_decode_kernel<FMT, D, NT, YT>, a) != cudaSuccess) return NVFP4_ERR_LAUNCH;
    return run_join<D, NT, YT>(a, sh.grid, st);
}

// Query columns per pass: 16 where the key head has more than 8 query heads
// and O^T fits the registers (D <= 128), else 8.
constexpr int cols_of(int G, int D) { return (G > 8 && D <= 128) ? 16 : 8; }

template <int FMT, typename YT>
static int run_fmt(const Args& a, const Shape& sh, cudaStream_t st) {
    const bool two = cols_of(a.G, a.c.head_dim) == 16;
    switch (a.c.head_dim) {
        case 64: return two ? run<FMT, 64, 2, YT>(a, sh, st) : run<FMT, 64, 1, YT>(a, sh, st);
        case 128: return two ? run<FMT, 128, 2, YT>(a, sh, st) : run<FMT, 128, 1, YT>(a, sh, st);
        case 256: return run<FMT, 256, 1, YT>(a, sh, st);
        default: return NVFP4_ERR_SHAPE;
    }
}

}  // namespace attn
}  // namespace nvfp4
