// Host side of the decode attention: workspace, grid and dispatch by format
// (the kernels are in attn_decode.cuh).
#include "attn_decode.cuh"

namespace nvfp4 {
namespace attn {

int run_bf16(const Args& a, const Shape& sh, int y_dtype, cudaStream_t st);
int run_e4m3(const Args& a, const Shape& sh, int y_dtype, cudaStream_t st);
int run_nvfp4(const Args& a, const Shape& sh, int y_dtype, cudaStream_t st);

struct Plan {
    int G, cols, chunks;
    Shape shape;
    size_t header, bytes;
};

// The grid: two CTAs per SM (one where a tile is 16 KB), fewer when even the longest
// sequences leave no tile for each warp.  The list takes 8 bytes of a CTA's shared
// memory per sequence, so beyond some 940 sequences (NVFP4, heads of 128) one CTA fits an
// SM and the grid runs in two waves: 1,024-token contexts, 16 / 8 heads, 900 sequences
// 238 us (4.5 TB/s), 1,024 sequences 360 us (3.4 TB/s).  False for shapes out of range.
static bool plan(const KvView& c, int64_t B, int q_heads, int64_t max_pages, Plan& p) {
    if (B < 1 || B > 4096 || q_heads < 1 || q_heads % c.heads || max_pages < 1 || max_pages > 0x7fffffff) return false;
    p.G = q_heads / c.heads;
    p.cols = cols_of(p.G, c.head_dim);
    p.chunks = (p.G + p.cols - 1) / p.cols;
    // tokens are int (a step may name 32 behind the last), list positions 32-bit:
    // tiles and the cost of segments
    if (max_pages > (int64_t)(0x7fffffff - 64) / c.page_size) return false;
    const int64_t seg = max_pages * (c.page_size / kKvTile) + kSegmentCost;
    if (seg > (int64_t)0x7fffffff / ((int64_t)c.heads * ((p.G + 7) / 8)) / B) return false;
    const int64_t tiles = B * max_pages * c.heads * p.chunks * (c.page_size / kKvTile);
    const int64_t most = kv_tile_bytes(c.format, c.head_dim) >= 16384 ? kMaxGrid / kCtasPerSm : kMaxGrid;
    p.shape.grid = (tiles + 3) / 4 < most ? (tiles + 3) / 4 : most;
    p.shape.seg_tiles = max_pages * (c.page_size / kKvTile);
    p.header = ((size_t)(2 * B + 4) * 4 + 255) / 256 * 256;
    p.bytes = p.header + (size_t)p.shape.grid * 2 * (p.cols * (c.head_dim + 4) + 3) / 4 * 4 * 4;
    return true;
}

}  // namespace attn

size_t attn_decode_workspace(const KvView& c, int64_t B, int q_heads, int64_t max_pages) {
    attn::Plan p;
    return attn::plan(c, B, q_heads, max_pages, p) ? p.bytes : 0;
}

int launch_attn_decode(const KvView& c, const AttnDecodeLaunch& L, cudaStream_t st) {
    attn::Plan p;
    if (!attn::plan(c, L.B, L.q_heads, L.max_pages, p)) return NVFP4_ERR_SHAPE;
    attn::Args a{};
    a.c = c;
    a.q = (const __nv_bfloat16*)L.q;
    a.q_ld = L.q_ld;
    a.B = (int)L.B;
    a.q_heads = L.q_heads;
    a.G = p.G;
    a.chunks = p.chunks;
    a.table = L.page_table;
    a.table_ld = L.table_ld;
    a.max_pages = (int)L.max_pages;
    a.lens = L.seq_lens;
    a.scale_log2 = L.scale * 1.44269504088896340736f;
    a.window = L.window;
    a.y = L.y;
    a.lse = L.lse;
    a.header = (uint32_t*)L.ws;
    a.partial = (float*)((char*)L.ws + p.header);
    a.status = L.status;
    a.zero = 0;
    // a window of w tokens lies in at most (w + 14) / 16 + 1 tiles
    attn::Shape shape = p.shape;
    if (L.window > 0 && ((int64_t)L.window + 14) / kKvTile + 1 < shape.seg_tiles)
        shape.seg_tiles = ((int64_t)L.window + 14) / kKvTile + 1;
    switch (c.format) {
        case NVFP4_KV_BF16: return attn::run_bf16(a, shape, L.y_dtype, st);
        case NVFP4_KV_E4M3: return attn::run_e4m3(a, shape, L.y_dtype, st);
        default: return attn::run_nvfp4(a, shape, L.y_dtype, st);
    }
}

}  // namespace nvfp4
