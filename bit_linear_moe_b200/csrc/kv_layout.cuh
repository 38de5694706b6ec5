// Layout of the paged key-value cache (include/nvfp4.h, nvfp4_kv_cache).
//
// The cache is [num_pages][heads][page_size / 16] tiles of 16 tokens.  A tile
// is one contiguous record, so that one bulk copy brings everything 16 tokens
// of one head need:
//     16 key rows, 16 value rows (kDb bytes each), then for NVFP4 the 16 + 16
//     rows of E4M3 block scales (D / 16 bytes each).
// Rows are token-major: a new token touches its own rows only.  The 16-byte
// pieces of row r are permuted, piece c at c ^ kv_turn(r, pieces), so that
// the attention kernel's fragment reads (8 rows x 4 threads for the keys,
// 4 rows two apart x 8 threads for the values) spread over the shared-memory
// banks without padding: r bit 0 moves a row by 64 bytes and bits 1..2 by 32
// and 64, which separates rows r, r + 1 and rows r, r + 2, r + 4, r + 6 of
// 128-byte and wider rows.
#pragma once

#include "common.cuh"

namespace nvfp4 {

constexpr int kKvTile = 16;  // tokens per tile

__host__ __device__ constexpr int kv_code_bytes(int fmt, int D) {
    return fmt == NVFP4_KV_BF16 ? 2 * D : fmt == NVFP4_KV_E4M3 ? D : D / 2;
}
__host__ __device__ constexpr int kv_scale_bytes(int fmt, int D) { return fmt == NVFP4_KV_NVFP4 ? D / 16 : 0; }
__host__ __device__ constexpr int kv_tile_bytes(int fmt, int D) {
    return 2 * kKvTile * (kv_code_bytes(fmt, D) + kv_scale_bytes(fmt, D));
}

// How far the 16-byte pieces of tile row r are turned (pieces: a power of two).
NVFP4_DEV int kv_turn(int r, int pieces) { return ((r & 6) ^ ((r & 1) << 2)) & (pieces - 1); }

// Byte offset, inside a row, of byte o of the row's codes.
NVFP4_DEV int kv_place(int r, int o, int pieces) { return (((o >> 4) ^ kv_turn(r, pieces)) << 4) | (o & 15); }

// The cache as the kernels take it (host-validated).
struct KvView {
    uint8_t* data;
    const float* k_gs;
    const float* v_gs;
    int64_t num_pages;
    int page_size;
    int heads;
    int head_dim;
    int format;
};

}  // namespace nvfp4
