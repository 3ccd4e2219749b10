// Layout of the FP4 key/value cache (declared in include/fp4gemm.h, section
// "FP4 key/value cache") and the register forms of one tile of it.
//
// A tile holds 32 tokens of one page and one KV head, in the order in which a
// wave's matrix-core fragments take them, so that a tile is read with whole
// 1 KiB wave loads and no value crosses lanes.  With lane = 16 j + r:
//   * keys: lane (r, j) holds D / 4 consecutive elements of tokens r and
//     r + 16: row r of the 16x16x32 product's left operand (S^T = K Q^T), the
//     elements being a permutation of the contraction that the query
//     fragments follow;
//   * values: lane (r, j) holds D / 16 consecutive elements (of each 128) of
//     tokens 4 j .. 4 j + 3 and 16 + 4 j .. : row r of O^T = V^T P^T, the
//     tokens being exactly those whose scores lane (., j) holds after S^T, so
//     the probabilities go from one product into the next in registers.
// Every byte belongs to one token: a token is written without reading.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace fp4 {

constexpr int kKvTile = 32;  // tokens of a tile; a page is a whole number of tiles

template <int FMT, int D>
struct KvTile {
    static constexpr int G = FMT == 0 ? 16 : 32;      // elements that share a scale
    static constexpr int CH = D < 128 ? D : 128;      // elements of one chunk of a row
    static constexpr int C = D / CH;                  // chunks
    static constexpr int KD = CH / 4;                 // elements of a key chunk that one lane holds
    static constexpr int VD = CH / 16;                // elements of a value chunk that one lane holds
    static constexpr int KG = KD >= G ? KD / G : 1;   // scales of a lane's key chunk
    static constexpr int F = D / 64;                  // 1 KiB fragments of the codes (keys or values)
    static constexpr int kCodes = 16 * D;             // bytes of the codes
    static constexpr int kScales = 32 * D / G;        // bytes of the scales
    static constexpr int kKs = 2 * kCodes, kVs = 2 * kCodes + kScales;
    static constexpr int kBytes = 2 * (kCodes + kScales);
    static constexpr int kKsLane = 2 * C * KG;        // key scale bytes of one lane

    // Byte offsets inside a tile of token t's elements d, d + 1 (d even) and of
    // the scale of group g.
    __host__ __device__ static constexpr int k_code(int t, int d) {
        const int u = t >> 4, r = t & 15;
        if constexpr (D == 64) return (d / 16 * 16 + r) * 16 + u * 8 + d % 16 / 2;
        return (d / CH * 2 + u) * 1024 + (d % CH / KD * 16 + r) * 16 + d % KD / 2;
    }
    __host__ __device__ static constexpr int v_code(int t, int d) {
        const int u = t >> 4, j = (t & 15) >> 2, i = t & 3;
        if constexpr (D == 64) return kCodes + (16 * j + d / VD) * 16 + u * 8 + i * 2 + d % VD / 2;
        return kCodes + (d / CH * 2 + u) * 1024 + (16 * j + d % CH / VD) * 16 + i * 4 + d % VD / 2;
    }
    __host__ __device__ static constexpr int k_scale(int t, int g) {
        const int u = t >> 4, r = t & 15;
        constexpr int per_chunk = CH / G;             // groups of a chunk
        const int c = g / per_chunk, q = g % per_chunk;
        return kKs + (q / KG * 16 + r) * kKsLane + c * 2 * KG + u * KG + q % KG;
    }
    __host__ __device__ static constexpr int v_scale(int t, int g) {
        const int u = t >> 4, j = (t & 15) >> 2, i = t & 3;
        return kVs + (g * 4 + j) * 8 + u * 4 + i;
    }
};

// Bytes of a tile, for the host.
inline int64_t kv_tile_bytes(int format, int64_t D) {
    const int64_t G = format == 0 ? 16 : 32;
    return 32 * D + 64 * D / G;
}

// The cache as the kernels see it.
struct KvArgs {
    uint8_t* data;
    int64_t slots;       // pages * page_size
    int page_size, tiles_per_page, kv_heads, pages;
    float k_alpha, v_alpha;
};

}  // namespace fp4
