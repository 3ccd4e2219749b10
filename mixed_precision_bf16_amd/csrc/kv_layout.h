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

// Tile that slot `slot` lies in, head h.
__device__ __forceinline__ uint8_t* kv_tile_of(const KvArgs& c, int64_t slot, int h, int tile_bytes, int& t) {
    int64_t page;
    int off;
    if (c.slots <= 0xFFFFFFFFll) {  // 32-bit division
        page = (uint32_t)slot / (uint32_t)c.page_size;
        off = (int)((uint32_t)slot - (uint32_t)page * (uint32_t)c.page_size);
    } else {
        page = slot / c.page_size;
        off = (int)(slot - page * c.page_size);
    }
    t = off % kKvTile;
    return c.data + ((page * c.kv_heads + h) * c.tiles_per_page + off / kKvTile) * (int64_t)tile_bytes;
}

// Quantizes one block of G elements x of a key or value row (quantize_block, the
// rule of fp4_quantize) and scatters its codes and scale into its tile.
template <int FMT, int D>
__device__ __forceinline__ void kv_store_block(const KvArgs& c, int64_t slot, int h, int g, bool is_v,
                                               const float (&x)[KvTile<FMT, D>::G]) {
    using L = KvTile<FMT, D>;
    constexpr int G = L::G;
    uint32_t out[G / 8];
    const uint32_t sb = quantize_block<FMT>(x, is_v ? c.v_alpha : c.k_alpha, out);
    int t;
    uint8_t* tile = kv_tile_of(c, slot, h, L::kBytes, t);
    if (!is_v) {
        if constexpr (FMT == 1 && D != 64) {
            *reinterpret_cast<u32x4*>(tile + L::k_code(t, g * G)) = u32x4{out[0], out[1], out[2], out[3]};
        } else {
#pragma unroll
            for (int w = 0; w < G / 16; ++w)
                *reinterpret_cast<u32x2*>(tile + L::k_code(t, g * G + 16 * w)) = u32x2{out[2 * w], out[2 * w + 1]};
        }
        tile[L::k_scale(t, g)] = (uint8_t)sb;
    } else {
#pragma unroll
        for (int w = 0; w < G / 8; ++w) {
            if constexpr (D == 64) {
                *reinterpret_cast<uint16_t*>(tile + L::v_code(t, g * G + 8 * w)) = (uint16_t)out[w];
                *reinterpret_cast<uint16_t*>(tile + L::v_code(t, g * G + 8 * w + 4)) = (uint16_t)(out[w] >> 16);
            } else {
                *reinterpret_cast<uint32_t*>(tile + L::v_code(t, g * G + 8 * w)) = out[w];
            }
        }
        tile[L::v_scale(t, g)] = (uint8_t)sb;
    }
}

// Calls F<FMT, ACT, D>(args...) for the run-time format, type and head size.
#define FP4_KV_DISPATCH(F, fmt, act, dim, ...)                                       \
    do {                                                                             \
        const int key_ = (int)(dim) * 4 + (fmt) * 2 + (act);                         \
        switch (key_) {                                                              \
            case 64 * 4 + 0: F<0, 0, 64>(__VA_ARGS__); break;                        \
            case 64 * 4 + 1: F<0, 1, 64>(__VA_ARGS__); break;                        \
            case 64 * 4 + 2: F<1, 0, 64>(__VA_ARGS__); break;                        \
            case 64 * 4 + 3: F<1, 1, 64>(__VA_ARGS__); break;                        \
            case 128 * 4 + 0: F<0, 0, 128>(__VA_ARGS__); break;                      \
            case 128 * 4 + 1: F<0, 1, 128>(__VA_ARGS__); break;                      \
            case 128 * 4 + 2: F<1, 0, 128>(__VA_ARGS__); break;                      \
            case 128 * 4 + 3: F<1, 1, 128>(__VA_ARGS__); break;                      \
            case 256 * 4 + 0: F<0, 0, 256>(__VA_ARGS__); break;                      \
            case 256 * 4 + 1: F<0, 1, 256>(__VA_ARGS__); break;                      \
            case 256 * 4 + 2: F<1, 0, 256>(__VA_ARGS__); break;                      \
            case 256 * 4 + 3: F<1, 1, 256>(__VA_ARGS__); break;                      \
        }                                                                            \
    } while (0)

}  // namespace fp4
