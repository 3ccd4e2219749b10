// Which kernel a product of 8-bit activations takes, and in how many shares of K
// (gemm_mx8.h, gemm_mx8.hip).  Host code alone.
#pragma once
#include <stddef.h>

#include <algorithm>

#include "layout.h"

namespace fp4 {

constexpr int64_t kMx8PadK = 128;  // rows are padded to whole matrix-core steps

inline int64_t mx8_padded(int64_t K) { return round_up(K, kMx8PadK); }

inline int64_t out_tiles_of(int64_t cols, int out_type) {
    return out_type == 2 ? mx8_padded(cols) / 16 : (cols + 15) / 16;
}

// Kernels of a product, in the order of Mx8Plan::shape: small m (16 mb rows, nwn x tn
// weight tiles, nwk shares of K a workgroup) and larger m (wm x wn waves of 16 mbw
// rows by 16 tnw weight rows).
struct DecodeMx8 {
    int mb, tn, nwn, nwk;
};
constexpr int kCus = 256;  // compute units of an MI355X
constexpr DecodeMx8 kDecode[] = {{1, 1, 1, 4}, {1, 2, 1, 4}, {1, 3, 1, 4}, {1, 2, 2, 2}, {1, 2, 4, 1}, {2, 1, 1, 4}, {2, 2, 1, 4},
                                 {2, 3, 1, 4}, {2, 2, 2, 2}, {2, 2, 4, 1}, {2, 2, 8, 1}, {4, 1, 2, 2}, {4, 2, 2, 2}, {4, 2, 8, 1}};
constexpr int kDecodes = sizeof(kDecode) / sizeof(kDecode[0]);
struct TiledMx8 {
    int wm, wn, mbw, tnw;
    double alone_us, share_us;  // 128 k of a tile: one tile a compute unit; each of several
};
constexpr TiledMx8 kTiled[] = {{1, 4, 4, 2, 0.31, 0.40}, {1, 4, 4, 4, 0.55, 0.48}, {2, 4, 4, 4, 0.82, 0.80},
                               {2, 4, 8, 4, 1.50, 1.48}};
constexpr int kTiles = sizeof(kTiled) / sizeof(kTiled[0]);

struct Mx8Plan {
    int shape, S;
    size_t workspace;
};

// The kernel and split with the least modelled time (us).  Measured on MI355X with every
// shape forced and the weights in HBM (copies of them in turn, 700 MB and more), N x K of
// 57344 x 8192, 10240 x 8192, 8192 x 28672, 8192 x 8192, 4096 x 14336, 1024 x 8192, 2880 x
// 2880, gated 57344 x 8192, 20480 x 4096 and 5760 x 2880, m = 1, 16, 24, 48, 64, 80, 160,
// 256, 700, 2048: the choice is 1 % off the best on average, 10 % at most (80 x 20480 x 4096 gated).
//   Small m: launch and first loads 3.5, then 128 k of a workgroup's tiles cost 0.03 a
//   tile (the weights of all 256 compute units arrive at 6.2 TB/s) and 0.022 for 16 rows of
//   activations.  16 x 10240 x 8192 takes 11.7 us with 3 tiles a workgroup (214
//   workgroups), 14.7 with 2 (320: two rounds), 11.6 with 4 and 18 with 8; 16 x 57344
//   x 8192 gated 51, 44 and 41 us with 2, 4 and 8.
//   Larger m: 3.0, then the tile's time, or that of the weights, of which a compute unit
//   takes its share of 6.2 TB/s at most; a split of K adds its partial sums' round trip
//   through the caches at 6 TB/s and the second launch, 4.0.  256 x 8192 x 28672: 61 us
//   as 128 x 256 tiles split four ways, 69 as 256 x 256 split eight ways, 75 as 64 x 128
//   unsplit; 2048 x 57344 x 8192 gated: 660 us as 256 x 256, 740 as 128 x 256, 785 as 64 x
//   256, 1470 as 64 x 128 tiles, which are for one round of workgroups: 256 x 8192 x 8192
//   23 us, 29 as 128 x 256 split four ways; 160 x 10240 x 8192 22, 29 and as 64 x 256 35;
//   64 x 8192 x 28672 split four ways 30, three ways 35, and 40 by the kernels for small m.
inline Mx8Plan mx8_plan(int64_t m, int64_t N, int64_t K, int out_type, int gate) {
    const int64_t out = out_tiles_of(gate ? N / 2 : N, out_type), chunks = mx8_padded(K) / kChunkK;
    const double bytes = (double)N * (double)K * 0.53125;
    Mx8Plan best{0, 1, 0};
    double best_us = 1e30;
    auto offer = [&](int shape, int S, double us) {
        if (us < best_us) {
            best_us = us;
            best = Mx8Plan{shape, S, 0};
        }
    };
    for (int i = 0; i < kDecodes && m <= 64; ++i) {
        const DecodeMx8& d = kDecode[i];
        const int tiles = d.tn * d.nwn, cols = gate ? tiles / 2 : tiles;
        if (d.mb != (m <= 16 ? 1 : m <= 32 ? 2 : 4) || (gate && tiles % 2) || (out_type == 2 && cols % 2)) continue;
        const int64_t groups = (out + cols - 1) / cols, rounds = (groups + kCus - 1) / kCus;
        offer(i, 1, 3.5 + std::max((double)(rounds * chunks) * (0.01 + 0.022 * d.mb + 0.03 * tiles),
                                   bytes / 6.2e6 * (1.0 + 0.3 / tiles)));
    }
    for (int i = 0; i < kTiles && m > 16; ++i) {
        const TiledMx8& t = kTiled[i];
        if (gate && out_type == 2 && t.tnw < 4) continue;  // a wave holds whole blocks of 32 columns
        const int64_t cols = t.wn * t.tnw / (gate ? 2 : 1), rows = 16 * t.wm * t.mbw;
        const int64_t tiles = ((out + cols - 1) / cols) * ((m + rows - 1) / rows), groups = (chunks + 3) / 4;
        for (int S : {1, 2, 3, 4, 6, 8}) {
            if (S > groups || (S > 1 && tiles * S > kCus)) break;  // a split fills the first round
            const int64_t rounds = (tiles * S + kCus - 1) / kCus, each = 4 * ((groups + S - 1) / S);
            const double stream = bytes / 6.2e6 * std::max(1.0, (double)kCus / (double)(tiles * S));
            double us = 3.0 + std::max((double)each * (rounds == 1 ? t.alone_us : (double)rounds * t.share_us), stream);
            if (S > 1) us += 4.0 + (double)S * (double)m * (double)N * 8.0 / 6e6;
            offer(kDecodes + i, S, us);
        }
    }
    if (best.S > 1)
        best.workspace = (size_t)best.S * (size_t)((m + 15) / 16) * (size_t)out * (gate ? 2 : 1) * 1024;
    return best;
}

}  // namespace fp4
