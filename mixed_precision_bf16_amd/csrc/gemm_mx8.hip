// C ABI and launches of the products of 8-bit activations (gemm_mx8.h).
#include <utility>

#include "gemm_mx8.h"

int fp4_check_weight_shape(int64_t N, int64_t K, int format);  // repack.cpp

namespace fp4 {

static int64_t out_tiles_of(int64_t cols, int out_type) {
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
static Mx8Plan mx8_plan(int64_t m, int64_t N, int64_t K, int out_type, int gate) {
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

template <int I>
static void decode_t(const Mx8Gemm& p, hipStream_t s) {
    constexpr DecodeMx8 d = kDecode[I];
    const int64_t tiles = d.tn * d.nwn / (p.up ? 2 : 1), out = out_tiles_of(p.cols, p.out_type);
    const dim3 grid((unsigned)((out + tiles - 1) / tiles), (unsigned)((p.M + 16 * d.mb - 1) / (16 * d.mb)));
    gemm_mx8_decode<d.mb, d.tn, d.nwn, d.nwk><<<grid, dim3(64 * d.nwn * d.nwk), 0, s>>>(p);
}

template <int I>
static void tiled_t(const Mx8Gemm& p, int S, void* workspace, hipStream_t s) {
    constexpr TiledMx8 t = kTiled[I];
    constexpr int TNW = t.tnw, BM = 16 * t.wm * t.mbw;
    const int64_t tiles = t.wn * TNW / (p.up ? 2 : 1), out = out_tiles_of(p.cols, p.out_type);
    const int64_t groups = (out + tiles - 1) / tiles, rows = (p.M + BM - 1) / BM;
    f32x4* P = S > 1 ? static_cast<f32x4*>(workspace) : nullptr;
    gemm_mx8_tiled<t.wm, t.wn, t.mbw, TNW><<<dim3((unsigned)(groups * rows * S)), dim3(64 * t.wm * t.wn), 0, s>>>(p, P, S);
    if (P) {
        const int64_t units = out / (p.out_type == 2 ? 2 : 1);
        const dim3 grid((unsigned)((units + 3) / 4), (unsigned)((p.M + 15) / 16));
        switch (S) {
            case 2: reduce_mx8<2><<<grid, dim3(256), 0, s>>>(p, P); break;
            case 3: reduce_mx8<3><<<grid, dim3(256), 0, s>>>(p, P); break;
            case 4: reduce_mx8<4><<<grid, dim3(256), 0, s>>>(p, P); break;
            case 6: reduce_mx8<6><<<grid, dim3(256), 0, s>>>(p, P); break;
            case 8: reduce_mx8<8><<<grid, dim3(256), 0, s>>>(p, P); break;
        }
    }
}

template <int... I>
static void launch_decode(int shape, const Mx8Gemm& p, hipStream_t s, std::integer_sequence<int, I...>) {
    (void)((shape == I && (decode_t<I>(p, s), true)) || ...);
}
template <int... I>
static void launch_tiled(int shape, const Mx8Gemm& p, int S, void* ws, hipStream_t s, std::integer_sequence<int, I...>) {
    (void)((shape == I && (tiled_t<I>(p, S, ws, s), true)) || ...);
}

static int gemm_mx8_check(int64_t m, int64_t N, int64_t K, int out_type, int gate) {
    if (out_type < 0 || out_type > 2 || gate < 0 || gate > 2) return FP4_ERR_FORMAT;
    int st = fp4_check_weight_shape(N, K, FP4_MXFP4);
    if (st != FP4_OK) return st;
    if (m < 0 || m > (int64_t(1) << 20)) return FP4_ERR_SHAPE;
    if (gate && N % 32) return FP4_ERR_SHAPE;  // the up rows begin at a weight tile
    const int64_t cols = gate ? N / 2 : N;
    if (out_type == 2 && cols % 32) return FP4_ERR_SHAPE;
    const int64_t rows = round_up(m, 256), most = int64_t(1) << 31;
    if (rows * mx8_padded(K) >= most || rows * cols * (out_type == 2 ? 1 : 2) >= most) return FP4_ERR_SHAPE;
    return FP4_OK;
}

// Whether what a call writes (output, its scales, workspace) lies apart from all else of it.
static bool gemm_mx8_apart(const fp4_gemm_mx8_args* q, size_t workspace) {
    const int64_t KA = mx8_padded(q->K), cols = q->gate ? q->N / 2 : q->N;
    const int64_t out = q->out_type == 2 ? q->m * mx8_padded(cols) : q->m * cols * 2;
    const int64_t weights = padded_n(q->N) * padded_k(q->K);
    const struct {
        const void* p;
        int64_t bytes;
    } part[] = {{q->out, out}, {q->out_scales, q->out_type == 2 ? out / 32 : 0}, {q->workspace, (int64_t)workspace},
                {q->codes, q->m * KA}, {q->scales, q->m * KA / 32}, {q->wq, weights / 2}, {q->sq, weights / 32}};
    for (int i = 0; i < 3; ++i)
        for (int k = i + 1; k < 7; ++k) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(part[i].p), b = reinterpret_cast<uintptr_t>(part[k].p);
            if (part[i].bytes && part[k].bytes && a < b + (uintptr_t)part[k].bytes && b < a + (uintptr_t)part[i].bytes)
                return false;
        }
    return true;
}

static int gemm_mx8_impl(const fp4_gemm_mx8_args* q, void* stream) {
    if (!q) return FP4_ERR_NULL;
    int st = gemm_mx8_check(q->m, q->N, q->K, q->out_type, q->gate);
    if (st != FP4_OK) return st;
    if (!alpha_ok(q->alpha)) return FP4_ERR_VALUE;
    if (q->m == 0) return FP4_OK;
    if (!q->codes || !q->scales || !q->wq || !q->sq || !q->out || (q->out_type == 2 && !q->out_scales))
        return FP4_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(q->codes) | reinterpret_cast<uintptr_t>(q->wq) |
         reinterpret_cast<uintptr_t>(q->sq) | reinterpret_cast<uintptr_t>(q->out)) & 15 ||
        (reinterpret_cast<uintptr_t>(q->scales) | reinterpret_cast<uintptr_t>(q->out_scales)) & 3)
        return FP4_ERR_SHAPE;
    const Mx8Plan plan = mx8_plan(q->m, q->N, q->K, q->out_type, q->gate);
    if (plan.workspace && (!q->workspace || q->workspace_bytes < plan.workspace ||
                           (reinterpret_cast<uintptr_t>(q->workspace) & 255)))
        return FP4_ERR_WORKSPACE;
    if (!gemm_mx8_apart(q, plan.workspace)) return FP4_ERR_SHAPE;
    st = check_device();
    if (st != FP4_OK) return st;
    Mx8Gemm p{};
    p.a = static_cast<const uint8_t*>(q->codes);
    p.as = static_cast<const uint8_t*>(q->scales);
    p.wq = static_cast<const uint8_t*>(q->wq);
    p.sq = static_cast<const uint8_t*>(q->sq);
    p.out = static_cast<uint8_t*>(q->out);
    p.out_scales = static_cast<uint8_t*>(q->out_scales);
    p.M = (int)q->m;
    p.KA = (int)mx8_padded(q->K);
    p.chunks = p.KA / kChunkK;
    p.KB = (int)(padded_k(q->K) / kChunkK);
    p.NT = (int)(padded_n(q->N) / kTileN);
    const int64_t cols = q->gate ? q->N / 2 : q->N;
    p.cols = (int)cols;
    p.cols_pad = (int)mx8_padded(cols);
    p.up = q->gate ? (int)(cols / kTileN) : 0;
    p.out_type = q->out_type;
    p.gate = q->gate;
    p.alpha = q->alpha;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (plan.shape < kDecodes)
        launch_decode(plan.shape, p, s, std::make_integer_sequence<int, kDecodes>{});
    else
        launch_tiled(plan.shape - kDecodes, p, plan.S, q->workspace, s, std::make_integer_sequence<int, kTiles>{});
    return launch_status();
}

}  // namespace fp4

extern "C" int fp4_gemm_mx8_workspace_size(int64_t m, int64_t N, int64_t K, int out_type, int gate, size_t* bytes) {
    int st = fp4::gemm_mx8_check(m, N, K, out_type, gate);
    if (st != FP4_OK) return st;
    if (!bytes) return FP4_ERR_NULL;
    *bytes = m == 0 ? 0 : fp4::mx8_plan(m, N, K, out_type, gate).workspace;
    return FP4_OK;
}

extern "C" int fp4_gemm_mx8(const fp4_gemm_mx8_args* args, void* stream) {
    return fp4::gemm_mx8_impl(args, stream);
}
