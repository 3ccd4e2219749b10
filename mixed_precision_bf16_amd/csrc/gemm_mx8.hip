// C ABI and launches of the products of 8-bit activations (gemm_mx8.h).
#include <utility>

#include "gemm_mx8.h"

int fp4_check_weight_shape(int64_t N, int64_t K, int format);  // repack.cpp

namespace fp4 {

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
