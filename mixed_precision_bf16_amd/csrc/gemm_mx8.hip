// C ABI and launches of the products of 8-bit activations (gemm_mx8.h).
#include "gemm_mx8.h"

int fp4_check_weight_shape(int64_t N, int64_t K, int format);  // repack.cpp

namespace fp4 {

template <int MB, int TN, int NWK, int PD>
static void stream_t(const Mx8Gemm& p, hipStream_t s) {
    const int tiles = p.up ? TN / 2 : TN;
    const int out_tiles = p.out_type == 2 ? p.cols_pad / 16 : (p.cols + 15) / 16;
    const dim3 grid((unsigned)((out_tiles + tiles - 1) / tiles), (unsigned)((p.M + 16 * MB - 1) / (16 * MB)));
    gemm_mx8_stream<MB, TN, NWK, PD><<<grid, dim3(64 * NWK), (size_t)NWK * TN * MB * 1024, s>>>(p);
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
    if (p.M <= 16) stream_t<1, 4, 8, 2>(p, s);
    else if (p.M <= 32) stream_t<2, 4, 8, 2>(p, s);
    else stream_t<4, 4, 4, 2>(p, s);
    return launch_status();
}

}  // namespace fp4

extern "C" int fp4_gemm_mx8_workspace_size(int64_t m, int64_t N, int64_t K, int out_type, int gate, size_t* bytes) {
    int st = fp4::gemm_mx8_check(m, N, K, out_type, gate);
    if (st != FP4_OK) return st;
    if (!bytes) return FP4_ERR_NULL;
    *bytes = 0;
    return FP4_OK;
}

extern "C" int fp4_gemm_mx8(const fp4_gemm_mx8_args* args, void* stream) {
    return fp4::gemm_mx8_impl(args, stream);
}
