// Root-mean-square norm with the residual's addition, in 16 or 8 bits, and the
// 8-bit quantizer of activations (include/fp4gemm.h, section "8-bit activations").
#include "apart.h"
#include "mx8.h"

namespace fp4 {

bool rows_apart(int64_t tokens, int64_t heads, int64_t D, int64_t ts, int64_t hs);  // kv_cache.hip

struct NormArgs {
    const uint16_t *x, *residual, *weight;
    uint8_t* out;          // 16-bit rows, or codes
    uint8_t* scales;
    uint16_t* sum;         // rounded x + residual, or null
    int64_t x_stride, residual_stride, sum_stride, out_stride;
    int rows, vecs, vecs_out;  // vectors of eight elements of a row; of an output row
    double inv_width, eps;
};

// h = x + residual of one vector, FP32.
template <int ACT>
__device__ __forceinline__ void norm_load(const NormArgs& a, int64_t row, int i, float (&h)[8]) {
    widen8<ACT>(load_once(a.x + row * a.x_stride + i * 8), h);
    if (a.residual) {
        float r[8];
        widen8<ACT>(load_once(a.residual + row * a.residual_stride + i * 8), r);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] += r[e];
    }
}

// Eight results y at vector i: 16-bit, or 8-bit with the block's scale taken
// over the four neighbouring lanes that hold its 32 elements.
template <int ACT, bool MX8>
__device__ __forceinline__ void norm_store(const NormArgs& a, int64_t row, int i, const float (&y)[8]) {
    if constexpr (!MX8) {
        *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(a.out) + row * a.out_stride + i * 8) = narrow8<ACT>(y);
    } else {
        float m = mx8_amax(y);
        m = fmaxf(m, __shfl_xor(m, 1));
        m = fmaxf(m, __shfl_xor(m, 2));
        const uint32_t sb = mx8_scale_byte(m);
        *reinterpret_cast<u32x2*>(a.out + (row * a.vecs_out + i) * 8) = mx8_codes(y, sb);
        if ((i & 3) == 0) a.scales[(row * a.vecs_out + i) / 4] = (uint8_t)sb;
    }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// y = h * root * weight with h = x + residual (FP32), root = 1 / sqrt(mean(h^2) +
// eps).  The squares, exact in FP64, are summed there, so that their size does not
// matter (BF16 values reach 1e38) and their order hardly does, and root, h * root and its
// product with the weight are each rounded to FP32 once: a result is the same on any
// split of the row unless the root lies within some 2^-52 of a border between FP32 values,
// about once in 2^28 rows.
// A team of T threads holds a row of up to 8 T V elements in registers and
// reads it once.  Bound by the bytes: 4095 x 8192 (BF16, a residual, 8-bit output;
// 236 MB) takes 42.5 us, 5.5 TB/s, with 512 threads a row and the nontemporal hint on
// the rows' loads; 48 us without the hint, 44 us with 256 threads (53 without either).
template <int ACT, bool MX8, int T, int V>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rms_norm_kernel(NormArgs a) {
    constexpr int kTeams = T < 256 ? 256 / T : 1, kWaves = T / 64;
    const int t = threadIdx.x % T, team = threadIdx.x / T;
    const int64_t row = (int64_t)blockIdx.x * kTeams + team;
    if (row >= a.rows) return;  // whole waves: a team is no smaller
    float h[V][8];
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = v * T + t;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] = 0.0f;
        if (i < a.vecs) norm_load<ACT>(a, row, i, h[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += (double)h[v][e] * (double)h[v][e];
    sum = wave_sum(sum);
    if constexpr (kWaves > 1) {
        __shared__ double part[kWaves];
        if (t % 64 == 0) part[t / 64] = sum;
        __syncthreads();
        sum = 0.0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += part[w];
    }
    const float root = (float)(1.0 / sqrt(sum * a.inv_width + a.eps));
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = v * T + t;
        if (i < a.vecs && a.sum)
            *reinterpret_cast<u32x4*>(a.sum + row * a.sum_stride + i * 8) = narrow8<ACT>(h[v]);
        if (i >= a.vecs_out) continue;  // blocks of 32, or the whole row: never part of a block
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = h[v][e] * root;
        if (a.weight && i < a.vecs) {
            float w[8];
            widen8<ACT>(*reinterpret_cast<const u32x4*>(a.weight + i * 8), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= w[e];
        }
        if (MX8 && i >= a.vecs) {  // the padding is zero whatever the row holds
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = 0.0f;
        }
        norm_store<ACT, MX8>(a, row, i, y);
    }
}

// Rows longer than the registers of a workgroup: read twice, the second time mostly from
// the caches (300 x 65536: 24 us, 3.3 TB/s of bytes read or written once; a row a
// compute unit, so that 300 rows take two rounds of the 256).
template <int ACT, bool MX8>
__global__ __launch_bounds__(1024) void rms_norm_long_kernel(NormArgs a) {
    __shared__ double part[16];
    const int64_t row = blockIdx.x;
    double sum = 0.0;
    for (int i = threadIdx.x; i < a.vecs; i += 1024) {
        float h[8];
        norm_load<ACT>(a, row, i, h);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += (double)h[e] * (double)h[e];
    }
    sum = wave_sum(sum);
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = sum;
    __syncthreads();
    sum = 0.0;
    for (int w = 0; w < 16; ++w) sum += part[w];
    const float root = (float)(1.0 / sqrt(sum * a.inv_width + a.eps));
    for (int i = threadIdx.x; i < a.vecs_out; i += 1024) {
        float y[8] = {};
        if (i < a.vecs) {
            norm_load<ACT>(a, row, i, y);  // before the sum is written: it may lie in x or the residual
            if (a.sum) *reinterpret_cast<u32x4*>(a.sum + row * a.sum_stride + i * 8) = narrow8<ACT>(y);
            float w[8];
            if (a.weight) widen8<ACT>(*reinterpret_cast<const u32x4*>(a.weight + i * 8), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = a.weight ? y[e] * root * w[e] : y[e] * root;
        }
        norm_store<ACT, MX8>(a, row, i, y);
    }
}

// Rows of 16-bit values to codes and scales, one vector a thread, four for a block.
// Bound by the bytes: 4096 x 8192 takes 21 us, 4.8 TB/s, its launch included.
template <int ACT>
__global__ __launch_bounds__(256) void quantize_mx8_kernel(NormArgs a) {
    const uint32_t n = blockIdx.x * 256u + threadIdx.x;  // at most 2^30
    if (n >= (uint32_t)a.rows * (uint32_t)a.vecs_out) return;  // whole blocks of 32
    const uint32_t row = n / (uint32_t)a.vecs_out;
    const int i = (int)(n - row * (uint32_t)a.vecs_out);
    float y[8] = {};
    if (i < a.vecs) widen8<ACT>(load_once(a.x + row * a.x_stride + i * 8), y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __builtin_canonicalizef(y[e]);  // a signalling NaN would hide other elements
    norm_store<ACT, true>(a, row, i, y);
}

// 16-bit rows: aligned, with strides of whole vectors.
static bool matrix_ok(const void* p, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride >= 0 && stride < (int64_t(1) << 40) && stride % 8 == 0;
}

static bool mx8_out_ok(const void* codes, const void* scales) {
    return (reinterpret_cast<uintptr_t>(codes) & 15) == 0 && (reinterpret_cast<uintptr_t>(scales) & 3) == 0;
}

// Rows of a launch: its work-items are counted in 32 bits.
constexpr int64_t kNormSliceRows = int64_t(1) << 20;

template <int ACT, bool MX8>
static void launch_norm(const NormArgs& a, hipStream_t s) {
    const int n = a.vecs_out;
    const unsigned rows = (unsigned)a.rows;
    if (n <= 64) rms_norm_kernel<ACT, MX8, 64, 1><<<dim3((rows + 3) / 4), dim3(256), 0, s>>>(a);
    else if (n <= 256) rms_norm_kernel<ACT, MX8, 256, 1><<<dim3(rows), dim3(256), 0, s>>>(a);
    else if (n <= 512) rms_norm_kernel<ACT, MX8, 512, 1><<<dim3(rows), dim3(512), 0, s>>>(a);
    else if (n <= 1024) rms_norm_kernel<ACT, MX8, 512, 2><<<dim3(rows), dim3(512), 0, s>>>(a);
    else if (n <= 4096) rms_norm_kernel<ACT, MX8, 1024, 4><<<dim3(rows), dim3(1024), 0, s>>>(a);
    else rms_norm_long_kernel<ACT, MX8><<<dim3(rows), dim3(1024), 0, s>>>(a);
}

static int norm_impl(const fp4_rms_norm_args* p, void* stream) {
    if (!p) return FP4_ERR_NULL;
    if ((p->act_type != 0 && p->act_type != 1) || (p->out_type != 0 && p->out_type != 1)) return FP4_ERR_FORMAT;
    const bool mx8 = p->out_type == 1;
    if (p->rows < 0 || p->rows > (int64_t(1) << 24) || p->width < 8 || p->width > (int64_t(1) << 20) ||
        p->width % (mx8 ? 32 : 8))
        return FP4_ERR_SHAPE;
    if (!(p->eps > 0.0f) || !(p->eps <= 1.0f)) return FP4_ERR_VALUE;
    if (p->rows == 0) return FP4_OK;
    if (!p->x || !p->out || (mx8 && !p->out_scales)) return FP4_ERR_NULL;
    if (!matrix_ok(p->x, p->x_stride) || (p->residual && !matrix_ok(p->residual, p->residual_stride)) ||
        (p->weight && !matrix_ok(p->weight, 0)))
        return FP4_ERR_SHAPE;
    if (p->sum && (!matrix_ok(p->sum, p->sum_stride) || !rows_apart(p->rows, 1, p->width, p->sum_stride, p->width)))
        return FP4_ERR_SHAPE;
    if (mx8 ? !mx8_out_ok(p->out, p->out_scales)
            : !matrix_ok(p->out, p->out_stride) || !rows_apart(p->rows, 1, p->width, p->out_stride, p->width))
        return FP4_ERR_SHAPE;
    // a row is read whole before it is written, so a 16-bit output may be an input, row on row;
    // else what is written lies apart from all other arrays
    const int64_t kp = mx8_padded(p->width);
    const Span x = span_of_rows(p->x, p->width, p->rows, p->x_stride);
    const Span residual = span_of_rows(p->residual, p->width, p->rows, p->residual_stride);
    const Span weight = span_of(p->weight, p->width * 2);
    const Span sum = span_of_rows(p->sum, p->width, p->rows, p->sum_stride);
    if (spans_meet(sum, weight) || !span_may_be(sum, x) || !span_may_be(sum, residual)) return FP4_ERR_SHAPE;
    if (mx8) {
        const Span codes = span_of(p->out, p->rows * kp), scales = span_of(p->out_scales, p->rows * kp / 32);
        if (spans_meet(codes, scales)) return FP4_ERR_SHAPE;
        for (const Span& from : {x, residual, weight, sum})
            if (spans_meet(codes, from) || spans_meet(scales, from)) return FP4_ERR_SHAPE;
    } else {
        const Span out = span_of_rows(p->out, p->width, p->rows, p->out_stride);
        if (spans_meet(out, weight) || spans_meet(out, sum) || !span_may_be(out, x) || !span_may_be(out, residual))
            return FP4_ERR_SHAPE;
    }
    int st = check_device();
    if (st != FP4_OK) return st;
    NormArgs a{};
    a.x = static_cast<const uint16_t*>(p->x);
    a.residual = static_cast<const uint16_t*>(p->residual);
    a.weight = static_cast<const uint16_t*>(p->weight);
    a.out = static_cast<uint8_t*>(p->out);
    a.scales = static_cast<uint8_t*>(p->out_scales);
    a.sum = static_cast<uint16_t*>(p->sum);
    a.x_stride = p->x_stride;
    a.residual_stride = p->residual_stride;
    a.sum_stride = p->sum_stride;
    a.out_stride = p->out_stride;
    a.vecs = (int)(p->width / 8);
    a.vecs_out = (int)((mx8 ? kp : p->width) / 8);
    a.inv_width = 1.0 / (double)p->width;
    a.eps = p->eps;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    const NormArgs all = a;
    for (int64_t r0 = 0; r0 < p->rows; r0 += kNormSliceRows) {
        a.rows = (int)std::min(kNormSliceRows, p->rows - r0);
        a.x = all.x + r0 * a.x_stride;
        if (all.residual) a.residual = all.residual + r0 * a.residual_stride;
        if (all.sum) a.sum = all.sum + r0 * a.sum_stride;
        a.out = all.out + (mx8 ? r0 * a.vecs_out * 8 : r0 * a.out_stride * 2);
        a.scales = all.scales + (mx8 ? r0 * a.vecs_out / 4 : 0);
        switch (p->act_type * 2 + (mx8 ? 1 : 0)) {
            case 0: launch_norm<0, false>(a, s); break;
            case 1: launch_norm<0, true>(a, s); break;
            case 2: launch_norm<1, false>(a, s); break;
            case 3: launch_norm<1, true>(a, s); break;
        }
        st = launch_status();
        if (st != FP4_OK) return st;
    }
    return FP4_OK;
}

static int quantize_mx8_impl(const void* x, int64_t rows, int64_t K, int64_t x_stride, int act_type, void* codes,
                             void* scales, void* stream) {
    if (act_type != 0 && act_type != 1) return FP4_ERR_FORMAT;
    if (rows < 0 || rows > (int64_t(1) << 24) || K < 32 || K > (int64_t(1) << 20) || K % 32) return FP4_ERR_SHAPE;
    if (rows == 0) return FP4_OK;
    if (!x || !codes || !scales) return FP4_ERR_NULL;
    if (!matrix_ok(x, x_stride) || !mx8_out_ok(codes, scales)) return FP4_ERR_SHAPE;
    const Span from = span_of_rows(x, K, rows, x_stride);
    const Span to = span_of(codes, rows * mx8_padded(K)), powers = span_of(scales, rows * mx8_padded(K) / 32);
    if (spans_meet(to, powers) || spans_meet(to, from) || spans_meet(powers, from)) return FP4_ERR_SHAPE;
    int st = check_device();
    if (st != FP4_OK) return st;
    NormArgs a{};
    a.x_stride = x_stride;
    a.vecs = (int)(K / 8);
    a.vecs_out = (int)(mx8_padded(K) / 8);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    // a launch counts its work-items in 32 bits
    const int64_t slice = std::max<int64_t>(1, (int64_t(1) << 30) / a.vecs_out);
    for (int64_t r0 = 0; r0 < rows; r0 += slice) {
        a.rows = (int)std::min(slice, rows - r0);
        a.x = static_cast<const uint16_t*>(x) + r0 * x_stride;
        a.out = static_cast<uint8_t*>(codes) + r0 * a.vecs_out * 8;
        a.scales = static_cast<uint8_t*>(scales) + r0 * a.vecs_out / 4;
        const dim3 grid((unsigned)(((int64_t)a.rows * a.vecs_out + 255) / 256)), block(256);
        if (act_type == 0) quantize_mx8_kernel<0><<<grid, block, 0, s>>>(a);
        else quantize_mx8_kernel<1><<<grid, block, 0, s>>>(a);
        st = launch_status();
        if (st != FP4_OK) return st;
    }
    return FP4_OK;
}

}  // namespace fp4

extern "C" int fp4_mx8_size(int64_t rows, int64_t K, size_t* codes_bytes, size_t* scales_bytes) {
    if (rows < 0 || rows > (int64_t(1) << 24) || K < 32 || K > (int64_t(1) << 20) || K % 32) return FP4_ERR_SHAPE;
    const int64_t n = rows * fp4::mx8_padded(K);
    if (codes_bytes) *codes_bytes = (size_t)n;
    if (scales_bytes) *scales_bytes = (size_t)(n / 32);
    return FP4_OK;
}

extern "C" int fp4_rms_norm(const fp4_rms_norm_args* args, void* stream) { return fp4::norm_impl(args, stream); }

extern "C" int fp4_quantize_mx8(const void* x, int64_t rows, int64_t K, int64_t x_stride, int act_type, void* codes,
                                void* scales, void* stream) {
    return fp4::quantize_mx8_impl(x, rows, K, x_stride, act_type, codes, scales, stream);
}
