// Products of 8-bit activations with MXFP4 weights on the scaled matrix cores
// (include/fp4gemm.h, section "8-bit activations").
//
//   Y[m][n] = alpha * sum_k a[m][k] w[n][k]
//   a = E4M3 code * 2^(scale - 127), one scale for 32 k; w the same with E2M1
//
// Up to 16 rows (bound by the weights' bytes): both operands become BF16, exactly,
// and the 16-bit matrix cores add their products in FP32.  More rows:
// One v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 weight rows by 16
// activation rows over 128 k.  Operand layout (checked on the device), lane =
// 16 j + r: row r of either operand; FP4: k = 32 j .. 32 j + 31 (the native
// weight layout, repack.cpp); FP8: k = 16 j .. 16 j + 15 and 64 + 16 j ..
// 64 + 16 j + 15; either scale: block j of the row's four.  The result: rows n =
// 4 j .. 4 j + 3, column m = r.
//
// With an FP8 operand this instruction cuts products off before it adds them (FP4 by
// FP4 and the 16-bit products lose nothing): of each eight k, 8 i .. 8 i + 7, a product
// loses, toward zero, what lies below 2^(e - 13), e being the largest sum of its two codes'
// exponents (E4M3 -6 at least, E2M1 0) that a nonzero product of the eight has.  A product
// has at most six bits, so one whose exponent is e - 9 or more loses nothing.  The sums lose
// less than 7 * 2^-13 of sum |a w|, and 6e-8 of it on average for Gaussian rows of 8192:
// 4e-6 of the result's size, a thousandth of a BF16 step; in 8-bit outputs it can move a
// code, and one block's scale in 15000, that lies next to a border.
// It is taken all the same: two such products, of the codes from 2 on and of those below,
// lose nothing, and cost 42 -> 45 us for 32 x 57344 x 8192 gated, 46 -> 76 for 61 rows, 63 ->
// 105 for 256 x 8192 x 28672 and 661 -> 1233 for 2048 x 57344 x 8192 gated; the 16-bit products
// of fp4_gemm take 103 us for the third and 1256 for the last's 57344 columns.
#pragma once
#include "mx8.h"

namespace fp4 {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Mx8Gemm {
    const uint8_t* a;   // codes [M][KA]
    const uint8_t* as;  // scales [M][KA / 32]
    const uint8_t* wq;
    const uint8_t* sq;
    uint8_t* out;         // 16-bit [M][cols], or codes [M][cols_pad]
    uint8_t* out_scales;  // [M][cols_pad / 32]
    int M, KA, chunks;    // chunks = KA / 128
    int KB;               // chunks of a weight tile (K padded to 512)
    int NT;               // weight tiles of 16 rows
    int cols, cols_pad;   // output columns; padded (8-bit output)
    int up;               // gated: weight tile of the first up row; else 0
    int out_type;         // 0 BF16, 1 FP16, 2 MX8
    int gate;             // 0 none, 1 SiLU, 2 GELU (tanh)
    float alpha;
};

// act(g) * u.  SiLU: g / (1 + e^-g).  GELU: g / (1 + e^-2z) with z = sqrt(2 / pi)
// (g + 0.044715 g^3), the same as g / 2 (1 + tanh z).
__device__ __forceinline__ float gated(float g, float u, int gate) {
    const float z = gate == 1 ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
    return g / (1.0f + __expf(-z)) * u;
}

__device__ __forceinline__ i32x8 fp4_operand(const u32x4& w) {
    return i32x8{(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
}
__device__ __forceinline__ i32x8 fp8_operand(const u32x4& lo, const u32x4& hi) {
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}
// Weight scale: byte T of its dword (chunk T of the 512 k); activation scale: the low byte.
template <int T>
__device__ __forceinline__ f32x4 mfma_fp4_fp8(const u32x4& w, const i32x8& a, const f32x4& c, uint32_t ws, uint32_t as) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(w), a, c, 4, 0, T, (int)ws, 0, (int)as);
}

// Output tile `t` (columns 16 t ..) of row m: the lane's four columns.
__device__ __forceinline__ void mx8_store16(const Mx8Gemm& p, const f32x4& v, int m, int t, int j) {
    if (p.out_type == 0) store_frag<0>(reinterpret_cast<uint16_t*>(p.out), v, m, t * 16 + 4 * j, p.M, p.cols);
    else store_frag<1>(reinterpret_cast<uint16_t*>(p.out), v, m, t * 16 + 4 * j, p.M, p.cols);
}

// Output tiles t and t + 1 (t even): one 8-bit block of row m, its 32 columns in
// the four lanes (r, 0 .. 3).
__device__ __forceinline__ void mx8_store8(const Mx8Gemm& p, f32x4 v0, f32x4 v1, int m, int t, int j) {
    float x[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    if (t * 16 >= p.cols) {  // columns is a multiple of 32: the whole block is padding
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    }
    float top = mx8_amax(x);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const uint32_t sb = mx8_scale_byte(top);
    const u32x2 c = mx8_codes(x, sb);
    if (m < p.M && t * 16 < p.cols_pad) {
        uint8_t* row = p.out + (int64_t)m * p.cols_pad + t * 16 + 4 * j;
        *reinterpret_cast<uint32_t*>(row) = c.x;
        *reinterpret_cast<uint32_t*>(row + 16) = c.y;
        if (j == 0) p.out_scales[(int64_t)m * (p.cols_pad / 32) + t / 2] = (uint8_t)sb;
    }
}

// The result of output tiles t (and with 8-bit output t + 1) from their sums.
// `sum(x)`: FP32 sums of weight tile x of the caller's group: output tiles first,
// gated: then the up tiles, `half` further on.
template <class Sum>
__device__ __forceinline__ void mx8_finish(const Mx8Gemm& p, Sum sum, int x, int half, int m, int t, int j) {
    auto result = [&](int y) {
        f32x4 v = sum(y) * p.alpha;
        if (p.up) {
            const f32x4 u = sum(y + half) * p.alpha;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = gated(v[e], u[e], p.gate);
        }
        return v;
    };
    if (p.out_type == 2) mx8_store8(p, result(x), result(x + 1), m, t, j);
    else mx8_store16(p, result(x), m, t, j);
}

// Eight E4M3 codes times a power of two (the exponent of `scale`): exact BF16 values.
__device__ __forceinline__ u32x4 bf16_of_fp8(uint32_t lo, uint32_t hi, float scale) {
    u32x4 o;
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
    return o;
}

// Place of workgroup x of `total` in the order of work: one band for each XCD, to which
// the workgroups are dealt in turn.
__device__ __forceinline__ int xcd_band(int x, int total) {
    const int xcd = x % kXcdCount, each = total / kXcdCount, more = total % kXcdCount;
    return xcd * each + min(xcd, more) + x / kXcdCount;
}

// Small m: bound by the weights' bytes.  A workgroup takes 16 MB rows and BT = NWN TN
// weight tiles (gated: BT / 2 gate tiles, then the up tiles of the same columns), as
// NWK groups of NWN waves; a group takes its share of K, a wave TN of the tiles.
// Weights go straight to registers, 512 k ahead (a wave load is 1 KiB in a row).  The
// activations of 512 k go to LDS by DMA, one buffer ahead, once for the NWN waves of a
// group and in whole lines: read straight into fragments (64-byte pieces of 16
// rows) they cost 1.4 times a weight tile's load, and 16 x 57344 x 8192 took 46 us
// instead of 41.  The columns of a row (16 bytes) are XOR-swizzled by row: fragment
// reads without bank conflicts.  The groups' sums meet in LDS, in their order.
// 16 rows: exact BF16 operands, 3 to 5 % slower than the 8-bit products (16 x 57344 x 8192
// gated 40.5 and 42.4 us) and free of their rounding; with 32 rows the conversions cost 6
// to 20 %, with 64 half, so those take the 8-bit products.
template <int MB, int TN, int NWN, int NWK>
__global__ __launch_bounds__(64 * NWN * NWK) void gemm_mx8_decode(Mx8Gemm p) {
    constexpr int BM = 16 * MB, BT = NWN * TN;
    constexpr bool kExact = MB == 1;
    constexpr int kBuf = BM * 512 + BM * 16;            // codes and scales of a group of 512 k
    constexpr int kStage = BM * 32 / (64 * NWN);        // 16-byte code pieces a lane brings per group
    static_assert(kStage >= 1 && kStage * 64 * NWN == BM * 32, "whole pieces");
    constexpr int kSums = NWK * BT * MB * 1024;
    constexpr int kLds = 2 * NWK * kBuf > kSums ? 2 * NWK * kBuf : kSums;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
    const int lane = threadIdx.x & 63, r = lane & 15, j = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave % NWN, kw = wave / NWN;
    const int half = p.up ? BT / 2 : BT;
    // in bands: 16 x 57344 x 8192 takes 41 us, dealt in turn 49.5 (gated 40.6 and 41.7)
    const int m0 = blockIdx.y * BM, t0 = xcd_band(blockIdx.x, gridDim.x) * half;
    const int Q = (p.chunks + 3) / 4, per = (Q + NWK - 1) / NWK;
    const int q0 = min(kw * per, Q), q1 = min(q0 + per, Q);   // every K group makes `per` turns

    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a, (uint32_t)p.M * (uint32_t)p.KA);
    const __amdgpu_buffer_rsrc_t rsa = make_rsrc(p.as, (uint32_t)p.M * (uint32_t)(p.KA / 32));
    __amdgpu_buffer_rsrc_t rw[TN], rs[TN];
#pragma unroll
    for (int tt = 0; tt < TN; ++tt) {
        const int y = wn * TN + tt;                     // weight tile of the workgroup: [gate | up]
        int t = t0 + y;
        if (p.up) t = y < BT / 2 ? min(t, p.up - 1) : p.up + t0 + y - BT / 2;
        t = min(t, p.NT - 1);
        rw[tt] = make_rsrc(p.wq + (size_t)t * p.KB * 1024, (uint32_t)p.KB * 1024u);
        rs[tt] = make_rsrc(p.sq + (size_t)t * p.KB * 64, (uint32_t)p.KB * 64u);
    }
    uint8_t* mine = lds + kw * 2 * kBuf;
    // piece n of a group: row n / 32, physical column n % 32 = column ^ (row % 8)
    uint32_t aoff[kStage];
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
        const int n = (i * NWN + wn) * 64 + lane, row = n >> 5, col = (n & 31) ^ (row & 7);
        aoff[i] = (uint32_t)(m0 + row) * (uint32_t)p.KA + col * 16;
    }
    const uint32_t soff = (uint32_t)(m0 + lane) * (uint32_t)(p.KA / 32);
    auto a_dma = [&](int q, int buf) {
        q = max(min(q, q1 - 1), 0);
#pragma unroll
        for (int i = 0; i < kStage; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra, (__attribute__((address_space(3))) void*)(mine + buf * kBuf + (i * NWN + wn) * 1024), 16,
                (int)(aoff[i] + (uint32_t)q * 512), 0, 0, 0);
        if (wn == 0 && lane < BM)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsa, (__attribute__((address_space(3))) void*)(mine + buf * kBuf + BM * 512), 16,
                (int)(soff + (uint32_t)q * 16), 0, 0, 0);
        asm volatile("" ::: "memory");  // the weights stay behind it: the waits count them
    };
    u32x4 w[4][TN];
    uint32_t sc[2][TN];
    auto w_issue = [&](auto t_c, int q) {
        constexpr int T = decltype(t_c)::value;
        const int c = max(min(4 * q + T, 4 * q1 - 1), 0);
#pragma unroll
        for (int tt = 0; tt < TN; ++tt)
            w[T][tt] = __builtin_amdgcn_raw_buffer_load_b128(rw[tt], lane * 16, c * 1024, kLoadStream);
    };
    auto s_issue = [&](int q, uint32_t (&s)[TN]) {
#pragma unroll
        for (int tt = 0; tt < TN; ++tt)
            s[tt] = __builtin_amdgcn_raw_buffer_load_b32(rs[tt], lane * 4, max(min(q, q1 - 1), 0) * 256, kLoadStream);
    };
    f32x4 acc[TN][MB];
#pragma unroll
    for (int tt = 0; tt < TN; ++tt)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) acc[tt][mb] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int frow = r * 512;
    auto compute = [&](auto t_c, int buf, const uint32_t (&s)[TN]) {
        constexpr int T = decltype(t_c)::value;
        const uint8_t* b = mine + buf * kBuf;
        if constexpr (kExact) {
            const u32x4 lo = *reinterpret_cast<const u32x4*>(b + frow + (((8 * T + 2 * j) ^ (r & 7)) << 4));
            const u32x4 hi = *reinterpret_cast<const u32x4*>(b + frow + (((8 * T + 2 * j + 1) ^ (r & 7)) << 4));
            const float sa = __uint_as_float((uint32_t)b[BM * 512 + r * 16 + T * 4 + j] << 23);
            const u32x4 a[4] = {bf16_of_fp8(lo.x, lo.y, sa), bf16_of_fp8(lo.z, lo.w, sa), bf16_of_fp8(hi.x, hi.y, sa),
                                bf16_of_fp8(hi.z, hi.w, sa)};
#pragma unroll
            for (int tt = 0; tt < TN; ++tt) {
                const float sw = __uint_as_float(((s[tt] >> (8 * T)) & 0xFFu) << 23);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[tt][0] = mfma<0>(dequant_mxfp4(w[T][tt][i], sw), a[i], acc[tt][0]);
            }
        } else {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                const u32x4 lo = *reinterpret_cast<const u32x4*>(b + mb * 8192 + frow + (((8 * T + j) ^ (r & 7)) << 4));
                const u32x4 hi = *reinterpret_cast<const u32x4*>(b + mb * 8192 + frow + (((8 * T + 4 + j) ^ (r & 7)) << 4));
                const uint32_t as = b[BM * 512 + (mb * 16 + r) * 16 + T * 4 + j];
                const i32x8 a = fp8_operand(lo, hi);
#pragma unroll
                for (int tt = 0; tt < TN; ++tt) acc[tt][mb] = mfma_fp4_fp8<T>(w[T][tt], a, acc[tt][mb], s[tt], as);
            }
        }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    a_dma(q0, 0);
    s_issue(q0, sc[0]);
    w_issue(I0{}, q0);
    w_issue(I1{}, q0);
    w_issue(I2{}, q0);
    w_issue(I3{}, q0);
    auto turn = [&](int i, const uint32_t (&cur)[TN], uint32_t (&nxt)[TN]) {
        const int q = q0 + i;
        // the DMA of this group is complete: after it came its weights alone
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(4 * TN) : "memory");
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        a_dma(q + 1, (i + 1) & 1);
        s_issue(q + 1, nxt);
        auto one = [&](auto t_c) {
            constexpr int T = decltype(t_c)::value;
            if (4 * q + T < min(p.chunks, 4 * q1)) compute(t_c, i & 1, cur);
            w_issue(t_c, q + 1);
        };
        one(I0{});
        one(I1{});
        one(I2{});
        one(I3{});
    };
    int i = 0;
    for (; i + 1 < per; i += 2) {
        turn(i, sc[0], sc[1]);
        turn(i + 1, sc[1], sc[0]);
    }
    if (i < per) turn(i, sc[0], sc[1]);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    f32x4* sums = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int tt = 0; tt < TN; ++tt)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) sums[((kw * BT + wn * TN + tt) * MB + mb) * 64 + lane] = acc[tt][mb];
    __syncthreads();
    const int unit = p.out_type == 2 ? 2 : 1, items = half / unit * MB;
    for (int it = wave; it < items; it += NWN * NWK) {
        const int y0 = it / MB * unit, mb = it % MB;
        auto sum = [&](int y) {
            f32x4 v = sums[(y * MB + mb) * 64 + lane];
#pragma unroll
            for (int k = 1; k < NWK; ++k) v += sums[((k * BT + y) * MB + mb) * 64 + lane];
            return v;
        };
        mx8_finish(p, sum, y0, BT / 2, m0 + mb * 16 + r, t0 + y0, j);
    }
}

// Larger m: a workgroup of WM x WN waves takes BM = 16 WM MBW rows and WN TNW
// weight tiles (gated: a wave's first TNW / 2 are gate tiles, the others the up
// tiles of the same columns), over groups of 512 k [ks Q / S, (ks + 1) Q / S).
// A goes to LDS by DMA, three chunks of 128 k in rotation, the 16-byte columns of a
// row XOR-swizzled by row / 2 (conflict-free fragment reads); its scales, 16 bytes a
// row and group, one group ahead in two buffers.  Weights go straight to registers,
// two chunks ahead.  Per chunk c: the fragments of each 16 rows are read one step
// ahead of their products; before the last products: wait for this wave's DMA of
// chunk c + 1, barrier (every wave has read chunk c, and chunk c + 1 is whole), DMA of
// chunk c + 3 into c's buffer.
// kDeep, the narrow tile (64 x 128) of few rows, whose weights come from HBM: buffers
// of two chunks, weights four chunks ahead past the caches, and a loop without a way
// out of it (37 -> 30 us for 61 x 8192 x 28672, 29 -> 23 for 256 x 8192 x 8192).  It
// leaves less room for other workgroups (1060 -> 1470 us for 2048 x 57344 x 8192 gated),
// and wider tiles lose by it in one round too (128 x 256: 61 -> 67 us for 256 x 8192 x
// 28672).
// Bound by the matrix cores where rows are many: 2048 x 57344 x 8192 gated 660 us, 2.9
// PFLOP/s (a library product of 8-bit floats of 8192 cubed reaches 2.7), the cores busy
// 65 % of the time at 1.86 GHz, what the power limit leaves; where they are few by the
// weights' way through the second-level cache: 256 x 8192 x 28672 61 us, 2.0 PFLOP/s,
// of which 7 are the shares' sums (with weights that lie in the cache 52).
// S > 1: FP32 partial sums in fragment order to P, for reduce_mx8.
template <int WM, int WN, int MBW, int TNW>
__global__ __launch_bounds__(64 * WM * WN) void gemm_mx8_tiled(Mx8Gemm p, f32x4* __restrict__ P, int S) {
    constexpr int kThreads = 64 * WM * WN;
    constexpr int BM = WM * MBW * 16;
    constexpr bool kDeep = TNW == 2;
    // chunks of a buffer, chunks the weights are ahead, and room for them
    constexpr int kPer = kDeep ? 2 : 1, kAhead = kDeep ? 4 : 2, kSlots = kDeep ? 8 : 4;
    constexpr int kChunk = BM * 128, kBuf = kPer * kChunk;
    constexpr int kStage = BM * 8 / kThreads;  // 16-byte pieces a thread brings per chunk
    static_assert(kStage * kThreads == BM * 8 && BM % 64 == 0 && BM <= kThreads, "whole pieces, whole waves");
    __shared__ __attribute__((aligned(16))) uint8_t lds[3 * kBuf + 2 * BM * 16];
    constexpr int kScales = 3 * kBuf;

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, j = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;

    // work item: K share innermost, then m tiles, then weight tiles, in one band
    // for each XCD: the workgroups of an XCD share weights and rows in its L2
    const int out_tiles = p.out_type == 2 ? p.cols_pad / 16 : (p.cols + 15) / 16;
    const int half = p.up ? TNW / 2 : TNW;         // output tiles of a wave
    const int MT = (p.M + BM - 1) / BM, NG = (out_tiles + WN * half - 1) / (WN * half);
    const int item = xcd_band(blockIdx.x, MT * NG * S);
    const int ks = item % S, mt = item / S % MT, ng = item / S / MT;
    const int m0 = mt * BM, t0 = (ng * WN + wn) * half;
    const int Q = (p.chunks + 3) / 4;
    const int q0 = (int)((int64_t)Q * ks / S), q1 = (int)((int64_t)Q * (ks + 1) / S);
    const int clast = min(4 * q1, p.chunks) - 1;

    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a, (uint32_t)p.M * (uint32_t)p.KA);
    const __amdgpu_buffer_rsrc_t rsa = make_rsrc(p.as, (uint32_t)p.M * (uint32_t)(p.KA / 32));
    __amdgpu_buffer_rsrc_t rw[TNW], rs[TNW];
#pragma unroll
    for (int tt = 0; tt < TNW; ++tt) {
        int t = t0 + tt;
        if (p.up) t = tt < TNW / 2 ? min(t, p.up - 1) : p.up + t0 + tt - TNW / 2;
        t = min(t, p.NT - 1);
        rw[tt] = make_rsrc(p.wq + (size_t)t * p.KB * 1024, (uint32_t)p.KB * 1024u);
        rs[tt] = make_rsrc(p.sq + (size_t)t * p.KB * 64, (uint32_t)p.KB * 64u);
    }

    // LDS slot n = row n / 8, physical column n % 8
    uint32_t aoff[kStage];
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
        const int n = tid + kThreads * i, row = n >> 3, col = (n & 7) ^ ((row >> 1) & 7);
        aoff[i] = (uint32_t)(m0 + row) * (uint32_t)p.KA + col * 16;
    }
    // chunks c .. c + kPer - 1 to the buffer at `buf` (past the range: into bytes nobody reads again)
    auto a_dma = [&](int c, int buf) {
#pragma unroll
        for (int u = 0; u < kPer; ++u)
#pragma unroll
            for (int i = 0; i < kStage; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    ra, (__attribute__((address_space(3))) void*)(lds + buf + u * kChunk + (i * kThreads + 64 * wave) * 16), 16,
                    (int)(aoff[i] + (uint32_t)min(c + u, clast) * 128), 0, 0, 0);
        asm volatile("" ::: "memory");  // later loads stay behind it: the waits count them
    };
    // scales of group q, 16 bytes a row (behind the row's last chunk: bytes that no
    // product takes), 64 rows a wave
    const uint32_t soff = (uint32_t)(m0 + 64 * (wave % (BM / 64)) + lane) * (uint32_t)(p.KA / 32);
    auto s_dma = [&](int q) {
        if (kDeep || wave < BM / 64)  // kDeep: every wave the same rows, no branch in a group
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsa, (__attribute__((address_space(3))) void*)(lds + kScales + (q & 1) * BM * 16 + 64 * (wave % (BM / 64)) * 16),
                16, (int)(soff + (uint32_t)min(q, q1 - 1) * 16), 0, 0, 0);
        asm volatile("" ::: "memory");  // the group's weights stay behind it: its last wait counts them
    };
    u32x4 w[kSlots][TNW];
    auto w_issue = [&](auto slot_c, int c) {
        constexpr int SL = decltype(slot_c)::value % kSlots;
        c = min(c, clast);
#pragma unroll
        for (int tt = 0; tt < TNW; ++tt)
            w[SL][tt] = __builtin_amdgcn_raw_buffer_load_b128(rw[tt], lane * 16, c * 1024, kDeep ? kLoadStream : kLoadReused);
    };
    // no fence: it would also wait for the newest DMA
    auto lds_barrier = [] {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    struct Frag {
        u32x4 lo, hi;
        uint32_t s;
    };
    const int frow = (wm * MBW * 16 + r) * 128, swz = (r >> 1) & 7;
    const int flo = frow + ((j ^ swz) << 4), fhi = frow + (((4 + j) ^ swz) << 4);
    const int fs = kScales + (wm * MBW * 16 + r) * 16 + j;
    auto read = [&](int buf, int mb, int t, int q, Frag& f) {
        f.lo = *reinterpret_cast<const u32x4*>(lds + buf + flo + mb * 2048);
        f.hi = *reinterpret_cast<const u32x4*>(lds + buf + fhi + mb * 2048);
        f.s = lds[fs + (q & 1) * BM * 16 + mb * 256 + t * 4];
    };
    f32x4 acc[TNW][MBW];
#pragma unroll
    for (int tt = 0; tt < TNW; ++tt)
#pragma unroll
        for (int mb = 0; mb < MBW; ++mb) acc[tt][mb] = f32x4{0.f, 0.f, 0.f, 0.f};

    int b_cur = 0, b_nxt = kBuf, b_far = 2 * kBuf;
    Frag fa, fb;
    uint32_t wsc[TNW], wsn[TNW];
    // chunk c = 4 q + T, its weights in slot E + T; fa holds its first fragment on entry
    auto step = [&](auto t_c, auto e_c, auto tail_c, int q, const uint32_t (&sc)[TNW]) {
        constexpr int T = decltype(t_c)::value, SL = (decltype(e_c)::value + T) % kSlots;
        constexpr bool kLast = T % kPer == kPer - 1;  // the last chunk of its buffer
        constexpr bool kTail = decltype(tail_c)::value;  // nothing follows the group
        const int c = 4 * q + T, at = b_cur + T % kPer * kChunk;
        if constexpr (!kTail || T + kAhead < 4) w_issue(std::integral_constant<int, SL + kAhead>{}, c + kAhead);
        if constexpr (!kLast) asm volatile("" ::: "memory");  // not put off to the next chunk
        auto mma = [&](const Frag& f, int mb) {
            const i32x8 a = fp8_operand(f.lo, f.hi);
#pragma unroll
            for (int tt = 0; tt < TNW; ++tt)
                acc[tt][mb] = mfma_fp4_fp8<T>(w[SL][tt], a, acc[tt][mb], sc[tt], f.s);
        };
#pragma unroll
        for (int mb = 0; mb + 1 < MBW; ++mb) {
            read(at, mb + 1, T, q, mb % 2 ? fa : fb);
            mma(mb % 2 ? fb : fa, mb);
        }
        if constexpr (kLast) {
            // Loads complete in issue order.  After the DMA of the next buffer came the
            // weights asked for in two buffers' steps, this one's included, and between
            // them the DMA of the buffer after it (before the first step too; a last group
            // asks for no weights behind it, and nothing is read after its T = 3).
            // The wait of T = 3 also completes the next group's scales, which are read
            // behind it: their DMA stands before the group's first step.  Behind it came
            // four steps' weights and, between them, one buffer's DMA (kPer 2: just what this
            // wait leaves under way) or three.
            constexpr int kSteps = kTail ? std::max(0, std::min(2 * kPer, 2 * kPer - (T + 1 - std::max(0, 4 - kAhead)))) : 2 * kPer;
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kPer * kStage + kSteps * TNW) : "memory");
            lds_barrier();
            a_dma(c + 1 + 2 * kPer, b_cur);
            const int b_free = b_cur;
            b_cur = b_nxt;
            b_nxt = b_far;
            b_far = b_free;
            if constexpr (!kTail || T < 3) read(b_cur, 0, (T + 1) % 4, T == 3 ? q + 1 : q, fa);
        } else {
            read(at + kChunk, 0, T + 1, q, fa);
        }
        mma(fb, MBW - 1);
        if constexpr (kDeep) __builtin_amdgcn_sched_barrier(0);  // products stay in their step
    };
    static_assert(MBW % 2 == 0, "fragments alternate");
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    using I4 = std::integral_constant<int, 4>;
    auto next_scales = [&](int q, uint32_t (&nxt)[TNW]) {
#pragma unroll
        for (int tt = 0; tt < TNW; ++tt)
            nxt[tt] = __builtin_amdgcn_raw_buffer_load_b32(rs[tt], lane * 4, min(q, q1 - 1) * 256, kLoadReused);
        s_dma(q);
    };
    auto group = [&](auto e_c, auto tail_c, int q, const uint32_t (&cur)[TNW]) {
        step(I0{}, e_c, tail_c, q, cur);
        if (4 * q + 1 > clast) return;
        step(I1{}, e_c, tail_c, q, cur);
        if (4 * q + 2 > clast) return;
        step(I2{}, e_c, tail_c, q, cur);
        if (4 * q + 3 > clast) return;
        step(I3{}, e_c, tail_c, q, cur);
    };
    // A group with another behind it: no way out of it, so that the compiler's own waits
    // for weights count the loads of the one way through (else of the shortest).
    auto whole_group = [&](auto e_c, int q, const uint32_t (&cur)[TNW]) {
        step(I0{}, e_c, std::false_type{}, q, cur);
        step(I1{}, e_c, std::false_type{}, q, cur);
        step(I2{}, e_c, std::false_type{}, q, cur);
        step(I3{}, e_c, std::false_type{}, q, cur);
    };
    s_dma(q0);
#pragma unroll
    for (int tt = 0; tt < TNW; ++tt) wsc[tt] = __builtin_amdgcn_raw_buffer_load_b32(rs[tt], lane * 4, q0 * 256, kLoadReused);
    // the first wait finds kAhead chunks of weights and one buffer behind the second DMA
    a_dma(4 * q0, 0);
    a_dma(4 * q0 + kPer, kBuf);
    w_issue(I0{}, 4 * q0);
    w_issue(I1{}, 4 * q0 + 1);
    if constexpr (kAhead > 2) {
        w_issue(I2{}, 4 * q0 + 2);
        w_issue(I3{}, 4 * q0 + 3);
    }
    a_dma(4 * q0 + 2 * kPer, 2 * kBuf);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kPer * kStage + kAhead * TNW) : "memory");  // the first DMA
    lds_barrier();
    read(b_cur, 0, 0, q0, fa);
    int q = q0;
    if constexpr (kDeep) {
        for (; q + 2 < q1; q += 2) {
            next_scales(q + 1, wsn);
            whole_group(I0{}, q, wsc);
            next_scales(q + 2, wsc);
            whole_group(I4{}, q + 1, wsn);
        }
        if (q + 2 == q1) {
            next_scales(q + 1, wsn);
            whole_group(I0{}, q, wsc);
            group(I4{}, std::true_type{}, q + 1, wsn);
        } else {
            group(I0{}, std::true_type{}, q, wsc);
        }
    } else {
        for (; q + 1 < q1; q += 2) {
            next_scales(q + 1, wsn);
            group(I0{}, std::false_type{}, q, wsc);
            next_scales(q + 2, wsc);
            group(I0{}, std::false_type{}, q + 1, wsn);
        }
        if (q < q1) group(I0{}, std::true_type{}, q, wsc);
    }
    // no DMA may still write this workgroup's LDS after it exits
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    if (P) {
        const int MB16 = (p.M + 15) / 16;
#pragma unroll
        for (int mb = 0; mb < MBW; ++mb) {
            const int b = m0 / 16 + wm * MBW + mb;
            if (b >= MB16) continue;
#pragma unroll
            for (int tt = 0; tt < TNW; ++tt) {
                // weight tiles in the order [output tile][gate, up]
                const int o = t0 + (p.up ? tt % (TNW / 2) : tt), ot = p.up ? 2 * out_tiles : out_tiles;
                const int at = p.up ? 2 * o + tt / (TNW / 2) : o;
                if (o < out_tiles) P[(((int64_t)ks * MB16 + b) * ot + at) * 64 + lane] = acc[tt][mb];
            }
        }
        return;
    }
#pragma unroll
    for (int mb = 0; mb < MBW; ++mb) {
        const int m = m0 + (wm * MBW + mb) * 16 + r;
#pragma unroll
        for (int tt = 0; tt < TNW; ++tt) {
            if (p.out_type == 2 && tt % 2) continue;
            if (p.up && tt >= TNW / 2) continue;
            mx8_finish(p, [&](int y) { return acc[y < TNW ? y : 0][mb]; }, tt, TNW / 2, m, t0 + tt, j);
        }
    }
}

// The partial sums of S shares of K, added in the order of the shares; one wave for
// 16 rows and one output tile (8-bit output: two).  All loads of a wave are under way
// at once.  256 x 8192 in four shares: 7.4 us, 5 TB/s; a last workgroup that adds in
// the product itself needs the shares' tiles in turn, and took twice the product's time.
template <int S>
__global__ __launch_bounds__(256) void reduce_mx8(Mx8Gemm p, const f32x4* __restrict__ P) {
    const int lane = threadIdx.x & 63, r = lane & 15, j = lane >> 4;
    const int unit = p.out_type == 2 ? 2 : 1;
    const int out_tiles = p.out_type == 2 ? p.cols_pad / 16 : (p.cols + 15) / 16;
    const int MB16 = (p.M + 15) / 16, ot = p.up ? 2 * out_tiles : out_tiles;
    const int t = (blockIdx.x * 4 + threadIdx.x / 64) * unit, b = blockIdx.y;
    if (t >= out_tiles) return;
    const int64_t plane = (int64_t)MB16 * ot * 64;
    auto sum = [&](int y) {  // y = tile, or gated: tile + (up ? half : 0) with half = 2
        const int at = p.up ? 2 * (t + y % 2) + y / 2 : t + y;
        const f32x4* src = P + ((int64_t)b * ot + at) * 64 + lane;
        f32x4 x[S];
#pragma unroll
        for (int k = 0; k < S; ++k) x[k] = src[k * plane];
        f32x4 v = x[0];
#pragma unroll
        for (int k = 1; k < S; ++k) v += x[k];
        return v;
    };
    mx8_finish(p, sum, 0, 2, b * 16 + r, t, j);
}

}  // namespace fp4
