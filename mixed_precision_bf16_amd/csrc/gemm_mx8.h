// Products of 8-bit activations with MXFP4 weights on the scaled matrix cores
// (include/fp4gemm.h, section "8-bit activations").
//
//   Y[m][n] = alpha * sum_k a[m][k] w[n][k]
//   a = E4M3 code * 2^(scale - 127), one scale for 32 k; w the same with E2M1
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 weight rows by 16
// activation rows over 128 k.  Operand layout (checked on the device), lane =
// 16 j + r: row r of either operand; FP4: k = 32 j .. 32 j + 31 (the native
// weight layout, repack.cpp); FP8: k = 16 j .. 16 j + 15 and 64 + 16 j ..
// 64 + 16 j + 15; either scale: block j of the row's four.  The result: rows n =
// 4 j .. 4 j + 3, column m = r.
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
__device__ __forceinline__ f32x4 mfma_fp4_fp8(const i32x8& w, const i32x8& a, const f32x4& c, uint32_t ws,
                                              uint32_t as) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 4, 0, 0, (int)ws, 0, (int)as);
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

// Small m.  A workgroup of NWK waves takes TN weight tiles (gated: TN / 2 gate
// tiles and the TN / 2 up tiles of the same columns) and 16 MB rows of A; each
// wave streams its share of K straight into registers, PD chunks ahead; the waves'
// sums meet in LDS, in the order of the waves.
template <int MB, int TN, int NWK, int PD>
__global__ __launch_bounds__(64 * NWK) void gemm_mx8_stream(Mx8Gemm p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds_raw[];
    f32x4* lds = reinterpret_cast<f32x4*>(lds_raw);
    const int lane = threadIdx.x & 63, r = lane & 15, j = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = blockIdx.y * 16 * MB;
    const int tiles = p.up ? TN / 2 : TN;  // output tiles of the workgroup
    const int t0 = blockIdx.x * tiles;
    const int c0 = (int)((int64_t)p.chunks * wave / NWK), c1 = (int)((int64_t)p.chunks * (wave + 1) / NWK);

    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a, (uint32_t)p.M * (uint32_t)p.KA);
    const __amdgpu_buffer_rsrc_t rsa = make_rsrc(p.as, (uint32_t)p.M * (uint32_t)(p.KA / 32));
    __amdgpu_buffer_rsrc_t rw[TN], rs[TN];
#pragma unroll
    for (int tt = 0; tt < TN; ++tt) {
        int t = t0 + tt;
        if (p.up) t = tt < TN / 2 ? min(t, p.up - 1) : p.up + t0 + tt - TN / 2;
        t = min(t, p.NT - 1);
        rw[tt] = make_rsrc(p.wq + (size_t)t * p.KB * 1024, (uint32_t)p.KB * 1024u);
        rs[tt] = make_rsrc(p.sq + (size_t)t * p.KB * 64, (uint32_t)p.KB * 64u);
    }
    uint32_t aoff[MB], soff[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        aoff[mb] = (uint32_t)(m0 + mb * 16 + r) * (uint32_t)p.KA + 16 * j;
        soff[mb] = (uint32_t)(m0 + mb * 16 + r) * (uint32_t)(p.KA / 32);
    }
    u32x4 w[PD][TN], alo[PD][MB], ahi[PD][MB];
    uint32_t ws[PD][TN], as[PD][MB];
    auto issue = [&](int s, int c) {
#pragma unroll
        for (int tt = 0; tt < TN; ++tt) {
            w[s][tt] = __builtin_amdgcn_raw_buffer_load_b128(rw[tt], lane * 16, c * 1024, kLoadStream);
            ws[s][tt] = __builtin_amdgcn_raw_buffer_load_b32(rs[tt], lane * 4, (c >> 2) * 256, kLoadReused);
        }
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            alo[s][mb] = __builtin_amdgcn_raw_buffer_load_b128(ra, aoff[mb] + c * 128, 0, kLoadReused);
            ahi[s][mb] = __builtin_amdgcn_raw_buffer_load_b128(ra, aoff[mb] + c * 128 + 64, 0, kLoadReused);
            as[s][mb] = __builtin_amdgcn_raw_buffer_load_b32(rsa, soff[mb] + c * 4, 0, kLoadReused);
        }
    };
    f32x4 acc[TN][MB];
#pragma unroll
    for (int tt = 0; tt < TN; ++tt)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) acc[tt][mb] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](int s, int c) {
        const int shift = 8 * (c & 3);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            const i32x8 a = fp8_operand(alo[s][mb], ahi[s][mb]);
            const uint32_t sc = as[s][mb] >> (8 * j);
#pragma unroll
            for (int tt = 0; tt < TN; ++tt)
                acc[tt][mb] = mfma_fp4_fp8(fp4_operand(w[s][tt]), a, acc[tt][mb], ws[s][tt] >> shift, sc);
        }
    };
#pragma unroll
    for (int s = 0; s < PD; ++s)
        if (c0 + s < c1) issue(s, c0 + s);
    int c = c0;
    for (; c + 2 * PD <= c1; c += PD) {
#pragma unroll
        for (int s = 0; s < PD; ++s) {
            compute(s, c + s);
            issue(s, c + s + PD);
        }
    }
#pragma unroll
    for (int s = 0; s < 2 * PD - 1; ++s) {
        if (c + s < c1) compute(s % PD, c + s);
        if (c + s + PD < c1 && s < PD) issue(s % PD, c + s + PD);
    }

    // the waves' sums
#pragma unroll
    for (int tt = 0; tt < TN; ++tt)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) lds[((wave * TN + tt) * MB + mb) * 64 + lane] = acc[tt][mb];
    __syncthreads();
    auto total = [&](int tt, int mb) {
        f32x4 v = lds[(tt * MB + mb) * 64 + lane];
#pragma unroll
        for (int k = 1; k < NWK; ++k) v += lds[((k * TN + tt) * MB + mb) * 64 + lane];
        return v * p.alpha;
    };
    auto result = [&](int tt, int mb) {
        f32x4 v = total(tt, mb);
        if (p.up) {
            const f32x4 u = total(tt + TN / 2, mb);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = gated(v[e], u[e], p.gate);
        }
        return v;
    };
    const int unit = p.out_type == 2 ? 2 : 1, items = tiles / unit * MB;
    for (int i = wave; i < items; i += NWK) {
        const int tt = i / MB * unit, mb = i % MB, m = m0 + mb * 16 + r;
        const f32x4 v = result(tt, mb);
        if (unit == 1) mx8_store16(p, v, m, t0 + tt, j);
        else mx8_store8(p, v, result(tt + 1, mb), m, t0 + tt, j);
    }
}

}  // namespace fp4
