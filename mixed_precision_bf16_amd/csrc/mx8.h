// 8-bit activations (include/fp4gemm.h, section "8-bit activations"): E4M3
// codes with one E8M0 scale for each 32 of them along a row.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "mx8_plan.h"

namespace fp4 {

// Scale byte of a block whose largest finite magnitude is amax (FP32 bits): the
// least power of two with amax / 2^(byte - 127) <= 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t mx8_scale_byte(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = int(b >> 23) - 8 + int((b & 0x007FFFFFu) > 0x00600000u);
    return (uint32_t)max(e, 0);
}

// Codes of eight elements under scale byte sb.  The gfx950 convert divides by
// its scale operand and rounds to nearest even, subnormal codes included; it
// gives NaN codes to NaN and infinite elements (E4M3 has no infinity), and no
// finite element of the block exceeds 448 scales.
__device__ __forceinline__ u32x2 mx8_codes(const float (&x)[8], uint32_t sb) {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    const float s = __uint_as_float(sb << 23);
    s16x2 lo = {0, 0}, hi = {0, 0};
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, x[0], x[1], s, false);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, x[2], x[3], s, true);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, x[4], x[5], s, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, x[6], x[7], s, true);
    return u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}

// Largest finite magnitude of eight elements; NaN elements are quiet.
__device__ __forceinline__ float mx8_amax(const float (&x)[8]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
    if (!(a < __builtin_inff())) {  // rare: an infinity among them
        a = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = fabsf(x[i]) < __builtin_inff() ? fmaxf(a, fabsf(x[i])) : a;
    }
    return a;
}

// Eight 16-bit elements that are read once: the nontemporal hint.
__device__ __forceinline__ u32x4 load_once(const uint16_t* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}

// Two 16-bit elements to FP32.
template <int ACT>
__device__ __forceinline__ void widen2(uint32_t p, float& lo, float& hi) {
    if constexpr (ACT == 0) {
        lo = __uint_as_float(p << 16);
        hi = __uint_as_float(p & 0xFFFF0000u);
    } else {
        lo = (float)__builtin_bit_cast(_Float16, (uint16_t)p);
        hi = (float)__builtin_bit_cast(_Float16, (uint16_t)(p >> 16));
    }
}

// Eight 16-bit elements to FP32 and back.
template <int ACT>
__device__ __forceinline__ void widen8(const u32x4& v, float (&x)[8]) {
    widen2<ACT>(v.x, x[0], x[1]);
    widen2<ACT>(v.y, x[2], x[3]);
    widen2<ACT>(v.z, x[4], x[5]);
    widen2<ACT>(v.w, x[6], x[7]);
}

template <int ACT>
__device__ __forceinline__ u32x4 narrow8(const float (&x)[8]) {
    return u32x4{pack_out<ACT>(x[0], x[1]), pack_out<ACT>(x[2], x[3]), pack_out<ACT>(x[4], x[5]),
                 pack_out<ACT>(x[6], x[7])};
}

}  // namespace fp4
