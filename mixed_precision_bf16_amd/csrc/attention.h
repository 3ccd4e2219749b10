// Attention over the FP4 key/value cache (include/fp4gemm.h, fp4_attention).
//
//   s_j = scale * q . k_j over the keys j that the query token sees,
//   m = max_j s_j,  p_j = exp(s_j - m),  l = sum_j p_j (+ exp(sink - m)),
//   out = sum_j p_j v_j / l,  lse = m + ln l.
//
// Both products run on the 16-bit matrix cores with FP32 accumulation, on
// keys and values dequantized in registers: FP16 for NVFP4 caches and for FP16
// activations, BF16 for MXFP4 caches with BF16 activations (E8M0 scales need
// its range).  Every NVFP4 code x scale product is exact in FP16.  An E8M0
// scale takes alpha's exponent e = floor(log2 alpha) along into the convert, so
// that the 16-bit values have the size of the rows themselves, whatever alpha
// is, and only alpha / 2^e, in [1, 2), is applied in FP32: exact in BF16, and in
// FP16 for every block whose largest element is at least 2^-20 and below 2^16.
// (In FP16 the codes of smaller blocks round to multiples of 2^-24, the step of
// FP16 rows themselves, and those of larger ones saturate.)
// The softmax runs in FP32 in base 2 with one pass over the keys: a running
// maximum m and sum l per query row.  Rows of the accumulators are rescaled
// only when a score exceeds the running maximum by more than kSlack binary
// orders, which a wave decides together: probabilities stay below
// 2^(kBias + kSlack), in range for FP16, and kBias moves the point where FP16
// probabilities vanish to 2^-(24 + kBias) of the largest one.  The one rounding
// below 32 bits before the output's is that of the probabilities to the
// matrix-core type (half a step: 2^-11, with BF16 2^-8, the size of the output's
// own); their sum takes them unrounded, so that the log-sum-exp keeps FP32.
#pragma once
#include <type_traits>
#include <utility>

#include "kv_layout.h"

namespace fp4 {

constexpr float kBias = 8.0f, kSlack = 7.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3.402823466e38f;  // running maximum before the first visible key: no score is lower
// Scores from here on (base 2) are taken relative to the running maximum before
// the exponential's own multiply-add, see far_scores.
constexpr float kFar = 0x1p20f;
constexpr int kAttnThreads = 256, kAttnWaves = 4;
// Waves per SIMD that the streaming kernel's registers allow; the GPU then holds
// 256 times as many of its workgroups (a workgroup has a wave on each SIMD).
constexpr int attn_waves(int D, int MT) { return D * MT <= 64 ? 4 : D * MT <= 128 ? 3 : D * MT <= 256 ? 2 : 1; }
// Units that the fixed cost of an item is worth (1: windowed layer 14.7 us, 3:
// 11.0, 5: 10.9; 64 sequences 76, 75, 77).
constexpr int kItemCost = 3;
constexpr int kAhead = 4;              // fragments of LDS read ahead by the tiled kernel
constexpr int kTeam = 16;              // shares of an item that are joined at a time
constexpr int kUnitTiles = kAttnWaves;  // tiles of a work unit: one per wave

// Matrix-core type of a format and activation type (0: BF16, 1: FP16).
constexpr int attn_type(int fmt, int act) { return fmt == 0 || act == 1 ? 1 : 0; }

struct AttnArgs {
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* q_offsets;  // null: every sequence has q_each query tokens
    const float* sinks;
    int64_t q_ts, q_hs, o_ts, o_hs, table_stride;
    int batch, q_rows, q_each, q_heads, group;
    int splits;                // tiled kernel: most shares of an item
    int max_keys;              // columns of the page table * page_size
    int window, causal;
    uint64_t tpp_magic;        // ceil(2^36 / tiles_per_page): the page of tile t < 2^26 is t * magic >> 36
    int k_exp, v_exp;          // MXFP4: exponents of k_alpha and v_alpha, which the block scales take along; else 0
    float scale;               // scale * k_alpha / 2^k_exp * log2(e)
    float v_alpha;             // v_alpha / 2^v_exp
    float inv_group;           // 1 / group
    int grid;                  // workgroups; in the streaming kernel as many as the GPU holds
    unsigned long long tag;    // of the arrival words
    float* ws_o;               // [2 * grid][rows][D]; tiled kernel: [grid][D / 4][rows][4] and so on
    float* ws_ml;              // [2 * grid][rows][2]
    unsigned long long* words; // [2 * grid]
};

// ------------------------------------------------------------ arrival words
// As split_arrive (the word is (launch tag, count), any other tag counts as 0,
// the last arrival leaves 0), with the tag installed well before the arrival,
// under the shadow of the first loads: the arrival itself is then one atomic.
// Every workgroup claims its words before it arrives, so they carry the tag.
__device__ __forceinline__ void claim_word(unsigned long long* w, unsigned long long seen, unsigned long long tag) {
    if (!carries_tag(seen, tag))  // the exchange fails only if another workgroup has installed the tag
        __hip_atomic_compare_exchange_strong(w, &seen, tag, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool arrive_word(unsigned long long* w, int count, unsigned long long tag) {
    const uint32_t n =
        (uint32_t)(__hip_atomic_fetch_add(w, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) - tag) + 1u;
    if (n == (uint32_t)count) __hip_atomic_store(w, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return n == (uint32_t)count;
}
__device__ __forceinline__ unsigned long long peek_word(unsigned long long* w) {
    return __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ------------------------------------------------------------ one key tile
template <int FMT, int D>
struct TileRegs {
    using L = KvTile<FMT, D>;
    u32x4 k[L::F], v[L::F];
    uint32_t ks[(L::kKsLane + 3) / 4];
    u32x2 vs[L::C];
};

// Offset of lane (r, j)'s key scales in their section: lanes j of one scale
// block (two, where a block is longer than a lane's elements) share them.
template <int FMT, int D>
__device__ __forceinline__ int key_scale_lane(int r, int j) {
    using L = KvTile<FMT, D>;
    return (j * L::KD / (L::G > L::KD ? L::G : L::KD) * 16 + r) * L::kKsLane;
}

// kOnce: codes that one workgroup reads once (a single row block, decode) go
// past the caches; with several row blocks they are read again.  64 sequences
// of 16 .. 8192 keys 75 -> 65 us, one of 131071 39 -> 36 us; four query tokens
// (two row tiles) would lose 3 %.
template <bool kOnce>
__device__ __forceinline__ u32x4 load_codes(const uint8_t* p) {
    if constexpr (kOnce) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    else return *reinterpret_cast<const u32x4*>(p);
}

template <int FMT, int D, bool kOnce>
__device__ __forceinline__ void load_tile(TileRegs<FMT, D>& t, const uint8_t* __restrict__ tile, int lane) {
    using L = KvTile<FMT, D>;
    const int r = lane & 15, j = lane >> 4;
#pragma unroll
    for (int f = 0; f < L::F; ++f) t.k[f] = load_codes<kOnce>(tile + f * 1024 + lane * 16);
#pragma unroll
    for (int f = 0; f < L::F; ++f) t.v[f] = load_codes<kOnce>(tile + L::kCodes + f * 1024 + lane * 16);
    const uint8_t* ks = tile + L::kKs + key_scale_lane<FMT, D>(r, j);
    if constexpr (L::kKsLane == 2) t.ks[0] = *reinterpret_cast<const uint16_t*>(ks);
    else if constexpr (L::kKsLane == 4) t.ks[0] = *reinterpret_cast<const uint32_t*>(ks);
    else {
        const u32x2 w = *reinterpret_cast<const u32x2*>(ks);
        t.ks[0] = w.x;
        t.ks[1] = w.y;
    }
#pragma unroll
    for (int c = 0; c < L::C; ++c) {
        const int g = c * (L::CH / L::G) + r * L::VD / L::G;
        t.vs[c] = *reinterpret_cast<const u32x2*>(tile + L::kVs + (g * 4 + j) * 8);
    }
}

// E8M0 byte b, times 2^e -> the convert's FP32 scale operand, of which it takes
// the exponent field (0 stands for 2^-127).  The scale saturates at the largest
// one whose products stay finite in the matrix-core type (2^125 in BF16, 2^13
// in FP16), so that a key that was written as an infinity cannot reach the
// queries that do not see it as 0 x Inf.
template <int CT>
__device__ __forceinline__ float e8m0_scale(uint32_t b, int e) {
    return __uint_as_float((uint32_t)min(max((int)b + e, 0), CT == 0 ? 252 : 140) << 23);
}

__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

template <int SEL>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, SEL));
}
template <int SEL>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, SEL));
}
template <int CT, int SEL>
__device__ __forceinline__ uint32_t codes16(uint32_t w, float s) {
    if constexpr (CT == 1) return codes_f16<SEL>(w, s);
    else return codes_bf16<SEL>(w, s);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, f16x2 s) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) * s);
}

// Eight codes times byte B of the lane's key scales (E8M0: and 2^e).
template <int FMT, int CT, int B, int N>
__device__ __forceinline__ u32x4 key_frag(uint32_t w, const uint32_t (&ks)[N], int e) {
    u32x4 o;
    if constexpr (FMT == 0) {
        // two E4M3 scales -> FP16 (exact), one of them for both halves; code x scale is exact in FP16
        const f16x2 p = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)ks[B / 4], 1.0f, (B & 2) != 0);
        const f16x2 s = (B & 1) ? f16x2{p.y, p.y} : f16x2{p.x, p.x};
        o.x = mul_f16x2(codes_f16<0>(w, 1.0f), s);
        o.y = mul_f16x2(codes_f16<1>(w, 1.0f), s);
        o.z = mul_f16x2(codes_f16<2>(w, 1.0f), s);
        o.w = mul_f16x2(codes_f16<3>(w, 1.0f), s);
    } else {
        const float s = e8m0_scale<CT>((ks[B / 4] >> (8 * (B % 4))) & 0xFFu, e);
        o.x = codes16<CT, 0>(w, s);
        o.y = codes16<CT, 1>(w, s);
        o.z = codes16<CT, 2>(w, s);
        o.w = codes16<CT, 3>(w, s);
    }
    return o;
}

// Key fragment of tokens 16 U .. , chunk CK, product step S (elements
// CH CK + KD j + 8 S .. + 7 of lane (r, j)).
template <int FMT, int CT, int D, int U, int CK, int S>
__device__ __forceinline__ u32x4 key_step(const TileRegs<FMT, D>& t, int e) {
    using L = KvTile<FMT, D>;
    constexpr int byte = CK * 2 * L::KG + U * L::KG + (S * 8 / L::G) % L::KG;
    if constexpr (D == 64) return key_frag<FMT, CT, byte>(t.k[0][2 * U + S], t.ks, e);
    else return key_frag<FMT, CT, byte>(t.k[CK * 2 + U][S], t.ks, e);
}

// Two d-fragments (elements VD r + 2 Q, + 1 of chunk CK) of O^T's left operand:
// lane (r, j) supplies tokens 4 j .. 4 j + 3 and 16 + 4 j .. .
template <int FMT, int CT, int D, int CK, int Q>
__device__ __forceinline__ void value_frags(const TileRegs<FMT, D>& t, int e, u32x4& even, u32x4& odd) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        uint32_t a[4];  // elements 2 Q, 2 Q + 1 of the four tokens
        const uint32_t sb = t.vs[CK][u];
        if constexpr (FMT == 0) {
            if constexpr (D == 64) {
                a[0] = codes_f16<Q>(t.v[0][2 * u], 1.0f);
                a[1] = codes_f16<Q + 2>(t.v[0][2 * u], 1.0f);
                a[2] = codes_f16<Q>(t.v[0][2 * u + 1], 1.0f);
                a[3] = codes_f16<Q + 2>(t.v[0][2 * u + 1], 1.0f);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = codes_f16<Q>(t.v[CK * 2 + u][i], 1.0f);
            }
            const f16x2 s01 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)sb, 1.0f, false);
            const f16x2 s23 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)sb, 1.0f, true);
            even[2 * u] = mul_f16x2(low_halves(a[0], a[1]), s01);
            even[2 * u + 1] = mul_f16x2(low_halves(a[2], a[3]), s23);
            odd[2 * u] = mul_f16x2(high_halves(a[0], a[1]), s01);
            odd[2 * u + 1] = mul_f16x2(high_halves(a[2], a[3]), s23);
        } else {
            float s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = e8m0_scale<CT>((sb >> (8 * i)) & 0xFFu, e);
            if constexpr (D == 64) {
                a[0] = codes16<CT, Q>(t.v[0][2 * u], s[0]);
                a[1] = codes16<CT, Q + 2>(t.v[0][2 * u], s[1]);
                a[2] = codes16<CT, Q>(t.v[0][2 * u + 1], s[2]);
                a[3] = codes16<CT, Q + 2>(t.v[0][2 * u + 1], s[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = codes16<CT, Q>(t.v[CK * 2 + u][i], s[i]);
            }
            even[2 * u] = low_halves(a[0], a[1]);
            even[2 * u + 1] = low_halves(a[2], a[3]);
            odd[2 * u] = high_halves(a[0], a[1]);
            odd[2 * u + 1] = high_halves(a[2], a[3]);
        }
    }
}

// Zero the scales of the value tokens at or past `end` (a slot that no token
// was written to holds anything: its probability is 0, and 0 x NaN is NaN).
template <int FMT, int D>
__device__ __forceinline__ void clear_values(TileRegs<FMT, D>& t, int tok0, int j, int end) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int left = end - (tok0 + 16 * u + 4 * j);  // tokens of this quad that exist
        const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
#pragma unroll
        for (int c = 0; c < KvTile<FMT, D>::C; ++c) t.vs[c][u] &= keep;
    }
}

// ------------------------------------------------------------ query rows
// Row of query-row block rb (R rows): token i and head g of the group.
template <int FMT, int ACT, int D>
struct QueryRow {
    using L = KvTile<FMT, D>;
    static constexpr int kFrags = D / 32;
    // Raw fragments of one row's query for lane (r, j).
    __device__ static __forceinline__ void load(u32x4 (&f)[kFrags], const uint16_t* __restrict__ row, bool valid,
                                                int j) {
        constexpr int S = L::KD / 8;
#pragma unroll
        for (int c = 0; c < L::C; ++c)
#pragma unroll
            for (int s = 0; s < S; ++s) {
                f[c * S + s] = u32x4{0u, 0u, 0u, 0u};
                if (valid) f[c * S + s] = *reinterpret_cast<const u32x4*>(row + c * L::CH + L::KD * j + 8 * s);
            }
    }
    // Converts them to the matrix-core type; returns the factor that turns the
    // accumulated products into base-2 scores (kept normal: a factor of 0
    // would turn a hidden key's -Inf into NaN).
    // A row lies in four lanes 16 apart (N = D / 32 fragments), or in two 32 apart.
    template <int N>
    __device__ static __forceinline__ float convert(u32x4 (&f)[N], float scale) {
        if constexpr (attn_type(FMT, ACT) == 1 && ACT == 0) {
            // BF16 queries on the FP16 matrix cores: a power of two brings the
            // row's largest element to 2^13 .. 2^14, so that every element
            // down to 2^-27 of it converts exactly.
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t p = f[i][e];
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(p << 16)), fabsf(__uint_as_float(p & 0xFFFF0000u))));
                }
            if constexpr (N == kFrags) top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127);
            const float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t p = f[i][x];
                    f[i][x] = pack_out<1>(__uint_as_float(p << 16) * up, __uint_as_float(p & 0xFFFF0000u) * up);
                }
            scale *= __uint_as_float((uint32_t)(127 - 13 + e) << 23);
        }
        return fmaxf(scale, 0x1p-126f);
    }
};

struct RowRange {
    int lo, hi;  // keys [lo, hi) that the row sees
};
// Keys that query token i of n sees in a sequence of `len` keys.
__device__ __forceinline__ RowRange row_range(int i, int n, int len, int causal, int window) {
    RowRange x{0, len};
    if (causal) {
        x.hi = max(0, len - n + i + 1);
        if (window > 0) x.lo = max(0, x.hi - window);
    }
    return x;
}

// ------------------------------------------------------------ streaming kernel
// Few query rows a sequence (decode, drafted tokens), any number of keys.
// An item is a (sequence, block of 16 MT query rows, KV head); its keys are cut
// into units of 128 (one tile a wave).  All units, with kItemCost places for
// the fixed cost of each item, are numbered item by item and dealt in equal
// contiguous ranges to the workgroups that the GPU holds, so that long and
// short sequences load it evenly, whatever the lengths on the device are.  An
// item that falls into several workgroups is joined by the one that arrives
// last, from the FP32 partial sums of all, in their order.
//
// Bound by HBM while it streams: up to 12 waves a CU, each with the next tile's
// 4.6 KB under way (64 sequences of 4000 keys of head size 256, 590 MB: 6.0 TB/s
// over the whole kernel); around that a workgroup spends 1.3 us on the scan of
// the sequences, 1.5 us to its first tile, 1 us to join its waves and 2 us to
// keep a partial sum and arrive.  Measured (MI355X, kernel time, 64 query and 8
// KV heads of 128): 64 sequences of 16 .. 8192 keys, NVFP4, 60 us (304 MB, 5.1
// TB/s); one sequence of 131071 keys, MXFP4, 35 us (143 MB, 4.1 TB/s; its 94
// partial sums a head are joined in two stages of sixteen, which costs 6 us
// against 11 us in one); one of 1000 keys 9 us, latency; four query tokens each
// over 16 sequences of 1000 .. 5000 keys 29 us, latency: two row tiles leave
// registers for two waves a SIMD, 1.3 are resident in the mean, the vector units
// are busy 34 % of the time and the matrix cores 9 %.  Tried: shares of equal
// length dispatched one a workgroup (77 us for the first case, where this took
// 75) and drawn from an atomic counter (115 us and more: all workgroups queue at it).
struct Seq {
    int q0, n;       // first query row, query tokens
    int len;         // keys
    int t0, t1;      // tiles [t0, t1) that some query sees
    int units;       // of one item
    int blocks;      // row blocks; 0 for a sequence without queries
};

template <int R>
__device__ __forceinline__ Seq sequence_from(const AttnArgs& a, int q0, int n, int len) {
    Seq x;
    x.q0 = q0;
    x.n = n;
    x.len = len;
    const RowRange f = row_range(0, n, len, a.causal, a.window);
    x.t0 = f.lo / kKvTile;
    x.t1 = max((len + kKvTile - 1) / kKvTile, x.t0);
    x.units = max(1, (x.t1 - x.t0 + kUnitTiles - 1) / kUnitTiles);
    x.blocks = (n * a.group + R - 1) / R;
    return x;
}

// Sequence b; one without queries for b past the batch.  `bad` is set where the
// query offsets decrease: their sequences would overlap, and the sums over all
// sequences that the host has bounded would not hold.
template <int R>
__device__ __forceinline__ Seq sequence_of(const AttnArgs& a, int b, bool& bad) {
    if (b >= a.batch) return Seq{};
    int q0 = b * a.q_each, n = a.q_each;
    if (a.q_offsets) {
        q0 = min(max(a.q_offsets[b], 0), a.q_rows);
        n = min(max(a.q_offsets[b + 1], 0), a.q_rows) - q0;
        bad |= n < 0;
        n = max(n, 0);
    }
    return sequence_from<R>(a, q0, n, min(max(a.seq_lens[b], 0), a.max_keys));
}

// Sum over lanes 0 .. lane.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15 into rows 1, 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast 31 into rows 2, 3
    return v;
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// Probabilities are exp2(s fac + (kBias - m)) with one multiply-add.  The running
// maximum m is the rounded product of the highest s: what the rounding took, and
// that of kBias - m, up to 2^-24 |m|, multiplies all probabilities of the row by
// one power of two, which the sum divides out.  Past 2^24 that factor would leave
// FP16's range, and then FP32's.  So where a row of the wave has |m| >= kFar, a
// branch that is not taken otherwise, scores become round(s fac) - m (0 at the
// maximum) first, and fac 1 and m 0 follow them.  True if some row is there; called
// when m has changed.
__device__ __forceinline__ bool far_scores(float m) { return __any(fabsf(m) >= kFar && m != kNoMax); }
__device__ __forceinline__ float near_score(float s, float fac, float m) {
#pragma clang fp contract(off)
    const float x = s * fac;
    return x - m;
}

// Final value factor and log-sum-exp of a row from its running maximum m,
// biased sum l and sink.
__device__ __forceinline__ float finish_row(float m, float l, bool has_sink, float sink, float& lse) {
    float top = m;
    if (has_sink) top = fmaxf(m, sink * kLog2e);
    const float f = exp2_(m - top - kBias);
    float sum = l * f;
    if (has_sink) sum += exp2_(sink * kLog2e - top);
    if (sum == 0.0f) {  // no key is seen, and the sink, if any, is below the range of base 2
        lse = has_sink ? sink : -__builtin_inff();
        return 0.0f;
    }
    lse = (top + __builtin_amdgcn_logf(sum)) * kLn2;
    return f / sum;
}

template <int FMT, int ACT, int D, int MT>
__global__ __launch_bounds__(kAttnThreads, attn_waves(D, MT)) void attention_stream(AttnArgs a, KvArgs cache) {
    using L = KvTile<FMT, D>;
    constexpr int CT = attn_type(FMT, ACT);
    constexpr int R = 16 * MT, F = D / 32, S = L::KD / 8, OT = D / 16;
    constexpr int kPad = D + 4;  // floats of a row in LDS
    __shared__ float lds_o[kAttnWaves][16][kPad];
    __shared__ float lds_m[kAttnWaves][16], lds_l[kAttnWaves][16];
    __shared__ int lds_scan[kAttnWaves];
    __shared__ int lds_found[5];
    __shared__ int lds_last;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, j = lane >> 4;
    const int kv_heads = cache.kv_heads;

    // ---- units of all sequences, and the shares of each
    auto scan = [&](int u, int& sum) {  // exclusive prefix of u over the workgroup, and its sum
        int p = wave_scan(u);
        __syncthreads();
        if (lane == 63) lds_scan[wave] = p;
        __syncthreads();
        p -= u;
        sum = 0;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) {
            p += w < wave ? lds_scan[w] : 0;
            sum += lds_scan[w];
        }
        return p;
    };
    // A position is a unit or one of the kItemCost places before an item's units.
    auto cost = [&](const Seq& x) { return (x.units + kItemCost) * x.blocks * kv_heads; };
    bool bad_offsets = false;
    const Seq own = sequence_of<R>(a, threadIdx.x, bad_offsets);
    const int own_cost = cost(own);
    int total;
    const int own_first = scan(own_cost, total);
    for (int base = kAttnThreads; base < a.batch; base += kAttnThreads) {
        int sum;
        scan(cost(sequence_of<R>(a, base + threadIdx.x, bad_offsets)), sum);
        total += sum;
    }
    if (a.q_offsets && __syncthreads_or(bad_offsets)) return;  // nothing is written
    const int per = (total + a.grid - 1) / a.grid;
    const int begin = blockIdx.x * per;  // grid * per < 2^31 (checked on the host)
    if (begin >= total) return;
    const int end = min(begin + per, total);

    // ---- the sequence that position `begin` lies in
    auto found = [&](const Seq& x, int b, int first) {
        lds_found[0] = b;
        lds_found[1] = x.q0;
        lds_found[2] = x.n;
        lds_found[3] = x.len;
        lds_found[4] = first;
    };
    if (a.batch <= kAttnThreads) {
        if (begin >= own_first && begin < own_first + own_cost) found(own, threadIdx.x, own_first);
    } else {
        for (int base = 0, before = 0; before <= begin; base += kAttnThreads) {  // ends: begin < total
            const Seq x = sequence_of<R>(a, base + threadIdx.x, bad_offsets);
            const int n = cost(x);
            int sum;
            const int first = before + scan(n, sum);
            if (begin >= first && begin < first + n) found(x, base + threadIdx.x, first);
            before += sum;
        }
    }
    __syncthreads();
    int b = __builtin_amdgcn_readfirstlane(lds_found[0]);
    int seq_first = __builtin_amdgcn_readfirstlane(lds_found[4]);
    Seq it = sequence_from<R>(a, __builtin_amdgcn_readfirstlane(lds_found[1]),
                              __builtin_amdgcn_readfirstlane(lds_found[2]),
                              __builtin_amdgcn_readfirstlane(lds_found[3]));
    int item = (begin - seq_first) / (it.units + kItemCost);

    for (;; ++item) {
        while (item >= it.blocks * kv_heads) {  // the next sequence that has work
            seq_first += cost(it);
            if (seq_first >= end) return;
            it = sequence_of<R>(a, ++b, bad_offsets);  // positions remain, so there is one
            item = 0;
        }
        const int unit0 = seq_first + item * (it.units + kItemCost) + kItemCost;  // position of the item's first unit
        const int u0 = max(begin - unit0, 0), u1 = min(end - unit0, it.units);
        if (unit0 >= end) return;
        if (u0 >= u1) continue;
        const int rb = item / kv_heads, h = item - rb * kv_heads;  // heads of a row block are neighbours
        const int wg0 = unit0 / per, parts = (unit0 + it.units - 1) / per - wg0 + 1, part = (int)blockIdx.x - wg0;
        // Partial sums: an item that goes on in the next workgroup is the last of
        // its first one (slot 2 wg0 + 1) and the first of the others.
        auto slot_of = [&](int p) { return 2 * (wg0 + p) + (p == 0 ? 1 : 0); };
        // words: the slot of the team's first part; for the teams, that of part 1
        const int p0 = part / kTeam * kTeam, teams = (parts + kTeam - 1) / kTeam, size = min(kTeam, parts - p0);
        unsigned long long *team_word = a.words + slot_of(p0), *teams_word = a.words + slot_of(1);
        unsigned long long seen_team = 0, seen_teams = 0;
        if (parts > 1 && threadIdx.x == 0) {
            seen_team = peek_word(team_word);
            seen_teams = peek_word(teams_word);
        }

        // ---- query rows and this wave's tiles.  The page numbers of the next
        // 64 tiles are one load (lane x: tile x), and the loads of a tile are
        // under way while the tile before it is computed.
        const int rows = min(R, it.n * a.group - rb * R);
        const int32_t* pages = a.page_table + (int64_t)b * a.table_stride;
        const int ta = it.t0 + u0 * kUnitTiles + wave;
        const int tb = min(it.t0 + u1 * kUnitTiles, it.t1);
        auto page_of = [&](int t) { return (int)(((uint64_t)(uint32_t)t * a.tpp_magic) >> 36); };
        auto load_pages = [&](int t) { return pages[page_of(max(0, min(t + kAttnWaves * lane, tb - 1)))]; };
        int window_pages = ta < tb ? load_pages(ta) : 0, window_first = ta;
        // row x of the block: token i0 + (x + g0) / group (below 2^11: exact in FP32)
        const int i0 = rb * R / a.group, g0 = rb * R - i0 * a.group;
        auto token_of = [&](int x) { return (int)(((float)(x + g0) + 0.5f) * a.inv_group); };
        u32x4 qf[MT][F];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const bool valid = 16 * mt + r < rows;
            const int di = token_of(16 * mt + r), i = i0 + di, g = 16 * mt + r + g0 - di * a.group;
            const uint16_t* src = a.q + (int64_t)(it.q0 + i) * a.q_ts + (int64_t)(h * a.group + g) * a.q_hs;
            QueryRow<FMT, ACT, D>::load(qf[mt], src, valid, j);
        }
        TileRegs<FMT, D> next;
        bool next_bad = false;
        auto fetch = [&](int t) {
            if (t - window_first >= 64 * kAttnWaves) {
                window_pages = load_pages(t);
                window_first = t;
            }
            int page = __builtin_amdgcn_readlane(window_pages, (t - window_first) / kAttnWaves);
            next_bad = (uint32_t)page >= (uint32_t)cache.pages;  // no keys there
            page = next_bad ? 0 : page;
            const uint8_t* tile = cache.data + (((int64_t)page * kv_heads + h) * cache.tiles_per_page +
                                                (t - page_of(t) * cache.tiles_per_page)) * (int64_t)L::kBytes;
            load_tile<FMT, D, MT == 1>(next, tile, lane);
        };
        if (ta < tb) fetch(ta);
        float fac[MT], m[MT], l[MT];
        RowRange range[MT];
        f32x4 o[MT][OT];
        int far_rows = 0;                 // bit mt: far_scores
        int lo_all = 0, hi_all = it.len;  // keys that every valid row sees
        {
            const int i1 = i0 + __builtin_amdgcn_readfirstlane(token_of(rows - 1));
            hi_all = row_range(i0, it.n, it.len, a.causal, a.window).hi;
            lo_all = row_range(i1, it.n, it.len, a.causal, a.window).lo;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            fac[mt] = QueryRow<FMT, ACT, D>::convert(qf[mt], a.scale);
            range[mt] = row_range(i0 + token_of(16 * mt + r), it.n, it.len, a.causal, a.window);
            m[mt] = kNoMax;
            l[mt] = 0.0f;
#pragma unroll
            for (int x = 0; x < OT; ++x) o[mt][x] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        if (parts > 1 && threadIdx.x == 0) {
            claim_word(team_word, seen_team, a.tag);
            if (teams > 1) claim_word(teams_word, seen_teams, a.tag);
        }

        for (int t = ta; t < tb; t += kAttnWaves) {
            TileRegs<FMT, D> x = next;
            const bool bad = next_bad;
            if (t + kAttnWaves < tb) fetch(t + kAttnWaves);
            const int tok0 = t * kKvTile;
            const int live = bad ? 0 : it.len;
            const bool edge = bad || tok0 + kKvTile > hi_all || tok0 < lo_all;
            if (edge) clear_values<FMT, D>(x, tok0, j, live);

            f32x4 sc[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int u = 0; u < 2; ++u) sc[mt][u] = f32x4{0.f, 0.f, 0.f, 0.f};
            auto keys = [&](auto uc, auto cc, auto stc) {
                const u32x4 kf =
                    key_step<FMT, CT, D, decltype(uc)::value, decltype(cc)::value, decltype(stc)::value>(x, a.k_exp);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    sc[mt][decltype(uc)::value] =
                        mfma<CT>(kf, qf[mt][decltype(cc)::value * S + decltype(stc)::value], sc[mt][decltype(uc)::value]);
            };
            auto keys_u = [&](auto uc) {
                auto keys_c = [&](auto cc) {
                    keys(uc, cc, std::integral_constant<int, 0>{});
                    keys(uc, cc, std::integral_constant<int, 1>{});
                    if constexpr (S == 4) {
                        keys(uc, cc, std::integral_constant<int, 2>{});
                        keys(uc, cc, std::integral_constant<int, 3>{});
                    }
                };
                keys_c(std::integral_constant<int, 0>{});
                if constexpr (L::C == 2) keys_c(std::integral_constant<int, 1>{});
            };
            keys_u(std::integral_constant<int, 0>{});
            keys_u(std::integral_constant<int, 1>{});

            u32x4 pf[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float s[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = sc[mt][e >> 2][e & 3];
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int tok = tok0 + 16 * (e >> 2) + 4 * j + (e & 3);
                        if (!(tok >= range[mt].lo && tok < range[mt].hi && tok < live)) s[e] = -__builtin_inff();
                    }
                }
                float top = s[0];
#pragma unroll
                for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e]);
                top *= fac[mt];
                if (__any(top > m[mt] + kSlack)) {
                    top = fmaxf(top, __shfl_xor(top, 16, 64));
                    top = fmaxf(top, __shfl_xor(top, 32, 64));
                    const float mn = fmaxf(m[mt], top);
                    const float down = exp2_(m[mt] - mn);
                    m[mt] = mn;
                    if (far_scores(mn)) far_rows |= 1 << mt;
                    l[mt] *= down;
#pragma unroll
                    for (int y = 0; y < OT; ++y) o[mt][y] *= down;
                }
                float f = fac[mt], off = kBias - m[mt];
                if (far_rows >> mt & 1) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] = near_score(s[e], f, m[mt]);
                    f = 1.0f;
                    off = kBias;
                }
                float p[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p[e] = exp2_(fmaf(s[e], f, off));
                    l[mt] += p[e];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) pf[mt][e] = pack_out<CT>(p[2 * e], p[2 * e + 1]);
            }

            auto values = [&](auto cc, auto qc) {
                constexpr int ck = decltype(cc)::value, q = decltype(qc)::value;
                u32x4 even, odd;
                value_frags<FMT, CT, D, ck, q>(x, a.v_exp, even, odd);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    o[mt][ck * L::VD + 2 * q] = mfma<CT>(even, pf[mt], o[mt][ck * L::VD + 2 * q]);
                    o[mt][ck * L::VD + 2 * q + 1] = mfma<CT>(odd, pf[mt], o[mt][ck * L::VD + 2 * q + 1]);
                }
            };
            auto values_c = [&](auto cc) {
                values(cc, std::integral_constant<int, 0>{});
                values(cc, std::integral_constant<int, 1>{});
                if constexpr (L::VD == 8) {
                    values(cc, std::integral_constant<int, 2>{});
                    values(cc, std::integral_constant<int, 3>{});
                }
            };
            values_c(std::integral_constant<int, 0>{});
            if constexpr (L::C == 2) values_c(std::integral_constant<int, 1>{});
        }

        // ---- join the four waves, 16 rows at a time
        const bool whole = parts == 1;
        // partial sums of all workgroups (below 2^28 bytes)
        const __amdgpu_buffer_rsrc_t ro = make_rsrc(a.ws_o, 2 * a.grid * R * D * 4);
        const __amdgpu_buffer_rsrc_t rm = make_rsrc(a.ws_ml, 2 * a.grid * R * 8);
        constexpr int E = D / 16;                       // outputs of a thread: 16 threads a row
        const int orow = threadIdx.x >> 4, od = (threadIdx.x & 15) * E;
        auto store_row = [&](int mt, int srow, float mx, float lx, const float (&ox)[E]) {
            const int di = token_of(16 * mt + srow), i = i0 + di;
            const int head = h * a.group + 16 * mt + srow + g0 - di * a.group;
            float lse;
            const float f = finish_row(mx, lx, a.sinks != nullptr, a.sinks ? a.sinks[head] : 0.0f, lse) * a.v_alpha;
            uint16_t* dst = a.out + (int64_t)(it.q0 + i) * a.o_ts + (int64_t)head * a.o_hs + od;
#pragma unroll
            for (int e = 0; e < E; e += 4)
                *reinterpret_cast<u32x2*>(dst + e) =
                    u32x2{pack_out<ACT>(ox[e] * f, ox[e + 1] * f), pack_out<ACT>(ox[e + 2] * f, ox[e + 3] * f)};
            if (a.lse && od == 0) a.lse[(int64_t)(it.q0 + i) * a.q_heads + head] = lse;
        };
        auto keep_row = [&](int slot, int row, float mx, float lx, const float (&ox)[E]) {
            const uint32_t at = slot * R + row;
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const f32x4 w = {ox[e], ox[e + 1], ox[e + 2], ox[e + 3]};
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, w), ro, (at * D + od + e) * 4, 0,
                                                       kDeviceCoherent);
            }
            if (od == 0)
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(mx), __float_as_uint(lx)}, rm, at * 8, 0,
                                                      kDeviceCoherent);
        };
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (16 * mt >= rows) break;
            l[mt] += __shfl_xor(l[mt], 16, 64);
            l[mt] += __shfl_xor(l[mt], 32, 64);
            __syncthreads();  // the LDS of the previous 16 rows is free
            if (j == 0) {
                lds_m[wave][r] = m[mt];
                lds_l[wave][r] = l[mt];
            }
#pragma unroll
            for (int c = 0; c < L::C; ++c)
#pragma unroll
                for (int reg = 0; reg < 4; ++reg)
#pragma unroll
                    for (int k = 0; k < L::VD; k += 4) {
                        f32x4 w;
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = o[mt][c * L::VD + k + e][reg];
                        *reinterpret_cast<f32x4*>(&lds_o[wave][r][c * L::CH + L::VD * (4 * j + reg) + k]) = w;
                    }
            __syncthreads();
            float mx = lds_m[0][orow];
#pragma unroll
            for (int w = 1; w < kAttnWaves; ++w) mx = fmaxf(mx, lds_m[w][orow]);
            float lx = 0.0f, ox[E];
#pragma unroll
            for (int e = 0; e < E; ++e) ox[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttnWaves; ++w) {
                const float f = exp2_(lds_m[w][orow] - mx);
                lx += lds_l[w][orow] * f;
#pragma unroll
                for (int e = 0; e < E; ++e) ox[e] += lds_o[w][orow][od + e] * f;
            }
            if (16 * mt + orow < rows) {
                if (whole) {
                    store_row(mt, orow, mx, lx, ox);
                } else {
                    keep_row(slot_of(part), 16 * mt + orow, mx, lx, ox);
                }
            }
        }
        if (!whole) {
            // ---- join the shares of the item: sixteen by their last workgroup, and
            // where there are more than sixteen, those sums by the last of all
            // as split_finish: this thread's stores are complete, then one arrival
            auto arrive = [&](unsigned long long* word, int count) {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                __syncthreads();
                if (threadIdx.x == 0) lds_last = arrive_word(word, count, a.tag);
                __syncthreads();
                asm volatile("" ::: "memory");
                return lds_last != 0;
            };
            // sum of `count` parts from p0 on, `step` apart, in their order
            auto join = [&](int p0, int step, int count, bool last) {
#pragma unroll 1
                for (int mt = 0; mt < MT; ++mt) {
                    const int left = rows - 16 * mt;
                    if (left <= 0) break;
                    // 16 threads a row; with at most 8 rows the two halves of the
                    // workgroup take every second batch of slots
                    const int halves = left <= 8 ? 2 : 1;
                    const int crow = halves == 2 ? orow & 7 : orow, half = halves == 2 ? orow >> 3 : 0;
                    constexpr int kBatch = D == 256 ? 4 : 8;
                    float mx = kNoMax, lx = 0.0f, ox[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) ox[e] = 0.0f;
                    if (crow < left) {
                        for (int s0 = half * kBatch; s0 < count; s0 += halves * kBatch) {
                            u32x2 ml[kBatch];
                            u32x4 po[kBatch][E / 4];
#pragma unroll
                            for (int s = 0; s < kBatch; ++s) {
                                // past the last slot: an offset past the buffer, which reads zeros
                                const bool there = s0 + s < count;
                                const uint32_t at = slot_of(p0 + (s0 + s) * step) * R + 16 * mt + crow;
                                ml[s] = __builtin_amdgcn_raw_buffer_load_b64(rm, there ? at * 8 : kOutOfRange, 0,
                                                                             kDeviceCoherent);
#pragma unroll
                                for (int e = 0; e < E / 4; ++e)
                                    po[s][e] = __builtin_amdgcn_raw_buffer_load_b128(
                                        ro, there ? (at * D + od + 4 * e) * 4 : kOutOfRange, 0, kDeviceCoherent);
                            }
                            float top = mx;
#pragma unroll
                            for (int s = 0; s < kBatch; ++s)
                                if (s0 + s < count) top = fmaxf(top, __uint_as_float(ml[s].x));
                            const float down = exp2_(mx - top);
                            mx = top;
                            lx *= down;
#pragma unroll
                            for (int e = 0; e < E; ++e) ox[e] *= down;
#pragma unroll
                            for (int s = 0; s < kBatch; ++s) {
                                const float w = s0 + s < count ? exp2_(__uint_as_float(ml[s].x) - mx) : 0.0f;
                                lx += w * __uint_as_float(ml[s].y);
#pragma unroll
                                for (int e = 0; e < E; ++e) ox[e] += w * __uint_as_float(po[s][e / 4][e % 4]);
                            }
                        }
                    }
                    __syncthreads();
                    if (halves == 2) {
                        if (half == 1) {
#pragma unroll
                            for (int e = 0; e < E; ++e) lds_o[0][crow][od + e] = ox[e];
                            if (od == 0) {
                                lds_m[0][crow] = mx;
                                lds_l[0][crow] = lx;
                            }
                        }
                        __syncthreads();
                        if (half == 0) {
                            const float m1 = lds_m[0][crow], top = fmaxf(mx, m1);
                            const float f0 = exp2_(mx - top), f1 = exp2_(m1 - top);
                            mx = top;
                            lx = lx * f0 + lds_l[0][crow] * f1;
#pragma unroll
                            for (int e = 0; e < E; ++e) ox[e] = ox[e] * f0 + lds_o[0][crow][od + e] * f1;
                        }
                    }
                    if (half == 0 && crow < left) {
                        if (last) store_row(mt, crow, mx, lx, ox);
                        else keep_row(slot_of(p0), 16 * mt + crow, mx, lx, ox);  // its own reads of the slot are done
                    }
                }
            };
            if (arrive(team_word, size)) {
                join(p0, 1, size, teams == 1);
                if (teams > 1 && arrive(teams_word, teams)) join(0, kTeam, teams, true);
            }
        }
    }
}

// f(0), f(1), .. f(N - 1) with the numbers as compile-time constants.
template <class Fn, int... I>
__device__ __forceinline__ void unrolled_(Fn&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class Fn>
__device__ __forceinline__ void unrolled(Fn&& f) {
    unrolled_(f, std::make_integer_sequence<int, N>{});
}

// ------------------------------------------------------------ tiled kernel
// Many query rows a sequence (prompts, chunks).  A workgroup takes 32 rows a
// wave of one (sequence, row block, KV head) and walks over the keys in steps
// of TT tiles.  Each key and value is dequantized once per workgroup: the
// waves share a step's fragments through LDS, where a fragment is the 1 KiB
// that a wave reads with one 16-byte load a lane, without bank conflicts.  Two
// LDS buffers and one barrier a step: while step i is multiplied, step i + 1 is
// dequantized into the other buffer and the codes of step i + 2 are loaded.
//
// The products are 32x32x16: on this GPU vector instructions of other waves run
// beside them, while beside the 16x16x32 form they mostly wait (measured with
// four waves a SIMD, per 16384 products: four FP4 converts alone 19.5 cycles,
// with the 16x16x32 form 27.8, with half a 32x32x16 one 23.4; two exponentials
// 19.2, 27.6, 21.7).  Head size 256 takes the 16x16x32 form with 16 rows a wave:
// the accumulators of 32 rows and their queries leave no registers for two
// waves a SIMD (six prompts: 253 us with one wave, 207 with spills, 180 so).
//
// Bound by power: a chunk of 2048 tokens over 8192 keys (NVFP4, 64 and 8 heads
// of 128) takes 435 .. 465 us in a row of calls, 1030 .. 1106 TFLOP/s against 1311
// of a large library product, with the clock down to 1.75 GHz; the matrix cores
// are busy 51 % of the cycles, the vector units as long.  So what saves work
// counts more than what overlaps it: 256 rows a workgroup instead of 128 (570 ->
// 537 us, half the dequantization) and steps of four tiles instead of two (-> 490 us).
//   S^T = K Q^T: with lane = 32 h + t, step i of a chunk takes the eight
//   elements of octet (j, s) of token t, j = 2 (i / S) + h, s = i mod S, where
//   octet (j, s) is dword s of the codes of lane (t mod 16, j);
//   O^T = V^T P^T: row 2 r + e of block q is element VD r + 2 q + e, product
//   step u takes tokens 16 u + 4 h .. + 3 and 16 u + 8 + 4 h .. + 3, whose
//   probabilities lane 32 h + . holds after S^T.
//
// A tile's dequantization is dealt to WPT waves by token half u (tokens 16 u ..
// 16 u + 15) and, with four waves (head size 256), by chunk.
template <int FMT, int D, int WPT>
struct TilePart {
    using L = KvTile<FMT, D>;
    static_assert(WPT == 2 || (WPT == 4 && L::C == 2), "two waves a tile, or two a chunk of it");
    static constexpr int N = 2 * L::C / WPT;    // chunks
    static constexpr int SP = L::KD / 8;        // octets of a lane and chunk
    static constexpr int VP = L::VD / 2;        // pairs of value elements of a chunk
    static constexpr int VW = D == 64 ? 2 : 4;  // dwords of a lane's value codes
    uint32_t k[N][SP], v[N][VW];
    uint32_t ks[N];  // the key scales of each chunk in the low bytes
    uint32_t vs[N];  // the scales of the four value tokens
};

typedef float f32x16 __attribute__((ext_vector_type(16)));
template <int CT>
__device__ __forceinline__ f32x16 mfma32(const u32x4& a, const u32x4& b, const f32x16& c) {
    if constexpr (CT == 0)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// Fragments of a part, chunk n: key steps, and the halves of the value
// fragments (two dwords: tokens 0, 1 and 2, 3 of the quad).
template <int FMT, int CT, int D, int S_>
__device__ __forceinline__ u32x4 part_key(uint32_t w, uint32_t ks, int e) {
    using L = KvTile<FMT, D>;
    const uint32_t a[1] = {ks};
    return key_frag<FMT, CT, (S_ * 8 / L::G) % L::KG>(w, a, e);
}
template <int FMT, int CT, int D, int Q>
__device__ __forceinline__ void part_value(const uint32_t* v, uint32_t vs, int e, u32x2& even, u32x2& odd) {
    float s[4] = {1.0f, 1.0f, 1.0f, 1.0f};
    if constexpr (FMT == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = e8m0_scale<CT>((vs >> (8 * i)) & 0xFFu, e);
    }
    uint32_t a[4];  // elements 2 Q, 2 Q + 1 of the four tokens
    if constexpr (D == 64) {
        a[0] = codes16<CT, Q>(v[0], s[0]);
        a[1] = codes16<CT, Q + 2>(v[0], s[1]);
        a[2] = codes16<CT, Q>(v[1], s[2]);
        a[3] = codes16<CT, Q + 2>(v[1], s[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = codes16<CT, Q>(v[i], s[i]);
    }
    even = u32x2{low_halves(a[0], a[1]), low_halves(a[2], a[3])};
    odd = u32x2{high_halves(a[0], a[1]), high_halves(a[2], a[3])};
    if constexpr (FMT == 0) {
        const f16x2 s01 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)vs, 1.0f, false);
        const f16x2 s23 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)vs, 1.0f, true);
        even = u32x2{mul_f16x2(even.x, s01), mul_f16x2(even.y, s23)};
        odd = u32x2{mul_f16x2(odd.x, s01), mul_f16x2(odd.y, s23)};
    }
}

template <int FMT, int ACT, int D, int RW, int NW, int TT, int WAVES>
__global__ __launch_bounds__(64 * NW, WAVES) void attention_tiled(AttnArgs a, KvArgs cache) {
    using L = KvTile<FMT, D>;
    constexpr int CT = attn_type(FMT, ACT);
    constexpr bool k32 = RW == 32;  // rows of a wave: 32x32x16 products, else 16x16x32
    constexpr int R = RW * NW, S = L::KD / 8, WPT = NW / TT;
    constexpr int F = D / 16;               // key fragments of a tile, and value fragments
    constexpr int QF = k32 ? F : F / 2;     // query fragments of a row: product steps
    constexpr int OB = k32 ? D / 32 : D / 16;  // blocks of the output's elements
    constexpr int NS = k32 ? 16 : 8;        // scores of a lane and tile
    using Acc = typename std::conditional<k32, f32x16, f32x4>::type;
    constexpr int kTileFrags = 2 * F;  // 1 KiB fragments of a tile
    __shared__ u32x4 lds[2][TT][kTileFrags][64];
    __shared__ int lds_scan[NW], lds_found[5];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, j = lane >> 4;         // as the codes lie in a tile
    const int prow = lane % RW, ph = lane / RW;     // as the products take them
    const int kv_heads = cache.kv_heads;

    // ---- the item, longest first: a block's level is its row block plus the
    // sequence's earlier keys, in row blocks; the KV heads of a block are next to
    // each other
    const int share = (int)blockIdx.x % a.splits, head_block = (int)blockIdx.x / a.splits;
    const int block = head_block / kv_heads, h = head_block - block * kv_heads;
    int b, rb;
    Seq it;
    if (a.batch <= 64) {  // every wave by itself, a sequence a lane
        bool bad_offsets = false;
        const Seq x = sequence_of<R>(a, lane, bad_offsets);
        if (__any(bad_offsets)) return;  // nothing is written
        const int base = min(max(x.len - x.n, 0) / (R / a.group + 1), 1 << 24);
        auto count = [&](int level) {  // blocks at this level or above
            return __builtin_amdgcn_readlane(wave_scan(min(max(x.blocks + base - level, 0), x.blocks)), 63);
        };
        int lo = 0, hi = x.blocks > 0 ? x.blocks + base : 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) hi = max(hi, __shfl_xor(hi, d, 64));
        if (block >= count(0)) return;
        while (hi - lo > 1) {  // the highest level `lo` with count(lo) > block
            const int mid = (lo + hi) >> 1;
            if (count(mid) > block) lo = mid;
            else hi = mid;
        }
        const unsigned long long at = __ballot(x.blocks + base > lo && base <= lo && x.blocks > 0);
        const int nth = block - count(lo + 1);
        const bool mine = (at >> lane & 1) && __popcll(at & ((1ull << lane) - 1)) == nth;
        b = __ffsll(__ballot(mine)) - 1;
        rb = lo - __shfl(base, b, 64);
        it = sequence_from<R>(a, __shfl(x.q0, b, 64), __shfl(x.n, b, 64), __shfl(x.len, b, 64));
    } else {  // sequences in order, their last blocks first
        int before = 0;
        bool there = false;
        for (int base = 0; base < a.batch && (!there || a.q_offsets); base += 64 * NW) {
            bool bad_offsets = false;
            const Seq x = sequence_of<R>(a, base + threadIdx.x, bad_offsets);
            if (__syncthreads_or(bad_offsets)) return;  // nothing is written: every block looks at all offsets
            if (there) continue;
            int p = wave_scan(x.blocks);
            __syncthreads();
            if (lane == 63) lds_scan[wave] = p;
            __syncthreads();
            p += before - x.blocks;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                p += w < wave ? lds_scan[w] : 0;
                before += lds_scan[w];
            }
            if (block >= p && block < p + x.blocks) {
                lds_found[0] = base + threadIdx.x;
                lds_found[1] = x.q0;
                lds_found[2] = x.n;
                lds_found[3] = x.len;
                lds_found[4] = p;
            }
            there = block < before;  // the same in every thread
        }
        if (!there) return;
        __syncthreads();
        b = lds_found[0];
        it = sequence_from<R>(a, lds_found[1], lds_found[2], lds_found[3]);
        rb = it.blocks - 1 - (block - lds_found[4]);
    }
    b = __builtin_amdgcn_readfirstlane(b);
    rb = __builtin_amdgcn_readfirstlane(rb);
    it = sequence_from<R>(a, __builtin_amdgcn_readfirstlane(it.q0), __builtin_amdgcn_readfirstlane(it.n),
                          __builtin_amdgcn_readfirstlane(it.len));
    const int rows = min(R, it.n * a.group - rb * R);
    const int i0 = rb * R / a.group, g0 = rb * R - i0 * a.group;
    auto token_of = [&](int x) { return (int)(((float)(x + g0) + 0.5f) * a.inv_group); };
    auto range_of = [&](int x) { return row_range(i0 + token_of(x), it.n, it.len, a.causal, a.window); };
    const int last_hi = __builtin_amdgcn_readfirstlane(range_of(rows - 1).hi);
    const int first_lo = __builtin_amdgcn_readfirstlane(range_of(0).lo);
    const int t0 = first_lo / kKvTile, t1 = (min(last_hi, it.len) + kKvTile - 1) / kKvTile;
    // Steps [s0, s1) of this share of the item; a share has four steps at least.
    const int all_steps = max(0, (t1 - t0 + TT - 1) / TT);
    const int shares = min(a.splits, max(1, all_steps / 4));
    if (share >= shares) return;
    const int s0 = all_steps * share / shares, steps = all_steps * (share + 1) / shares - s0;

    // ---- query row of this lane
    const int my0 = wave * RW, my = my0 + prow;
    u32x4 qf[QF];
    {
        const int di = token_of(my), i = i0 + di, g = my + g0 - di * a.group;
        const uint16_t* src = a.q + (int64_t)(it.q0 + i) * a.q_ts + (int64_t)(h * a.group + g) * a.q_hs;
#pragma unroll
        for (int f = 0; f < QF; ++f) {
            constexpr int per = k32 ? 2 * S : S;  // product steps of a chunk
            const int c = f / per, x = f % per, lane_j = k32 ? 2 * (x / S) + ph : ph;
            qf[f] = u32x4{0u, 0u, 0u, 0u};
            if (my < rows) qf[f] = *reinterpret_cast<const u32x4*>(src + c * L::CH + L::KD * lane_j + 8 * (x % S));
        }
    }

    unsigned long long* word = a.words + head_block;
    unsigned long long seen = 0;
    if (shares > 1 && threadIdx.x == 0) seen = peek_word(word);

    // ---- loads of this wave's part of a step
    const int32_t* pages = a.page_table + (int64_t)b * a.table_stride;
    const int my_tile = wave / WPT, sub = wave % WPT;
    auto page_of = [&](int t) { return (int)(((uint64_t)(uint32_t)t * a.tpp_magic) >> 36); };
    auto load_pages = [&](int t) { return pages[page_of(max(0, min(t + lane, t1 - 1)))]; };
    int window_pages = steps > 0 ? load_pages(t0 + s0 * TT) : 0, window_first = t0 + s0 * TT;
    using Part = TilePart<FMT, D, WPT>;
    Part raw;
    const int half = sub & 1, chunk0 = sub >> 1;  // this wave's token half and first chunk
    int raw_bad = 0, raw_left = 0;  // tiles of the step without keys; keys that this wave's tile holds from its start
    auto fetch = [&](int step) {
        const int ts = t0 + (s0 + step) * TT;
        if (ts + TT - window_first > 64) {
            window_pages = load_pages(ts);
            window_first = ts;
        }
        raw_bad = 0;
        int page = 0;
#pragma unroll
        for (int x = 0; x < TT; ++x) {
            const int p = __builtin_amdgcn_readlane(window_pages, ts + x - window_first);
            const bool bad = ts + x >= t1 || (uint32_t)p >= (uint32_t)cache.pages;
            raw_bad |= bad ? 1 << x : 0;
            if (x == my_tile) page = bad ? 0 : p;
        }
        const int t = min(ts + my_tile, t1 - 1);
        raw_left = (raw_bad >> my_tile & 1) ? 0 : it.len - t * kKvTile;
        const uint8_t* tile = cache.data + (((int64_t)page * kv_heads + h) * cache.tiles_per_page +
                                            (t - page_of(t) * cache.tiles_per_page)) * (int64_t)L::kBytes;
#pragma unroll
        for (int n = 0; n < Part::N; ++n) {
            const int c = chunk0 + n;
            const uint8_t* kc = tile + (D == 64 ? half * 8 : (c * 2 + half) * 1024) + lane * 16;
            if constexpr (Part::SP == 2) {
                const u32x2 k = *reinterpret_cast<const u32x2*>(kc);
                raw.k[n][0] = k.x;
                raw.k[n][1] = k.y;
            } else {
                const u32x4 k = *reinterpret_cast<const u32x4*>(kc);
#pragma unroll
                for (int e = 0; e < 4; ++e) raw.k[n][e] = k[e];
            }
            const uint8_t* vc = tile + L::kCodes + (D == 64 ? half * 8 : (c * 2 + half) * 1024) + lane * 16;
            if constexpr (D == 64) {
                const u32x2 v = *reinterpret_cast<const u32x2*>(vc);
                raw.v[n][0] = v.x;
                raw.v[n][1] = v.y;
            } else {
                const u32x4 v = *reinterpret_cast<const u32x4*>(vc);
#pragma unroll
                for (int e = 0; e < 4; ++e) raw.v[n][e] = v[e];
            }
            const uint8_t* ks = tile + L::kKs + key_scale_lane<FMT, D>(r, j) + (c * 2 + half) * L::KG;
            if constexpr (L::KG == 2) raw.ks[n] = *reinterpret_cast<const uint16_t*>(ks);
            else raw.ks[n] = *ks;
            const int g = c * (L::CH / L::G) + r * L::VD / L::G;
            raw.vs[n] = *reinterpret_cast<const uint32_t*>(tile + L::kVs + (g * 4 + j) * 8 + half * 4);
        }
    };
    // raw -> fragments in LDS buffer `buf`, in kPieces pieces: the key steps, then
    // pairs of value fragments, of each chunk
    constexpr int kPieces = Part::N * (Part::SP + Part::VP);
    auto spread = [&](int buf, auto piece) {
        constexpr int n = decltype(piece)::value / (Part::SP + Part::VP), p = decltype(piece)::value % (Part::SP + Part::VP);
        u32x4(*out)[64] = lds[buf][my_tile];
        const int c = chunk0 + n;
        if constexpr (p < Part::SP) {
            // octet (j, p) of token 16 half + r
            const u32x4 f = part_key<FMT, CT, D, p>(raw.k[n][p], raw.ks[n], a.k_exp);
            if constexpr (k32) out[c * 2 * S + (j >> 1) * S + p][32 * (j & 1) + 16 * half + r] = f;
            else out[half * (F / 2) + c * S + p][lane] = f;
        } else {
            constexpr int q = p - Part::SP;
            const int left = raw_left - 16 * half - 4 * j;  // value tokens of the quad that exist (clear_values)
            const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
            u32x2 even, odd;
            part_value<FMT, CT, D, q>(raw.v[n], raw.vs[n] & keep, a.v_exp, even, odd);
            const int block = c * Part::VP + q;
            if constexpr (k32) {
                u32x2* vo = reinterpret_cast<u32x2*>(&out[F + block * 2 + half][32 * (j & 1) + 2 * r]) + (j >> 1);
                vo[0] = even;
                vo[2] = odd;
            } else {
                u32x2* vo = reinterpret_cast<u32x2*>(&out[F + 2 * block][lane]) + half;
                vo[0] = even;
                vo[128] = odd;
            }
        }
    };

    if (steps > 0) fetch(0);
    const float fac = QueryRow<FMT, ACT, D>::convert(qf, a.scale);
    const RowRange range = range_of(my);
    float m = kNoMax, l = 0.0f;
    bool far = false;  // far_scores
    Acc o[OB];
#pragma unroll
    for (int x = 0; x < OB; ++x) o[x] = Acc(0.0f);
    // keys that every row of this wave sees
    const int my_rows = min(RW, rows - my0);  // may be below 1
    const int hi_all = __builtin_amdgcn_readfirstlane(range_of(min(my0, rows - 1)).hi);
    const int lo_all = __builtin_amdgcn_readfirstlane(range_of(max(0, my0 + max(my_rows, 1) - 1)).lo);
    int cur_bad = 0;
    if (steps > 0) {
        unrolled<kPieces>([&](auto p) { spread(0, p); });
        cur_bad = raw_bad;
        fetch(min(1, steps - 1));
    }

    if (shares > 1 && threadIdx.x == 0) claim_word(word, seen, a.tag);

    for (int step = 0; step < steps; ++step) {
        __syncthreads();  // buffer `step` is written, the other one is read out
        const int buf = step & 1, tok0 = (t0 + (s0 + step) * TT) * kKvTile;
        const u32x4(*in)[kTileFrags][64] = lds[buf];
        // The order is fixed by hand: fragments are read kAhead before their
        // products, and the next step's dequantization goes in between.  (The
        // last step spreads a step again that nothing reads.)
        constexpr int kFrags = TT * F;
        Acc sc[k32 ? TT : 2 * TT];  // k32: a tile, else 16 keys each
        u32x4 ring[kAhead];
        // value fragments, k32: for each tile and half u the blocks
        auto key_at = [&](int e) { return in[e / F][e % F][lane]; };
        auto value_at = [&](int e) { return in[e / F][F + (k32 ? (e % OB) * 2 + e / OB % 2 : e % F)][lane]; };
#pragma unroll
        for (int e = 0; e < kAhead; ++e) ring[e] = key_at(e);
        __builtin_amdgcn_sched_barrier(0);
        unrolled<kFrags>([&](auto ec) {
            constexpr int e = decltype(ec)::value, x = e / QF, f = e % QF;
            constexpr int p0 = e * kPieces / kFrags, p1 = (e + 1) * kPieces / kFrags;
            if constexpr (f == 0) sc[x] = Acc(0.0f);
            if constexpr (k32) sc[x] = mfma32<CT>(ring[e % kAhead], qf[f], sc[x]);
            else sc[x] = mfma<CT>(ring[e % kAhead], qf[f], sc[x]);
            if constexpr (e + kAhead < kFrags) ring[e % kAhead] = key_at(e + kAhead);
            unrolled<p1 - p0>([&](auto p) { spread(buf ^ 1, std::integral_constant<int, p0 + decltype(p)::value>{}); });
            __builtin_amdgcn_sched_barrier(0);
        });
#pragma unroll
        for (int e = 0; e < kAhead; ++e) ring[e] = value_at(e);
        const int bad = cur_bad;
        const bool edge = bad || tok0 + TT * kKvTile > hi_all || tok0 < lo_all;
        cur_bad = raw_bad;
        fetch(min(step + 2, steps - 1));

        constexpr int A = k32 ? 16 : 4;  // scores of an accumulator
        if (edge) {
#pragma unroll
            for (int e = 0; e < NS * TT; ++e) {
                const int key = tok0 + (k32 ? 8 : 16) * (e >> 2) + 4 * ph + (e & 3);
                const bool see = key >= range.lo && key < range.hi && key < it.len && !(bad >> (e / NS) & 1);
                if (!see) sc[e / A][e % A] = -__builtin_inff();
            }
        }
        float top = sc[0][0];
#pragma unroll
        for (int e = 1; e < NS * TT; ++e) top = fmaxf(top, sc[e / A][e % A]);
        top *= fac;
        if (__any(top > m + kSlack)) {
            if constexpr (!k32) top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float mn = fmaxf(m, top);
            const float down = exp2_(m - mn);
            m = mn;
            far = far_scores(mn);
            l *= down;
#pragma unroll
            for (int y = 0; y < OB; ++y) o[y] *= down;
        }
        // Probabilities of a lane's first eight keys, then the products of eight
        // with the next ones' probabilities in between.
        float f = fac, off = kBias - m;
        if (far) {
#pragma unroll
            for (int e = 0; e < NS * TT; ++e) sc[e / A][e % A] = near_score(sc[e / A][e % A], f, m);
            f = 1.0f;
            off = kBias;
        }
        constexpr int kEights = NS * TT / 8;
        u32x4 pf[kEights];
        auto weigh = [&](int u, int pair) {  // two of eight keys
            const int e = 8 * u + 2 * pair;
            const float p0 = exp2_(fmaf(sc[e / A][e % A], f, off)), p1 = exp2_(fmaf(sc[e / A][e % A + 1], f, off));
            l += p0 + p1;
            pf[u][pair] = pack_out<CT>(p0, p1);
        };
#pragma unroll
        for (int pair = 0; pair < 4; ++pair) weigh(0, pair);
        __builtin_amdgcn_sched_barrier(0);
        unrolled<kFrags>([&](auto ec) {
            constexpr int e = decltype(ec)::value, u = e / OB, y = e % OB;
            constexpr int w0 = y * 4 / OB, w1 = (y + 1) * 4 / OB;
            if constexpr (k32) o[y] = mfma32<CT>(ring[e % kAhead], pf[u], o[y]);
            else o[y] = mfma<CT>(ring[e % kAhead], pf[u], o[y]);
            if constexpr (e + kAhead < kFrags) ring[e % kAhead] = value_at(e + kAhead);
            if constexpr (u + 1 < kEights) unrolled<w1 - w0>([&](auto w) { weigh(u + 1, w0 + decltype(w)::value); });
            __builtin_amdgcn_sched_barrier(0);
        });
    }

    // ---- join the shares of an item: each keeps its sums as they lie in its
    // threads, and the last to arrive adds them in their order
    if (shares > 1) {
        constexpr int kQuads = OB * (k32 ? 4 : 1), T = 64 * NW;
        const __amdgpu_buffer_rsrc_t ro = make_rsrc(a.ws_o, a.grid * kQuads * T * 16);  // below 2^31 bytes
        const __amdgpu_buffer_rsrc_t rm = make_rsrc(a.ws_ml, a.grid * T * 8);
        const int first = head_block * a.splits;  // slot of share 0
        unrolled<kQuads>([&](auto qc) {
            constexpr int q = decltype(qc)::value, y = k32 ? q / 4 : q, e = k32 ? q % 4 * 4 : 0;
            const f32x4 w = {o[y][e], o[y][e + 1], o[y][e + 2], o[y][e + 3]};
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, w), ro,
                                                   (((first + share) * kQuads + q) * T + threadIdx.x) * 16, 0,
                                                   kDeviceCoherent);
        });
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(m), __float_as_uint(l)}, rm,
                                              ((first + share) * T + threadIdx.x) * 8, 0, kDeviceCoherent);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0) lds_scan[0] = arrive_word(word, shares, a.tag);
        __syncthreads();
        if (!lds_scan[0]) return;
        asm volatile("" ::: "memory");
        float top = kNoMax;
        for (int x = 0; x < shares; ++x)
            top = fmaxf(top, __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                                 rm, ((first + x) * T + threadIdx.x) * 8, 0, kDeviceCoherent)));
        m = top;
        l = 0.0f;
#pragma unroll
        for (int y = 0; y < OB; ++y) o[y] = Acc(0.0f);
        for (int x = 0; x < shares; ++x) {
            const u32x2 ml = __builtin_amdgcn_raw_buffer_load_b64(rm, ((first + x) * T + threadIdx.x) * 8, 0,
                                                                  kDeviceCoherent);
            const float w = exp2_(__uint_as_float(ml.x) - top);
            l += w * __uint_as_float(ml.y);
            unrolled<kQuads>([&](auto qc) {
                constexpr int q = decltype(qc)::value, y = k32 ? q / 4 : q, e = k32 ? q % 4 * 4 : 0;
                const f32x4 v = __builtin_bit_cast(
                    f32x4, __builtin_amdgcn_raw_buffer_load_b128(ro, (((first + x) * kQuads + q) * T + threadIdx.x) * 16, 0,
                                                                 kDeviceCoherent));
#pragma unroll
                for (int z = 0; z < 4; ++z) o[y][e + z] += w * v[z];
            });
        }
    }

    // ---- outputs.  k32: row 2 r + e of block q is element VD r + 2 q + e of its
    // chunk, and lane 32 h + . holds rows 8 g + 4 h + i; else row r of block q is
    // element VD r + q, and lane 16 h + . holds rows 4 h + i.
    if constexpr (!k32) l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (my < rows) {
        const int di = token_of(my), i = i0 + di, head = h * a.group + my + g0 - di * a.group;
        float lse;
        const float f = finish_row(m, l, a.sinks != nullptr, a.sinks ? a.sinks[head] : 0.0f, lse) * a.v_alpha;
        uint16_t* dst = a.out + (int64_t)(it.q0 + i) * a.o_ts + (int64_t)head * a.o_hs;
        constexpr int V = L::VD;
#pragma unroll
        for (int c = 0; c < L::C; ++c)
#pragma unroll
            for (int x = 0; x < (k32 ? 8 : 4); ++x) {
                uint32_t w[V / 2];
#pragma unroll
                for (int q = 0; q < V / 2; ++q) {
                    if constexpr (k32)
                        w[q] = pack_out<ACT>(o[c * V / 2 + q][2 * x] * f, o[c * V / 2 + q][2 * x + 1] * f);
                    else
                        w[q] = pack_out<ACT>(o[c * V + 2 * q][x] * f, o[c * V + 2 * q + 1][x] * f);
                }
                const int r0 = k32 ? 4 * (x / 2) + 2 * ph + x % 2 : 4 * ph + x;
                uint16_t* to = dst + c * L::CH + V * r0;
                if constexpr (V == 8) *reinterpret_cast<u32x4*>(to) = u32x4{w[0], w[1], w[2], w[3]};
                else *reinterpret_cast<u32x2*>(to) = u32x2{w[0], w[1]};
            }
        if (a.lse && ph == 0) a.lse[(int64_t)(it.q0 + i) * a.q_heads + head] = lse;
    }
}

// Compiled shapes of the tiled kernel: X(D, RW, NW, TT, WAVES): NW
// waves of RW rows, TT tiles a step.
#define FP4_ATTN_TILED(X) X(64, 32, 8, 4, 2) X(128, 32, 8, 4, 2) X(256, 16, 8, 2, 2)
constexpr int tiled_rows(int D) { return D == 256 ? 128 : 256; }

// Compiled shapes of the streaming kernel: X(D, MT), blocks of 16 MT query rows.
#define FP4_ATTN_SHAPES(X) X(64, 1) X(64, 2) X(64, 4) X(128, 1) X(128, 2) X(128, 4) X(256, 1) X(256, 2)

// Launches of one (format, activation type), in a translation unit each.
// False when the shape is not compiled.
bool launch_attention_nv_bf16(int D, int MT, bool tiled, const AttnArgs& a, const KvArgs& c, hipStream_t s);
bool launch_attention_nv_f16(int D, int MT, bool tiled, const AttnArgs& a, const KvArgs& c, hipStream_t s);
bool launch_attention_mx_bf16(int D, int MT, bool tiled, const AttnArgs& a, const KvArgs& c, hipStream_t s);
bool launch_attention_mx_f16(int D, int MT, bool tiled, const AttnArgs& a, const KvArgs& c, hipStream_t s);

}  // namespace fp4
