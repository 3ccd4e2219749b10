// FP4 key/value cache: its size, the quantizing write, the read-back
// (include/fp4gemm.h, section "FP4 key/value cache").
#include "kv_layout.h"

namespace fp4 {

// Checks shared by every entry that takes a cache; fills `a`.
int kv_check(const fp4_kv_cache* c, KvArgs* a) {
    if (!c) return FP4_ERR_NULL;
    size_t bytes;
    int st = fp4_kv_cache_size(c->pages, c->page_size, c->kv_heads, c->head_dim, c->format, &bytes);
    if (st != FP4_OK) return st;
    if (!(c->k_alpha > 0.0f) || !alpha_ok(c->k_alpha) || !(c->v_alpha > 0.0f) || !alpha_ok(c->v_alpha))
        return FP4_ERR_VALUE;
    if (!c->data) return FP4_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(c->data) & 15) return FP4_ERR_SHAPE;
    a->data = static_cast<uint8_t*>(c->data);
    a->slots = c->pages * c->page_size;
    a->page_size = (int)c->page_size;
    a->tiles_per_page = (int)(c->page_size / kKvTile);
    a->kv_heads = (int)c->kv_heads;
    a->pages = (int)c->pages;
    a->k_alpha = c->k_alpha;
    a->v_alpha = c->v_alpha;
    return FP4_OK;
}

template <int ACT>
__device__ __forceinline__ void widen2(uint32_t p, float& lo, float& hi) {
    if constexpr (ACT == 0) {
        lo = __uint_as_float(p << 16);
        hi = __uint_as_float(p & 0xFFFF0000u);
    } else {
        const f16x2 h = __builtin_bit_cast(f16x2, p);
        lo = (float)h.x;
        hi = (float)h.y;
    }
}

// One thread quantizes one block of G elements of a key or value row
// (quantize_block, the rule of fp4_quantize) and scatters its codes and scale
// into the tile.  Four neighbouring lanes take four consecutive tokens, whose
// value codes are neighbours in the tile, so that the four-byte (D = 64:
// two-byte) pieces of a wave merge into whole lines in L2.  8192 tokens of 8
// heads of 128 (43 MB) take 12.7 us, 3.4 TB/s: bound by those scattered stores;
// one token takes 6.2 us, latency (slot, row, scale, one division an element
// where alpha is no power of two).
template <int FMT, int ACT, int D>
__global__ __launch_bounds__(256) void kv_append_kernel(KvArgs c, const uint16_t* __restrict__ k,
                                                        const uint16_t* __restrict__ v,
                                                        const int64_t* __restrict__ slots, int tokens,
                                                        int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs) {
    constexpr int G = KvTile<FMT, D>::G, GP = D / G;
    const uint32_t n = blockIdx.x * 256u + threadIdx.x;
    const int token = (int)(n / (4 * GP) * 4 + n % 4), g = (int)(n / 4 % GP);
    const int h = blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    if (token >= tokens) return;
    const int64_t slot = slots[token];  // used only after the rows' loads are under way
    const uint16_t* src = is_v ? v + token * v_ts + h * v_hs : k + token * k_ts + h * k_hs;
    const u32x4* p = reinterpret_cast<const u32x4*>(src + g * G);
    u32x4 raw[G / 8];
#pragma unroll
    for (int i = 0; i < G / 8; ++i) raw[i] = p[i];
    if (slot < 0 || slot >= c.slots) return;
    float x[G];
#pragma unroll
    for (int i = 0; i < G / 2; ++i) widen2<ACT>(raw[i / 4][i % 4], x[2 * i], x[2 * i + 1]);
    kv_store_block<FMT, D>(c, slot, h, g, is_v, x);
}

// Eight codes times their scale and alpha, rounded to the output type.
template <int FMT, int ACT>
__device__ __forceinline__ u32x4 read_eight(uint32_t w, uint32_t sb, float alpha) {
    float s;
    if constexpr (FMT == 0) s = __builtin_amdgcn_cvt_f32_fp8((int)sb, 0);
    else s = __uint_as_float(sb != 0 ? sb << 23 : 0x00400000u);
    const f32x2 f0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const f32x2 f1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2 f2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const f32x2 f3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    u32x4 o;
    o.x = pack_out<ACT>(f0.x * s * alpha, f0.y * s * alpha);
    o.y = pack_out<ACT>(f1.x * s * alpha, f1.y * s * alpha);
    o.z = pack_out<ACT>(f2.x * s * alpha, f2.y * s * alpha);
    o.w = pack_out<ACT>(f3.x * s * alpha, f3.y * s * alpha);
    return o;
}

// One thread reads eight elements of a key row and of a value row: a wave
// writes whole rows with 16-byte stores.  Bound by the bytes: 65536 tokens of 8
// heads of 128 (NVFP4 to BF16, 344 MB) take 49 us, 7.0 TB/s.  kFar: outputs too
// large for the caches go past them (81 us otherwise); 8192 tokens take 8.9 us
// either way, and their reader finds them.  Two and four rows a thread were no
// faster (52 us past the caches, 67 and 72 us through them).
template <int FMT, int ACT, int D, bool kFar>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs c, const int64_t* __restrict__ slots, int tokens,
                                                      uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                                                      int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs) {
    using L = KvTile<FMT, D>;
    constexpr int P = D / 8;
    const uint32_t n = blockIdx.x * 256u + threadIdx.x;
    const int token = (int)(n / P), d = (int)(n % P) * 8, g = d / L::G;
    const int h = blockIdx.y;
    if (token >= tokens) return;
    const int64_t slot = slots[token];
    uint32_t kw = 0, vw = 0, ks = 0, vs = 0;  // zeros for a slot outside the cache
    if (slot >= 0 && slot < c.slots) {
        int t;
        const uint8_t* tile = kv_tile_of(c, slot, h, L::kBytes, t);
        if (k) {
            kw = *reinterpret_cast<const uint32_t*>(tile + L::k_code(t, d));
            ks = tile[L::k_scale(t, g)];
        }
        if (v) {
            if constexpr (D == 64)
                vw = *reinterpret_cast<const uint16_t*>(tile + L::v_code(t, d)) |
                     ((uint32_t)*reinterpret_cast<const uint16_t*>(tile + L::v_code(t, d + 4)) << 16);
            else
                vw = *reinterpret_cast<const uint32_t*>(tile + L::v_code(t, d));
            vs = tile[L::v_scale(t, g)];
        }
    }
    auto store = [](uint16_t* p, const u32x4& x) {
        if constexpr (kFar) __builtin_nontemporal_store(x, reinterpret_cast<u32x4*>(p));
        else *reinterpret_cast<u32x4*>(p) = x;
    };
    if (k) store(k + token * k_ts + h * k_hs + d, read_eight<FMT, ACT>(kw, ks, c.k_alpha));
    if (v) store(v + token * v_ts + h * v_hs + d, read_eight<FMT, ACT>(vw, vs, c.v_alpha));
}

// Row strides (elements) of a [tokens][heads][D] array: 16-byte aligned rows.
bool rows_ok(const void* p, int64_t ts, int64_t hs) {
    const int64_t most = int64_t(1) << 40;
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ts >= 0 && hs >= 0 && ts < most && hs < most && ts % 8 == 0 &&
           hs % 8 == 0;
}

// No two rows of a written array share an element.
bool rows_apart(int64_t tokens, int64_t heads, int64_t D, int64_t ts, int64_t hs) {
    const bool token_major = (heads == 1 || hs >= D) && (tokens == 1 || ts >= (heads - 1) * hs + D);
    const bool head_major = (tokens == 1 || ts >= D) && (heads == 1 || hs >= (tokens - 1) * ts + D);
    return token_major || head_major;
}

// Outputs above this many bytes are stored past the caches.
constexpr int64_t kReadFar = int64_t(64) << 20;

// Tokens a launch covers: its work-items are counted in 32 bits.
constexpr int64_t kKvSliceTokens = int64_t(1) << 20;

template <int FMT, int ACT, int D>
static void append_t(const KvArgs& c, const uint16_t* k, const uint16_t* v, const int64_t* slots, int tokens,
                     int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs, hipStream_t s) {
    constexpr int GP = D / KvTile<FMT, D>::G;
    const int64_t threads = (int64_t)((tokens + 3) / 4 * 4) * GP;
    kv_append_kernel<FMT, ACT, D><<<dim3((unsigned)((threads + 255) / 256), 2 * c.kv_heads), dim3(256), 0, s>>>(
        c, k, v, slots, tokens, k_ts, k_hs, v_ts, v_hs);
}

template <int FMT, int ACT, int D>
static void read_t(const KvArgs& c, const int64_t* slots, int tokens, uint16_t* k, uint16_t* v, int64_t k_ts,
                   int64_t k_hs, int64_t v_ts, int64_t v_hs, hipStream_t s) {
    const int64_t threads = (int64_t)tokens * (D / 8);
    const dim3 grid((unsigned)((threads + 255) / 256), c.kv_heads), block(256);
    const int64_t bytes = (int64_t)tokens * c.kv_heads * D * 2 * ((k != nullptr) + (v != nullptr));
    if (bytes > kReadFar)
        kv_read_kernel<FMT, ACT, D, true><<<grid, block, 0, s>>>(c, slots, tokens, k, v, k_ts, k_hs, v_ts, v_hs);
    else
        kv_read_kernel<FMT, ACT, D, false><<<grid, block, 0, s>>>(c, slots, tokens, k, v, k_ts, k_hs, v_ts, v_hs);
}

static int append_impl(const fp4_kv_cache* cache, const void* k, const void* v, const int64_t* slots, int64_t tokens,
                       int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs, int act_type, void* stream) {
    KvArgs c;
    int st = kv_check(cache, &c);
    if (st != FP4_OK) return st;
    if (act_type != 0 && act_type != 1) return FP4_ERR_FORMAT;
    if (tokens < 0 || tokens > (int64_t(1) << 24)) return FP4_ERR_SHAPE;
    if (tokens == 0) return FP4_OK;
    if (!k || !v || !slots) return FP4_ERR_NULL;
    if (!rows_ok(k, k_ts, k_hs) || !rows_ok(v, v_ts, v_hs) || (reinterpret_cast<uintptr_t>(slots) & 7))
        return FP4_ERR_SHAPE;
    st = check_device();
    if (st != FP4_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    for (int64_t t0 = 0; t0 < tokens; t0 += kKvSliceTokens) {
        const int n = (int)std::min(kKvSliceTokens, tokens - t0);
        const uint16_t* kp = static_cast<const uint16_t*>(k) + t0 * k_ts;
        const uint16_t* vp = static_cast<const uint16_t*>(v) + t0 * v_ts;
        FP4_KV_DISPATCH(append_t, cache->format, act_type, cache->head_dim, c, kp, vp, slots + t0, n, k_ts, k_hs, v_ts,
                        v_hs, s);
        st = launch_status();
        if (st != FP4_OK) return st;
    }
    return FP4_OK;
}

static int read_impl(const fp4_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k, void* v, int64_t k_ts,
                     int64_t k_hs, int64_t v_ts, int64_t v_hs, int act_type, void* stream) {
    KvArgs c;
    int st = kv_check(cache, &c);
    if (st != FP4_OK) return st;
    if (act_type != 0 && act_type != 1) return FP4_ERR_FORMAT;
    if (tokens < 0 || tokens > (int64_t(1) << 24)) return FP4_ERR_SHAPE;
    if (tokens == 0) return FP4_OK;
    if ((!k && !v) || !slots) return FP4_ERR_NULL;
    if ((k && (!rows_ok(k, k_ts, k_hs) || !rows_apart(tokens, c.kv_heads, cache->head_dim, k_ts, k_hs))) ||
        (v && (!rows_ok(v, v_ts, v_hs) || !rows_apart(tokens, c.kv_heads, cache->head_dim, v_ts, v_hs))) ||
        (reinterpret_cast<uintptr_t>(slots) & 7))
        return FP4_ERR_SHAPE;
    st = check_device();
    if (st != FP4_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    for (int64_t t0 = 0; t0 < tokens; t0 += kKvSliceTokens) {
        const int n = (int)std::min(kKvSliceTokens, tokens - t0);
        uint16_t* kp = k ? static_cast<uint16_t*>(k) + t0 * k_ts : nullptr;
        uint16_t* vp = v ? static_cast<uint16_t*>(v) + t0 * v_ts : nullptr;
        FP4_KV_DISPATCH(read_t, cache->format, act_type, cache->head_dim, c, slots + t0, n, kp, vp, k_ts, k_hs, v_ts,
                        v_hs, s);
        st = launch_status();
        if (st != FP4_OK) return st;
    }
    return FP4_OK;
}

}  // namespace fp4

extern "C" int fp4_kv_cache_size(int64_t pages, int64_t page_size, int64_t kv_heads, int64_t head_dim, int format,
                                 size_t* bytes) {
    if (format != FP4_NVFP4 && format != FP4_MXFP4) return FP4_ERR_FORMAT;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return FP4_ERR_SHAPE;
    if (pages < 1 || pages > (int64_t(1) << 30) || page_size < fp4::kKvTile || page_size > 4096 ||
        page_size % fp4::kKvTile || kv_heads < 1 || kv_heads > 256)
        return FP4_ERR_SHAPE;
    if (!bytes) return FP4_ERR_NULL;
    *bytes = (size_t)(pages * kv_heads * (page_size / fp4::kKvTile) * fp4::kv_tile_bytes(format, head_dim));
    return FP4_OK;
}

extern "C" int fp4_kv_append(const fp4_kv_cache* cache, const void* k, const void* v, const int64_t* slots,
                             int64_t tokens, int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                             int64_t v_head_stride, int act_type, void* stream) {
    return fp4::append_impl(cache, k, v, slots, tokens, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                            act_type, stream);
}

extern "C" int fp4_kv_read(const fp4_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k, void* v,
                           int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                           int64_t v_head_stride, int act_type, void* stream) {
    return fp4::read_impl(cache, slots, tokens, k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                          act_type, stream);
}
