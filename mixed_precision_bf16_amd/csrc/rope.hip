// Rotary positions (include/fp4gemm.h, section "Rotary positions"): alone, and
// with the write of the rotated keys into the FP4 cache.
#include "kv_layout.h"
#include "mx8.h"

namespace fp4 {

int kv_check(const fp4_kv_cache* c, KvArgs* a);                                              // kv_cache.hip
bool rows_ok(const void* p, int64_t ts, int64_t hs);
bool rows_apart(int64_t tokens, int64_t heads, int64_t D, int64_t ts, int64_t hs);

struct RopeArgs {
    const int64_t* positions;
    const float* frequencies;
    int rotary;  // elements rotated: the first ones of a head
    int pairs;   // rotary / 2
    double amplitude;
};

// Strided [tokens][heads][head_dim] rows.
struct Rows {
    const uint16_t* p;
    int64_t ts, hs;
};
struct RowsOut {
    uint16_t* p;
    int64_t ts, hs;
};

// sin and cos of an angle in FP64: the nearest multiple n of pi/2 is taken off in
// two steps with fused products (pi/2 = hi + lo to 2^-107; the method of Cody and
// Waite), then the Taylor series of both to x^17 and x^16 on [-pi/4, pi/4]
// (the first terms left out are below 3e-18), and n mod 4 gives the quadrant.
// Angles up to 2^31 keep an absolute error below 2^-51, so that rounded to FP32
// the result is the correctly rounded one but for one angle in 2^26.
__device__ __forceinline__ void sincos64(double angle, double& s, double& c) {
    const double n = rint(angle * 0.63661977236758134308);  // 2 / pi
    double x = fma(-n, 1.57079632679489655800, angle);
    x = fma(-n, 6.12323399573676603587e-17, x);
    const double z = x * x;
    double ps = 1.0 / 355687428096000.0;  // 1 / 17!
    ps = fma(ps, z, -1.0 / 1307674368000.0);
    ps = fma(ps, z, 1.0 / 6227020800.0);
    ps = fma(ps, z, -1.0 / 39916800.0);
    ps = fma(ps, z, 1.0 / 362880.0);
    ps = fma(ps, z, -1.0 / 5040.0);
    ps = fma(ps, z, 1.0 / 120.0);
    ps = fma(ps, z, -1.0 / 6.0);
    const double sx = fma(ps * z, x, x);
    double pc = 1.0 / 20922789888000.0;  // 1 / 16!
    pc = fma(pc, z, -1.0 / 87178291200.0);
    pc = fma(pc, z, 1.0 / 479001600.0);
    pc = fma(pc, z, -1.0 / 3628800.0);
    pc = fma(pc, z, 1.0 / 40320.0);
    pc = fma(pc, z, -1.0 / 720.0);
    pc = fma(pc, z, 1.0 / 24.0);
    pc = fma(pc, z, -0.5);
    const double cx = fma(pc, z, 1.0);
    const int q = (int)(n - 4.0 * floor(n * 0.25));
    s = q & 1 ? cx : sx;
    c = q & 1 ? sx : cx;
    if (q & 2) s = -s;
    if (q == 1 || q == 2) c = -c;
}

// The workgroup's table of {cos, sin} [tokens][pairs], times the amplitude,
// rounded to FP32: computed once for all heads of its tokens.
__device__ __forceinline__ void rope_table(const RopeArgs& r, int token0, int tokens, f32x2* table) {
    for (int i = threadIdx.x; i < tokens * r.pairs; i += 256) {
        const int t = i / r.pairs;
        double s, c;
        sincos64((double)r.positions[token0 + t] * (double)r.frequencies[i - t * r.pairs], s, c);
        table[i] = f32x2{(float)(c * r.amplitude), (float)(s * r.amplitude)};
    }
}

// One pair: every product and sum rounded to FP32, none fused, so that the
// rotated keys, and with them their FP4 codes, are the same everywhere.
__device__ __forceinline__ void rotate(float a, float b, f32x2 cs, float& x, float& y) {
#pragma clang fp contract(off)
    const float ac = a * cs.x, bs = b * cs.y, bc = b * cs.x, as = a * cs.y;
    x = ac - bs;
    y = bc + as;
}

template <int ACT>
__device__ __forceinline__ float widen1(uint16_t v) {
    if constexpr (ACT == 0) return __uint_as_float((uint32_t)v << 16);
    else return (float)__builtin_bit_cast(_Float16, v);
}
template <int ACT>
__device__ __forceinline__ uint16_t narrow1(float v) {
    return (uint16_t)(pack_out<ACT>(v, 0.0f) & 0xFFFFu);
}

// How the two elements of a pair lie: neighbours; halves whose distance is a
// whole number of 16-byte vectors; halves at any distance.
enum { kPairs = 0, kHalves = 1, kHalvesAny = 2 };

// Work items of a head: item p rotates what it reads and writes it, so that the
// output may be the input.
template <int KIND>
__device__ __forceinline__ int rope_items(int head_dim, int rotary) {
    if constexpr (KIND == kPairs) return head_dim / 8;
    if constexpr (KIND == kHalves) return rotary / 16 + (head_dim - rotary) / 8;
    return rotary / 2 + (head_dim - rotary);
}

template <int ACT, int KIND>
__device__ __forceinline__ void rope_item(const uint16_t* x, uint16_t* y, int p, const RopeArgs& r,
                                          const f32x2* cs) {
    if constexpr (KIND == kPairs) {
        u32x4 v = *reinterpret_cast<const u32x4*>(x + 8 * p);
        if (8 * p < r.rotary) {
            float f[8];
            widen8<ACT>(v, f);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * p + i < r.pairs) {
                    rotate(f[2 * i], f[2 * i + 1], cs[4 * p + i], f[2 * i], f[2 * i + 1]);
                    v[i] = pack_out<ACT>(f[2 * i], f[2 * i + 1]);
                }
        }
        *reinterpret_cast<u32x4*>(y + 8 * p) = v;
    } else if constexpr (KIND == kHalves) {
        const int n = r.pairs / 8;
        if (p < n) {
            float a[8], b[8];
            widen8<ACT>(*reinterpret_cast<const u32x4*>(x + 8 * p), a);
            widen8<ACT>(*reinterpret_cast<const u32x4*>(x + r.pairs + 8 * p), b);
#pragma unroll
            for (int i = 0; i < 8; ++i) rotate(a[i], b[i], cs[8 * p + i], a[i], b[i]);
            *reinterpret_cast<u32x4*>(y + 8 * p) = narrow8<ACT>(a);
            *reinterpret_cast<u32x4*>(y + r.pairs + 8 * p) = narrow8<ACT>(b);
        } else {
            const int d = r.rotary + 8 * (p - n);
            *reinterpret_cast<u32x4*>(y + d) = *reinterpret_cast<const u32x4*>(x + d);
        }
    } else {
        if (p < r.pairs) {
            float a, b;
            rotate(widen1<ACT>(x[p]), widen1<ACT>(x[p + r.pairs]), cs[p], a, b);
            y[p] = narrow1<ACT>(a);
            y[p + r.pairs] = narrow1<ACT>(b);
        } else {
            y[p + r.pairs] = x[p + r.pairs];
        }
    }
}

// Heads [h0, h1) of `tokens` tokens.
template <int ACT, int KIND>
__device__ __forceinline__ void rope_heads(const Rows& x, const RowsOut& y, int head_dim, int token0, int tokens,
                                           int h0, int h1, const RopeArgs& r, const f32x2* table) {
    const uint32_t per = (uint32_t)rope_items<KIND>(head_dim, r.rotary), heads = (uint32_t)(h1 - h0);
    for (uint32_t i = threadIdx.x; i < tokens * heads * per; i += 256) {
        const uint32_t th = i / per, t = th / heads;
        const int h = h0 + (int)(th - t * heads), p = (int)(i - th * per);
        rope_item<ACT, KIND>(x.p + (token0 + t) * x.ts + h * x.hs, y.p + (token0 + t) * y.ts + h * y.hs, p, r,
                             table + t * r.pairs);
    }
}

// Elements d .. d + 7 of a rotated key row, rounded to the row's type: what
// rope_item writes.
template <int ACT, int KIND>
__device__ __forceinline__ void rope_eight(const uint16_t* x, int d, const RopeArgs& r, const f32x2* cs,
                                           float (&f)[8]) {
    const u32x4 own = *reinterpret_cast<const u32x4*>(x + d);
    widen8<ACT>(own, f);
    if (d >= r.rotary) return;
    if constexpr (KIND == kPairs) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (d / 2 + i < r.pairs) rotate(f[2 * i], f[2 * i + 1], cs[d / 2 + i], f[2 * i], f[2 * i + 1]);
    } else if constexpr (KIND == kHalves) {
        const bool first = d < r.pairs;
        const int other = first ? d + r.pairs : d - r.pairs, p = first ? d : other;
        float g[8];
        widen8<ACT>(*reinterpret_cast<const u32x4*>(x + other), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float u, v;
            rotate(first ? f[i] : g[i], first ? g[i] : f[i], cs[p + i], u, v);
            f[i] = first ? u : v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = d + i;
            if (e < r.rotary) {
                const bool first = e < r.pairs;
                const int p = first ? e : e - r.pairs;
                float u, v;
                rotate(widen1<ACT>(x[p]), widen1<ACT>(x[p + r.pairs]), cs[p], u, v);
                f[i] = first ? u : v;
            }
        }
    }
    widen8<ACT>(narrow8<ACT>(f), f);
}

// A workgroup takes `tile` tokens and the heads of its share (blockIdx.y).
template <int ACT, int KIND>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs r, Rows x, RowsOut y, int tokens, int tile, int heads,
                                                   int head_dim) {
    extern __shared__ f32x2 table[];
    const int token0 = blockIdx.x * tile, n = min(tile, tokens - token0);
    rope_table(r, token0, n, table);
    __syncthreads();
    const int h0 = (int)((int64_t)heads * blockIdx.y / gridDim.y);
    const int h1 = (int)((int64_t)heads * (blockIdx.y + 1) / gridDim.y);
    rope_heads<ACT, KIND>(x, y, head_dim, token0, n, h0, h1, r, table);
}

// One block of G elements of one token and head, keys rotated first, quantized
// and scattered as kv_append does.
template <int FMT, int ACT, int D, int KIND>
__device__ __forceinline__ void append_block(const KvArgs& c, const RopeArgs& r, const Rows& x, bool is_v, int token,
                                             int64_t slot, int h, int g, const f32x2* cs) {
    constexpr int G = KvTile<FMT, D>::G;
    const uint16_t* row = x.p + token * x.ts + h * x.hs;
    float f[G];
#pragma unroll
    for (int w = 0; w < G / 8; ++w) {
        float e[8];
        if (is_v) widen8<ACT>(*reinterpret_cast<const u32x4*>(row + g * G + 8 * w), e);
        else rope_eight<ACT, KIND>(row, g * G + 8 * w, r, cs, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[8 * w + i] = e[i];
    }
    kv_store_block<FMT, D>(c, slot, h, g, is_v, f);
}

// Shares of blockIdx.y: first the query heads' (q_parts), then the KV heads'.
// The 4 GP threads of four tokens and one head lie together (kv_append_kernel).
template <int FMT, int ACT, int D, int KIND>
__global__ __launch_bounds__(256) void append_rope_kernel(KvArgs c, RopeArgs r, Rows q, RowsOut qo, Rows k, Rows v,
                                                          const int64_t* __restrict__ slots, int tokens, int tile,
                                                          int q_heads, int q_parts) {
    extern __shared__ f32x2 table[];
    constexpr int GP = D / KvTile<FMT, D>::G;
    const int token0 = blockIdx.x * tile, n = min(tile, tokens - token0);
    rope_table(r, token0, n, table);
    __syncthreads();
    int part = blockIdx.y;
    if (part < q_parts) {
        const int h0 = (int)((int64_t)q_heads * part / q_parts), h1 = (int)((int64_t)q_heads * (part + 1) / q_parts);
        rope_heads<ACT, KIND>(q, qo, D, token0, n, h0, h1, r, table);
        return;
    }
    part -= q_parts;
    const int parts = gridDim.y - q_parts;
    const int b0 = (int)((int64_t)2 * c.kv_heads * part / parts), b1 = (int)((int64_t)2 * c.kv_heads * (part + 1) / parts);
    const int per = (n + 3) / 4 * 4 * GP;
    for (int i = threadIdx.x; i < (b1 - b0) * per; i += 256) {
        const int hv = i / per, m = i - hv * per;  // keys of all heads, then values
        const int t = m / (4 * GP) * 4 + m % 4, g = m / 4 % GP;
        if (t >= n) continue;
        const int64_t slot = slots[token0 + t];
        if (slot < 0 || slot >= c.slots) continue;
        const bool is_v = b0 + hv >= c.kv_heads;
        append_block<FMT, ACT, D, KIND>(c, r, is_v ? v : k, is_v, token0 + t, slot,
                                        is_v ? b0 + hv - c.kv_heads : b0 + hv, g, table + t * r.pairs);
    }
}

static int rope_kind(const fp4_rope_args* r) {
    return r->interleaved ? kPairs : r->rotary % 16 == 0 ? kHalves : kHalvesAny;
}

static int rope_check(const fp4_rope_args* r, int64_t tokens, int64_t head_dim, RopeArgs* a) {
    if (!r) return FP4_ERR_NULL;
    if (r->rotary < 2 || r->rotary > head_dim || r->rotary % 2) return FP4_ERR_SHAPE;
    if (!(r->amplitude >= 0x1p-20f) || !(r->amplitude <= 0x1p20f)) return FP4_ERR_VALUE;
    if (tokens < 0 || tokens > (int64_t(1) << 24)) return FP4_ERR_SHAPE;
    a->positions = r->positions;
    a->frequencies = r->frequencies;
    a->rotary = (int)r->rotary;
    a->pairs = (int)(r->rotary / 2);
    a->amplitude = r->amplitude;
    return FP4_OK;
}

static int rope_pointers(const RopeArgs& a) {
    if (!a.positions || !a.frequencies) return FP4_ERR_NULL;
    return (reinterpret_cast<uintptr_t>(a.positions) & 7) || (reinterpret_cast<uintptr_t>(a.frequencies) & 3)
               ? FP4_ERR_SHAPE : FP4_OK;
}

// Tokens a launch covers: its work-items are counted in 32 bits.
constexpr int64_t kRopeSliceTokens = int64_t(1) << 20;

// Tokens of a workgroup and shares of the heads.
static int rope_tile(int64_t tokens) { return tokens >= 2048 ? 8 : 4; }

static int rope_parts(int64_t tokens, int tile, int64_t items) {
    // enough workgroups for the GPU, each with 256 items at least
    const int64_t groups = (tokens + tile - 1) / tile, want = (2048 + groups - 1) / groups;
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, items * tile / 256));
}

template <int ACT>
static void rope_t(int kind, const RopeArgs& r, const Rows& x, const RowsOut& y, int tokens, int heads, int head_dim,
                   hipStream_t s) {
    const int tile = rope_tile(tokens);
    const dim3 grid((unsigned)((tokens + tile - 1) / tile),
                    (unsigned)std::min(heads, rope_parts(tokens, tile, (int64_t)heads * (head_dim / 8)))),
        block(256);
    const size_t lds = (size_t)tile * r.pairs * sizeof(f32x2);
    if (kind == kPairs) rope_kernel<ACT, kPairs><<<grid, block, lds, s>>>(r, x, y, tokens, tile, heads, head_dim);
    else if (kind == kHalves) rope_kernel<ACT, kHalves><<<grid, block, lds, s>>>(r, x, y, tokens, tile, heads, head_dim);
    else rope_kernel<ACT, kHalvesAny><<<grid, block, lds, s>>>(r, x, y, tokens, tile, heads, head_dim);
}

static int rope_impl(const fp4_rope_args* rope, const void* x, void* out, int64_t tokens, int64_t heads,
                     int64_t head_dim, int64_t x_ts, int64_t x_hs, int64_t out_ts, int64_t out_hs, int act_type,
                     void* stream) {
    if (act_type != 0 && act_type != 1) return FP4_ERR_FORMAT;
    if (heads < 0 || heads > 65536 || head_dim < 8 || head_dim > 1024 || head_dim % 8) return FP4_ERR_SHAPE;
    RopeArgs r;
    int st = rope_check(rope, tokens, head_dim, &r);
    if (st != FP4_OK) return st;
    if (tokens == 0 || heads == 0) return FP4_OK;
    if (!x || !out) return FP4_ERR_NULL;
    st = rope_pointers(r);
    if (st != FP4_OK) return st;
    if (!rows_ok(x, x_ts, x_hs) || !rows_ok(out, out_ts, out_hs) || !rows_apart(tokens, heads, head_dim, out_ts, out_hs))
        return FP4_ERR_SHAPE;
    st = check_device();
    if (st != FP4_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    for (int64_t t0 = 0; t0 < tokens; t0 += kRopeSliceTokens) {
        const int n = (int)std::min(kRopeSliceTokens, tokens - t0);
        const Rows in{static_cast<const uint16_t*>(x) + t0 * x_ts, x_ts, x_hs};
        const RowsOut to{static_cast<uint16_t*>(out) + t0 * out_ts, out_ts, out_hs};
        if (act_type == 0) rope_t<0>(rope_kind(rope), r, in, to, n, (int)heads, (int)head_dim, s);
        else rope_t<1>(rope_kind(rope), r, in, to, n, (int)heads, (int)head_dim, s);
        st = launch_status();
        if (st != FP4_OK) return st;
        r.positions += kRopeSliceTokens;
    }
    return FP4_OK;
}

struct AppendRope {
    KvArgs c;
    RopeArgs r;
    Rows q, k, v;
    RowsOut qo;
    const int64_t* slots;
    int tokens, q_heads, kind;
};

template <int FMT, int ACT, int D>
static void append_rope_t(const AppendRope& a, hipStream_t s) {
    constexpr int GP = D / KvTile<FMT, D>::G;
    const int tile = rope_tile(a.tokens);
    const int qp = a.q_heads ? std::min(a.q_heads, rope_parts(a.tokens, tile, (int64_t)a.q_heads * (D / 8))) : 0;
    const int kp = std::min(2 * a.c.kv_heads, rope_parts(a.tokens, tile, (int64_t)2 * a.c.kv_heads * GP));
    const dim3 grid((unsigned)((a.tokens + tile - 1) / tile), (unsigned)(qp + kp)), block(256);
    const size_t lds = (size_t)tile * a.r.pairs * sizeof(f32x2);
    if (a.kind == kPairs)
        append_rope_kernel<FMT, ACT, D, kPairs><<<grid, block, lds, s>>>(a.c, a.r, a.q, a.qo, a.k, a.v, a.slots,
                                                                         a.tokens, tile, a.q_heads, qp);
    else if (a.kind == kHalves)
        append_rope_kernel<FMT, ACT, D, kHalves><<<grid, block, lds, s>>>(a.c, a.r, a.q, a.qo, a.k, a.v, a.slots,
                                                                          a.tokens, tile, a.q_heads, qp);
    else
        append_rope_kernel<FMT, ACT, D, kHalvesAny><<<grid, block, lds, s>>>(a.c, a.r, a.q, a.qo, a.k, a.v, a.slots,
                                                                             a.tokens, tile, a.q_heads, qp);
}

static int append_rope_impl(const fp4_kv_cache* cache, const fp4_rope_args* rope, const fp4_append_rope_args* p,
                            void* stream) {
    AppendRope a{};
    int st = kv_check(cache, &a.c);
    if (st != FP4_OK) return st;
    if (!p) return FP4_ERR_NULL;
    if (p->act_type != 0 && p->act_type != 1) return FP4_ERR_FORMAT;
    st = rope_check(rope, p->tokens, cache->head_dim, &a.r);
    if (st != FP4_OK) return st;
    if (p->q_heads < 0 || p->q_heads > 65536) return FP4_ERR_SHAPE;
    if (p->tokens == 0) return FP4_OK;
    if (!p->k || !p->v || !p->slots || (p->q_heads && (!p->q || !p->q_out))) return FP4_ERR_NULL;
    st = rope_pointers(a.r);
    if (st != FP4_OK) return st;
    if (!rows_ok(p->k, p->k_token_stride, p->k_head_stride) || !rows_ok(p->v, p->v_token_stride, p->v_head_stride) ||
        (reinterpret_cast<uintptr_t>(p->slots) & 7))
        return FP4_ERR_SHAPE;
    if (p->q_heads && (!rows_ok(p->q, p->q_token_stride, p->q_head_stride) ||
                       !rows_ok(p->q_out, p->q_out_token_stride, p->q_out_head_stride) ||
                       !rows_apart(p->tokens, p->q_heads, cache->head_dim, p->q_out_token_stride, p->q_out_head_stride)))
        return FP4_ERR_SHAPE;
    st = check_device();
    if (st != FP4_OK) return st;
    a.q_heads = (int)p->q_heads;
    a.kind = rope_kind(rope);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    for (int64_t t0 = 0; t0 < p->tokens; t0 += kRopeSliceTokens) {
        a.tokens = (int)std::min(kRopeSliceTokens, p->tokens - t0);
        auto rows = [&](const void* x, int64_t ts, int64_t hs) {
            return Rows{static_cast<const uint16_t*>(x) + (x ? t0 * ts : 0), ts, hs};
        };
        a.q = rows(p->q, p->q_token_stride, p->q_head_stride);
        a.k = rows(p->k, p->k_token_stride, p->k_head_stride);
        a.v = rows(p->v, p->v_token_stride, p->v_head_stride);
        a.qo = RowsOut{static_cast<uint16_t*>(p->q_out) + (p->q_out ? t0 * p->q_out_token_stride : 0),
                       p->q_out_token_stride, p->q_out_head_stride};
        a.slots = p->slots + t0;
        FP4_KV_DISPATCH(append_rope_t, cache->format, p->act_type, cache->head_dim, a, s);
        st = launch_status();
        if (st != FP4_OK) return st;
        a.r.positions += kRopeSliceTokens;
    }
    return FP4_OK;
}

}  // namespace fp4

extern "C" int fp4_rope(const fp4_rope_args* rope, const void* x, void* out, int64_t tokens, int64_t heads,
                        int64_t head_dim, int64_t x_token_stride, int64_t x_head_stride, int64_t out_token_stride,
                        int64_t out_head_stride, int act_type, void* stream) {
    return fp4::rope_impl(rope, x, out, tokens, heads, head_dim, x_token_stride, x_head_stride, out_token_stride,
                          out_head_stride, act_type, stream);
}

extern "C" int fp4_kv_append_rope(const fp4_kv_cache* cache, const fp4_rope_args* rope,
                                  const fp4_append_rope_args* args, void* stream) {
    return fp4::append_rope_impl(cache, rope, args, stream);
}
