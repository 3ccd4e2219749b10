// Rotary positions (include/fp4gemm.h, section "Rotary positions"): alone, and
// with the write of the rotated keys into the FP4 cache.
#include "apart.h"
#include "kv_layout.h"
#include "mx8.h"

namespace fp4 {

int kv_check(const fp4_kv_cache* c, KvArgs* a);                                              // kv_cache.hip
bool rows_ok(const void* p, int64_t ts, int64_t hs);
bool rows_apart(int64_t tokens, int64_t heads, int64_t D, int64_t ts, int64_t hs);

// Tokens of a workgroup (whole quads: the value codes of four tokens are neighbours),
// and its shares of the heads: enough workgroups for the GPU, each with 256 items at
// least.  8191 tokens of 64 + 8 heads of 128: 65.6 us with 4 tokens, 70 with 8, 73 with 16;
// with 4 tokens and twice the workgroups 71 us.
constexpr int kRopeTile = 4;

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

// kFar: outputs too large for the caches go past them.
template <bool kFar>
__device__ __forceinline__ void store16(uint16_t* p, const u32x4& v) {
    if constexpr (kFar) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
    else *reinterpret_cast<u32x4*>(p) = v;
}

template <int ACT, int KIND, bool kFar>
__device__ __forceinline__ void rope_item(const uint16_t* x, uint16_t* y, int p, const RopeArgs& r,
                                          const f32x2* cs) {
    if constexpr (KIND == kPairs) {
        u32x4 v = load_once(x + 8 * p);
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
        store16<kFar>(y + 8 * p, v);
    } else if constexpr (KIND == kHalves) {
        const int n = r.pairs / 8;
        if (p < n) {
            float a[8], b[8];
            widen8<ACT>(load_once(x + 8 * p), a);
            widen8<ACT>(load_once(x + r.pairs + 8 * p), b);
#pragma unroll
            for (int i = 0; i < 8; ++i) rotate(a[i], b[i], cs[8 * p + i], a[i], b[i]);
            store16<kFar>(y + 8 * p, narrow8<ACT>(a));
            store16<kFar>(y + r.pairs + 8 * p, narrow8<ACT>(b));
        } else {
            const int d = r.rotary + 8 * (p - n);
            store16<kFar>(y + d, load_once(x + d));
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

// Heads [h0, h1) of `tokens` tokens: a thread keeps its item of a head and goes
// through the heads of all tokens.
template <int ACT, int KIND, bool kFar>
__device__ __forceinline__ void rope_heads(const Rows& x, const RowsOut& y, int head_dim, int token0, int tokens,
                                           int h0, int h1, const RopeArgs& r, const f32x2* table) {
    const int per = rope_items<KIND>(head_dim, r.rotary), heads = h1 - h0;
    const int side = min(per, 256), step = 256 / side;  // threads on a head, heads at a time
    if ((int)threadIdx.x >= side * step) return;
    const int row = threadIdx.x / side;
    int t = row / heads, h = row - t * heads;
    while (t < tokens) {
        for (int p = threadIdx.x - row * side; p < per; p += side)
            rope_item<ACT, KIND, kFar>(x.p + (token0 + t) * x.ts + (h0 + h) * x.hs,
                                       y.p + (token0 + t) * y.ts + (h0 + h) * y.hs, p, r, table + t * r.pairs);
        for (h += step; h >= heads; h -= heads) ++t;
    }
}

// What turns the block of G elements from d0 on of one token's keys: element e
// becomes own c[e] + other s[e], other being its pair's other element and s signed
// (a - b s and a + b (-s) round alike).
template <int G, int KIND>
struct BlockTurn {
    float c[G], s[G];
    __device__ __forceinline__ void load(const RopeArgs& r, const f32x2* cs, int d0) {
#pragma unroll
        for (int e = 0; e < G; ++e) {
            const int d = d0 + e;
            const bool first = KIND == kPairs ? d % 2 == 0 : d < r.pairs;
            const f32x2 v = cs[min(KIND == kPairs ? d / 2 : first ? d : d - r.pairs, r.pairs - 1)];
            c[e] = v.x;
            s[e] = first ? -v.y : v.y;
        }
    }
};

// Elements d0 .. d0 + G - 1 of a key row, turned and rounded to the row's type: what
// rope_item writes.
template <int ACT, int KIND, int G>
__device__ __forceinline__ void turned_block(const uint16_t* x, int d0, const RopeArgs& r, const BlockTurn<G, KIND>& turn,
                                             float (&out)[G]) {
#pragma clang fp contract(off)
#pragma unroll
    for (int w = 0; w < G; w += 8) {
        const int d = d0 + w;
        float own[8], other[8] = {};
        widen8<ACT>(*reinterpret_cast<const u32x4*>(x + d), own);
        if constexpr (KIND == kHalves) {
            if (d < r.rotary)
                widen8<ACT>(*reinterpret_cast<const u32x4*>(d < r.pairs ? x + d + r.pairs : x + d - r.pairs), other);
        } else if constexpr (KIND == kPairs) {
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] = own[i ^ 1];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (d + i < r.rotary) other[i] = widen1<ACT>(d + i < r.pairs ? x[d + i + r.pairs] : x[d + i - r.pairs]);
        }
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float oc = own[i] * turn.c[w + i], ts = other[i] * turn.s[w + i];
            y[i] = d + i < r.rotary ? oc + ts : own[i];
        }
        widen8<ACT>(narrow8<ACT>(y), y);
#pragma unroll
        for (int i = 0; i < 8; ++i) out[w + i] = y[i];
    }
}

// A workgroup takes kRopeTile tokens and the heads of its share (blockIdx.y).  Bound by
// the bytes where tokens are many: 64 heads of 128 of 8191 tokens take 51.5 us, 5.2 TB/s;
// where they are few by what one workgroup does in turn: positions and frequencies from
// memory, the table in FP64, a barrier, and only then the first rows (1001 tokens of 36
// heads of 128 in FP16, 64 elements of each turned in pairs: 8.2 us, bytes for 3.5).
// Halves at any distance move single elements: 8191 tokens of 40 heads of 80 take 84 us
// with 20 elements turned, 29 with 32.
template <int ACT, int KIND, bool kFar>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs r, Rows x, RowsOut y, int tokens, int heads,
                                                   int head_dim) {
    extern __shared__ f32x2 table[];
    const int token0 = blockIdx.x * kRopeTile, n = min(kRopeTile, tokens - token0);
    rope_table(r, token0, n, table);
    __syncthreads();
    const int h0 = (int)((int64_t)heads * blockIdx.y / gridDim.y);
    const int h1 = (int)((int64_t)heads * (blockIdx.y + 1) / gridDim.y);
    rope_heads<ACT, KIND, kFar>(x, y, head_dim, token0, n, h0, h1, r, table);
}

// The bytes again, and the scattered stores of the values' codes: 8191 tokens of 64 + 8
// heads of 128 take 65 us; 1 token takes 6.5, the latencies of rope_kernel in turn and
// the slot's behind the table.
// Shares of blockIdx.y: first the KV heads' (kv_parts; their scattered stores take
// longest), then the query heads'.  The 4 GP threads of four tokens and one head lie
// together (kv_append_kernel).
template <int FMT, int ACT, int D, int KIND, bool kFar>
__global__ __launch_bounds__(256) void append_rope_kernel(KvArgs c, RopeArgs r, Rows q, RowsOut qo, Rows k, Rows v,
                                                          const int64_t* __restrict__ slots, int tokens,
                                                          int q_heads, int kv_parts) {
    extern __shared__ f32x2 table[];
    constexpr int GP = D / KvTile<FMT, D>::G;
    const int token0 = blockIdx.x * kRopeTile, n = min(kRopeTile, tokens - token0);
    rope_table(r, token0, n, table);
    __syncthreads();
    int part = blockIdx.y;
    if (part >= kv_parts) {
        part -= kv_parts;
        const int parts = gridDim.y - kv_parts;
        const int h0 = (int)((int64_t)q_heads * part / parts), h1 = (int)((int64_t)q_heads * (part + 1) / parts);
        rope_heads<ACT, KIND, kFar>(q, qo, D, token0, n, h0, h1, r, table);
        return;
    }
    // a thread keeps its token and block, and goes through the heads: keys, then values
    constexpr int G = KvTile<FMT, D>::G;
    const int b0 = 2 * c.kv_heads * part / kv_parts, b1 = 2 * c.kv_heads * (part + 1) / kv_parts;
    const int per = (n + 3) / 4 * 4 * GP, step = 256 / per;
    const int row = threadIdx.x / per, m = threadIdx.x - row * per;
    const int t = m / (4 * GP) * 4 + m % 4, g = m / 4 % GP;
    if (row >= step || t >= n) return;
    const int64_t slot = slots[token0 + t];
    if (slot < 0 || slot >= c.slots) return;
    BlockTurn<G, KIND> turn;
    turn.load(r, table + t * r.pairs, g * G);
    for (int b = b0 + row; b < b1; b += step) {
        const bool is_v = b >= c.kv_heads;
        const int h = is_v ? b - c.kv_heads : b;
        float f[G];
        if (is_v) {
            const uint16_t* x = v.p + (token0 + t) * v.ts + h * v.hs + g * G;
#pragma unroll
            for (int w = 0; w < G; w += 8) {
                float e[8];
                widen8<ACT>(*reinterpret_cast<const u32x4*>(x + w), e);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[w + i] = e[i];
            }
        } else {
            turned_block<ACT, KIND, G>(k.p + (token0 + t) * k.ts + h * k.hs, g * G, r, turn, f);
        }
        kv_store_block<FMT, D>(c, slot, h, g, is_v, f);
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

static int rope_parts(int64_t tokens, int64_t items) {
    const int64_t groups = (tokens + kRopeTile - 1) / kRopeTile, want = (2048 + groups - 1) / groups;
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, items * kRopeTile / 256));
}

// Outputs above this many bytes are stored past the caches.
constexpr int64_t kRopeFar = int64_t(64) << 20;

template <int ACT>
static void rope_t(int kind, const RopeArgs& r, const Rows& x, const RowsOut& y, int tokens, int heads, int head_dim,
                   hipStream_t s) {
    const dim3 grid((unsigned)((tokens + kRopeTile - 1) / kRopeTile),
                    (unsigned)std::min(heads, rope_parts(tokens, (int64_t)heads * (head_dim / 8)))),
        block(256);
    const size_t lds = (size_t)kRopeTile * r.pairs * sizeof(f32x2);
    const bool far = (int64_t)tokens * heads * head_dim * 2 > kRopeFar;
    if (kind == kHalvesAny) rope_kernel<ACT, kHalvesAny, false><<<grid, block, lds, s>>>(r, x, y, tokens, heads, head_dim);
    else if (kind == kPairs && far) rope_kernel<ACT, kPairs, true><<<grid, block, lds, s>>>(r, x, y, tokens, heads, head_dim);
    else if (kind == kPairs) rope_kernel<ACT, kPairs, false><<<grid, block, lds, s>>>(r, x, y, tokens, heads, head_dim);
    else if (far) rope_kernel<ACT, kHalves, true><<<grid, block, lds, s>>>(r, x, y, tokens, heads, head_dim);
    else rope_kernel<ACT, kHalves, false><<<grid, block, lds, s>>>(r, x, y, tokens, heads, head_dim);
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
    const Span to = span_of_rows(out, head_dim, tokens, out_ts, heads, out_hs);
    if (!span_may_be(to, span_of_rows(x, head_dim, tokens, x_ts, heads, x_hs)) ||
        spans_meet(to, span_of(r.positions, tokens * 8)) || spans_meet(to, span_of(r.frequencies, (int64_t)r.pairs * 4)))
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

template <int FMT, int ACT, int D, int KIND, bool kFar>
static void launch_append_rope(const AppendRope& a, hipStream_t s) {
    constexpr int GP = D / KvTile<FMT, D>::G;
    const int qp = a.q_heads ? std::min(a.q_heads, rope_parts(a.tokens, (int64_t)a.q_heads * (D / 8))) : 0;
    const int kp = std::min(2 * a.c.kv_heads, rope_parts(a.tokens, (int64_t)2 * a.c.kv_heads * GP));
    const dim3 grid((unsigned)((a.tokens + kRopeTile - 1) / kRopeTile), (unsigned)(qp + kp)), block(256);
    append_rope_kernel<FMT, ACT, D, KIND, kFar><<<grid, block, (size_t)kRopeTile * a.r.pairs * sizeof(f32x2), s>>>(
        a.c, a.r, a.q, a.qo, a.k, a.v, a.slots, a.tokens, a.q_heads, kp);
}

template <int FMT, int ACT, int D>
static void append_rope_t(const AppendRope& a, hipStream_t s) {
    const bool far = (int64_t)a.tokens * a.q_heads * D * 2 > kRopeFar;
    if (a.kind == kHalvesAny) launch_append_rope<FMT, ACT, D, kHalvesAny, false>(a, s);
    else if (a.kind == kPairs && far) launch_append_rope<FMT, ACT, D, kPairs, true>(a, s);
    else if (a.kind == kPairs) launch_append_rope<FMT, ACT, D, kPairs, false>(a, s);
    else if (far) launch_append_rope<FMT, ACT, D, kHalves, true>(a, s);
    else launch_append_rope<FMT, ACT, D, kHalves, false>(a, s);
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
    // what is written (queries, cache) lies apart from all else of the call
    auto span = [&](const void* x, int64_t ts, int64_t heads, int64_t hs) {
        return span_of_rows(x, cache->head_dim, p->tokens, ts, heads, hs);
    };
    const Span q = span(p->q, p->q_token_stride, p->q_heads, p->q_head_stride);
    const Span qo = span(p->q_out, p->q_out_token_stride, p->q_heads, p->q_out_head_stride);
    const Span held = span_of(a.c.data, (int64_t)a.c.pages * a.c.tiles_per_page * a.c.kv_heads *
                                            kv_tile_bytes(cache->format, cache->head_dim));
    if (!span_may_be(qo, q) || spans_meet(qo, held) || spans_meet(held, q)) return FP4_ERR_SHAPE;
    for (const Span& from : {span(p->k, p->k_token_stride, a.c.kv_heads, p->k_head_stride),
                             span(p->v, p->v_token_stride, a.c.kv_heads, p->v_head_stride), span_of(p->slots, p->tokens * 8),
                             span_of(a.r.positions, p->tokens * 8), span_of(a.r.frequencies, (int64_t)a.r.pairs * 4)})
        if (spans_meet(qo, from) || spans_meet(held, from)) return FP4_ERR_SHAPE;
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
