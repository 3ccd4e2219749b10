// C entry of the attention over the FP4 key/value cache: checks, shape choice,
// launch (include/fp4gemm.h, fp4_attention).
#include <cmath>

#include "attention.h"

namespace fp4 {

int kv_check(const fp4_kv_cache* c, KvArgs* a);  // kv_cache.hip
bool rows_apart(int64_t tokens, int64_t heads, int64_t D, int64_t ts, int64_t hs);

struct AttnPlan {
    bool tiled;
    int MT, grid, splits;
    size_t ml_off, word_off, ws_bytes;
};

// Checks of everything that the plan depends on, and the plan.
static int attn_plan(const KvArgs& c, int64_t D, const fp4_attention_args& x, AttnPlan* p) {
    if (x.batch < 0 || x.batch > (int64_t(1) << 24) || x.q_rows < 0 || x.q_rows > (int64_t(1) << 24) ||
        x.q_heads < c.kv_heads || x.q_heads % c.kv_heads || x.q_heads / c.kv_heads > 1024 ||
        x.q_rows * x.q_heads >= (int64_t(1) << 31) || x.max_q < 0 || x.page_columns < 1 ||
        x.page_columns > (int64_t(1) << 31) || x.page_columns * c.page_size >= (int64_t(1) << 31))
        return FP4_ERR_SHAPE;
    const int64_t group = x.q_heads / c.kv_heads;
    int64_t each = x.max_q > 0 ? std::min(x.max_q, x.q_rows) : x.q_rows;
    if (!x.q_offsets && x.batch > 0) each = x.q_rows / x.batch;
    const int64_t rows = each * group;
    p->MT = rows <= 16 ? 1 : (rows <= 32 || D == 256) ? 2 : 4;
    // The tiled kernel, its items cut into shares where they do not fill the
    // GPU.  Measured (us, streaming / tiled; 64 query and 8 KV heads, 8192 keys):
    // head size 128: 32 query tokens 40 / 43, 64 (512 rows) 60 / 53, 128 103 / 67,
    // 512 361 / 138; head size 64: 32 25 / 33, 64 35 / 35, 128 60 / 46, 512 184 / 88;
    // head size 256 (16, 4): 64 (256 rows) 46 / 43, 128 64 / 55, 192 (768 rows)
    // 84 / 86, 256 104 / 72, uneven as the numbers of shares are.  With many
    // sequences its partly filled blocks pay earlier: 32 sequences of 16 tokens (128
    // rows), 4000 keys 207 / 120 (head size 64: 106 / 83); but 16 of 8 tokens (64
    // rows) 61 / 70.
    const int64_t tiled = tiled_rows((int)D);
    const int64_t tiled_items = (x.q_rows * group / tiled + x.batch) * c.kv_heads;
    p->tiled = rows >= (D == 256 ? 768 : 512) || (rows >= 128 && x.batch * c.kv_heads >= 128);
    if (p->tiled) {
        p->splits = (int)std::min<int64_t>(16, std::max<int64_t>(1, 320 / tiled_items));
        if (tiled_items * p->splits >= (int64_t(1) << 23)) return FP4_ERR_SHAPE;  // a launch's work-items fit 32 bits
        p->grid = (int)(tiled_items * p->splits);
        const size_t slots = p->splits > 1 ? (size_t)p->grid : 0;
        p->ml_off = slots * tiled * D * 4;
        p->word_off = p->ml_off + slots * 512 * 8;
        p->ws_bytes = p->word_off + (p->splits > 1 ? (size_t)tiled_items * 8 : 0);
        return FP4_OK;
    }
    p->splits = 1;
    const int64_t R = 16 * p->MT;
    // every sequence has at most one partly filled row block
    const int64_t items = (x.q_rows * group / R + x.batch) * c.kv_heads;
    const int64_t unit_keys = kUnitTiles * kKvTile;
    const int64_t units = (x.page_columns * c.page_size + unit_keys - 1) / unit_keys + 1;
    // as many workgroups as the GPU holds at a time
    const int64_t most = 256 * attn_waves((int)D, p->MT);
    if (items > (int64_t(1) << 30) || items * (units + kItemCost) >= (int64_t(1) << 31) - most) return FP4_ERR_SHAPE;
    p->grid = (int)std::max<int64_t>(1, std::min(most, items * units));
    static_assert(256 * attn_waves(64, 1) / kTeam < 1 << kCountBits && kTeam < 1 << kCountBits, "arrivals at a word");
    const size_t slots = 2 * (size_t)p->grid;
    p->ml_off = slots * R * D * 4;
    p->word_off = p->ml_off + slots * R * 8;
    p->ws_bytes = p->word_off + slots * 8;
    return FP4_OK;
}

static bool attn_rows_ok(const void* p, int64_t ts, int64_t hs) {
    const int64_t most = int64_t(1) << 40;
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ts >= 0 && hs >= 0 && ts < most && hs < most && ts % 8 == 0 &&
           hs % 8 == 0;
}

static int attention_impl(const fp4_kv_cache* cache, const fp4_attention_args* x, void* stream) {
    if (!x) return FP4_ERR_NULL;
    KvArgs c;
    int st = kv_check(cache, &c);
    if (st != FP4_OK) return st;
    AttnPlan p;
    st = attn_plan(c, cache->head_dim, *x, &p);
    if (st != FP4_OK) return st;
    if (x->act_type != 0 && x->act_type != 1) return FP4_ERR_FORMAT;
    if ((x->causal != 0 && x->causal != 1) || x->window < 0 || (x->window > 0 && !x->causal) || !(x->scale > 0.0f) ||
        !alpha_ok(x->scale))
        return FP4_ERR_VALUE;
    // the factor of a BF16 query row scaled to FP16 (up to 2^114) stays finite
    const double factor = (double)x->scale * c.k_alpha;
    if (factor < 0x1p-100 || factor > 0x1p12) return FP4_ERR_VALUE;
    if (x->batch == 0 || x->q_rows == 0) return FP4_OK;
    if (!x->q || !x->out || !x->page_table || !x->seq_lens) return FP4_ERR_NULL;
    const int64_t D = cache->head_dim;
    if (!attn_rows_ok(x->q, x->q_token_stride, x->q_head_stride) ||
        !attn_rows_ok(x->out, x->out_token_stride, x->out_head_stride) ||
        !rows_apart(x->q_rows, x->q_heads, D, x->out_token_stride, x->out_head_stride) ||
        (x->page_stride < x->page_columns && x->page_stride != 0) || x->page_stride > (int64_t(1) << 40) ||
        (!x->q_offsets && x->q_rows % x->batch) ||
        ((reinterpret_cast<uintptr_t>(x->lse) | reinterpret_cast<uintptr_t>(x->page_table) |
          reinterpret_cast<uintptr_t>(x->seq_lens) | reinterpret_cast<uintptr_t>(x->q_offsets) |
          reinterpret_cast<uintptr_t>(x->sinks)) & 3))
        return FP4_ERR_SHAPE;
    if (p.ws_bytes > 0 &&
        (!x->workspace || x->workspace_bytes < p.ws_bytes || (reinterpret_cast<uintptr_t>(x->workspace) & 15)))
        return FP4_ERR_WORKSPACE;
    st = check_device();
    if (st != FP4_OK) return st;
    AttnArgs a;
    a.q = static_cast<const uint16_t*>(x->q);
    a.out = static_cast<uint16_t*>(x->out);
    a.lse = x->lse;
    a.page_table = x->page_table;
    a.seq_lens = x->seq_lens;
    a.q_offsets = x->q_offsets;
    a.sinks = x->sinks;
    a.q_ts = x->q_token_stride;
    a.q_hs = x->q_head_stride;
    a.o_ts = x->out_token_stride;
    a.o_hs = x->out_head_stride;
    a.table_stride = x->page_stride;
    a.batch = (int)x->batch;
    a.q_rows = (int)x->q_rows;
    a.q_each = (int)(x->q_rows / x->batch);
    a.q_heads = (int)x->q_heads;
    a.group = (int)(x->q_heads / c.kv_heads);
    a.max_keys = (int)(x->page_columns * c.page_size);
    a.window = (int)std::min<int64_t>(x->window, a.max_keys);
    a.causal = x->causal;
    a.tpp_magic = ((uint64_t(1) << 36) + c.tiles_per_page - 1) / c.tiles_per_page;
    const bool nv = cache->format == FP4_NVFP4;
    a.k_exp = nv ? 0 : std::ilogb(c.k_alpha);
    a.v_exp = nv ? 0 : std::ilogb(c.v_alpha);
    a.scale = x->scale * std::ldexp(c.k_alpha, -a.k_exp) * kLog2e;
    a.v_alpha = std::ldexp(c.v_alpha, -a.v_exp);
    a.inv_group = 1.0f / a.group;
    a.grid = p.grid;
    a.splits = p.splits;
    a.tag = next_split_tag();
    char* ws = static_cast<char*>(x->workspace);
    a.ws_o = reinterpret_cast<float*>(ws);
    a.ws_ml = reinterpret_cast<float*>(ws + p.ml_off);
    a.words = reinterpret_cast<unsigned long long*>(ws + p.word_off);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    const auto launch = nv ? (x->act_type == 0 ? launch_attention_nv_bf16 : launch_attention_nv_f16)
                           : (x->act_type == 0 ? launch_attention_mx_bf16 : launch_attention_mx_f16);
    if (!launch((int)D, p.MT, p.tiled, a, c, s)) return FP4_ERR_SHAPE;
    return launch_status();
}

}  // namespace fp4

extern "C" int fp4_attention_workspace_size(const fp4_kv_cache* cache, const fp4_attention_args* args, size_t* bytes) {
    if (!cache || !args || !bytes) return FP4_ERR_NULL;
    size_t unused;
    int st = fp4_kv_cache_size(cache->pages, cache->page_size, cache->kv_heads, cache->head_dim, cache->format, &unused);
    if (st != FP4_OK) return st;
    fp4::KvArgs c{};
    c.kv_heads = (int)cache->kv_heads;
    c.page_size = (int)cache->page_size;
    fp4::AttnPlan p;
    st = fp4::attn_plan(c, cache->head_dim, *args, &p);
    if (st != FP4_OK) return st;
    *bytes = p.ws_bytes;
    return FP4_OK;
}

extern "C" int fp4_attention(const fp4_kv_cache* cache, const fp4_attention_args* args, void* stream) {
    return fp4::attention_impl(cache, args, stream);
}
