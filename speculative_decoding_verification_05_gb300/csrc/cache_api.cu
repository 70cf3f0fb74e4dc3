// C ABI of the paged cache: argument validation, workspace layout and launch
// configuration of the attention, append, compact, resize and fork calls.
// Every call checks its arguments before touching CUDA.

#include <algorithm>
#include <cmath>

#include "attention.cuh"
#include "cache.cuh"
#include "specverify.h"

namespace sv {
spec_status note_cuda_error(cudaError_t e);
}

namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxB = 65535;
constexpr int kSms = 152;  // of a GB300; a fixed grid keeps results independent of the device's count

size_t al(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

spec_status done(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : sv::note_cuda_error(e); }

int esize(spec_dtype d) { return d == SPEC_F32 ? 4 : 2; }

bool dtype_ok(spec_dtype d) { return d == SPEC_F32 || d == SPEC_BF16; }

bool page_ok(int page_size) {
    return page_size >= 8 && page_size <= SPEC_MAX_PAGE && (page_size & (page_size - 1)) == 0;
}

int shift_of(int page_size) {
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

// Whether n ints from a and m ints from b (null: none) share any.
bool overlap(const int32_t* a, size_t n, const int32_t* b, size_t m) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + 4 * m && y < x + 4 * n;
}

bool dim_ok(int D) { return D >= 8 && D <= SPEC_MAX_HEAD_DIM && D % 8 == 0; }

bool cache_ok(const spec_cache* c, spec_dtype dtype) {
    if (!c || !dtype_ok(dtype) || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16) ||
        !aligned(c->page_refs, 4))
        return false;
    if (c->layers < 1 || c->num_pages < 1 || c->num_pages > (1 << 30) || !page_ok(c->page_size) || c->kv_heads < 1 ||
        c->kv_heads > 1024 || !dim_ok(c->head_dim))
        return false;
    const int64_t per16 = 16 / esize(dtype);
    for (const int64_t s : {c->layer_stride, c->page_stride, c->token_stride, c->head_stride})
        if (s < 0 || s % per16 != 0) return false;
    return true;
}

bool table_ok(const int32_t* table, int64_t stride, int max_pages) {
    return table && aligned(table, 4) && max_pages >= 1 && max_pages <= (1 << 26) && stride >= max_pages;
}

sv::CacheView view_of(const spec_cache* c, spec_dtype dtype) {
    const int es = esize(dtype);
    sv::CacheView v = {};
    v.k = static_cast<char*>(c->k);
    v.v = static_cast<char*>(c->v);
    v.layer_stride = c->layer_stride * es;
    v.page_stride = c->page_stride * es;
    v.token_stride = c->token_stride * es;
    v.head_stride = c->head_stride * es;
    v.layers = c->layers;
    v.num_pages = c->num_pages;
    v.page_shift = shift_of(c->page_size);
    v.heads = c->kv_heads;
    v.row_bytes = c->head_dim * es;
    v.refs = c->page_refs;
    return v;
}

// The attention's grid and workspace: functions of the shape alone.
sv::AttnPlan attention_layout(sv::AttnPlan a, int D) {
    size_t o = 0;
    a.part_o = o;
    o = al(o + (size_t)2 * a.grid * a.rows * D * sizeof(float));
    a.part_ml = o;
    o = al(o + (size_t)2 * a.grid * a.rows * sizeof(float2));
    a.joins = o;
    o = al(o + (size_t)a.grid * sizeof(sv::AttnJoin));
    a.total = o;
    return a;
}

sv::AttnPlan simt_plan(int D, spec_dtype dtype, bool many) {
    const int dt = dtype == SPEC_F32 ? 0 : 1;
    sv::AttnPlan a = {};
    a.rows = sv::attention_simt_rows(many);
    a.kv = sv::attention_simt_kv(dt, D, many);
    a.grid = kSms * sv::attention_simt_ctas(dt, D, many);
    a.extra = sv::attention_simt_extra();
    return attention_layout(a, D);
}

sv::AttnPlan tc_plan(int D, int group, int N) {
    sv::AttnPlan a = {};
    a.rows = sv::attention_tc_rows(group);
    a.kv = sv::attention_tc_kv();
    a.grid = kSms;
    a.extra = sv::attention_tc_extra(group, N);
    return attention_layout(a, D);
}

bool tc_shape(int D, spec_dtype dtype) { return dtype == SPEC_BF16 && (D == 64 || D == 128); }

size_t attention_bytes(int D, int group, spec_dtype dtype) {
    const size_t simt = std::max(simt_plan(D, dtype, false).total, simt_plan(D, dtype, true).total);
    return tc_shape(D, dtype) ? std::max(simt, tc_plan(D, group, 1).total) : simt;
}

bool attention_shape_ok(int B, int N, int q_heads, int kv_heads, int D) {
    return B >= 1 && B <= kMaxB && N >= 1 && N <= SPEC_MAX_TREE_N && kv_heads >= 1 && kv_heads <= 1024 &&
           q_heads >= kv_heads && q_heads % kv_heads == 0 && q_heads / kv_heads <= SPEC_MAX_GROUP && dim_ok(D);
}

}  // namespace

extern "C" {

size_t spec_tree_attention_workspace_size(int B, int N, int q_heads, int kv_heads, int head_dim, spec_dtype dtype) {
    if (!attention_shape_ok(B, N, q_heads, kv_heads, head_dim) || !dtype_ok(dtype)) return 0;
    return attention_bytes(head_dim, q_heads / kv_heads, dtype);
}

spec_status spec_tree_attention(const void* q, const spec_cache* cache, spec_dtype dtype,
                                const int32_t* page_table, int64_t table_stride, int max_pages,
                                const int32_t* cache_len, const uint8_t* mask, const int32_t* n_nodes,
                                int B, int N, int q_heads, float scale, void* out, float* lse, int32_t* status,
                                void* workspace, size_t ws_bytes, spec_stream stream) {
    if (!cache_ok(cache, dtype) || cache->layers != 1 || !table_ok(page_table, table_stride, max_pages))
        return SPEC_EINVAL;
    if (!attention_shape_ok(B, N, q_heads, cache->kv_heads, cache->head_dim)) return SPEC_EINVAL;
    if (!q || !out || !cache_len || !workspace || !aligned(q, 16) || !aligned(out, 16) || !aligned(cache_len, 4) ||
        !aligned(n_nodes, 4) || !aligned(lse, 4) || !aligned(status, 4) || !aligned(workspace, kAlign))
        return SPEC_EINVAL;
    const float c2 = scale * 1.4426950408889634f;
    if (!std::isfinite(scale) || !std::isfinite(c2)) return SPEC_EINVAL;
    // a sequence's tiles (16 rows x 32 positions at the least) are counted in 32 bits
    const double row_tiles = (double)cache->kv_heads * ((N * (q_heads / cache->kv_heads) + 15) / 16);
    if (row_tiles * ((double)max_pages * cache->page_size / 32 + 8) >= 2147483648.0) return SPEC_EINVAL;
    if (ws_bytes < attention_bytes(cache->head_dim, q_heads / cache->kv_heads, dtype)) return SPEC_EINVAL;
    sv::AttnParams p = {};
    p.q = q;
    p.k = cache->k;
    p.v = cache->v;
    p.page_stride = cache->page_stride;
    p.token_stride = cache->token_stride;
    p.head_stride = cache->head_stride;
    p.table = page_table;
    p.table_stride = table_stride;
    p.cache_len = cache_len;
    p.mask = mask;
    p.n_nodes = n_nodes;
    p.B = B;
    p.N = N;
    p.Hkv = cache->kv_heads;
    p.G = q_heads / cache->kv_heads;
    p.D = cache->head_dim;
    p.num_pages = cache->num_pages;
    p.max_pages = max_pages;
    p.page_shift = shift_of(cache->page_size);
    p.c2 = c2;
    p.out = out;
    p.lse = lse;
    p.status = status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto use = [&](const sv::AttnPlan& plan) {
        p.tile_rows = plan.rows;
        p.extra = plan.extra;
        p.whole = plan.whole;
        p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.part_o);
        p.part_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + plan.part_ml);
        p.joins = reinterpret_cast<sv::AttnJoin*>(static_cast<char*>(workspace) + plan.joins);
    };
    // Whole units: no more of them than CTAs, of `most` tiles at the most, and not
    // so few that a shared unit's part would be three tiles less (a join costs as
    // much). bf16, units of 8 rows and 128 columns, split and whole: 96 of 2 tiles
    // 14.2 and 11.1 us, of 4 17.4 and 13.6; 40 of 4 13.9 and 13.1; 8 of 2 11.8 and
    // 9.7. float32 tiles take longer than a join: 96 units of 2 tiles (64 columns)
    // 11.8 and 10.0, of 4 14.1 and 17.8. The tiles are those that the page table's
    // width allows (lengths are known on the device only): a table as wide as the
    // longest sequence may get has its units split.
    auto whole = [&](sv::AttnPlan plan, int most) {
        const double units = (double)B * p.Hkv * ((N * p.G + plan.rows - 1) / plan.rows);
        const double tiles = std::ceil((double)max_pages * cache->page_size / plan.kv);
        plan.whole = units <= plan.grid && tiles <= most && tiles - units * (tiles + plan.extra) / plan.grid <= 3.0;
        return plan;
    };
    sv::AttnMaps maps;
    // (that kernel takes the maximum before the scale: it has to be positive)
    if (tc_shape(p.D, dtype) && scale > 0.f && sv::attention_tc_maps(p, &maps)) {
        const sv::AttnPlan plan = whole(tc_plan(p.D, p.G, N), sv::attention_tc_whole());
        use(plan);
        return done(sv::launch_attention_tc(p, plan, maps, st));
    }
    const sv::AttnPlan plan = whole(simt_plan(p.D, dtype, sv::attention_simt_many(N * p.G, p.D)), sv::attention_simt_whole());
    use(plan);
    return done(sv::launch_attention_simt(p, dtype == SPEC_F32 ? 0 : 1, plan, st));
}

spec_status spec_cache_append(const void* k, const void* v, const spec_cache* cache, spec_dtype dtype,
                              const int32_t* page_table, int64_t table_stride, int max_pages,
                              const int32_t* cache_len, const int32_t* n_nodes, int B, int N, int32_t* status,
                              spec_stream stream) {
    if (!cache_ok(cache, dtype) || cache->layers != 1 || !table_ok(page_table, table_stride, max_pages))
        return SPEC_EINVAL;
    if (B < 1 || B > kMaxB || N < 1 || N > (1 << 20) || !k || !v || !cache_len || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(cache_len, 4) || !aligned(n_nodes, 4) || !aligned(status, 4))
        return SPEC_EINVAL;
    sv::AppendParams p = {};
    p.c = view_of(cache, dtype);
    p.k = static_cast<const char*>(k);
    p.v = static_cast<const char*>(v);
    p.table = page_table;
    p.table_stride = table_stride;
    p.cache_len = cache_len;
    p.n_nodes = n_nodes;
    p.status = status;
    p.B = B;
    p.N = N;
    p.max_pages = max_pages;
    return done(sv::launch_append(p, reinterpret_cast<cudaStream_t>(stream)));
}

spec_status spec_cache_compact(const spec_cache* cache, spec_dtype dtype, const int32_t* page_table,
                               int64_t table_stride, int max_pages, const int32_t* cache_len,
                               const int32_t* accept_len, const int32_t* path_nodes, int B, int W,
                               int32_t* new_len, int32_t* status, spec_stream stream) {
    if (!cache_ok(cache, dtype) || !table_ok(page_table, table_stride, max_pages)) return SPEC_EINVAL;
    if (B < 1 || B > kMaxB || W < 1 || W > SPEC_MAX_TREE_N || !cache_len || !accept_len || !new_len ||
        !aligned(cache_len, 4) || !aligned(accept_len, 4) || !aligned(path_nodes, 4) || !aligned(new_len, 4) ||
        !aligned(status, 4))
        return SPEC_EINVAL;
    // (one block of a sequence writes these while its others still read those)
    const int32_t* const in[] = {cache_len, accept_len, path_nodes};
    for (int i = 0; i < 3; ++i) {
        const size_t n = (size_t)B * (i == 2 ? W : 1);
        if (overlap(in[i], n, new_len, B) || overlap(in[i], n, status, B)) return SPEC_EINVAL;
    }
    if (overlap(new_len, B, status, B)) return SPEC_EINVAL;
    sv::CompactParams p = {};
    p.c = view_of(cache, dtype);
    p.table = page_table;
    p.table_stride = table_stride;
    p.cache_len = cache_len;
    p.accept_len = accept_len;
    p.path = path_nodes;
    p.new_len = new_len;
    p.status = status;
    p.B = B;
    p.W = W;
    p.max_pages = max_pages;
    return done(sv::launch_compact(p, reinterpret_cast<cudaStream_t>(stream)));
}

spec_status spec_cache_resize(int32_t* page_table, int64_t table_stride, int max_pages, int num_seqs,
                              int32_t* page_refs, int num_pages, int page_size, const int32_t* seqs,
                              const int32_t* tokens, int F, int32_t* status, spec_stream stream) {
    if (!table_ok(page_table, table_stride, max_pages) || num_seqs < 1 || num_pages < 1 || num_pages > (1 << 30) ||
        !page_ok(page_size) || F < 1 || F > SPEC_MAX_POOL_SEQS || F > num_seqs)
        return SPEC_EINVAL;
    if (!page_refs || !tokens || !aligned(page_refs, 4) || !aligned(tokens, 4) || !aligned(seqs, 4) ||
        !aligned(status, 4))
        return SPEC_EINVAL;
    sv::PoolParams p = {};
    p.table = page_table;
    p.table_stride = table_stride;
    p.refs = page_refs;
    p.status = status;
    p.S = num_seqs;
    p.F = F;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.page_shift = shift_of(page_size);
    p.seqs = seqs;
    p.tokens = tokens;
    return done(sv::launch_resize(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t spec_cache_fork_workspace_size(int F) {
    if (F < 1 || F > SPEC_MAX_POOL_SEQS) return 0;
    return al((size_t)F * sizeof(int4));
}

spec_status spec_cache_fork(const spec_cache* cache, spec_dtype dtype, int32_t* page_table, int64_t table_stride,
                            int max_pages, int num_seqs, int32_t* page_refs, int32_t* cache_len, const int32_t* src,
                            const int32_t* dst, int F, int32_t* status, void* workspace, size_t ws_bytes,
                            spec_stream stream) {
    if (!cache_ok(cache, dtype) || !table_ok(page_table, table_stride, max_pages) || num_seqs < 1 || F < 1 ||
        F > SPEC_MAX_POOL_SEQS || F > num_seqs)
        return SPEC_EINVAL;
    if (!page_refs || !cache_len || !src || !dst || !workspace || !aligned(page_refs, 4) || !aligned(cache_len, 4) ||
        !aligned(src, 4) || !aligned(dst, 4) || !aligned(status, 4) || !aligned(workspace, kAlign) ||
        ws_bytes < spec_cache_fork_workspace_size(F))
        return SPEC_EINVAL;
    sv::PoolParams p = {};
    p.table = page_table;
    p.table_stride = table_stride;
    p.refs = page_refs;
    p.status = status;
    p.S = num_seqs;
    p.F = F;
    p.max_pages = max_pages;
    p.num_pages = cache->num_pages;
    p.page_shift = shift_of(cache->page_size);
    p.cache_len = cache_len;
    p.src = src;
    p.dst = dst;
    p.copies = static_cast<int4*>(workspace);
    return done(sv::launch_fork(p, view_of(cache, dtype), reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
