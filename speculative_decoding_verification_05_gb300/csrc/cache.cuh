// Parameters of the paged-cache kernels (cache.cu).
#pragma once

#include "common.cuh"

namespace sv {

// A cache of `layers` layers: page p, slot s, head h of layer y starts at
// y * layer_stride + p * page_stride + s * token_stride + h * head_stride
// bytes, in k and in v; a head's row is row_bytes long.
struct CacheView {
    char* k;
    char* v;
    long long layer_stride, page_stride, token_stride, head_stride;  // bytes
    int layers, num_pages, page_shift, heads, row_bytes;
    const int32_t* refs;  // [num_pages], or null: not checked
};

struct AppendParams {
    CacheView c;
    const char* k;  // [B, N, heads, D]
    const char* v;
    const int32_t* table;
    long long table_stride;
    const int32_t* cache_len;
    const int32_t* n_nodes;
    int32_t* status;
    int B, N, max_pages;
};

struct RotaryParams {
    CacheView c;
    const char* q;  // [B, N, q_heads, D]
    const char* k;  // [B, N, heads, D]
    const char* v;
    char* q_out;
    const unsigned long long* turns;  // [half] 2^-64 of a turn a position
    float factor;
    int half, interleaved, q_heads;
    const int32_t* table;
    long long table_stride;
    const int32_t* cache_len;
    const int32_t* positions;  // [B] or null (cache_len)
    const int32_t* depth;      // [B, N] or null (the node's number)
    const int32_t* n_nodes;
    int32_t* status;
    int B, N, max_pages;
    int tokens;  // of a block (set by the launcher)
};

struct CompactParams {
    CacheView c;
    const int32_t* table;
    long long table_stride;
    const int32_t* cache_len;
    const int32_t* accept_len;  // [B]
    const int32_t* path;        // [B, W] or null (a chain: nothing moves)
    int32_t* new_len;
    int32_t* status;
    int B, W, max_pages;
};

struct EvictParams {
    CacheView c;
    const int32_t* table;
    long long table_stride;
    const int32_t* cache_len;  // [B]
    const int32_t* budget;     // [B]
    int sink, recent;
    float* weights;      // [layers, B, heads, capacity]
    long long capacity;
    int32_t* new_len;
    int32_t* status;
    int32_t* list;  // [layers, B, heads, capacity] kept positions
    int2* jobs;     // [layers, B, heads] first entry of the list that moves, entries
    int B, max_pages;
};

struct PoolParams {
    int32_t* table;  // [S] rows of table_stride entries
    long long table_stride;
    int32_t* refs;   // [num_pages]
    int32_t* status;
    int S, F, max_pages, num_pages, page_shift;
    // resize
    const int32_t* seqs;    // [F] or null (0 .. F - 1)
    const int32_t* tokens;  // [F]
    // fork
    int32_t* cache_len;  // [S]
    const int32_t* src;  // [F]
    const int32_t* dst;  // [F]
    int4* copies;        // [F] (page from, page to, slots, length)
};

cudaError_t launch_append(const AppendParams& p, cudaStream_t st);
cudaError_t launch_append_rotary(RotaryParams p, int dtype, cudaStream_t st);
cudaError_t launch_compact(const CompactParams& p, cudaStream_t st);
cudaError_t launch_evict(const EvictParams& p, cudaStream_t st);
cudaError_t launch_resize(const PoolParams& p, cudaStream_t st);
cudaError_t launch_fork(const PoolParams& p, const CacheView& c, cudaStream_t st);
cudaError_t debug_read_rotary(unsigned int* count, unsigned int* line);
cudaError_t debug_read_evict(unsigned int* count, unsigned int* line);
cudaError_t debug_read_cache(unsigned int* count, unsigned int* line);

}  // namespace sv
