// The paged key / value cache around a verification step: appending the
// drafted nodes' keys and values, moving an accepted path's entries together,
// and the pages themselves (growing, releasing, sharing).
//
// A page is free iff its reference count is zero; pages are taken lowest
// number first, in the order of the call's sequences, so a table depends on
// the calls alone and no free list is kept. Everything here moves bytes: the
// element type only sets a row's length, and rows are copied as 16-byte words.

#include <algorithm>

#include "cache.cuh"
#include "specverify.h"

namespace sv {
namespace {

constexpr int kENoPages = SPEC_ENOPAGES;
constexpr int CT = 256;

SV_DEV uint4 ldg16(const char* p) { return *reinterpret_cast<const uint4*>(p); }
SV_DEV void stg16(char* p, uint4 x) { *reinterpret_cast<uint4*>(p) = x; }

// Whether pages [first, last] of a sequence exist and, with refs, are its own
// (all threads of the block).
SV_DEV bool pages_ok(const int32_t* table, int first, int last, int num_pages, const int32_t* refs) {
    bool bad = false;
    for (int i = first + (int)threadIdx.x; i <= last; i += blockDim.x) {
        const int id = __ldg(table + i);
        if (id < 0 || id >= num_pages) bad = true;
        else if (refs) bad |= __ldg(refs + id) != 1;
    }
    return !__syncthreads_or(bad);
}

// ---- appending ---------------------------------------------------------------
// Block (x, b) copies a run of sequence b's new rows. A row is a token's
// heads x head_dim elements in the input and heads rows of the page. Bound by
// memory where there is enough of it (8 x 1000 tokens, 32 heads of 128 columns,
// bf16: 40.2 us, 6.0 TB/s read and written), below that by the two dependent
// lookups before the first copy (64 x 8 tokens, 8 heads: 2.4 us).
constexpr int kAppendTokens = 4;

__global__ void __launch_bounds__(CT) append_kernel(const __grid_constant__ AppendParams p) {
    const int b = blockIdx.y, tid = threadIdx.x;
    const long long L = p.cache_len[b];
    const int n = p.n_nodes ? p.n_nodes[b] : p.N;
    const int sh = p.c.page_shift;
    const int32_t* table = p.table + b * p.table_stride;
    bool ok = L >= 0 && n >= 0 && n <= p.N && L + n <= ((long long)p.max_pages << sh);
    if (ok && n > 0) ok = pages_ok(table, (int)(L >> sh), (int)((L + n - 1) >> sh), p.c.num_pages, p.c.refs);
    if (blockIdx.x == 0 && tid == 0 && p.status) p.status[b] = ok ? kOk : kEData;
    if (!ok) return;
    const int per_head = p.c.row_bytes / 16, per_token = p.c.heads * per_head;
    const int t0 = blockIdx.x * kAppendTokens, t1 = min(t0 + kAppendTokens, n);
    for (int i = tid; i < (t1 - t0) * per_token; i += CT) {
        const int t = t0 + i / per_token, c = i % per_token, h = c / per_head;
        const long long pos = L + t;
        const int id = table[pos >> sh];
        if (!SV_IN(id, p.c.num_pages) || !SV_IN(h, p.c.heads)) continue;
        const long long to = (long long)id * p.c.page_stride + (pos & ((1 << sh) - 1)) * p.c.token_stride +
                             h * p.c.head_stride + (c - h * per_head) * 16;
        const long long from = (((long long)b * p.N + t) * per_token + c) * 16;
        const uint4 x = ldg16(p.k + from), y = ldg16(p.v + from);
        stg16(p.c.k + to, x);
        stg16(p.c.v + to, y);
    }
}

// ---- compacting ---------------------------------------------------------------
// The path's nodes ascend (0 = path[0] < path[1] < ...), so node i's place
// L + i is never after its source L + path[i], and a batch of entries read
// before it is written never overwrites a later source. A thread owns one
// 16-byte column of one layer's K or V and walks the path in such batches:
// eight rows in flight a thread, no barrier between them. Bound by latency: the
// path, its pages, the rows (16 sequences, paths to 7, 32 layers, 8 heads of 128
// columns, bf16: 4.4 us; 61 sequences, paths to 17, 12 layers, float32: 5.8 us).
constexpr int kMoves = 8;

__global__ void __launch_bounds__(CT) compact_kernel(const __grid_constant__ CompactParams p) {
    __shared__ long long from[SPEC_MAX_TREE_N], to[SPEC_MAX_TREE_N];
    const int b = blockIdx.y, tid = threadIdx.x;
    const long long L = p.cache_len[b];
    const int a = p.accept_len[b], sh = p.c.page_shift;
    const int32_t* table = p.table + b * p.table_stride;
    const int32_t* path = p.path ? p.path + (long long)b * p.W : nullptr;
    bool ok = L >= 0 && a >= 0 && a < p.W;
    if (ok && path) {
        bool bad = false;
        for (int i = tid; i <= a; i += CT) bad |= i == 0 ? path[0] != 0 : path[i] <= path[i - 1];
        ok = !__syncthreads_or(bad);
    }
    const long long end = ok ? L + (path ? path[a] : a) + 1 : 0;
    if (ok) ok = end <= ((long long)p.max_pages << sh);
    if (ok) ok = pages_ok(table, (int)(L >> sh), (int)((end - 1) >> sh), p.c.num_pages, nullptr);
    int stay = 1;  // the path's first entries may be in place already
    if (ok && path)
        while (stay <= a && path[stay] == stay) ++stay;
    const bool moves = ok && path && stay <= a;
    if (moves && p.c.refs) ok = pages_ok(table, (int)((L + stay) >> sh), (int)((L + a) >> sh), p.c.num_pages, p.c.refs);
    if (blockIdx.x == 0 && tid == 0) {
        p.new_len[b] = ok ? (int)(L + a + 1) : -1;
        if (p.status) p.status[b] = ok ? kOk : kEData;
    }
    if (!ok || !moves) return;
    auto place = [&](long long pos) {
        const int id = SV_IN(pos, (long long)p.max_pages << sh) ? table[pos >> sh] : -1;
        return SV_IN(id, p.c.num_pages) ? (long long)id * p.c.page_stride + (pos & ((1 << sh) - 1)) * p.c.token_stride : -1LL;
    };
    for (int i = tid; i <= a && SV_IN(i, SPEC_MAX_TREE_N); i += CT) {
        from[i] = place(L + path[i]);
        to[i] = place(L + i);
    }
    __syncthreads();
    const int per_head = p.c.row_bytes / 16, cols = p.c.heads * per_head;
    const long long units = (long long)p.c.layers * 2 * cols;
    for (long long u = (long long)blockIdx.x * CT + tid; u < units; u += (long long)gridDim.x * CT) {
        const int y = (int)(u / (2 * cols)), r = (int)(u - (long long)y * 2 * cols), kv = r / cols, c = r - kv * cols;
        const int h = c / per_head;
        char* base = (kv ? p.c.v : p.c.k) + y * p.c.layer_stride + h * p.c.head_stride + (c - h * per_head) * 16;
        for (int i = stay; i <= a; i += kMoves) {
            uint4 x[kMoves];
#pragma unroll
            for (int j = 0; j < kMoves; ++j)
                if (i + j <= a && SV_PLACE(from[i + j])) x[j] = ldg16(base + from[i + j]);
#pragma unroll
            for (int j = 0; j < kMoves; ++j)
                if (i + j <= a && SV_PLACE(from[i + j]) && SV_PLACE(to[i + j])) stg16(base + to[i + j], x[j]);
        }
    }
}

// ---- pages ----------------------------------------------------------------------
constexpr int PT = 1024;
constexpr int kMaxF = SPEC_MAX_POOL_SEQS;

// Exclusive prefix of v over the block's threads; *total: the sum.
SV_DEV int block_exclusive(int v, int* scratch, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < PT / 32; ++w) {
        const int u = scratch[w];
        if (w < warp) before += u;
        sum += u;
    }
    *total = sum;
    return before + inc - v;
}

// offs[0 .. F]: prefix sums of need[0 .. F - 1] (offs holds the needs on entry).
SV_DEV int prefix_needs(int* offs, int F, int* scratch) {
    int carry = 0;
    for (int f0 = 0; f0 < F; f0 += PT) {
        const int f = f0 + (int)threadIdx.x;
        const int v = f < F ? offs[f] : 0;
        int sum;
        const int ex = block_exclusive(v, scratch, &sum);
        if (f < F) offs[f] = carry + ex;
        carry += sum;
    }
    if (threadIdx.x == 0) offs[F] = carry;
    __syncthreads();
    return carry;
}

// Sequence that the rank-th new page goes to: the last f with offs[f] <= rank
// (sequences that need none share their successor's offset).
SV_DEV int owner_of(const int* offs, int F, int rank) {
    int lo = 0, hi = F;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (offs[mid] <= rank) lo = mid; else hi = mid;
    }
    return lo;
}

// Calls give(rank, page) for the lowest free pages in order until `need` are
// given; returns how many there were (at most need). A thread looks at four
// neighbouring pages at a time, the block at 4096; those that are free go to a
// list and are given out a thread each (by their finder, a window's first few
// threads gave out one page after the other: a fork of 12 took 13.0 us, not 9.8).
// Stretches of 32768 pages without a free one are passed with one barrier.
// Bound by the latency of a window's loads and scan: 64 sequences that take a
// page each at the end of a pool of 1000, 20000 and 200000, and the call that
// releases them: 10.9, 18.3 and 21.9 us (9.8, 31.1 and 228 with one page a
// thread and a scan for every window).
constexpr int kLook = 4, kStretch = 8;

SV_DEV int4 four_refs(const int32_t* refs, int pg, int num_pages) {  // (nothing past the end is free)
    if (pg + 4 <= num_pages && (reinterpret_cast<size_t>(refs) & 15) == 0)
        return __ldcg(reinterpret_cast<const int4*>(refs + pg));
    int4 x = make_int4(1, 1, 1, 1);
    if (pg < num_pages) x.x = __ldcg(refs + pg);
    if (pg + 1 < num_pages) x.y = __ldcg(refs + pg + 1);
    if (pg + 2 < num_pages) x.z = __ldcg(refs + pg + 2);
    if (pg + 3 < num_pages) x.w = __ldcg(refs + pg + 3);
    return x;
}

template <typename Give>
SV_DEV int take_free(const int32_t* refs, int num_pages, int need, int* scratch, Give give) {
    constexpr int kWindow = PT * kLook;
    __shared__ int list[kWindow];
    const int tid = threadIdx.x;
    int found = 0;
    for (int p0 = 0; p0 < num_pages && found < need; p0 += kWindow) {
        if (p0 % (kWindow * kStretch) == 0 && num_pages - p0 > kWindow) {
            bool any = false;
#pragma unroll
            for (int j = 0; j < kStretch; ++j) {
                const int4 x = four_refs(refs, min(p0 + j * kWindow, num_pages) + tid * kLook, num_pages);
                any |= x.x == 0 || x.y == 0 || x.z == 0 || x.w == 0;
            }
            if (!__syncthreads_or(any)) {
                if (num_pages - p0 <= kWindow * kStretch) break;
                p0 += kWindow * (kStretch - 1);
                continue;
            }
        }
        const int pg = p0 + tid * kLook;
        const int4 x = four_refs(refs, pg, num_pages);
        const bool f0 = x.x == 0, f1 = x.y == 0, f2 = x.z == 0, f3 = x.w == 0;
        int sum, at = block_exclusive(f0 + f1 + f2 + f3, scratch, &sum);
        if (f0) list[at++] = pg;
        if (f1) list[at++] = pg + 1;
        if (f2) list[at++] = pg + 2;
        if (f3) list[at++] = pg + 3;
        __syncthreads();
        for (int r = tid; r < min(sum, need - found); r += PT) give(found + r, list[r]);
        found += sum;
    }
    __syncthreads();
    return min(found, need);
}

// First -1 of a table row (the pages that the sequence holds), by one warp;
// -1 where a held entry names no page.
SV_DEV int held_pages(const int32_t* row, int max_pages, int num_pages) {
    const int lane = threadIdx.x & 31;
    for (int i0 = 0; i0 < max_pages; i0 += 32) {
        const int i = i0 + lane;
        const int id = i < max_pages ? row[i] : -1;
        const unsigned ends = __ballot_sync(0xFFFFFFFFu, id == -1);
        const unsigned bad = __ballot_sync(0xFFFFFFFFu, id < -1 || id >= num_pages);
        const int stop = ends ? __ffs(ends) - 1 : 32;
        if (bad & (stop == 32 ? 0xFFFFFFFFu : (1u << stop) - 1u)) return -1;
        if (ends) return i0 + stop;
    }
    return max_pages;
}

// One CTA: the order of the free pages is one scan's, and a call's tables are
// small. Releases come first (so their pages can be taken in the same
// call), then the growing sequences take pages in order. A sequence whose
// pages do not all fit beside those before it gets none.
__global__ void __launch_bounds__(PT) resize_kernel(const __grid_constant__ PoolParams p) {
    __shared__ int offs[kMaxF + 1];
    __shared__ int scratch[PT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int f = warp; f < p.F; f += PT / 32) {
        const int s = p.seqs ? p.seqs[f] : f, want_tokens = p.tokens[f];
        const long long want = ((long long)want_tokens + (1 << p.page_shift) - 1) >> p.page_shift;
        bool ok = s >= 0 && s < p.S && want_tokens >= 0 && want <= p.max_pages;
        int32_t* row = p.table + (long long)(ok ? s : 0) * p.table_stride;
        const int have = ok ? held_pages(row, p.max_pages, p.num_pages) : -1;
        ok = ok && have >= 0;
        if (ok)
            for (int i = (int)want + lane; i < have; i += 32) {
                atomicSub(p.refs + row[i], 1);
                row[i] = -1;
            }
        if (lane == 0) {
            offs[f] = ok && want > have ? (int)want - have : 0;
            if (p.status) p.status[f] = ok ? kOk : kEData;
        }
    }
    __syncthreads();
    __threadfence_block();
    const int need = prefix_needs(offs, p.F, scratch);
    if (need == 0) return;
    auto entry = [&](int f, int i) {  // the i-th new page of sequence f
        const int s = p.seqs ? p.seqs[f] : f;
        const int want = (int)(((long long)p.tokens[f] + (1 << p.page_shift) - 1) >> p.page_shift);
        return p.table + (long long)s * p.table_stride + want - (offs[f + 1] - offs[f]) + i;
    };
    const int got = take_free(p.refs, p.num_pages, need, scratch, [&](int rank, int pg) {
        const int f = owner_of(offs, p.F, rank);
        if (SV_IN(entry(f, rank - offs[f]) - p.table, p.S * p.table_stride) && SV_IN(pg, p.num_pages)) {
            *entry(f, rank - offs[f]) = pg;
            p.refs[pg] = 1;
        }
    });
    if (got == need) return;
    // too few: the sequences that were not served whole give theirs back
    for (int f = warp; f < p.F; f += PT / 32) {
        if (offs[f + 1] == offs[f] || offs[f + 1] <= got) continue;
        for (int r = offs[f] + lane; r < got; r += 32) {
            int32_t* e = entry(f, r - offs[f]);
            if (!SV_IN(e - p.table, p.S * p.table_stride) || !SV_IN(*e, p.num_pages)) continue;
            p.refs[*e] = 0;
            *e = -1;
        }
        if (lane == 0 && p.status) p.status[f] = kENoPages;
    }
}

// One CTA: the tables, counts and lengths of the forks, and for each the page
// copy that is left to do. Its chain of dependent steps (lengths, tables, free
// pages, tables again) bounds a small fork: 11.0 us of 12 forks with their copies
// (8 layers).
__global__ void __launch_bounds__(PT) fork_kernel(const __grid_constant__ PoolParams p) {
    __shared__ int offs[kMaxF + 1];
    __shared__ int scratch[PT / 32];
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto check = [&](int f, int* len, int* full) {  // a warp: whether fork f can be made
        const int s = p.src[f], d = p.dst[f];
        if (s < 0 || s >= p.S || d < 0 || d >= p.S || s == d) return false;
        const int L = p.cache_len[s];
        if (L < 0 || L > ((long long)p.max_pages << p.page_shift)) return false;
        const int32_t* row = p.table + (long long)s * p.table_stride;
        const int pages = (int)(((long long)L + (1 << p.page_shift) - 1) >> p.page_shift);
        bool bad = p.table[(long long)d * p.table_stride] != -1;
        for (int i = lane; i < pages; i += 32) bad |= row[i] < 0 || row[i] >= p.num_pages;
        *len = L;
        *full = L >> p.page_shift;
        return __any_sync(0xFFFFFFFFu, bad) == 0;
    };
    for (int f = warp; f < p.F; f += PT / 32) {
        int L = 0, full = 0;
        const bool ok = check(f, &L, &full);
        const int rest = ok ? L - (full << p.page_shift) : 0;
        if (lane == 0) {
            offs[f] = rest > 0;
            p.copies[f] = ok ? make_int4(rest > 0 ? p.table[(long long)p.src[f] * p.table_stride + full] : -1, -1, rest, L)
                             : make_int4(-1, -2, 0, 0);
            if (p.status) p.status[f] = ok ? kOk : kEData;
        }
    }
    __syncthreads();
    const int need = prefix_needs(offs, p.F, scratch);
    take_free(p.refs, p.num_pages, need, scratch, [&](int rank, int pg) { 
        const int f = owner_of(offs, p.F, rank);
        if (SV_IN(f, p.F)) p.copies[f].y = pg;
    });
    __syncthreads();
    for (int f = warp; f < p.F; f += PT / 32) {
        const int4 c = p.copies[f];
        if (c.y == -2) continue;  // bad data
        if (c.z > 0 && c.y < 0) {
            if (lane == 0 && p.status) p.status[f] = kENoPages;
            continue;
        }
        const int s = p.src[f], d = p.dst[f], L = c.w, full = L >> p.page_shift;
        const int32_t* from = p.table + (long long)s * p.table_stride;
        int32_t* to = p.table + (long long)d * p.table_stride;
        for (int i = lane; i < full; i += 32) {
            const int id = from[i];
            if (!SV_IN(id, p.num_pages) || !SV_IN(i, p.max_pages)) continue;
            to[i] = id;
            atomicAdd(p.refs + id, 1);
        }
        if (lane == 0) {
            if (c.z > 0 && SV_IN(full, p.max_pages) && SV_IN(c.y, p.num_pages)) {
                to[full] = c.y;
                p.refs[c.y] = 1;
            }
            p.cache_len[d] = L;
        }
    }
}

// Block (y, f): the used slots of fork f's last page in one layer's K (y even)
// or V. dense: a page's slots lie one after the other, heads within a slot too.
// Bound by memory; a thread keeps eight words in flight (64 forks, 32 layers, 8
// heads of 128 columns: 37.6 us, the floor of the bytes alone 34).
template <bool DENSE>
__global__ void __launch_bounds__(CT) fork_copy_kernel(const __grid_constant__ CacheView c, const int4* copies) {
    const int y = blockIdx.x >> 1;
    char* base = (blockIdx.x & 1 ? c.v : c.k) + y * c.layer_stride;
    const int per_head = c.row_bytes / 16, per_token = c.heads * per_head;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 job = __ldcg(copies + blockIdx.y);
    if (job.z <= 0 || job.y < 0) return;
    if (!SV_IN(job.x, c.num_pages) || !SV_IN(job.y, c.num_pages) || !SV_IN(job.z, 1 << c.page_shift)) return;
    const char* from = base + job.x * c.page_stride;
    char* to = base + job.y * c.page_stride;
    const int words = job.z * per_token;
    constexpr int U = 8;
    for (int i0 = threadIdx.x; i0 < words; i0 += CT * U) {
        uint4 x[U];
        long long at[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = min(i0 + j * CT, words - 1);
            if (DENSE) {
                at[j] = (long long)i * 16;
            } else {
                const int t = i / per_token, e = i - t * per_token, h = e / per_head;
                at[j] = t * c.token_stride + h * c.head_stride + (e - h * per_head) * 16;
            }
            x[j] = ldg16(from + at[j]);
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i0 + j * CT < words) stg16(to + at[j], x[j]);
    }
}

int blocks_for(long long units, int per_block, int others) {
    const long long n = (units + per_block - 1) / per_block;
    const long long most = std::max(1LL, 152LL * 16 / std::max(1, others));
    return (int)std::max(1LL, std::min(n, most));
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t st) {
    append_kernel<<<dim3((p.N + kAppendTokens - 1) / kAppendTokens, p.B), CT, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t st) {
    const long long units = p.path ? (long long)p.c.layers * 2 * p.c.heads * (p.c.row_bytes / 16) : 1;
    compact_kernel<<<dim3(blocks_for(units, CT, p.B), p.B), CT, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_resize(const PoolParams& p, cudaStream_t st) {
    resize_kernel<<<1, PT, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_fork(const PoolParams& p, const CacheView& c, cudaStream_t st) {
    fork_kernel<<<1, PT, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // starts while the bookkeeping ends (it waits for it before it reads a copy)
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * c.layers, p.F);
    cfg.blockDim = dim3(CT);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const bool dense = c.head_stride == c.row_bytes && c.token_stride == (long long)c.heads * c.row_bytes;
    const int4* copies = p.copies;
    return dense ? cudaLaunchKernelEx(&cfg, fork_copy_kernel<true>, c, copies)
                 : cudaLaunchKernelEx(&cfg, fork_copy_kernel<false>, c, copies);
}

SV_DEBUG_READER(cache)

}  // namespace sv
