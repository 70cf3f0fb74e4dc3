// Eviction from the paged cache by accumulated attention weight: a sequence
// longer than its budget keeps, for every layer and key / value head by itself,
// its first `sink` positions, its last `recent` ones and of the rest those of the
// largest weight (ties: the lowest position; NaN counts as larger than all), in
// their order, and their keys, values and weights move together to the front.
//
// Two launches. One block a (layer, sequence, head) finds the weight of rank m
// among the n middle positions - the largest key that at least m of them reach,
// digit by digit of the ordered 32-bit keys (11, 11 and 10 bits), each by a
// histogram of the positions that share the digits before it -, lists the kept
// positions by one prefix sum, and moves the weights. Then one
// block a list and K or V moves the rows: as a kept position's new place is never
// behind its old one, rows are read a batch at a time and written when the whole
// block has read its batch, and no later batch's row is overwritten.
//
// Bound by memory where there is enough of it: 16 sequences of 1500-4000 positions,
// 32 layers, 8 heads of 128 columns, bf16, to 1600: 1044 us, 6.1 TB/s over both
// launches (the moves alone 895 us, 7.0 TB/s of what has to move; the selection 122,
// 137 with the keys formed anew for every digit: its instructions, two blocks an
// SM). One sequence, 12 layers, 4 heads of 64, float32, 1501 to 1003: 17.2 us, the chain of dependent steps (with
// the bound found bit by bit, a count of the block each, 34).

#include <algorithm>

#include "cache.cuh"
#include "specverify.h"

namespace sv {
namespace {

constexpr int ST = 512;   // threads of a selecting block
constexpr int kItems = 8;  // positions of a thread: neighbours
constexpr int kBins = 2048;  // values of a digit of a key
constexpr int CT = 256;
constexpr int kMoves = 8;
constexpr int kMostRows = 64;  // rows that a block reads at once, an eighth of a batch

SV_DEV uint4 ldg16(const char* p) { return *reinterpret_cast<const uint4*>(p); }
SV_DEV void stg16(char* p, uint4 x) { *reinterpret_cast<uint4*>(p) = x; }

// Ordered keys of weights; NaN above everything.
SV_DEV uint32_t weight_key(float w) { return w != w ? 0xFFFFFFFFu : f32_key(w); }

// Exclusive prefixes of two counts over the block's threads, and their sums.
SV_DEV void block_prefix2(int a, int b, int* pa, int* pb, int* sa, int* sb, int2* scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, x, o), v = __shfl_up_sync(0xFFFFFFFFu, y, o);
        if (lane >= o) x += u, y += v;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = make_int2(x, y);
    __syncthreads();
    int bx = 0, by = 0, tx = 0, ty = 0;
#pragma unroll
    for (int w = 0; w < ST / 32; ++w) {
        const int2 u = scratch[w];
        if (w < warp) bx += u.x, by += u.y;
        tx += u.x, ty += u.y;
    }
    *pa = bx + x - a;
    *pb = by + y - b;
    *sa = tx;
    *sb = ty;
}

__global__ void __launch_bounds__(ST, 2) evict_select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ union {
        int hist[kBins];
        int2 kept[ST * kItems];  // positions and weights that one round keeps
    } u;
    __shared__ int2 scratch[ST / 32];
    __shared__ int first_moved, found, rest;
    asm volatile("griddepcontrol.launch_dependents;");
    const long long unit = blockIdx.x;  // (layer, sequence, head)
    [[maybe_unused]] const long long units = (long long)p.c.layers * p.B * p.c.heads;
    const int h = (int)(unit % p.c.heads), b = (int)(unit / p.c.heads % p.B), tid = threadIdx.x, sh = p.c.page_shift;
    const long long L = p.cache_len[b], budget = p.budget[b], least = (long long)p.sink + p.recent;
    const int32_t* table = p.table + b * p.table_stride;
    bool ok = L >= 0 && L <= ((long long)p.max_pages << sh) && L <= p.capacity && budget >= least;
    const bool over = ok && L > budget;
    if (over) {
        bool bad = false;
        const int own0 = (int)(p.sink >> sh), own1 = budget > p.sink ? (int)((budget - 1) >> sh) : -1;
        for (int i = tid; i <= (int)((L - 1) >> sh); i += ST) {
            const int id = __ldg(table + i);
            if (id < 0 || id >= p.c.num_pages) bad = true;
            else if (p.c.refs && i >= own0 && i <= own1) bad |= __ldg(p.c.refs + id) != 1;
        }
        ok = !__syncthreads_or(bad);
    }
    if (h == 0 && unit < (long long)p.B * p.c.heads && tid == 0) {
        p.new_len[b] = ok ? (int)min(L, budget) : -1;
        if (p.status) p.status[b] = ok ? kOk : kEData;
    }
    if (!ok || !over) {
        if (tid == 0 && SV_IN(unit, units)) p.jobs[unit] = make_int2(0, 0);
        return;
    }

    const int len = (int)L, keep = (int)budget, mid0 = min(p.sink, len), mid1 = len - p.recent, m = keep - p.sink - p.recent;
    float* w = p.weights + unit * p.capacity;
    int32_t* list = p.list + unit * p.capacity;
    const bool fits = len <= ST * kItems;  // the block's registers hold all weights
    const bool vec = (p.capacity & 3) == 0 && (reinterpret_cast<size_t>(p.weights) & 15) == 0;
    float x[kItems];
    uint32_t key[kItems];
    auto load = [&](int at) {
        const int t = at + tid * kItems;
        if (vec && t + kItems <= len) {
#pragma unroll
            for (int j = 0; j < kItems; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(w + t + j);
                x[j] = f.x, x[j + 1] = f.y, x[j + 2] = f.z, x[j + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kItems; ++j) x[j] = t + j < len ? w[t + j] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kItems; ++j) key[j] = weight_key(x[j]);
    };
    if (tid == 0) first_moved = keep;
    if (fits) load(0);
    // The m-th key from above, and how many of its ties are kept (m = 0: a bound
    // above all keys).
    unsigned long long bound = 1ull << 32;
    int ties = m;
    if (m > 0) {
        uint32_t prefix = 0;  // the digits so far
#pragma unroll 1
        for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift - 10) {
            const uint32_t mask = shift ? kBins - 1 : 1023;
            const int before = shift == 21 ? 32 : shift + (shift ? 11 : 10);  // bits that the prefix leaves
            for (int i = tid; i < kBins; i += ST) u.hist[i] = 0;
            __syncthreads();
            for (int at = 0; at < len; at += ST * kItems) {
                if (!fits) load(at);
                const int t = at + tid * kItems;
#pragma unroll
                for (int j = 0; j < kItems; ++j) {
                    const uint32_t k = key[j];
                    if (t + j >= mid0 && t + j < mid1 && (before == 32 || k >> before == prefix))
                        atomicAdd(&u.hist[k >> shift & mask], 1);
                }
            }
            __syncthreads();
            // from the largest digit down, kBins / ST a thread
            const int top = kBins - 1 - tid * (kBins / ST);
            int n[kBins / ST], sum = 0;
#pragma unroll
            for (int j = 0; j < kBins / ST; ++j) sum += n[j] = u.hist[top - j];
            int above, unused, s0, s1;
            block_prefix2(sum, 0, &above, &unused, &s0, &s1, scratch);
            if (above < ties && ties <= above + sum) {
#pragma unroll
                for (int j = 0; j < kBins / ST; ++j) {
                    if (above < ties && ties <= above + n[j]) {
                        found = top - j;
                        rest = ties - above;
                    }
                    above += n[j];
                }
            }
            __syncthreads();
            prefix = prefix << (shift ? 11 : 10) | (uint32_t)found;
            ties = rest;
        }
        bound = prefix;
    }
    // kept so far: those above the bound or always kept, and ties
    int above0 = 0, tied0 = 0, moved = keep;  // (moved: the first entry that changes its place)
    __syncthreads();
    for (int at = 0; at < len; at += ST * kItems) {
        if (!fits) load(at);
        const int t = at + tid * kItems;
        uint32_t above = 0, tied = 0;
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int i = t + j;
            const unsigned long long k = key[j];
            const bool in = i < len, always = i < mid0 || i >= mid1;
            if (in && (always || k > bound)) above |= 1u << j;
            else if (in && k == bound) tied |= 1u << j;
        }
        int a, e, sa, se;
        block_prefix2(__popc(above), __popc(tied), &a, &e, &sa, &se, scratch);  // (its barriers: all have read)
        // (in shared memory first: the threads' places lie apart, and each is one word)
        const int start = above0 + min(tied0, ties);
        a += above0;
        e += tied0;
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const bool is = above >> j & 1, tie = tied >> j & 1;
            const int to = a + min(e, ties);
            if (is || (tie && e < ties)) {
                if (SV_IN(to - start, ST * kItems)) u.kept[to - start] = make_int2(t + j, __float_as_int(x[j]));
                if (to != t + j) moved = min(moved, to);
            }
            a += is;
            e += tie;
        }
        above0 += sa;
        tied0 += se;
        __syncthreads();
        const int n = above0 + min(tied0, ties) - start;
        for (int i = tid; i < n; i += ST) {
            const int2 k = u.kept[i];
            if (SV_IN(start + i, keep) && SV_IN(start + i, p.capacity)) {
                list[start + i] = k.x;
                w[start + i] = __int_as_float(k.y);
            }
        }
    }
    moved = __reduce_min_sync(0xFFFFFFFFu, moved);
    if ((tid & 31) == 0 && moved < keep) atomicMin(&first_moved, moved);
    __syncthreads();
    for (int i = keep + tid; i < len; i += ST)
        if (SV_IN(i, p.capacity)) w[i] = 0.f;
    if (tid == 0 && SV_IN(unit, units)) p.jobs[unit] = make_int2(first_moved, keep);
}

__global__ void __launch_bounds__(CT) evict_move_kernel(const __grid_constant__ EvictParams p) {
    // from, to; three batches': warps that still write the last one, the one that is
    // read, the next
    __shared__ longlong2 place[3][kMostRows * kMoves];
    const long long unit = blockIdx.x >> 1;
    const int h = (int)(unit % p.c.heads), b = (int)(unit / p.c.heads % p.B), tid = threadIdx.x, sh = p.c.page_shift;
    char* base = (blockIdx.x & 1 ? p.c.v : p.c.k) + unit / p.c.heads / p.B * p.c.layer_stride + h * p.c.head_stride;
    const int32_t* table = p.table + b * p.table_stride;
    const int words = p.c.row_bytes / 16 / gridDim.y, width = min(CT / words, kMostRows), r0 = tid / words;
    const int col = blockIdx.y * words + tid - r0 * words;
    const int batch = width * kMoves;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int2 job = __ldcg(p.jobs + unit);
    const int32_t* list = p.list + unit * p.capacity;
    auto row = [&](int pos) {
        if (!SV_IN(pos, (long long)p.max_pages << sh)) return -1LL;
        const int id = __ldg(table + (pos >> sh));
        return SV_IN(id, p.c.num_pages) ? (long long)id * p.c.page_stride + (pos & ((1 << sh) - 1)) * p.c.token_stride : -1LL;
    };
    auto places = [&](int at, int buf) {
        for (int i = tid; i < batch; i += CT)
            if (at + i < job.y) place[buf][i] = make_longlong2(row(__ldcg(list + at + i)), row(at + i));
    };
    places(job.x, 0);
    __syncthreads();
    int buf = 0;
    for (int at = job.x; at < job.y; at += batch) {
        const int next = buf == 2 ? 0 : buf + 1;
        uint4 x[kMoves];
        const int n = job.y - at;
        const bool mine = r0 < width;
#pragma unroll
        for (int j = 0; j < kMoves; ++j)
            if (mine && r0 + j * width < n && SV_PLACE(place[buf][r0 + j * width].x)) x[j] = ldg16(base + place[buf][r0 + j * width].x + col * 16);
        places(at + batch, next);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kMoves; ++j)
            if (mine && r0 + j * width < n && SV_PLACE(place[buf][r0 + j * width].x) && SV_PLACE(place[buf][r0 + j * width].y))
                stg16(base + place[buf][r0 + j * width].y + col * 16, x[j]);
        buf = next;
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t st) {
    const long long units = (long long)p.c.layers * p.B * p.c.heads;
    evict_select_kernel<<<(unsigned)units, ST, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // starts while the selection ends (it waits for it before it reads a list)
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // few lists: a row's columns are shared out too, down to 64 bytes
    int split = 1;
    while (split < 4 && p.c.row_bytes % (128 * split) == 0 && 2 * units * split < 152 * 4) split *= 2;
    cfg.gridDim = dim3((unsigned)(2 * units), split);
    cfg.blockDim = dim3(CT);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, p);
}

SV_DEBUG_READER(evict)

}  // namespace sv
