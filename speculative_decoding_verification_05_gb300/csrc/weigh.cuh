// Parameters and the division of the work of the weighing kernels: the attention
// weights of a step's accepted rows added up for every position and key / value
// head,
//   weights[b, g, t] += sum_{r < n, heads h of g, t <= L + r} exp(scale q_rh . k_t - lse_rh),
// row r being node path[r] (no path: r), whose accepted ancestors' entries lie
// at L .. L + r. With the rows' log-sums known from the attention no softmax is
// needed and a position's sum is one CTA's: no atomics, the same order always.
//
// A unit is (sequence, head, tile of KV positions) with all its rows; it costs as
// much as it has blocks of ROWS rows. All units in order form one range that is
// cut into equal parts, one a CTA; a unit is its first part's.
#pragma once

#include "common.cuh"

namespace sv {

struct WeighParams {
    const void* q;    // [B, N, Hkv * G, D]
    const float* lse;  // [B, N, Hkv * G]
    const void* k;    // page p, slot s, head h at p * page_stride + s * token_stride + h * head_stride
    long long page_stride, token_stride, head_stride;  // elements
    const int32_t* table;
    long long table_stride;
    const int32_t* cache_len;  // [B]
    const int32_t* accept;     // [B] rows less one, or null (N rows)
    const int32_t* path;       // [B, W] or null
    int B, N, W, Hkv, G, D, num_pages, max_pages, page_shift;
    long long capacity;  // of a head's weights
    float c2;            // scale * log2(e)
    float* weights;      // [B, Hkv, capacity]
    int32_t* status;     // [B] or null
};

// A sequence's rows and context; n = 0: none, or bad data (bad set).
struct WeighSeq {
    int n, L;
    bool bad;
};

SV_DEV WeighSeq weigh_seq(const WeighParams& p, int b) {
    WeighSeq s;
    s.L = __ldg(p.cache_len + b);
    const int most = p.path ? min(p.N, p.W) : p.N;
    const int a = p.accept ? __ldg(p.accept + b) : most - 1;
    const long long end = (long long)s.L + a + 1;
    s.bad = s.L < 0 || a < -1 || a >= most || end > ((long long)p.max_pages << p.page_shift) || end > p.capacity;
    s.n = s.bad ? 0 : a + 1;
    return s;
}

template <int KV, int ROWS>
SV_DEV long long weigh_cost(const WeighParams& p, const WeighSeq& s) {  // of one unit
    return ((long long)s.n * p.G + ROWS - 1) / ROWS;
}
template <int KV>
SV_DEV long long weigh_units(const WeighParams& p, const WeighSeq& s) {
    return s.n > 0 ? ((long long)s.L + s.n + KV - 1) / KV * p.Hkv : 0;
}

struct WeighScan {
    long long warp_sum[32];
    long long base;
    int b;
};

// This CTA's units: called by all NT threads of the block (nothing if b = -1).
struct WeighPart {
    long long at, end, base;  // places in the range; base: where sequence b begins
    int b;
};

template <int KV, int ROWS, int NT>
SV_DEV WeighPart weigh_locate(const WeighParams& p, WeighScan* sc) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int run = (p.B + NT - 1) / NT, b0 = min(tid * run, p.B), b1 = min(b0 + run, p.B);
    auto work = [&](int b) {
        const WeighSeq s = weigh_seq(p, b);
        return weigh_units<KV>(p, s) * weigh_cost<KV, ROWS>(p, s);
    };
    long long mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += work(b);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) sc->warp_sum[warp] = inc;
    if (tid == 0) sc->b = -1;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const long long u = sc->warp_sum[w];
        if (w < warp) before += u;
        total += u;
    }
    const long long lo = before + inc - mine, each = total / gridDim.x, more = total - each * gridDim.x;
    const long long c = blockIdx.x, at = each * c + min(c, more), end = at + each + (c < more);
    if (at < end && at >= lo && at < lo + mine) {
        long long base = lo;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const long long w = work(b);
            if (at < base + w) {
                sc->b = b;
                sc->base = base;
                break;
            }
            base += w;
        }
    }
    __syncthreads();
    return WeighPart{at, end, sc->base, sc->b};
}

// The units that begin in the part, one after the other: tiles of one (sequence,
// head) at a time.
struct WeighStay {
    int b, h, n, L, first, last;  // tiles [first, last) of head h
};

template <int KV, int ROWS>
SV_DEV bool weigh_next(const WeighParams& p, WeighPart* w, WeighStay* s) {
    if (w->b < 0) return false;
#pragma unroll 1
    while (w->at < w->end && w->b < p.B) {
        const WeighSeq q = weigh_seq(p, w->b);
        const long long cost = weigh_cost<KV, ROWS>(p, q), units = weigh_units<KV>(p, q);
        const long long u0 = cost ? (w->at - w->base + cost - 1) / cost : 0;  // the first that begins at `at` or later
        if (u0 >= units) {
            w->base += cost * units;
            w->at = max(w->at, w->base);
            ++w->b;
            continue;
        }
        const long long tiles = units / p.Hkv;
        s->h = (int)(u0 / tiles);
        // units of this head that begin before the part's end
        const long long stop = min((w->end - w->base + cost - 1) / cost, (s->h + 1) * tiles);
        if (u0 >= stop) return false;
        s->b = w->b;
        s->n = q.n;
        s->L = q.L;
        s->first = (int)(u0 - s->h * tiles);
        s->last = (int)(stop - s->h * tiles);
        w->at = w->base + stop * cost;
        return true;
    }
    return false;
}

// Whether a sequence's data are good: its path's nodes and its pages (one warp).
SV_DEV bool weigh_check(const WeighParams& p, int b) {
    const int lane = threadIdx.x & 31;
    const WeighSeq s = weigh_seq(p, b);
    bool bad = s.bad;
    if (s.n > 0) {
        if (p.path)
            for (int r = lane; r < s.n; r += 32) {
                const int i = __ldg(p.path + (long long)b * p.W + r);
                bad |= i < 0 || i >= p.N;
            }
        for (long long i = lane; i <= ((long long)s.L + s.n - 1) >> p.page_shift; i += 32) {
            const int id = __ldg(p.table + b * p.table_stride + i);
            bad |= id < 0 || id >= p.num_pages;
        }
    }
    return !__any_sync(0xFFFFFFFFu, bad);
}

// Statuses of all sequences, shared out over the grid's warps. RAISE: they are zero
// before, and are only ever raised, as those of a part that gave up are.
template <bool RAISE>
SV_DEV void weigh_statuses(const WeighParams& p, int gw, int warps) {
    if (!p.status) return;
#pragma unroll 1
    for (int b = gw; b < p.B; b += warps) {
        const bool ok = weigh_check(p, b);
        if ((threadIdx.x & 31) != 0) continue;
        if (!RAISE) p.status[b] = ok ? kOk : kEData;
        else if (!ok) atomicMax(p.status + b, kEData);
    }
}

// The tensor-core kernel (bf16, D 64 or 128) reads the keys through a tensor map;
// *took: false where the cache's strides have none (nothing was launched).
cudaError_t launch_weigh_tc(const WeighParams& p, cudaStream_t st, bool* took);
int debug_withhold_weigh_tile(int j);
cudaError_t debug_read_weigh_tc(unsigned int* count, unsigned int* line);
cudaError_t launch_weigh_simt(const WeighParams& p, int dtype, cudaStream_t st);
cudaError_t debug_read_weigh(unsigned int* count, unsigned int* line);

}  // namespace sv
