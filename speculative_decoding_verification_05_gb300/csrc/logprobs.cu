// Log probabilities of given tokens, their ranks, the rows' entropies and the
// likeliest alternatives, in one pass over the logits.
//
// With y_i = (z_i - m) / T, m the row's maximum and S = sum e^{y_i}:
//   log p(x) = y_x - ln S,   H = ln S - (sum e^{y_i} y_i) / S,
//   rank(x) = #{z_i > z_x} + #{i < x: z_i = z_x},
// and the alternatives are the first K in the order (z descending, i ascending).
//
// A row is split over a cluster of CTAs (one to eight); a thread holds its share
// of the part in registers, so the exponentials follow the maximum without a
// second read. Parts leave (m, S, sum e^y y, count above z_x) against their own
// maximum and their K best in the first CTA's shared memory, which joins them
// in the order of the parts: results depend on the shape alone.
//
// The K best of a part: any key that K threads' maxima reach is a bound that no
// better element lies below, so a search over the threads' maxima (one count of
// the block a step) ends at a bound that K to 2 K of them reach; only those
// threads look at their elements, and the few that reach it are ranked by
// comparing all with all. Where that finds more than fit (rows of equal logits) the
// bound is taken over the elements themselves, then over the indices of the ties.

#include <algorithm>

#include "attention.cuh"
#include "logprobs.cuh"
#include "specverify.h"

namespace sv {
namespace {

typedef unsigned long long u64;

constexpr int kMaxTop = SPEC_MAX_TOP;
constexpr int kMaxParts = 8;
constexpr int kCap = 1024;  // elements that are ranked at once

SV_DEV u64 cand_key(float z, int i) { return ((u64)f32_key(z) << 32) | (0xFFFFFFFFu - (uint32_t)i); }

// What a part of a row leaves for the join.
struct Part {
    float m, S, U;  // maximum, sum 2^t, sum 2^t t with t = (z - m) log2(e) / T
    int above;      // elements before the token in the order
};

template <int NT>
struct Shared {
    Part parts[kMaxParts];            // (of the cluster: the first CTA's)
    u64 best[kMaxParts * kMaxTop];    // each part's K best, descending
    u64 mine[kMaxTop];                // this part's
    u64 cand[kCap + kMaxTop];
    float red[3][NT / 32];
    int cnt[NT / 32];
    int found;
};

SV_DEV uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
SV_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
SV_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The address of the first CTA's copy of a shared variable.
template <typename T>
SV_DEV uint32_t in_first(T* p) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)));
    return a;
}
SV_DEV void st_cluster(uint32_t a, u64 x) { asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(x) : "memory"); }

template <int NT>
SV_DEV int block_sum(int v, int* scratch) {
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) s += scratch[w];
    return s;
}

// How far a part's maximum lies below the row's, in octaves (2^-200 is 0; a part
// of nothing but -inf has no maximum).
SV_DEV float octaves(float m, float top, float c2) { return m == -INFINITY ? -200.f : fmaxf((m - top) * c2, -200.f); }

// The n keys in cand (distinct) ranked against one another; the first k, in
// descending order, to best.
template <int NT>
SV_DEV void rank_keys(const u64* cand, int n, int k, u64* best) {
    for (int i = threadIdx.x; i < n; i += NT) {
        const u64 key = cand[i];
        int r = 0;
        for (int j = 0; j < n; ++j) r += cand[j] > key;
        if (r < k) best[r] = key;
    }
}

// Stops the compiler from keeping what it unpacked from a word for the next pass
// (it needs more registers than the thread has).
SV_DEV void forget(uint4& x) { asm volatile("" : "+r"(x.x), "+r"(x.y), "+r"(x.z), "+r"(x.w)); }

// The largest of a granule's elements (NaN loses).
template <typename E>
SV_DEV float granule_max(const uint4& x) {
    if constexpr (sizeof(E) == 4) {
        float r;
        asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(__uint_as_float(x.x)), "f"(__uint_as_float(x.y)), "f"(__uint_as_float(x.z)));
        return fmaxf(r, __uint_as_float(x.w));
    } else {
        uint32_t a, b;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(x.x), "r"(x.y));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(x.z), "r"(x.w));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
        return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
    }
}

// A thread's sums, two at a time.
struct Sums {
    uint64_t S, U;
};

// Adds a granule's 2^t and 2^t t, t = (v - ref) c2; NaN in S for a NaN or +inf.
template <int VN>
SV_DEV void add_granule(const float (&v)[VN], float ref, float c2, Sums* a) {
    const uint64_t rr = pack2(-ref, -ref), cc = pack2(c2, c2);
    uint64_t u = 0ull;
#pragma unroll
    for (int e = 0; e < VN; e += 2) {
        const uint64_t t = mul2(add2(pack2(v[e], v[e + 1]), rr), cc);
        float t0, t1;
        unpack2(t, &t0, &t1);
        const uint64_t w = pack2(ex2(t0), ex2(t1));
        a->S = add2(a->S, w);
        u = fma2(w, t, u);
    }
    float u0, u1;
    unpack2(u, &u0, &u1);
    if (!(u0 + u1 <= 0.f)) {  // a logit of -inf gave 0 times infinity (or the row is bad): again, with an end
        u0 = u1 = 0.f;
#pragma unroll
        for (int e = 0; e < VN; ++e) {
            const float t = fmaxf((v[e] - ref) * c2, -200.f);  // (2^-200 is 0)
            u0 = fmaf(ex2(t), t, u0);
        }
        u = pack2(u0, u1);
    }
    a->U = add2(a->U, u);
}

// How many of a granule's elements lie above t: the signs of t - v.
template <int VN>
SV_DEV int count_above(const float (&v)[VN], float t) {
    const uint64_t tt = pack2(t, t), minus = pack2(-1.f, -1.f);
    uint32_t n = 0;
#pragma unroll
    for (int e = 0; e < VN; e += 2) {
        float a, b;
        unpack2(fma2(pack2(v[e], v[e + 1]), minus, tt), &a, &b);
        n += (__float_as_uint(a) >> 31) + (__float_as_uint(b) >> 31);
    }
    return (int)n;
}

template <typename E, int NT, int NV>
__global__ void __launch_bounds__(NT, 1024 / NT) logprob_kernel(const __grid_constant__ LogprobParams p) {
    constexpr int VN = VecTraits<E>::kN;
    __shared__ Shared<NT> s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part = p.parts > 1 ? (int)cluster_rank() : 0;
    const long long row = blockIdx.x / p.parts;
    const int b = (int)(row / p.P), tok = __ldg(p.tokens + row), K = p.top;
    const bool first = part == 0;

    // rows without a token, or with a bad one (the whole cluster leaves)
    if (tok < 0 || tok >= p.V) {
        const bool bad = tok != -1;
        if (!first) return;
        const float nan = __int_as_float(0x7FC00000);
        if (tid == 0) {
            p.logprob[row] = bad ? nan : 0.f;
            if (p.entropy) p.entropy[row] = bad ? nan : 0.f;
            if (p.rank) p.rank[row] = -1;
            if (p.status && (bad || p.P == 1)) {
                if (p.P == 1) p.status[b] = bad ? kEData : kOk;
                else atomicMax(p.status + b, kEData);
            }
        }
        if (tid < K) {
            p.top_tokens[row * K + tid] = -1;
            p.top_logprobs[row * K + tid] = bad ? nan : -INFINITY;
        }
        return;
    }
    if (p.parts > 1) cluster_arrive();  // (waited for before the first CTA's memory is written)

    // Granules of 16 bytes: granule g holds the elements [g VN - h, (g + 1) VN - h).
    const E* z0 = reinterpret_cast<const E*>(p.logits) + row * p.V;
    const int h = (int)(reinterpret_cast<size_t>(z0) & 15) / (int)sizeof(E);
    const uint4* g0 = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(z0) - h * sizeof(E));
    const int granules = (p.V + h + VN - 1) / VN;
    const int lo = part * p.part_granules, hi = min(lo + p.part_granules, granules);
    // a granule; the row's edges element by element, -inf outside of it
    auto granule = [&](int g) {
        const int at = g * VN - h;
        if (at >= 0 && at + VN <= p.V) return ld_stream_v4(g0 + g);
        constexpr uint32_t fill = sizeof(E) == 4 ? 0xFF800000u : 0xFF80FF80u;
        uint32_t w[4] = {fill, fill, fill, fill};
#pragma unroll
        for (int e = 0; e < VN; ++e)
            if (at + e >= 0 && at + e < p.V) {
                const uint32_t bits = __float_as_uint(VecTraits<E>::load1(z0 + at + e));
                if (sizeof(E) == 4) w[e & 3] = bits;
                else w[(e >> 1) & 3] = e & 1 ? (w[(e >> 1) & 3] & 0xFFFFu) | bits : (w[(e >> 1) & 3] & 0xFFFF0000u) | bits >> 16;
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    const float zx = VecTraits<E>::load1(z0 + tok) + 0.f;  // (-0 becomes +0: signs of differences are counted)
    // the next value below z_x: z > below where z >= z_x (-inf: none, its ties are counted one by one)
    const float below = zx == -INFINITY ? zx : zx == 0.f ? -0x1p-149f : key_to_f32(f32_key(zx) - 1);

    Part acc = {-INFINITY, 0.f, 0.f, 0};
    bool listed = false;
#pragma unroll 1
    for (int r0 = lo; r0 < hi || r0 == lo; r0 += NT * NV) {
        const int end = min(hi, r0 + NT * NV);
        uint4 x[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (r0 + j * NT + tid < end) x[j] = granule(r0 + j * NT + tid);
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (r0 + j * NT + tid < end) mx = fmaxf(mx, granule_max<E>(x[j]));
        const float wm = warp_max(mx);
        __syncthreads();
        if (lane == 0) s.red[0][warp] = wm;
        if (tid == 0) s.found = listed ? K : 0;
        if (listed && tid < K) s.cand[tid] = s.mine[tid];
        __syncthreads();
        float m = s.red[0][0];
#pragma unroll
        for (int w = 1; w < NT / 32; ++w) m = fmaxf(m, s.red[0][w]);
        const float ref = m == -INFINITY ? 0.f : m;
        const bool ranked = p.rank && __any_sync(0xFFFFFFFFu, mx >= zx);
        Sums sums = {0ull, 0ull};
        int above = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int g = r0 + j * NT + tid, at = g * VN - h;
            if (g < end) {
                forget(x[j]);
                float v[VN];
                VecTraits<E>::unpack(x[j], v);
                add_granule<VN>(v, ref, p.c2, &sums);
                if (ranked) {
                    above += count_above<VN>(v, at + VN <= tok ? below : zx);
                    if (at < tok && (at + VN > tok || zx == -INFINITY)) {  // the token's own granule
#pragma unroll
                        for (int e = 0; e < VN; ++e) above += at + e >= 0 && at + e < tok && v[e] == zx;
                    }
                }
                forget(x[j]);
            }
        }
        float S, U, S1, U1;
        unpack2(sums.S, &S, &S1);
        unpack2(sums.U, &U, &U1);
        S += S1;
        U += U1;

        if (K > 0) {
            // a bound that at least K threads' maxima reach: downwards from the
            // maximum by growing steps, then between the last two
            const uint32_t key = f32_key(mx);
            uint32_t lo_k = f32_key(m), hi_k = lo_k + 1, step = 1u << 19;
            int n = __syncthreads_count(key >= lo_k);
            while (n < K && lo_k > 0) {
                hi_k = lo_k;
                lo_k = lo_k > step ? lo_k - step : 0;
                step <<= 1;
                n = __syncthreads_count(key >= lo_k);
            }
            while (n > 2 * K && hi_k - lo_k > 1) {
                const uint32_t mid = lo_k + (hi_k - lo_k) / 2;
                const int c = __syncthreads_count(key >= mid);
                if (c >= K) {
                    lo_k = mid;
                    n = c;
                } else {
                    hi_k = mid;
                }
            }
            if (key >= lo_k) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int g = r0 + j * NT + tid, at = g * VN - h;
                    if (g < end && f32_key(granule_max<E>(x[j])) >= lo_k) {
                        float v[VN];
                        VecTraits<E>::unpack(x[j], v);
#pragma unroll
                        for (int e = 0; e < VN; ++e)
                            if (f32_key(v[e]) >= lo_k && at + e >= 0 && at + e < p.V) {
                                const int to = atomicAdd(&s.found, 1);
                                if (to < kCap) s.cand[to] = cand_key(v[e], at + e);
                            }
                    }
                }
            }
            __syncthreads();
            int n_cand = s.found;
            if (n_cand > kCap) {
                // many equal ones: the K-th key of all elements, then the K-th
                // index among its ties (the elements read again)
                auto count = [&](auto is) {
                    int c = 0;
#pragma unroll 1
                    for (int g = r0 + tid; g < end; g += NT) {
                        float v[VN];
                        VecTraits<E>::unpack(granule(g), v);
#pragma unroll
                        for (int e = 0; e < VN; ++e) {
                            const int i = g * VN - h + e;
                            c += i >= 0 && i < p.V && is(f32_key(v[e]), i);
                        }
                    }
                    return block_sum<NT>(c, s.cnt);
                };
                const int want = min(K, count([](uint32_t, int) { return true; }));
                uint32_t a = 0, z = 0xFFFFFFFFu;  // reached by `want` or more, and by fewer
                while (z - a > 1) {
                    const uint32_t mid = a + (z - a) / 2;
                    if (count([&](uint32_t k, int) { return k >= mid; }) >= want) a = mid;
                    else z = mid;
                }
                int ia = -1, iz = p.V - 1;  // up to iz are enough, up to ia are not
                while (iz - ia > 1) {
                    const int mid = ia + (iz - ia) / 2;
                    if (count([&](uint32_t k, int i) { return k > a || (k == a && i <= mid); }) >= want) iz = mid;
                    else ia = mid;
                }
                const int before = listed ? K : 0;
                __syncthreads();
                if (tid == 0) s.found = before;
                if (tid < before) s.cand[tid] = s.mine[tid];
                __syncthreads();
                count([&](uint32_t k, int i) {
                    if (k > a || (k == a && i <= iz)) s.cand[atomicAdd(&s.found, 1)] = ((u64)k << 32) | (0xFFFFFFFFu - (uint32_t)i);
                    return false;
                });
                __syncthreads();
                n_cand = s.found;
            }
            if (tid < K && n_cand < K) s.mine[tid] = 0;  // (a part of fewer elements)
            if (n_cand < K) __syncthreads();
            rank_keys<NT>(s.cand, n_cand, K, s.mine);
            listed = true;
        }

        // this round joined to the ones before it
        S = warp_sum(S);
        U = warp_sum(U);
        above = __reduce_add_sync(0xFFFFFFFFu, above);
        __syncthreads();
        if (lane == 0) {
            s.red[1][warp] = S;
            s.red[2][warp] = U;
            s.cnt[warp] = above;
        }
        __syncthreads();
        S = U = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            S += s.red[1][w];
            U += s.red[2][w];
            acc.above += s.cnt[w];
        }
        if (r0 == lo) {
            acc.m = m;
            acc.S = S;
            acc.U = U;
        } else {
            const float top = fmaxf(acc.m, m), at = top == -INFINITY ? 0.f : top;
            const float da = octaves(acc.m, at, p.c2), db = octaves(m, at, p.c2), wa = ex2(da), wb = ex2(db);
            acc.U = wa * fmaf(acc.S, da, acc.U) + wb * fmaf(S, db, U);
            acc.S = wa * acc.S + wb * S;
            acc.m = top;
        }
    }

    if (p.parts > 1) {
        cluster_wait();
        if (tid == 0) {
            const uint32_t a = in_first(&s.parts[part]);
            st_cluster(a, ((u64)__float_as_uint(acc.S) << 32) | __float_as_uint(acc.m));
            st_cluster(a + 8, ((u64)(uint32_t)acc.above << 32) | __float_as_uint(acc.U));
        }
        if (tid < K) st_cluster(in_first(&s.best[part * K + tid]), s.mine[tid]);
        cluster_arrive();
        cluster_wait();
        if (!first) return;
    } else {
        if (tid == 0) s.parts[0] = acc;
        if (tid < K) s.best[tid] = s.mine[tid];
        __syncthreads();
    }

    float m = -INFINITY;
    for (int c = 0; c < p.parts; ++c) m = fmaxf(m, s.parts[c].m);
    float S = 0.f, U = 0.f;
    int above = 0;
    for (int c = 0; c < p.parts; ++c) {
        const Part q = s.parts[c];
        const float d = octaves(q.m, m, p.c2), w = ex2(d);
        S = fmaf(w, q.S, S);
        U += w * fmaf(q.S, d, q.U);
        above += q.above;
    }
    // (S is 0 where all are -inf, NaN with a NaN or +inf among them)
    const bool bad = !(S > 0.f) || m == INFINITY;
    const float log_s = logf(S), nan = __int_as_float(0x7FC00000);
    if (tid == 0) {
        p.logprob[row] = bad ? nan : (zx - m) * p.inv_t - log_s;
        if (p.entropy) p.entropy[row] = bad ? nan : fmaxf(0.f, log_s - U / S * 0.69314718055994531f);
        if (p.rank) p.rank[row] = bad ? -1 : above;
        if (p.status) {
            if (p.P == 1) p.status[b] = bad ? kEData : kOk;
            else if (bad) atomicMax(p.status + b, kEData);
        }
    }
    if (bad) {
        if (tid < K) {
            p.top_tokens[row * K + tid] = -1;
            p.top_logprobs[row * K + tid] = nan;
        }
    } else if (K > 0) {
        const int n = p.parts * K;
        for (int i = tid; i < n; i += NT) {
            const u64 key = s.best[i];
            int r = 0;
            for (int j = 0; j < n; ++j) r += s.best[j] > key;
            // (0: a part of fewer elements had none to give)
            if (key != 0 && r < K && SV_IN(row * K + r, p.rows * K)) {
                const float z = key_to_f32((uint32_t)(key >> 32));
                p.top_tokens[row * K + r] = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
                p.top_logprobs[row * K + r] = (z - m) * p.inv_t - log_s;
            }
        }
    }
}

template <typename E, int NT, int NV>
cudaError_t launch(LogprobParams p, cudaStream_t st) {
    constexpr int VN = VecTraits<E>::kN;
    const long long granules = ((long long)p.V + VN - 1) / VN + 1;  // (one more where the row starts inside one)
    // as few CTAs a row as hold it in their registers; more where there are few
    // rows, down to parts of four granules a thread
    int parts = 1;
    while (parts < kMaxParts && granules > (long long)parts * NT * NV) parts *= 2;
    while (parts < kMaxParts && p.rows * parts < 152 * 2 && granules / parts > NT * 2) parts *= 2;
    p.parts = parts;
    p.part_granules = (int)((granules + parts - 1) / parts);
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = parts;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.rows * parts));
    cfg.blockDim = dim3(NT);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprob_kernel<E, NT, NV>, p);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, int dtype, cudaStream_t st) {
    return dtype == 0 ? launch<float, 512, 8>(p, st) : launch<bf16_t, 256, 8>(p, st);
}

SV_DEBUG_READER(logprobs)

}  // namespace sv
