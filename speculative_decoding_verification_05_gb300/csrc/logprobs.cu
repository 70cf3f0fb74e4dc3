// Log probabilities of given tokens, their ranks, the rows' entropies and the
// likeliest alternatives, in one pass over the logits.
//
// With y_i = (z_i - m) / T, m the row's maximum and S = sum e^{y_i}:
//   log p(x) = y_x - ln S,   H = ln S - (sum e^{y_i} y_i) / S,
//   rank(x) = #{z_i > z_x} + #{i < x: z_i = z_x},
// and the alternatives are the first K in the order (z descending, i ascending).
//
// A row is split over a cluster of CTAs (one to eight). A thread streams its
// share in batches of a few 16-byte granules, the next batch on its way, and adds
// up against its own maximum so far, so no thread waits for another before the
// part's end. Exponents are t = z c2 - M, c2 = log2(e) / T, with one rounding, M
// the rounded product of the maximum and c2: whatever M's rounding is, it is the
// same for all terms and drops out of t_x - log2 S. Parts leave (m, sum 2^t, sum
// 2^t t, count above z_x) and their K best in the first CTA's shared memory, which
// joins them in the order of the parts: results depend on the shape alone.
//
// The K best of a part: any key that K threads' maxima reach is a bound that no
// better element lies below, so a search over the threads' maxima (one count of
// the block a step) ends at a bound that K to 5 K / 4 of them reach; only those
// threads' granules are read again (from L2, shared out over the block), and the
// few elements that reach the bound are ranked by comparing all with all. Where
// they are more than fit (rows of equal logits) the bound is taken over the
// elements themselves, then over the indices of the ties.
//
// What bounds it: latency and issue, no longer memory. float32 takes 14 warp
// instructions for 32 elements (an exponential, 2.5 for the sums, 1.5 for the
// rank, the rest loads and batches' ends), bf16 15; the scheduler issues in half
// to two thirds of the cycles. 288 rows of 128256 float32 logits: 37.0 us without
// alternatives (4.0 TB/s; 28.8 in parts of half a row), 45.7 with 20; 2000 rows of
// 32016 bf16: 37.4 us (3.4 TB/s); five rows of 32000 bf16, five alternatives: 10.4
// us. Tried: a part held in registers whole, the maximum first (a barrier between
// every two passes; 59 us for the 288 rows), the parts' granules through shared
// memory by asynchronous copies, 6 to 12 a thread in flight (33 to 41 us), four
// granules a batch for bf16 (spills; 47 us for the 2000 rows).

#include <algorithm>

#include "attention.cuh"
#include "logprobs.cuh"
#include "specverify.h"

namespace sv {
namespace {

typedef unsigned long long u64;

constexpr int kMaxTop = SPEC_MAX_TOP;
constexpr int kMaxParts = 8;
constexpr float kLn2 = 0.69314718055994531f;
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
    u64 cand[kCap];
    float red[3][NT / 32];
    int cnt[NT / 32], sum[NT / 32];
    int found, flagged;
    int who[NT];  // threads whose maximum reaches the bound
};

SV_DEV uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// (not the aligned forms: a warp's threads come to the second arrival from branches)
SV_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
SV_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

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

// Whether exponents against the maximum m are taken from its rounded product M = m
// c2. Its rounding, which all terms of a sum share, is then below 2^-4; past that (low
// temperatures, masks of the type's lowest value) the difference v - m comes first.
SV_DEV bool by_product(float m, float c2) { return fabsf(m * c2) < 0x1p20f; }

// The exponent of v against the reference m, from -200 on (2^-200 is 0).
SV_DEV float exponent(float v, float m, float c2) {
    return fmaxf(by_product(m, c2) ? fmaf(v, c2, -__fmul_rn(m, c2)) : (v - m) * c2, -200.f);
}
// How far one reference lies below another (a part of nothing but -inf has none).
SV_DEV float octaves(float m, float top, float c2) {
    if (m == -INFINITY) return -200.f;
    const float a = __fmul_rn(m, c2), b = __fmul_rn(top, c2);
    const float d = by_product(m, c2) ? (by_product(top, c2) ? a - b : fmaf(-top, c2, a))
                                      : (by_product(top, c2) ? fmaf(m, c2, -b) : (m - top) * c2);
    return fmaxf(d, -200.f);
}

// The n keys in cand (distinct) ranked against one another; the first k, in
// descending order, to best.
template <int NT>
SV_DEV void rank_keys(const u64* cand, int n, int k, u64* best) {
    for (int i = threadIdx.x; i < n; i += NT) {
        const u64 key = cand[i];
        int r = 0;
        for (int j = 0; j < n; ++j) r += cand[j] > key;
        if (r < k && SV_IN(r, kMaxTop)) best[r] = key;
    }
}

// Stops the compiler from keeping what it unpacked from a word for the next pass
// (it needs more registers than the thread has).
SV_DEV void forget(uint4& x) { asm volatile("" : "+r"(x.x), "+r"(x.y), "+r"(x.z), "+r"(x.w)); }

SV_DEV void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

SV_DEV float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
SV_DEV uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The largest of a granule's elements and of `m` (NaN loses).
template <typename E>
SV_DEV float granule_max(const uint4& x, float m) {
    if constexpr (sizeof(E) == 4) {
        return max3(max3(m, __uint_as_float(x.x), __uint_as_float(x.y)), __uint_as_float(x.z), __uint_as_float(x.w));
    } else {
        const uint32_t a = max_bf16x2(max_bf16x2(x.x, x.y), max_bf16x2(x.z, x.w));
        return max3(m, __uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
    }
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

// A thread's sums against its maximum so far.
template <typename E>
struct Stream {
    static constexpr int VN = VecTraits<E>::kN;
    float m = -INFINITY, c2;
    float M = __builtin_nanf("");  // of m; NaN where exponents are not taken from it
    uint64_t S = 0ull, U = 0ull;  // 2^t, 2^t t, two at a time
    int above = 0;

    // n granules; z_x is `zx`, `t` what counts as above it in all of them (ranked).
    template <int n>
    SV_DEV void add(uint4 (&x)[n], bool rank, float zx, float t) {
        float top = m;
#pragma unroll
        for (int j = 0; j < n; ++j) top = granule_max<E>(x[j], top);
        if (top > m) {
            float to = __fmul_rn(top, c2);
            to = fabsf(to) < 0x1p20f ? to : __builtin_nanf("");
            float d = M - to;
            d = d == d ? fmaxf(d, -200.f) : octaves(m, top, c2);
            const float w = ex2(d);
            const uint64_t dd = pack2(d, d), ww = pack2(w, w);
            U = mul2(ww, fma2(dd, S, U));
            S = mul2(ww, S);
            m = top;
            M = to;
        }
        const uint64_t cc = pack2(c2, c2), mm = pack2(-M, -M);
        const bool count = rank && __any_sync(__activemask(), m >= zx);
        uint64_t s = 0ull, u = 0ull;
#pragma unroll
        for (int j = 0; j < n; ++j) {
            forget(x[j]);
            float v[VN];
            VecTraits<E>::unpack(x[j], v);
#pragma unroll
            for (int e = 0; e < VN; e += 2) {
                const uint64_t tt = fma2(pack2(v[e], v[e + 1]), cc, mm);
                float t0, t1;
                unpack2(tt, &t0, &t1);
                const uint64_t w = pack2(ex2(t0), ex2(t1));
                s = add2(s, w);
                u = fma2(w, tt, u);
            }
            if (count) above += count_above<VN>(v, t);
        }
        float u0, u1;
        unpack2(u, &u0, &u1);
        u0 += u1;
        if (!(fabsf(u0) < INFINITY)) {  // a logit of -inf gave 0 times infinity, or M is NaN, or the row is bad: one by one
            float s0 = 0.f;
            u0 = 0.f;
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int j = 0; j < n; ++j) {
                float v[VN];
                VecTraits<E>::unpack(x[j], v);
#pragma unroll
                for (int e = 0; e < VN; ++e) {
                    const float e2 = exponent(v[e], ref, c2), w = v[e] != v[e] || v[e] == INFINITY ? v[e] - v[e] : ex2(e2);
                    s0 += w;
                    u0 = fmaf(w, e2, u0);
                }
            }
            s = pack2(s0, 0.f);
            u = pack2(u0, 0.f);
        }
        S = add2(S, s);
        U = add2(U, u);
    }
};

template <typename E, int NT, int U>
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
        if (tid == 0 && SV_IN(row, p.rows)) {
            p.logprob[row] = bad ? nan : 0.f;
            if (p.entropy) p.entropy[row] = bad ? nan : 0.f;
            if (p.rank) p.rank[row] = -1;
            if (p.status && (bad || p.P == 1)) {
                if (p.P == 1) p.status[b] = bad ? kEData : kOk;
                else atomicMax(p.status + b, kEData);
            }
        }
        if (tid < K && SV_IN(row * K + tid, p.rows * K)) {
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

    // Whole granules [in, out) of the part lie inside the row; the row's first and
    // last may not.
    const int in = lo + (lo == 0 && h > 0), out = min(hi, (p.V + h) / VN), mine = (tok + h) / VN;  // (the token's granule)
    // (a row inside one granule has one edge: the first)
    const bool head = in > lo, tail = out < hi && out >= in, rank = p.rank != nullptr;
    Stream<E> a;
    a.c2 = p.c2;
    // granules from g on, NT apart: added, those before the token's counted as
    // above it with ties. `base`: the block's first, `n` of them a thread
    auto add = [&](auto& x, int base, int n) {
        const int g = base + tid;
        if (base > mine || base + n * NT <= mine) {
            a.add(x, rank, zx, base > mine ? zx : below);
            return;
        }
        // (the batch that holds the token's granule)
        a.add(x, false, zx, zx);
        for (int j = 0; rank && j < n; ++j) {
            float v[VN];
            uint4 y = x[0];
#pragma unroll
            for (int k = 1; k < n; ++k)
                if (k == j) y = x[k];
            VecTraits<E>::unpack(y, v);
            a.above += count_above<VN>(v, g + j * NT < mine ? below : zx);
            const int at = (g + j * NT) * VN - h;
            if (g + j * NT == mine)
#pragma unroll
                for (int e = 0; e < VN; ++e) a.above += at + e >= 0 && at + e < tok && v[e] == zx;
        }
    };
    {
        const uint4* z = g0 + in + tid;
        const int full = max(0, (out - in) / (NT * U)), base = in + full * (NT * U);
        // (what comes last, less than a batch and the edges, is called for now)
        for (int g = base + tid; g < out; g += NT) prefetch_l2(g0 + g);
        uint4 x[U], y[U];
        auto fetch = [&](uint4 (&to)[U], int i) {
#pragma unroll
            for (int j = 0; j < U; ++j) to[j] = ld_stream_v4(z + (long long)i * (NT * U) + j * NT);
        };
        if (full > 0) fetch(x, 0);
#pragma unroll 1
        for (int i = 0; i < full; i += 2) {
            if (i + 1 < full) fetch(y, i + 1);
            add(x, in + i * (NT * U), U);
            if (i + 1 < full) {
                if (i + 2 < full) fetch(x, i + 2);
                add(y, in + (i + 1) * (NT * U), U);
            }
        }
#pragma unroll 1
        for (int j = base < out ? 0 : U; j < U + 2; ++j) {
            // the row's edges: one thread each
            const int g = j < U ? base + j * NT + tid : j == U ? (tid == 0 && head ? lo : hi) : (tid == 0 && tail ? out : hi);
            if (g < (j < U ? out : hi)) {
                uint4 one[1] = {granule(g)};
                add(one, g - tid, 1);
            }
        }
    }
    __syncwarp();
    if (rank && zx == -INFINITY) {  // a token without probability: its ties before it
#pragma unroll 1
        for (int g = lo + tid; g < min(hi, mine + 1); g += NT) {
            float v[VN];
            VecTraits<E>::unpack(granule(g), v);
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                const int i = g * VN - h + e;
                // (the token's own granule has counted its ties already)
                a.above += g != mine && i >= 0 && v[e] == zx;
            }
        }
        __syncwarp();
    }
    float m = a.m;
    int above = a.above;

    // The part's maximum, and the sums against it.
    Part acc;
    {
        const float wm = warp_max(m);
        if (lane == 0) s.red[0][warp] = wm;
        if (tid == 0) s.found = s.flagged = 0;
        __syncthreads();
        acc.m = s.red[0][0];
#pragma unroll
        for (int w = 1; w < NT / 32; ++w) acc.m = fmaxf(acc.m, s.red[0][w]);
        float S, T, S1, T1;
        unpack2(a.S, &S, &S1);
        unpack2(a.U, &T, &T1);
        const float d = octaves(m, acc.m, p.c2), w = ex2(d);
        S += S1;
        T = w * fmaf(d, S, T + T1);
        S *= w;
        S = warp_sum(S);
        T = warp_sum(T);
        above = __reduce_add_sync(0xFFFFFFFFu, above);
        if (lane == 0) {
            s.red[1][warp] = S;
            s.red[2][warp] = T;
            s.cnt[warp] = above;
        }
    }

    if (K > 0) {
        // a bound that at least K threads' maxima reach: downwards from the
        // maximum by growing steps, then between the last two
        const uint32_t key = f32_key(m);
        uint32_t lo_k = f32_key(acc.m), hi_k = lo_k + 1, step = 1u << 19;
        int n = __syncthreads_count(key >= lo_k);
        while (n < K && lo_k > 0) {
            hi_k = lo_k;
            lo_k = lo_k > step ? lo_k - step : 0;
            step <<= 1;
            n = __syncthreads_count(key >= lo_k);
        }
        // (up to 2 K of them: 41.4 us for 38.7 where the granules that are read again come
        // from DRAM, 512 rows of 128256 float32 logits, 288 with a token, 20 alternatives)
        while (n > K + K / 4 && hi_k - lo_k > 1) {
            const uint32_t mid = lo_k + (hi_k - lo_k) / 2;
            const int c = __syncthreads_count(key >= mid);
            if (c >= K) {
                lo_k = mid;
                n = c;
            } else {
                hi_k = mid;
            }
        }
        auto gather = [&](const uint4& x, int g) {
            if (f32_key(granule_max<E>(x, -INFINITY)) < lo_k) return;
            float v[VN];
            VecTraits<E>::unpack(x, v);
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                const int i = g * VN - h + e;
                if (f32_key(v[e]) >= lo_k && i >= 0 && i < p.V) {
                    const int to = atomicAdd(&s.found, 1);
                    if (to < kCap) s.cand[to] = cand_key(v[e], i);
                }
            }
        };
        if (tid == 0 && head) gather(granule(lo), lo);
        if (tid == 0 && tail) gather(granule(out), out);
        if (key >= lo_k) {
            const int to = atomicAdd(&s.flagged, 1);
            if (SV_IN(to, NT)) s.who[to] = tid;
        }
        __syncthreads();
        const int who = s.flagged, jobs = who * max(0, (out - in + NT - 1) / NT);
#pragma unroll 1
        for (int i0 = tid; i0 < jobs; i0 += NT * U) {
            uint4 x[U];
            int g[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int i = i0 + j * NT, k = i / who;
                g[j] = i < jobs ? in + k * NT + s.who[i - k * who] : out;
                if (g[j] < out) x[j] = ld_stream_v4(g0 + g[j]);
            }
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (g[j] < out) gather(x[j], g[j]);
        }
        __syncthreads();
        int n_cand = s.found;
        if (n_cand > kCap) {
            // many equal ones: the K-th key of all elements, then the K-th index
            // among its ties
            auto count = [&](auto is) {
                int c = 0;
#pragma unroll 1
                for (int g = lo + tid; g < hi; g += NT) {
                    float v[VN];
                    VecTraits<E>::unpack(granule(g), v);
#pragma unroll
                    for (int e = 0; e < VN; ++e) {
                        const int i = g * VN - h + e;
                        c += i >= 0 && i < p.V && is(f32_key(v[e]), i);
                    }
                }
                return block_sum<NT>(c, s.sum);
            };
            const int want = min(K, count([](uint32_t, int) { return true; }));
            // reached by `want` or more, and by fewer (by none: the key of the NaN 0x7FFFFFFF is
            // 2^32 - 1)
            u64 k0 = 0, k1 = 1ull << 32;
            while (k1 - k0 > 1) {
                const u64 mid = k0 + (k1 - k0) / 2;
                if (count([&](uint32_t k, int) { return k >= mid; }) >= want) k0 = mid;
                else k1 = mid;
            }
            int i0 = -1, i1 = p.V - 1;  // up to i1 are enough, up to i0 are not
            while (i1 - i0 > 1) {
                const int mid = i0 + (i1 - i0) / 2;
                if (count([&](uint32_t k, int i) { return k > k0 || (k == k0 && i <= mid); }) >= want) i1 = mid;
                else i0 = mid;
            }
            if (tid == 0) s.found = 0;
            __syncthreads();
            count([&](uint32_t k, int i) {
                if (k > k0 || (k == k0 && i <= i1)) {
                    const int to = atomicAdd(&s.found, 1);  // (`want` of them in all)
                    if (to < kCap && SV_IN(to, kMaxTop)) s.cand[to] = ((u64)k << 32) | (0xFFFFFFFFu - (uint32_t)i);
                }
                return false;
            });
            __syncthreads();
            n_cand = min(s.found, kCap);
        }
        if (n_cand < K) {  // (a part of fewer elements)
            if (tid < K) s.mine[tid] = 0;
            __syncthreads();
        }
        rank_keys<NT>(s.cand, n_cand, K, s.mine);
    }
    __syncthreads();
    acc.S = acc.U = 0.f;
    acc.above = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        acc.S += s.red[1][w];
        acc.U += s.red[2][w];
        acc.above += s.cnt[w];
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

    m = -INFINITY;
    for (int c = 0; c < p.parts; ++c) m = fmaxf(m, s.parts[c].m);
    float S = 0.f, T = 0.f;
    above = 0;
    for (int c = 0; c < p.parts; ++c) {
        const Part q = s.parts[c];
        const float d = octaves(q.m, m, p.c2), w = ex2(d);
        S = fmaf(w, q.S, S);
        T += w * fmaf(q.S, d, q.U);
        above += q.above;
    }
    // (S is 0 where all are -inf, NaN with a NaN or +inf among them)
    const bool bad = !(S > 0.f) || m == INFINITY;
    const float log_s = logf(S), nan = __int_as_float(0x7FC00000);
    const float M = m * p.c2;
    // (not above 0 by a rounding)
    auto log_of = [&](float z) {
        const float t = fmaf(z, p.c2, -M);
        return fminf(0.f, (by_product(m, p.c2) && fabsf(t) < INFINITY ? t * kLn2 : (z - m) * p.inv_t) - log_s);
    };
    if (tid == 0 && SV_IN(row, p.rows)) {
        p.logprob[row] = bad ? nan : log_of(zx);
        if (p.entropy) p.entropy[row] = bad ? nan : fmaxf(0.f, log_s - T / S * kLn2);
        if (p.rank) p.rank[row] = bad ? -1 : above;
        if (p.status) {
            if (p.P == 1) p.status[b] = bad ? kEData : kOk;
            else if (bad) atomicMax(p.status + b, kEData);
        }
    }
    if (bad) {
        if (tid < K && SV_IN(row * K + tid, p.rows * K)) {
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
                p.top_logprobs[row * K + r] = log_of(z);
            }
        }
    }
}

template <typename E, int NT, int U>
cudaError_t launch(LogprobParams p, cudaStream_t st) {
    constexpr int VN = VecTraits<E>::kN;
    const long long granules = ((long long)p.V + VN - 1) / VN + 1;  // (one more where the row starts inside one)
    // Few rows are split, until there are four CTAs an SM, down to parts of two
    // granules a thread: a part's end costs as much as 30 KB of it. 288 rows of
    // 128256 float32 logits, no alternatives (and 20): 32.9 (43.0) us whole, 28.8
    // (36.1) in two parts, 37.0 (45.5) in four. Half of a step's rows have no token
    // as a rule (512 rows, 288 with one, 20 alternatives: 49.0 us whole, 38.5 in two
    // parts, 46.7 in four), hence four and not two, which a few hundred rows that all
    // have a token pay for.
    int parts = 1;
    while (parts < kMaxParts && p.rows * parts < 152 * 4 && granules / parts > NT * 2) parts *= 2;
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
    return cudaLaunchKernelEx(&cfg, logprob_kernel<E, NT, U>, p);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, int dtype, cudaStream_t st) {
    // bf16 rows by blocks of 128 threads (of 256): 2000 rows of 32016 37.3 us (43.1), with
    // five alternatives 46.4 (53.3); 256 of 128256 22.1 (24.6), with 20 30.8 (34.9). float32
    // rows by 256 (128): of 128256 with 20 alternatives, 288 of 512 with a token, 39.0 us
    // (54.5), five with five 12.6 (14.4); but 2000 of 32000 54.5 (49.0), which this rule by
    // type leaves.
    return dtype == 0 ? launch<float, 256, 4>(p, st) : launch<bf16_t, 128, 2>(p, st);
}

SV_DEBUG_READER(logprobs)

}  // namespace sv
