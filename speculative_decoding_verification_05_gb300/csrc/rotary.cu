// Rotary positions of a step's nodes, fused with the cache's append: queries
// rotated, keys rotated into their pages, values copied into theirs, one pass.
//
// Pair j of a head's first `dim` columns is turned by the angle pos f_j:
//   (a, b) -> factor (a cos - b sin, b cos + a sin),
// columns (j, j + dim / 2) or, interleaved, (2 j, 2 j + 1). f_j is kept as a
// fraction of a full turn in units of 2^-64, so pos f_j modulo a turn is one
// integer product that wraps, exact for every position (a float32 angle at
// position 10^6 is off by 0.06 radians); what is left of it after the nearest
// quarter turn goes through sinpi and cospi. Products are fp32, rounded once.
//
// A block takes a few tokens: their cosines and sines once in shared memory for
// all heads, then a thread a 16-byte column (or a pair of them) of one token, its
// cosines in registers, and every few heads of it, two to four rows in flight; the
// first rows and values are under way before the cosines are computed. Neighbouring
// threads have neighbouring heads (neighbouring tokens: 36.2 us for 32.4 then).
//
// Bound by memory where there is enough of it: 8 x 1000 tokens, 32 query and 8 key
// heads of 128 columns, bf16: 32.6 us, 5.5 TB/s read and written (the append alone,
// which has no queries to write, 6.0). Below that by the chain of lengths, table,
// cosines and rows: 16 trees of 61 nodes, 12 heads of 64, float32: 7.5 us, one chain
// of 5: 3.9 us.

#include <algorithm>

#include "cache.cuh"
#include "specverify.h"

namespace sv {
namespace {

constexpr int CT = 256;
constexpr int kMostTokens = 4;

SV_DEV uint4 ldg16(const char* p) { return *reinterpret_cast<const uint4*>(p); }
SV_DEV void stg16(char* p, uint4 x) { *reinterpret_cast<uint4*>(p) = x; }

template <typename E>
SV_DEV uint4 pack(const float (&x)[VecTraits<E>::kN]) {
    if constexpr (sizeof(E) == 4) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// (cos, sin) of pos turns 2^-64 of a turn, times factor.
SV_DEV float2 turn(unsigned long long turns, long long pos, float factor) {
    const unsigned long long ph = turns * (unsigned long long)pos;
    const uint32_t quarter = (uint32_t)((ph + (1ull << 61)) >> 62);
    const float x = (float)(long long)(ph - ((unsigned long long)quarter << 62)) * 0x1p-63f;  // half turns, in [-1/4, 1/4]
    float s, c;
    sincospif(x, &s, &c);
    const float a = quarter & 1 ? -s : c, b = quarter & 1 ? c : s;
    return quarter & 2 ? make_float2(-a * factor, -b * factor) : make_float2(a * factor, b * factor);
}

SV_DEV void rotate(float a, float b, float2 cs, float* x, float* y) {
    *x = fmaf(a, cs.x, -(b * cs.y));
    *y = fmaf(b, cs.x, a * cs.y);
}

// How a head's rotated columns lie in 16-byte words.
enum Layout : int {
    kHalves,    // word j and word j + dim / 2 columns later hold pairs
    kNeighbours,  // a word holds whole pairs
    kSplit      // halves that do not begin at a word: the partners one by one
};

// Word c of a row (kHalves: the words c and c + half of its rotated columns
// where c < half): the result's one or two words. cs: the token's pairs.
template <typename E, int LAYOUT>
struct Row {
    static constexpr int VN = VecTraits<E>::kN, kPairs = LAYOUT == kNeighbours ? VN / 2 : VN;
    uint4 x, y;
    // The word's pairs of a token's (cs).
    SV_DEV static void pairs(const RotaryParams& p, const float2* cs, int c, float2 (&z)[kPairs]) {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            int j = c * kPairs + e;
            if (LAYOUT == kSplit && j >= p.half) j -= p.half;
            if (j < p.half) z[e] = cs[j];
        }
    }
    SV_DEV void load(const RotaryParams& p, const char* from, int c) {
        x = ldg16(from + c * 16);
        if (LAYOUT == kHalves && c * VN < p.half) y = ldg16(from + c * 16 + p.half * (int)sizeof(E));
    }
    SV_DEV void store(const RotaryParams& p, const char* from, char* to, int c, const float2 (&cs)[kPairs]) {
        float a[VN], b[VN], u[VN], v[VN];
        VecTraits<E>::unpack(x, a);
        if (LAYOUT == kHalves) {
            if (c * VN >= p.half) return stg16(to + c * 16, x);
            VecTraits<E>::unpack(y, b);
#pragma unroll
            for (int e = 0; e < VN; ++e) rotate(a[e], b[e], cs[e], &u[e], &v[e]);
            stg16(to + c * 16, pack<E>(u));
            stg16(to + c * 16 + p.half * (int)sizeof(E), pack<E>(v));
        } else if (LAYOUT == kNeighbours) {
#pragma unroll
            for (int e = 0; e < VN; e += 2) {
                const int j = (c * VN + e) >> 1;
                u[e] = a[e];
                u[e + 1] = a[e + 1];
                if (j < p.half) rotate(a[e], a[e + 1], cs[e >> 1], &u[e], &u[e + 1]);
            }
            stg16(to + c * 16, pack<E>(u));
        } else {
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                const int i = c * VN + e, j = i < p.half ? i : i - p.half;
                u[e] = a[e];
                if (j < p.half) {
                    const float other = VecTraits<E>::load1(from + (i < p.half ? i + p.half : j) * (int)sizeof(E));
                    float w;
                    if (i < p.half) rotate(a[e], other, cs[e], &u[e], &w);
                    else rotate(other, a[e], cs[e], &w, &u[e]);
                }
            }
            stg16(to + c * 16, pack<E>(u));
        }
    }
};

template <typename E, int LAYOUT>
__global__ void __launch_bounds__(CT, 4) append_rotary_kernel(const __grid_constant__ RotaryParams p) {
    constexpr int VN = VecTraits<E>::kN;
    __shared__ float2 cs[kMostTokens * SPEC_MAX_HEAD_DIM / 2];
    __shared__ long long place[kMostTokens];
    const int b = blockIdx.y, tid = threadIdx.x, sh = p.c.page_shift, D = p.c.row_bytes / (int)sizeof(E);
    const long long L = p.cache_len[b], pos0 = p.positions ? p.positions[b] : L;
    const int n = p.n_nodes ? p.n_nodes[b] : p.N;
    const int32_t* table = p.table + b * p.table_stride;
    const int32_t* depth = p.depth ? p.depth + (long long)b * p.N : nullptr;
    bool ok = L >= 0 && n >= 0 && n <= p.N && L + n <= ((long long)p.max_pages << sh) && pos0 >= 0;
    if (ok && n > 0) {
        bool bad = false;
        for (int i = (int)(L >> sh) + tid; i <= (int)((L + n - 1) >> sh); i += CT) {
            const int id = __ldg(table + i);
            if (id < 0 || id >= p.c.num_pages) bad = true;
            else if (p.c.refs) bad |= __ldg(p.c.refs + id) != 1;
        }
        if (depth) {
            for (int i = tid; i < n; i += CT) bad |= depth[i] < 0 || pos0 + depth[i] > 0x7FFFFFFFLL;
        } else {
            bad |= pos0 + n - 1 > 0x7FFFFFFFLL;
        }
        ok = !__syncthreads_or(bad);
    }
    if (blockIdx.x == 0 && tid == 0 && p.status) p.status[b] = ok ? kOk : kEData;

    const int t0 = blockIdx.x * p.tokens, t1 = min(t0 + p.tokens, p.N), used = ok ? min(t1, max(n, t0)) : t0;
    // queries of nodes that are not there: zeros; of a sequence with bad data: NaN
    {
        const uint32_t fill = ok ? 0u : (sizeof(E) == 4 ? 0x7FC00000u : 0x7FC07FC0u);
        const long long words = (long long)(t1 - used) * p.q_heads * (D / VN);
        char* o = p.q_out + ((long long)b * p.N + used) * p.q_heads * p.c.row_bytes;
        const long long at = ((long long)b * p.N + used) * p.q_heads * (D / VN), all = (long long)p.B * p.N * p.q_heads * (D / VN);
        for (long long i = tid; i < words; i += CT)
            if (SV_IN(at + i, all)) stg16(o + i * 16, make_uint4(fill, fill, fill, fill));
    }
    if (used == t0) return;  // (the same for the whole block)
    // rotated rows, the queries' heads, then the keys': a thread has one column of
    // one token (its cosines stay in registers) and every `slots`-th head
    const int heads = p.q_heads + p.c.heads;
    const int cols = LAYOUT == kHalves ? (D - p.half) / VN : D / VN, slots = CT / cols / p.tokens;
    const int r0 = tid / cols, c0 = tid - r0 * cols, t = r0 / slots, h0 = r0 - t * slots;
    // (kHalves: columns from half on are the ones that are not rotated)
    const int c = LAYOUT == kHalves && c0 * VN >= p.half ? c0 + p.half / VN : c0;
    const bool mine = t < used - t0;
    const long long token = (long long)b * p.N + t0 + t;
    auto from = [&](int h) {
        return h < p.q_heads ? p.q + (token * p.q_heads + h) * p.c.row_bytes : p.k + (token * p.c.heads + h - p.q_heads) * p.c.row_bytes;
    };
    constexpr int U = LAYOUT == kHalves ? 2 : 4;  // rows in flight
    Row<E, LAYOUT> row[U];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h + u * slots < heads) row[u].load(p, from(h + u * slots), c);
    };
    // the values, as they are: the first ones, and the first rows, are on their way
    // while the cosines are computed
    const int per_head = D / VN, per_token = p.c.heads * per_head, words = (used - t0) * per_token;
    const char* v = p.v + ((long long)b * p.N + t0) * per_token * 16;
    constexpr int VU = 2;
    uint4 x[VU];
#pragma unroll
    for (int u = 0; u < VU; ++u)
        if (tid + u * CT < words) x[u] = ldg16(v + (long long)(tid + u * CT) * 16);
    if (mine) load(h0);
    for (int i = tid; i < (used - t0) * p.half; i += CT) {
        const int t = i / p.half, j = i - t * p.half;
        cs[i] = turn(__ldg(p.turns + j), pos0 + (depth ? depth[t0 + t] : t0 + t), p.factor);
    }
    if (tid < used - t0) {
        const long long pos = L + t0 + tid;
        const int id = table[pos >> sh];
        place[tid] = SV_IN(id, p.c.num_pages) ? (long long)id * p.c.page_stride + (pos & ((1 << sh) - 1)) * p.c.token_stride : -1;
    }
    __syncthreads();
    auto put = [&](int i, uint4 y) {
        const int t = i / per_token, e = i - t * per_token, h = e / per_head;
        if (SV_IN(h, p.c.heads) && SV_PLACE(place[t]))
            stg16(p.c.v + place[t] + h * p.c.head_stride + (e - h * per_head) * 16, y);
    };
#pragma unroll
    for (int u = 0; u < VU; ++u)
        if (tid + u * CT < words) put(tid + u * CT, x[u]);
    if (mine) {
        float2 z[Row<E, LAYOUT>::kPairs];
        Row<E, LAYOUT>::pairs(p, cs + t * p.half, c, z);
        char* const k = p.c.k + place[t];
        for (int h = h0; h < heads; h += U * slots) {
            if (h != h0) load(h);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = h + u * slots;
                if (i < heads && SV_PLACE(place[t]) && SV_IN(token * p.q_heads, (long long)p.B * p.N * p.q_heads) && SV_IN(c, D / VN))
                    row[u].store(p, from(i),
                                 i < p.q_heads ? p.q_out + (token * p.q_heads + i) * p.c.row_bytes : k + (i - p.q_heads) * p.c.head_stride,
                                 c, z);
            }
        }
    }
    for (int i = tid + VU * CT; i < words; i += CT) put(i, ldg16(v + (long long)i * 16));
}

template <typename E>
cudaError_t launch(const RotaryParams& p, dim3 grid, cudaStream_t st) {
    if (p.interleaved) append_rotary_kernel<E, kNeighbours><<<grid, CT, 0, st>>>(p);
    else if (p.half % VecTraits<E>::kN == 0) append_rotary_kernel<E, kHalves><<<grid, CT, 0, st>>>(p);
    else append_rotary_kernel<E, kSplit><<<grid, CT, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_rotary(RotaryParams p, int dtype, cudaStream_t st) {
    // four tokens a block where that leaves every SM four blocks (one: the first
    // steps of a block, its lengths and page, would be taken four times)
    p.tokens = (long long)p.B * p.N >= 152 * 4 * kMostTokens ? kMostTokens : 1;
    const dim3 grid((p.N + p.tokens - 1) / p.tokens, p.B);
    return dtype == 0 ? launch<float>(p, grid, st) : launch<bf16_t>(p, grid, st);
}

SV_DEBUG_READER(rotary)

}  // namespace sv
