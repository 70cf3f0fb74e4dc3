// Tree attention over a paged cache on the CUDA cores, in two kernels for few and
// for many rows, and the kernel that joins partial results (attention.cuh: the mathematics and the division of
// the work). Takes every type and head size; float32 caches and head sizes
// that the tensor-core kernel lacks come here.
//
// One CTA of eight warps takes 16 rows of a unit, two a warp; where a unit has
// fewer, the warps share out a tile's positions as well (8 rows: two warps a
// pair of rows, half the positions each; 2 rows: eight). Tiles of 64 positions
// (32 where a cache row is longer than 256 bytes) of K and V are staged by
// 16-byte asynchronous copies, two tiles deep and across the stays in units. A
// lane scores two positions, one, or a part of one's columns, for both rows of
// its warp; the weights go through a warp-private strip of shared memory, and a
// lane accumulates four (eight: D > 128) output columns in registers, narrow
// heads (D <= 64) two or more positions at a time, in packed pairs. Warps meet
// at the tile's arrival and release, and to add up what the warps of a row
// have. fp32 throughout.
//
// Bound by issued instructions (some 800 a warp and tile of 64 positions, 190
// of them products and their loads) from a few tiles a CTA on, by start-up and
// the join below that: 8 sequences of 8 nodes, 12 heads of 64 columns, float32:
// 9.2 us at contexts of 20, 21.0 at 760, 183 at 12000 (3.3 TB/s of K and V). With
// two warps idle of every four there, a row maximum by shuffles each tile and
// single products it took 24.7 and 234. Tiles of 32 positions with two, three or
// four CTAs an SM took 254, 264 and 339.

#include <algorithm>

#include "attention.cuh"
#include "mbar.cuh"
#include "per_device.h"
#include "specverify.h"

namespace sv {
namespace {

constexpr int NT = 256;
constexpr int kRows = 16;
constexpr int kExtra = 1;  // tiles that a unit's start and end count for
constexpr int kWhole = 2;  // tiles of a unit that is not split

template <typename E>
constexpr int row_bytes(int D) {  // a K row in shared memory: 16 bytes of padding against bank conflicts
    return D * (int)sizeof(E) + 16;
}

template <typename E, int KV>
size_t simt_smem(int D) {
    return (size_t)2 * KV * (row_bytes<E>(D) + D * sizeof(E)) + (size_t)kRows * D * (2 * sizeof(E) + 4) +
           (size_t)kRows * KV * 4;
}

template <typename E>
SV_DEV float4 lds4(const unsigned char* p);
template <>
SV_DEV float4 lds4<float>(const unsigned char* p) {
    return *reinterpret_cast<const float4*>(p);
}
template <>
SV_DEV float4 lds4<bf16_t>(const unsigned char* p) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xFFFF0000u));
}

// Four columns in two packed pairs.
struct Two {
    uint64_t a, b;
};
SV_DEV float lo2(uint64_t x) { return __uint_as_float((uint32_t)x); }
SV_DEV float hi2(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
SV_DEV uint64_t mul1(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
SV_DEV Two axpy2(uint64_t ww, Two x, Two c) {
    return Two{fma2(ww, x.a, c.a), fma2(ww, x.b, c.b)};
}
SV_DEV Two mul2(float f, Two x) {
    const uint64_t ff = pack2(f, f);
    return Two{mul1(ff, x.a), mul1(ff, x.b)};
}
template <typename E>
SV_DEV Two lds4x2(const unsigned char* p) {
    const float4 x = lds4<E>(p);
    return Two{pack2(x.x, x.y), pack2(x.z, x.w)};
}
template <>
SV_DEV Two lds4x2<float>(const unsigned char* p) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(p);
    return Two{x.x, x.y};
}

SV_DEV float4 fma4(float a, float4 v, float4 c) {
    return make_float4(fmaf(a, v.x, c.x), fmaf(a, v.y, c.y), fmaf(a, v.z, c.z), fmaf(a, v.w, c.w));
}

SV_DEV void cp16(uint32_t dst, const void* src, int bytes) {  // the rest of 16 is filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// One tile's K and V rows into a stage, 2^lv lanes a row (its 16-byte words,
// rounded up). Rows past the sequence's end and rows of a page that does not
// exist are zero. Returns whether a page id was bad.
template <typename E, int KV>
SV_DEV bool load_tile(const AttnParams& p, const AttnStay& s, int tile, uint32_t ks, uint32_t vs, int lv) {
    const int vec = p.D * (int)sizeof(E) / 16, ps1 = (1 << p.page_shift) - 1, c = threadIdx.x & ((1 << lv) - 1);
    if (c >= vec) return false;
    const uint32_t pos0 = (uint32_t)tile * KV;
    const int upto = (int)min((long long)KV, s.len - pos0);
    const int32_t* table = p.table + s.b * p.table_stride;
    const long long in = s.h * p.head_stride + c * (16 / (int)sizeof(E));
    const E* kc = static_cast<const E*>(p.k) + in;
    const E* vc = static_cast<const E*>(p.v) + in;
    ks += c * 16;
    vs += c * 16;
    bool bad = false;
#pragma unroll 4
    for (int t = threadIdx.x >> lv; t < KV; t += NT >> lv) {
        const uint32_t pos = pos0 + t;
        int id = t < upto ? __ldg(table + (pos >> p.page_shift)) : 0;
        const bool ok = (uint32_t)id < (uint32_t)p.num_pages;
        bad |= !ok;
        if (!ok) id = 0;
        const long long at = id * p.page_stride + (int)(pos & ps1) * p.token_stride;
        const int bytes = ok && t < upto ? 16 : 0;
        cp16(ks + t * row_bytes<E>(p.D), kc + at, bytes);
        cp16(vs + t * p.D * (int)sizeof(E), vc + at, bytes);
    }
    return bad;
}

template <typename E, int KV>
__global__ void __launch_bounds__(NT, 2) attn_simt_kernel(const __grid_constant__ AttnParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ AttnScan scan;
    __shared__ float2 sums[kRows];  // running maximum and sum by part and row
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = p.D, D4 = D / 4, kstride = row_bytes<E>(D);
    unsigned char* ks = smem;
    unsigned char* vs = ks + 2 * KV * kstride;
    unsigned char* qs = vs + (size_t)2 * KV * D * sizeof(E);               // two stays' queries
    float* os = reinterpret_cast<float*>(qs + 2 * kRows * D * sizeof(E));  // the warps' sums, by part and row
    float* ws = os + kRows * D + warp * 2 * KV;                            // the warp's weights [2][KV]
    const float none = __uint_as_float(0xFF800000u);

    constexpr int NG = KV == 64 ? 1 : 2;  // tiles of 64 positions have rows of 128 columns at most
    // for the product with V a warp's lanes are PG groups of W lanes, a lane a
    // column of four, and every group takes its share of the positions
    const int lw = D4 <= 8 ? 3 : D4 <= 16 ? 4 : 5, W = 1 << lw, PG = 32 >> lw, pg = lane >> lw, vc = lane & (W - 1);
    int col[NG];  // (lanes without a column go along with the last)
#pragma unroll
    for (int g = 0; g < NG; ++g) col[g] = 4 * min(vc + 32 * g, D4 - 1);
    const int lv = 32 - __clz(D * (int)sizeof(E) / 16 - 1);

    asm volatile("griddepcontrol.launch_dependents;");
    const AttnCut cut = attn_locate<KV, NT>(p, &scan);
    AttnWalk<KV> walk(scan, cut);

    // One flat sequence of tiles, whatever stays they belong to: a tile's copies
    // go out, then the one before it is worked on.
    AttnStay sq = {}, next = {};  // that of the tile worked on, of the tile copied
    int tile = 0, ahead = 0;      // of sq, of next
    bool bad, next_bad = false, have = false, more = true;
    // A row's weights are 2^(s - ref), ref the maximum so far, raised only where a
    // score lies more than 8 octaves above it (fp32 sums scale without loss); a
    // lane's l is the sum of its own positions' weights.
    float ref[2], l[2];
    Two acc[2][NG];
#pragma unroll 1
    for (int st = 0, qb = 0; more; st ^= 1) {
        const bool fresh = ahead >= next.last;
        bad = next_bad;
        if (fresh) {
            more = walk.next(p, &next);
            ahead = next.first;
            next_bad = false;
        }
        if (more) {
            next_bad |= load_tile<E, KV>(p, next, ahead, smem_u32(ks) + st * KV * kstride,
                                         smem_u32(vs) + st * KV * D * (int)sizeof(E), lv);
            if (fresh) {
                const int vec = D * (int)sizeof(E) / 16;
                const E* q = static_cast<const E*>(p.q);
#pragma unroll 1
                for (int i = tid; i < next.rows * vec; i += NT) {
                    const int r = i / vec, c = i - r * vec, node = (next.row0 + r) / p.G, g = (next.row0 + r) - node * p.G;
                    const long long row = ((long long)next.b * p.N + node) * (p.Hkv * p.G) + next.h * p.G + g;
                    cp16(smem_u32(qs) + ((qb ^ 1) * kRows * vec + i) * 16, q + row * D + c * (16 / (int)sizeof(E)), 16);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (!have) {  // while the first tile is on its way
            if (tid == 0) attn_join<KV>(p, scan, cut);
            attn_edges<E>(p, blockIdx.x * (NT / 32) + warp, gridDim.x * (NT / 32));
        } else {
            const int rows = sq.rows, sd = st ^ 1;
            // pairs of rows, rounded up to 2^lg; a tile's positions shared out over 8 >> lg warps, P each
            const int lg = rows <= 2 ? 0 : 32 - __clz((rows - 1) >> 1), part = warp >> lg, r0 = 2 * (warp - (part << lg));
            const int lp = (KV == 64 ? 3 : 2) + lg, P = 1 << lp, LP = max(1, 32 >> lp), pos_l = lane & (P - 1), dq = lane >> lp;
            if (tile == sq.first) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    ref[r] = none;
                    l[r] = 0.f;
                    for (int g = 0; g < NG; ++g) acc[r][g] = Two{0ull, 0ull};
                }
            }
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();
            const long long pos0 = (long long)tile * KV + part * P;
            if (r0 < rows && pos0 < sq.len) {
                const unsigned char* k0 = ks + (sd * KV + part * P + pos_l) * kstride;
                const unsigned char* vt0 = vs + ((size_t)(sd * KV + part * P) * D) * sizeof(E);
                const unsigned char* q0 = qs + (qb * kRows + r0) * D * sizeof(E);
                const unsigned char* q1 = r0 + 1 < rows ? q0 + D * sizeof(E) : q0;
                const bool two = KV == 64 && P == 64;
                uint64_t d[2][2] = {};  // even and odd columns' sums
                auto dot = [&](int j, uint64_t& d0, uint64_t& d1, int c) {
                    const Two a0 = lds4x2<E>(q0 + c * 4 * sizeof(E)), a1 = lds4x2<E>(q1 + c * 4 * sizeof(E));
                    const Two x = lds4x2<E>(k0 + j * 32 * kstride + c * 4 * sizeof(E));
                    d0 = fma2(a0.a, x.a, fma2(a0.b, x.b, d0));
                    d1 = fma2(a1.a, x.a, fma2(a1.b, x.b, d1));
                };
                if (two) {
#pragma unroll 4
                    for (int c = 0; c < D4; ++c) {
                        dot(0, d[0][0], d[1][0], c);
                        dot(1, d[0][1], d[1][1], c);
                    }
                } else {
#pragma unroll 4
                    for (int c = dq; c < D4; c += LP) dot(0, d[0][0], d[1][0], c);
                }
                float s[2][2];
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int j = 0; j < 2; ++j) s[r][j] = lo2(d[r][j]) + hi2(d[r][j]);
                for (int o = P; o < 32; o <<= 1) {
                    s[0][0] += __shfl_xor_sync(0xFFFFFFFFu, s[0][0], o);
                    s[1][0] += __shfl_xor_sync(0xFFFFFFFFu, s[1][0], o);
                }
                const int ctx = (int)min((long long)P, sq.L - pos0);  // of these positions
                const bool tail = ctx < P;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    s[r][0] *= p.c2;
                    s[r][1] *= p.c2;
                    if (tail) {
                        const int node = (sq.row0 + min(r0 + r, rows - 1)) / p.G;
                        const uint8_t* mask = p.mask ? p.mask + ((long long)sq.b * p.N + node) * p.N : nullptr;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int nd = pos_l + 32 * j - ctx;
                            if (nd >= 0 && (nd >= sq.n || (mask ? __ldg(mask + nd) == 0 : nd > node))) s[r][j] = none;
                        }
                    }
                    if (!two) s[r][1] = none;
                    // (a NaN score raises nothing and makes the row NaN)
                    const float top = fmaxf(s[r][0], s[r][1]);
                    if (__any_sync(0xFFFFFFFFu, top > ref[r] + 8.f)) {
                        const float to = fmaxf(ref[r], warp_max(top)), f = ex2(ref[r] - to);
                        ref[r] = to;
                        l[r] *= f;
#pragma unroll
                        for (int g = 0; g < NG; ++g) acc[r][g] = mul2(f, acc[r][g]);
                    }
                    const float base = ref[r] == none ? 0.f : ref[r];
                    const float w0 = ex2(s[r][0] - base), w1 = ex2(s[r][1] - base);
                    ws[r * KV + pos_l] = w0;  // (lanes of one position write the same)
                    if (two) ws[r * KV + pos_l + 32] = w1;
                    l[r] += w0 + w1;
                }
                __syncwarp();
                if (!tail) {
#pragma unroll 2
                    for (int t2 = 4 * pg; t2 < P; t2 += 4 * PG) {
                        const float4 w0 = *reinterpret_cast<const float4*>(ws + t2);
                        const float4 w1 = *reinterpret_cast<const float4*>(ws + KV + t2);
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const unsigned char* v = vt0 + (t2 * D + col[g]) * sizeof(E);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const Two x = lds4x2<E>(v + e * D * sizeof(E));
                                const float a = e == 0 ? w0.x : e == 1 ? w0.y : e == 2 ? w0.z : w0.w;
                                const float b = e == 0 ? w1.x : e == 1 ? w1.y : e == 2 ? w1.z : w1.w;
                                acc[0][g] = axpy2(pack2(a, a), x, acc[0][g]);
                                acc[1][g] = axpy2(pack2(b, b), x, acc[1][g]);
                            }
                        }
                    }
                } else {
                    // an unseen node's values may be anything: a zero weight leaves them out
                    const Two zero = {0ull, 0ull};
#pragma unroll 2
                    for (int t2 = pg; t2 < P; t2 += PG) {
                        const float w0 = ws[t2], w1 = ws[KV + t2];
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const Two x = lds4x2<E>(vt0 + (t2 * D + col[g]) * sizeof(E));
                            acc[0][g] = axpy2(pack2(w0, w0), w0 != 0.f ? x : zero, acc[0][g]);
                            acc[1][g] = axpy2(pack2(w1, w1), w1 != 0.f ? x : zero, acc[1][g]);
                        }
                    }
                }
                __syncwarp();
            }
            __syncthreads();
            if (tile + 1 == sq.last) {
                if (r0 < rows) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int at = (part << (lg + 1)) + r0 + r;
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            float4 a = make_float4(lo2(acc[r][g].a), hi2(acc[r][g].a), lo2(acc[r][g].b), hi2(acc[r][g].b));
#pragma unroll 1
                            for (int o = W; o < 32; o <<= 1) {
                                a.x += __shfl_xor_sync(0xFFFFFFFFu, a.x, o);
                                a.y += __shfl_xor_sync(0xFFFFFFFFu, a.y, o);
                                a.z += __shfl_xor_sync(0xFFFFFFFFu, a.z, o);
                                a.w += __shfl_xor_sync(0xFFFFFFFFu, a.w, o);
                            }
                            if (pg == 0 && vc + 32 * g < D4) *reinterpret_cast<float4*>(os + at * D + (vc + 32 * g) * 4) = a;
                        }
                        const float sum = warp_sum(lane < P ? l[r] : 0.f);
                        if (lane == 0) sums[at] = make_float2(ref[r], sum);
                    }
                }
                bad = __syncthreads_or(bad);
#pragma unroll 1
                for (int i = tid; i < rows * D4; i += NT) {
                    const int r = i / D4, c = i - r * D4;
                    float mr = none, lr = 0.f;
#pragma unroll 1
                    for (int at = r; at < kRows; at += 2 << lg) mr = fmaxf(mr, sums[at].x);
                    const float ref = mr == none ? 0.f : mr;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                    for (int at = r; at < kRows; at += 2 << lg) {
                        const float f = ex2(sums[at].x - ref);
                        lr += sums[at].y * f;
                        o = fma4(f, *reinterpret_cast<const float4*>(os + at * D + c * 4), o);
                    }
                    if (bad) lr = __uint_as_float(0x7FC00000u);
                    const int node = (sq.row0 + r) / p.G, head = sq.h * p.G + (sq.row0 + r) - node * p.G;
                    const long long row = ((long long)sq.b * p.N + node) * (p.Hkv * p.G) + head;
                    if (sq.whole) {
                        const float inv = lr == 0.f ? 0.f : 1.f / lr;
                        if (SV_IN(row, (long long)p.B * p.N * p.Hkv * p.G))
                            store4<E>(reinterpret_cast<E*>(p.out) + row * D + c * 4,
                                      make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
                        if (c == 0 && p.lse) p.lse[row] = lse_of(mr, lr);
                    } else {
                        const long long at = (long long)sq.slot * kRows + r;
                        *reinterpret_cast<float4*>(p.part_o + at * D + c * 4) = o;
                        if (c == 0) p.part_ml[at] = make_float2(mr, lr);
                    }
                }
            }
        }
        if (fresh) {
            sq = next;
            tile = next.first;
            qb ^= 1;
        } else {
            ++tile;
        }
        ++ahead;
        have = true;
    }
}

// ---- many rows ---------------------------------------------------------------------
//
// Units of more rows: 64 a CTA, in register tiles. Thread (ty, tx) of 16 x 16 has
// rows 4 ty .. 4 ty + 3: first their scores at positions tx + 16 j of a tile (four
// rows by four positions, so that eight loads of four columns serve 64 products),
// then their outputs' columns 4 (tx + 16 g). The rows of a thread are the same
// both times, and the weights pass between the 16 threads of a row through shared
// memory of their warp's own: warps meet at a tile's arrival and release
// alone. Bound by latency at two warps a scheduler (the products' pipe is 49 % busy,
// shared memory 54 %): 16 trees of 60 nodes, 8 heads of 4 query
// heads of 128 columns, contexts to 1000, float32: 403 us, 29 TFLOP/s (821 us with
// 16 rows a CTA); 16 nodes, 8 x 8 heads, 20000 positions: 301 us, 35 TFLOP/s (687).
constexpr int kMany = 64;

template <typename E, int KV>
size_t many_smem(int D) {
    return (size_t)2 * KV * (row_bytes<E>(D) + D * sizeof(E)) + (size_t)kMany * row_bytes<E>(D) +
           (size_t)KV * (kMany + 4) * 4;
}

template <typename E, int KV, int NG>
__global__ void __launch_bounds__(NT, NG == 1 ? 2 : 1) attn_many_kernel(const __grid_constant__ AttnParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ AttnScan scan;
    constexpr int J = KV / 16, PS = kMany + 4;
    const int tid = threadIdx.x, warp = tid >> 5, tx = tid & 15, ty = tid >> 4;
    const int D = p.D, D4 = D / 4, stride = row_bytes<E>(D);
    unsigned char* ks = smem;
    unsigned char* vs = ks + 2 * KV * stride;
    unsigned char* qs = vs + (size_t)2 * KV * D * sizeof(E);
    float* ws = reinterpret_cast<float*>(qs + kMany * stride) + 4 * ty;  // weights [KV][PS], this thread's rows
    const float none = __uint_as_float(0xFF800000u);
    int col[NG];  // (threads without a column go along with the last)
#pragma unroll
    for (int g = 0; g < NG; ++g) col[g] = 4 * min(tx + 16 * g, D4 - 1);
    const int lv = 32 - __clz(D * (int)sizeof(E) / 16 - 1);

    asm volatile("griddepcontrol.launch_dependents;");
    const AttnCut cut = attn_locate<KV, NT>(p, &scan);
    AttnWalk<KV> walk(scan, cut);

    AttnStay sq = {}, next = {};  // that of the tile worked on, of the tile copied
    int tile = 0, ahead = 0;      // of sq, of next
    bool bad, next_bad = false, have = false, more = true;
    float ref[4], l[4];  // (as above: weights against a maximum with slack, a thread's own sums)
    Two acc[4][NG];
#pragma unroll 1
    for (int st = 0; more; st ^= 1) {
        const bool fresh = ahead >= next.last;
        bad = next_bad;
        if (fresh) {
            more = walk.next(p, &next);
            ahead = next.first;
            next_bad = false;
        }
        if (more) {
            next_bad |= load_tile<E, KV>(p, next, ahead, smem_u32(ks) + st * KV * stride,
                                         smem_u32(vs) + st * KV * D * (int)sizeof(E), lv);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (!have) {  // while the first tile is on its way
            if (tid == 0) attn_join<KV>(p, scan, cut);
            attn_edges<E>(p, blockIdx.x * (NT / 32) + warp, gridDim.x * (NT / 32));
        } else {
            if (tile == sq.first) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    ref[r] = none;
                    l[r] = 0.f;
#pragma unroll
                    for (int g = 0; g < NG; ++g) acc[r][g] = Two{0ull, 0ull};
                }
            }
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();
            if (warp * 8 < sq.rows) {
                const long long pos0 = (long long)tile * KV;
                const unsigned char* q0 = qs + 4 * ty * stride;
                const unsigned char* k0 = ks + ((st ^ 1) * KV + tx) * stride;
                const unsigned char* v0 = vs + (size_t)(st ^ 1) * KV * D * sizeof(E);
                float s[4][J];
                {
                    uint64_t d[4][J] = {};  // even and odd columns' sums
#pragma unroll 2
                    for (int c = 0; c < D4; ++c) {
                        Two a[4], x[J];
#pragma unroll
                        for (int r = 0; r < 4; ++r) a[r] = lds4x2<E>(q0 + r * stride + c * 4 * sizeof(E));
#pragma unroll
                        for (int j = 0; j < J; ++j) x[j] = lds4x2<E>(k0 + 16 * j * stride + c * 4 * sizeof(E));
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int j = 0; j < J; ++j) d[r][j] = fma2(a[r].a, x[j].a, fma2(a[r].b, x[j].b, d[r][j]));
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int j = 0; j < J; ++j) s[r][j] = (lo2(d[r][j]) + hi2(d[r][j])) * p.c2;
                }
                const bool tail = pos0 + KV > sq.L;
                if (tail) {
                    const int ctx = (int)max(-(1LL << 30), sq.L - pos0);  // context among these positions
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int node = (sq.row0 + min(4 * ty + r, sq.rows - 1)) / p.G;
                        const uint8_t* mask = p.mask ? p.mask + ((long long)sq.b * p.N + node) * p.N : nullptr;
#pragma unroll
                        for (int j = 0; j < J; ++j) {
                            const int nd = tx + 16 * j - ctx;
                            if (nd >= 0 && (nd >= sq.n || (mask ? __ldg(mask + nd) == 0 : nd > node))) s[r][j] = none;
                        }
                    }
                }
                float top[4];
                bool raise = false;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    top[r] = s[r][0];
#pragma unroll
                    for (int j = 1; j < J; ++j) top[r] = fmaxf(top[r], s[r][j]);
                    // (an absent row's queries are whatever lay there: it takes no part in the vote)
                    raise |= 4 * ty + r < sq.rows && top[r] > ref[r] + 8.f;
                }
                if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float to = top[r];
#pragma unroll
                        for (int o = 8; o > 0; o >>= 1) to = fmaxf(to, __shfl_xor_sync(0xFFFFFFFFu, to, o));
                        to = fmaxf(to, ref[r]);
                        const float f = to == none ? 1.f : ex2(ref[r] - to);
                        ref[r] = to;
                        l[r] *= f;
#pragma unroll
                        for (int g = 0; g < NG; ++g) acc[r][g] = mul2(f, acc[r][g]);
                    }
                }
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    float w[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        w[r] = ex2(s[r][j] - (ref[r] == none ? 0.f : ref[r]));
                        l[r] += w[r];
                    }
                    *reinterpret_cast<float4*>(ws + (tx + 16 * j) * PS) = make_float4(w[0], w[1], w[2], w[3]);
                }
                __syncwarp();
                if (!tail) {
#pragma unroll 4
                    for (int t = 0; t < KV; ++t) {
                        const float4 w = *reinterpret_cast<const float4*>(ws + t * PS);
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const Two x = lds4x2<E>(v0 + (t * D + col[g]) * sizeof(E));
                            acc[0][g] = axpy2(pack2(w.x, w.x), x, acc[0][g]);
                            acc[1][g] = axpy2(pack2(w.y, w.y), x, acc[1][g]);
                            acc[2][g] = axpy2(pack2(w.z, w.z), x, acc[2][g]);
                            acc[3][g] = axpy2(pack2(w.w, w.w), x, acc[3][g]);
                        }
                    }
                } else {
                    // an unseen node's values may be anything: a zero weight leaves them out
                    const Two zero = {0ull, 0ull};
#pragma unroll 1
                    for (int t = 0; t < KV; ++t) {
                        const float4 w = *reinterpret_cast<const float4*>(ws + t * PS);
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const Two x = lds4x2<E>(v0 + (t * D + col[g]) * sizeof(E));
                            acc[0][g] = axpy2(pack2(w.x, w.x), w.x != 0.f ? x : zero, acc[0][g]);
                            acc[1][g] = axpy2(pack2(w.y, w.y), w.y != 0.f ? x : zero, acc[1][g]);
                            acc[2][g] = axpy2(pack2(w.z, w.z), w.z != 0.f ? x : zero, acc[2][g]);
                            acc[3][g] = axpy2(pack2(w.w, w.w), w.w != 0.f ? x : zero, acc[3][g]);
                        }
                    }
                }
                __syncwarp();
            }
            if (tile + 1 < sq.last) {
                __syncthreads();
            } else {
                bad = __syncthreads_or(bad);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int rr = 4 * ty + r;
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], o);
                    if (rr >= sq.rows) continue;
                    if (bad) l[r] = __uint_as_float(0x7FC00000u);
                    const int node = (sq.row0 + rr) / p.G, head = sq.h * p.G + (sq.row0 + rr) - node * p.G;
                    const long long row = ((long long)sq.b * p.N + node) * (p.Hkv * p.G) + head;
                    const long long part = (long long)sq.slot * kMany + rr;
                    const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        if (tx + 16 * g >= D4) continue;
                        if (sq.whole) {
                            const Two o = mul2(inv, acc[r][g]);
                            if (SV_IN(row, (long long)p.B * p.N * p.Hkv * p.G))
                                store4<E>(reinterpret_cast<E*>(p.out) + row * D + col[g],
                                          make_float4(lo2(o.a), hi2(o.a), lo2(o.b), hi2(o.b)));
                        } else {
                            const Two o = acc[r][g];
                            *reinterpret_cast<float4*>(p.part_o + part * D + col[g]) =
                                make_float4(lo2(o.a), hi2(o.a), lo2(o.b), hi2(o.b));
                        }
                    }
                    if (tx == 0) {
                        if (!sq.whole) p.part_ml[part] = make_float2(ref[r], l[r]);
                        else if (p.lse) p.lse[row] = lse_of(ref[r], l[r]);
                    }
                }
            }
        }
        if (fresh) {
            sq = next;
            tile = next.first;
            // (the last stay's queries are done with)
            if (more) {
                const int vec = D * (int)sizeof(E) / 16;
                const E* q = static_cast<const E*>(p.q);
#pragma unroll 1
                for (int i = tid; i < sq.rows * vec; i += NT) {
                    const int r = i / vec, c = i - r * vec, node = (sq.row0 + r) / p.G, g = (sq.row0 + r) - node * p.G;
                    const long long row = ((long long)sq.b * p.N + node) * (p.Hkv * p.G) + sq.h * p.G + g;
                    cp16(smem_u32(qs) + r * stride + c * 16, q + row * D + c * (16 / (int)sizeof(E)), 16);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
        } else {
            ++tile;
        }
        ++ahead;
        have = true;
    }
}

// Joins the pieces of the units that several parts share: block (c, y) takes
// JR rows of joins[c]. A row's weights 2^(m_i - max m) / sum of its pieces are
// formed by 256 / JR lanes; a thread adds up four columns of JR / 8 rows (128
// columns), eight loads in flight, the first of them while the weights are
// formed. The sums' order is that of the parts. With few rows (JR = 8) it is
// bound by the latency of dependent loads (the pieces come from L2), and a
// thread's eight loads are a row's pieces; with many (JR = 32) by instructions,
// and they are two pieces of four rows, so that a block's start is shared by
// more. Calls with JR = 8 and 32: 16 trees of 512 rows 117.7 and 109.3 us; 16 of
// 64 rows and 32 heads 80.0 and 78.5; 30 of 150 rows 35.1 and 33.0; one of 4000
// rows 182 and 173; one chain of 20 rows 13.2 and 15.2; five of 28 rows 19.3 and
// 21.1; one tree of 244 rows in 19 pieces 124 and 131 (8 units: 64 blocks).
constexpr int kJoinNT = 256;
constexpr int kJoinFew = 152 * 4;  // blocks of 8 rows that an SM runs side by side

template <typename E, int JR>
__global__ void __launch_bounds__(kJoinNT) attn_join_kernel(const __grid_constant__ AttnParams p) {
    constexpr int LANES = kJoinNT / JR, RT = JR / 8, PT = 8 / RT, MOST = 32;  // MOST: weights of a row that are kept
    __shared__ float weight[JR][MOST];
    __shared__ float top[JR];
    __shared__ long long out_row[JR];
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4* src = reinterpret_cast<const int4*>(p.joins + blockIdx.x + 1);
    const int4 u = __ldcg(src), v = __ldcg(src + 1);  // b, h, row0, rows; slot0, first, last, lost
    // parts that gave up (the first one's entry, which joins nothing, by the first block)
    const uint32_t lost0 = blockIdx.x == 0 ? __ldcg(&p.joins->lost) : 0u;
    if ((lost0 | (uint32_t)v.w) && tid == 0 && blockIdx.y == 0 && p.status) {
        if (lost0) attn_lost(p, (int)(lost0 & 0xFFFF) - 1, (int)(lost0 >> 16));
        if (v.w) attn_lost(p, (v.w & 0xFFFF) - 1, (int)((uint32_t)v.w >> 16));
    }
    const int r0 = blockIdx.y * JR, rows = min(JR, u.w - r0);
    if (rows <= 0) return;
    const int pieces = v.z - v.y + 2, D4 = p.D / 4, lw = D4 <= 1 ? 0 : 32 - __clz(D4 - 1);
    const int step = kJoinNT >> lw, d = (tid & ((1 << lw) - 1)) * 4;  // rows at a time, this thread's columns
    auto at = [&](int i, int r) { return (long long)(i == 0 ? v.x : 2 * (v.y + i - 1)) * p.tile_rows + r0 + r; };
    float4 x[RT][PT];
    auto load = [&](int ra, int i0) {
#pragma unroll
        for (int k = 0; k < RT; ++k)
#pragma unroll
            for (int e = 0; e < PT; ++e)
                x[k][e] = ra + k * step < rows && i0 + e < pieces
                              ? __ldcg(reinterpret_cast<const float4*>(p.part_o + at(i0 + e, ra + k * step) * p.D + d))
                              : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    const int ra0 = d < p.D ? tid >> lw : rows;
    load(ra0, 0);
    {
        const int r = tid / LANES, lane = tid % LANES;
        const float2 none = make_float2(__uint_as_float(0xFF800000u), 0.f);
        float m = none.x, l = 0.f;
        float2 ml = none;
#pragma unroll 1
        for (int i = lane; r < rows && i < pieces; i += LANES) {
            ml = __ldcg(p.part_ml + at(i, r));
            m = fmaxf(m, ml.x);
        }
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float ref = m == none.x ? 0.f : m;
#pragma unroll 1
        for (int i = lane; r < rows && i < pieces; i += LANES) {
            if (pieces > LANES) ml = __ldcg(p.part_ml + at(i, r));
            const float w = ex2(ml.x - ref);
            if (i < MOST) weight[r][i] = w;
            l += w * ml.y;
        }
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        if (lane == 0 && r < rows) {
            const int rr = u.z + r0 + r, node = rr / p.G;
            const long long row = ((long long)u.x * p.N + node) * (p.Hkv * p.G) + u.y * p.G + (rr - node * p.G);
            out_row[r] = row;
            top[r] = ref;
            if (p.lse) p.lse[row] = lse_of(m, l);
        }
        __syncwarp();
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int i = lane; r < rows && i < min(pieces, MOST); i += LANES) weight[r][i] *= inv;
        if (pieces > MOST && r < rows) {  // kept for the pieces past MOST: the sum's inverse
            __syncwarp();
            if (lane == 0) weight[r][0] = inv;
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int ra = ra0; ra < rows; ra += RT * step) {
        float4 acc[RT];
#pragma unroll
        for (int k = 0; k < RT; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i0 = 0; i0 < pieces; i0 += PT) {
            if (i0 || ra != ra0) load(ra, i0);
#pragma unroll
            for (int k = 0; k < RT; ++k) {
                const int r = ra + k * step;
                if (r >= rows) break;
#pragma unroll
                for (int e = 0; e < PT; ++e)
                    if (i0 + e < pieces) {
                        const float w = pieces <= MOST ? weight[r][i0 + e]
                                                       : weight[r][0] * ex2(__ldcg(p.part_ml + at(i0 + e, r)).x - top[r]);
                        acc[k] = fma4(w, x[k][e], acc[k]);
                    }
            }
        }
#pragma unroll
        for (int k = 0; k < RT; ++k) {
            const int r = ra + k * step;
            if (r >= rows) break;
            if (SV_IN(out_row[r], (long long)p.B * p.N * p.Hkv * p.G))
                store4<E>(reinterpret_cast<E*>(p.out) + out_row[r] * p.D + d, acc[k]);
        }
    }
}

template <typename E>
cudaError_t launch_join(const AttnParams& p, const AttnPlan& plan, cudaStream_t st) {
    if (plan.whole) return cudaSuccess;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    const int rows = std::min(plan.rows, p.N * p.G);
    // (a join a unit at the most)
    const long long units = (long long)p.B * p.Hkv * ((p.N * p.G + plan.rows - 1) / plan.rows);
    const bool many = std::min<long long>(units, plan.grid - 1) * ((rows + 7) / 8) > kJoinFew;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.grid - 1, many ? (rows + 31) / 32 : (rows + 7) / 8);
    cfg.blockDim = dim3(kJoinNT);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return many ? cudaLaunchKernelEx(&cfg, attn_join_kernel<E, 32>, p) : cudaLaunchKernelEx(&cfg, attn_join_kernel<E, 8>, p);
}

template <typename E, int KV>
cudaError_t launch_simt(const AttnParams& p, const AttnPlan& plan, cudaStream_t st) {
    constexpr int widest = KV == 64 ? 256 / (int)sizeof(E) : SPEC_MAX_HEAD_DIM;  // (attention_simt_kv)
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(attn_simt_kernel<E, KV>), simt_smem<E, KV>(widest));
    if (e != cudaSuccess) return e;
    attn_simt_kernel<E, KV><<<plan.grid, NT, simt_smem<E, KV>(p.D), st>>>(p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join<E>(p, plan, st);
}

}  // namespace

cudaError_t allow_smem(const void* kernel, size_t most) {
    static OncePerDevice once;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return (cudaError_t)once.run(kernel, dev, [&] {
        return (int)cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    });
}

cudaError_t launch_attention_join(const AttnParams& p, int dtype, const AttnPlan& plan, cudaStream_t st) {
    return dtype == 0 ? launch_join<float>(p, plan, st) : launch_join<bf16_t>(p, plan, st);
}

int attention_simt_rows(bool many) { return many ? kMany : kRows; }
// Which of the two kernels. float32, 8 sequences, 8 heads, contexts to 1000, of
// 16 and of 64 rows a CTA: 128 columns, 17 rows 58.8 and 47.9 us, 48 rows 90.0
// and 66.7; 64 columns, 24 rows 28.8 and 31.9, 48 rows 42.2 and 46.9, and 4
// sequences of 300 rows, contexts to 2000, 240 and 178.
bool attention_simt_many(int rows, int D) { return rows >= (D > 64 ? kRows + 1 : kMany); }

int attention_simt_extra() { return kExtra; }
int attention_simt_whole() { return kWhole; }

int attention_simt_kv(int dtype, int D, bool many) { return D * (dtype == 0 ? 4 : 2) > (many ? 512 : 256) ? 32 : 64; }

template <typename E, int KV, int NG>
cudaError_t launch_many(const AttnParams& p, const AttnPlan& plan, cudaStream_t st) {
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(attn_many_kernel<E, KV, NG>), many_smem<E, KV>(64 * NG));
    if (e != cudaSuccess) return e;
    attn_many_kernel<E, KV, NG><<<plan.grid, NT, many_smem<E, KV>(p.D), st>>>(p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join<E>(p, plan, st);
}

template <typename E>
cudaError_t launch_cores(const AttnParams& p, const AttnPlan& plan, cudaStream_t st) {
    if (plan.rows == kRows) return plan.kv == 64 ? launch_simt<E, 64>(p, plan, st) : launch_simt<E, 32>(p, plan, st);
    if (p.D <= 64) return launch_many<E, 64, 1>(p, plan, st);
    if (p.D <= 128) return launch_many<E, 64, 2>(p, plan, st);
    return launch_many<E, sizeof(E) == 4 ? 32 : 64, 4>(p, plan, st);
}

cudaError_t launch_attention_simt(const AttnParams& p, int dtype, const AttnPlan& plan, cudaStream_t st) {
    return dtype == 0 ? launch_cores<float>(p, plan, st) : launch_cores<bf16_t>(p, plan, st);
}

// CTAs of an SM: what its shared memory and its registers hold.
int attention_simt_ctas(int dtype, int D, bool many) {
    const bool wide = attention_simt_kv(dtype, D, many) == 64;
    size_t smem;
    if (many) smem = dtype != 0 ? many_smem<bf16_t, 64>(D) : wide ? many_smem<float, 64>(D) : many_smem<float, 32>(D);
    else if (dtype != 0) smem = wide ? simt_smem<bf16_t, 64>(D) : simt_smem<bf16_t, 32>(D);
    else smem = wide ? simt_smem<float, 64>(D) : simt_smem<float, 32>(D);
    return (int)std::max<size_t>(1, std::min<size_t>(many && D > 64 ? 1 : 2, (size_t)227 * 1024 / (smem + 2048)));
}

SV_DEBUG_READER(attention)

}  // namespace sv
