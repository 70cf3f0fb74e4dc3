// Tree attention over a paged cache on the CUDA cores, and the kernel that
// joins partial results (attention.cuh: the mathematics and the division of
// the work). Takes every type and head size; float32 caches and head sizes
// that the tensor-core kernel lacks come here.
//
// One CTA of eight warps takes 16 rows of a unit, two a warp. Tiles of 64
// positions (32 where a float32 head is wider than 128) of K and V are staged
// by 16-byte asynchronous copies, two tiles deep. A lane scores two positions
// (one) for both rows of its warp; the running
// maximum and sum are the warp's (shuffles), the weights go through a
// warp-private strip of shared memory, and a lane accumulates four (eight:
// D > 128) output columns in registers. Warps meet only at the tile's arrival
// and release. fp32 throughout.

#include <algorithm>
#include <atomic>
#include <mutex>

#include "attention.cuh"

namespace sv {
namespace {

constexpr int NT = 256;
constexpr int kRows = 16;
constexpr int kExtra = 1;  // tiles that a unit's start and end count for

template <typename E>
constexpr int row_bytes(int D) {  // a K row in shared memory: 16 bytes of padding against bank conflicts
    return D * (int)sizeof(E) + 16;
}

template <typename E, int KV>
size_t simt_smem(int D) {
    return (size_t)2 * KV * (row_bytes<E>(D) + D * sizeof(E)) + (size_t)kRows * D * 4 + (size_t)kRows * KV * 4;
}

SV_DEV void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
SV_DEV uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

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

SV_DEV float4 fma4(float a, float4 v, float4 c) {
    return make_float4(fmaf(a, v.x, c.x), fmaf(a, v.y, c.y), fmaf(a, v.z, c.z), fmaf(a, v.w, c.w));
}

// One tile's K and V rows into a stage. Rows past the sequence's end and rows
// of a page that does not exist are zero. Returns whether a page id was bad.
template <typename E, int KV>
SV_DEV bool load_tile(const AttnParams& p, int b, int h, long long pos0, long long end, unsigned char* ks,
                      unsigned char* vs) {
    const int vec = p.D * (int)sizeof(E) / 16;
    const E* kc = reinterpret_cast<const E*>(p.k) + h * p.head_stride;
    const E* vc = reinterpret_cast<const E*>(p.v) + h * p.head_stride;
    const int ps1 = (1 << p.page_shift) - 1;
    const int32_t* table = p.table + b * p.table_stride;
    bool bad = false;
    for (int i = threadIdx.x; i < KV * vec; i += NT) {
        const int t = i / vec, c = i - t * vec;
        const long long pos = pos0 + t;
        unsigned char* kd = ks + t * row_bytes<E>(p.D) + c * 16;
        unsigned char* vd = vs + (t * vec + c) * 16;
        int id = -1;
        if (pos < end) {
            id = __ldg(table + (pos >> p.page_shift));
            if (id < 0 || id >= p.num_pages) {
                bad = true;
                id = -1;
            }
        }
        if (id >= 0) {
            const long long at = id * p.page_stride + (pos & ps1) * p.token_stride + c * (16 / (int)sizeof(E));
            cp16(smem_addr(kd), kc + at);
            cp16(smem_addr(vd), vc + at);
        } else {
            *reinterpret_cast<uint4*>(kd) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(vd) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return bad;
}

template <typename E, int KV>
__global__ void __launch_bounds__(NT) attn_simt_kernel(const __grid_constant__ AttnParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ AttnScan scan;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int J = KV / 32;
    const int D = p.D, D4 = D / 4, kstride = row_bytes<E>(D);
    unsigned char* ks = smem;
    unsigned char* vs = ks + 2 * KV * kstride;
    float* qs = reinterpret_cast<float*>(vs + (size_t)2 * KV * D * sizeof(E));
    float* ws = qs + kRows * D + warp * 2 * KV;  // the warp's weights [2][KV]

    attn_edges<E>(p, blockIdx.x * (NT / 32) + warp, gridDim.x * (NT / 32));
    asm volatile("griddepcontrol.launch_dependents;");
    const AttnCut cut = attn_locate<KV, kExtra, NT>(p, &scan);
    if (tid == 0) attn_join<KV, kExtra>(p, scan, cut);
    AttnWalk<KV, kExtra> walk(scan, cut);
    AttnStay sq;
    while (walk.next(p, &sq)) {
        const int b = sq.b, h = sq.h, first = sq.first, last = sq.last, row_base = sq.row0, rows = sq.rows;
        const long long len = (long long)sq.L + sq.n;

        // queries, in octaves of the score
        const E* q = reinterpret_cast<const E*>(p.q);
        for (int i = tid; i < rows * D4; i += NT) {
            const int r = i / D4, c = i - r * D4, node = (row_base + r) / p.G, g = (row_base + r) % p.G;
            const E* src = q + (((long long)b * p.N + node) * (p.Hkv * p.G) + h * p.G + g) * D + c * 4;
            float4 x = lds4<E>(reinterpret_cast<const unsigned char*>(src));
            *reinterpret_cast<float4*>(qs + r * D + c * 4) =
                make_float4(x.x * p.c2, x.y * p.c2, x.z * p.c2, x.w * p.c2);
        }
        bool bad = load_tile<E, KV>(p, b, h, (long long)first * KV, len, ks, vs);

        const int r0 = warp * 2;
        float m[2], l[2];
        float4 acc[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            m[r] = __uint_as_float(0xFF800000u);
            l[r] = 0.f;
            acc[r][0] = acc[r][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int tile = first; tile < last; ++tile) {
            const int st = (tile - first) & 1;
            if (tile + 1 < last) {
                bad |= load_tile<E, KV>(p, b, h, (long long)(tile + 1) * KV, len, ks + (st ^ 1) * KV * kstride,
                                    vs + (size_t)(st ^ 1) * KV * D * sizeof(E));
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncthreads();
            if (r0 < rows) {
                const unsigned char* kt0 = ks + st * KV * kstride;
                const unsigned char* vt0 = vs + (size_t)st * KV * D * sizeof(E);
                float s[2][J] = {};
                const float* q0 = qs + r0 * D;
                const float* q1 = r0 + 1 < rows ? q0 + D : q0;
                for (int c = 0; c < D4; ++c) {
                    const float4 a0 = *reinterpret_cast<const float4*>(q0 + c * 4);
                    const float4 a1 = *reinterpret_cast<const float4*>(q1 + c * 4);
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const float4 x = lds4<E>(kt0 + (lane + 32 * j) * kstride + c * 4 * sizeof(E));
                        s[0][j] = fmaf(a0.x, x.x, fmaf(a0.y, x.y, fmaf(a0.z, x.z, fmaf(a0.w, x.w, s[0][j]))));
                        s[1][j] = fmaf(a1.x, x.x, fmaf(a1.y, x.y, fmaf(a1.z, x.z, fmaf(a1.w, x.w, s[1][j]))));
                    }
                }
                const long long pos0 = (long long)tile * KV;
                const bool tail = pos0 + KV > sq.L;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int node = (row_base + min(r0 + r, rows - 1)) / p.G;
                    if (tail) {
#pragma unroll
                        for (int j = 0; j < J; ++j) {
                            const long long nd = pos0 + lane + 32 * j - sq.L;
                            const bool see = nd < 0 || (nd < sq.n && (p.mask ? __ldg(p.mask + ((long long)b * p.N + node) * p.N + nd) != 0
                                                                             : nd <= node));
                            if (!see) s[r][j] = __uint_as_float(0xFF800000u);
                        }
                    }
                    // a NaN score makes the row NaN (fmaxf drops it, the exponential keeps it)
                    const float mn = fmaxf(m[r], warp_max(J == 2 ? fmaxf(s[r][0], s[r][J - 1]) : s[r][0]));
                    const float ref = mn == __uint_as_float(0xFF800000u) ? 0.f : mn;
                    const float f = ex2(m[r] - ref);
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const float w = ex2(s[r][j] - ref);
                        ws[r * KV + 32 * j + lane] = w;
                        sum += w;
                    }
                    l[r] = l[r] * f + warp_sum(sum);
                    m[r] = mn;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        acc[r][g].x *= f;
                        acc[r][g].y *= f;
                        acc[r][g].z *= f;
                        acc[r][g].w *= f;
                    }
                }
                __syncwarp();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int c = lane + 32 * g;
                    if (c < D4) {
                        if (!tail) {
#pragma unroll 8
                            for (int t2 = 0; t2 < KV; ++t2) {
                                const float4 x = lds4<E>(vt0 + ((size_t)t2 * D + c * 4) * sizeof(E));
                                acc[0][g] = fma4(ws[t2], x, acc[0][g]);
                                acc[1][g] = fma4(ws[KV + t2], x, acc[1][g]);
                            }
                        } else {
                            // an unseen node's values may be anything: a zero weight leaves them out
                            for (int t2 = 0; t2 < KV; ++t2) {
                                const float4 x = lds4<E>(vt0 + ((size_t)t2 * D + c * 4) * sizeof(E));
                                const float w0 = ws[t2], w1 = ws[KV + t2];
                                if (w0 != 0.f) acc[0][g] = fma4(w0, x, acc[0][g]);
                                if (w1 != 0.f) acc[1][g] = fma4(w1, x, acc[1][g]);
                            }
                        }
                    }
                }
                __syncwarp();
            }
            __syncthreads();
        }
        bad = __syncthreads_or(bad);
        const bool whole = sq.whole;
        const int slot = sq.slot;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (r0 + r >= rows) break;
            if (bad) l[r] = __uint_as_float(0x7FC00000u);
            const int node = (row_base + r0 + r) / p.G, head = h * p.G + (row_base + r0 + r) % p.G;
            const long long row = ((long long)b * p.N + node) * (p.Hkv * p.G) + head;
            const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int c = lane + 32 * g;
                if (c >= D4) break;
                if (whole) {
                    const float4 o = make_float4(acc[r][g].x * inv, acc[r][g].y * inv, acc[r][g].z * inv,
                                                 acc[r][g].w * inv);
                    if (SV_IN(row, (long long)p.B * p.N * p.Hkv * p.G))
                        store4<E>(reinterpret_cast<E*>(p.out) + row * D + c * 4, o);
                } else {
                    *reinterpret_cast<float4*>(p.part_o + ((long long)slot * kRows + r0 + r) * D + c * 4) = acc[r][g];
                }
            }
            if (lane == 0) {
                if (!whole)
                    p.part_ml[(long long)slot * kRows + r0 + r] = make_float2(m[r], l[r]);
                else if (p.lse)
                    p.lse[row] = lse_of(m[r], l[r]);
            }
        }
    }
}

// Joins the pieces of the units that several parts share: block (c, y) takes
// kJoinRows rows of joins[c]. A warp forms the weights 2^(m_i - max m) / sum of
// a row's pieces, a lane a piece; every thread adds up four columns of a row,
// eight pieces in flight (the first eight while the weights are formed). The
// sums' order is that of the parts. Bound by the latency of dependent loads;
// the pieces come from L2.
constexpr int kJoinRows = 8, kJoinNT = 256;

template <typename E>
__global__ void __launch_bounds__(kJoinNT) attn_join_kernel(const __grid_constant__ AttnParams p) {
    __shared__ float weight[kJoinRows][32];
    __shared__ float top[kJoinRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4* src = reinterpret_cast<const int4*>(p.joins + blockIdx.x + 1);
    const int4 u = __ldcg(src), v = __ldcg(src + 1);  // b, h, row0, rows; slot0, first, last
    const int r0 = blockIdx.y * kJoinRows, rows = min(kJoinRows, u.w - r0);
    if (rows <= 0) return;
    const int pieces = v.z - v.y + 2, D4 = p.D / 4;
    auto at = [&](int i, int r) { return (long long)(i == 0 ? v.x : 2 * (v.y + i - 1)) * p.tile_rows + r0 + r; };
    const float2 none = make_float2(__uint_as_float(0xFF800000u), 0.f);
    float4 x[8];
    auto load = [&](int i0, int r, int d) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = i0 + k < pieces ? __ldcg(reinterpret_cast<const float4*>(p.part_o + at(i0 + k, r) * p.D + d))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    if (tid < rows * D4) load(0, tid / D4, tid % D4 * 4);
    if (warp < rows) {
        const int r = warp;
        float2 ml = none;
        float m = none.x, l = 0.f;
        for (int i = lane; i < pieces; i += 32) {
            ml = __ldcg(p.part_ml + at(i, r));
            m = fmaxf(m, ml.x);
        }
        m = warp_max(m);
        const float ref = m == none.x ? 0.f : m;
        for (int i = lane; i < pieces; i += 32) {
            if (pieces > 32) ml = __ldcg(p.part_ml + at(i, r));
            l += ex2(ml.x - ref) * ml.y;
        }
        l = warp_sum(l);
        if (pieces <= 32) weight[r][lane] = lane < pieces ? ex2(ml.x - ref) * (l == 0.f ? 0.f : 1.f / l) : 0.f;
        if (lane == 0) {
            if (pieces > 32) weight[r][0] = l == 0.f ? 0.f : 1.f / l;
            top[r] = ref;
            if (p.lse) {
                const int rr = u.z + r0 + r, node = rr / p.G;
                p.lse[((long long)u.x * p.N + node) * (p.Hkv * p.G) + u.y * p.G + (rr - node * p.G)] = lse_of(m, l);
            }
        }
    }
    __syncthreads();
    for (int j = tid; j < rows * D4; j += kJoinNT) {
        const int r = j / D4, d = (j - r * D4) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < pieces; i0 += 8) {
            if (i0 || j != tid) load(i0, r, d);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i0 + k < pieces) {
                    const float w = pieces <= 32 ? weight[r][i0 + k]
                                                 : weight[r][0] * ex2(__ldcg(p.part_ml + at(i0 + k, r)).x - top[r]);
                    acc = fma4(w, x[k], acc);
                }
        }
        const int rr = u.z + r0 + r, node = rr / p.G;
        const long long row = ((long long)u.x * p.N + node) * (p.Hkv * p.G) + u.y * p.G + (rr - node * p.G);
        if (SV_IN(row, (long long)p.B * p.N * p.Hkv * p.G)) store4<E>(reinterpret_cast<E*>(p.out) + row * p.D + d, acc);
    }
}

template <typename E>
cudaError_t launch_join(const AttnParams& p, const AttnPlan& plan, cudaStream_t st) {
    if (plan.grid == 1) return cudaSuccess;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.grid - 1, (std::min(plan.rows, p.N * p.G) + kJoinRows - 1) / kJoinRows);
    cfg.blockDim = dim3(kJoinNT);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<E>, p);
}

template <typename E, int KV>
cudaError_t launch_simt(const AttnParams& p, const AttnPlan& plan, cudaStream_t st) {
    const size_t smem = simt_smem<E, KV>(p.D);
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(attn_simt_kernel<E, KV>), smem);
    if (e != cudaSuccess) return e;
    attn_simt_kernel<E, KV><<<plan.grid, NT, smem, st>>>(p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join<E>(p, plan, st);
}

}  // namespace

cudaError_t allow_smem(const void* kernel, size_t bytes) {
    constexpr int kMost = 16;
    struct Entry {
        std::atomic<const void*> kernel{nullptr};
        std::atomic<size_t> bytes{0};
        std::atomic<int> dev{-1};
    };
    static Entry seen[kMost];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    for (Entry& s : seen)
        if (s.kernel.load(std::memory_order_acquire) == kernel && s.dev.load(std::memory_order_relaxed) == dev &&
            s.bytes.load(std::memory_order_relaxed) >= bytes)
            return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    static std::mutex mu;
    std::lock_guard<std::mutex> g(mu);
    for (Entry& s : seen) {
        const void* k = s.kernel.load(std::memory_order_relaxed);
        if (k && (k != kernel || s.dev.load(std::memory_order_relaxed) != dev)) continue;
        s.dev.store(dev, std::memory_order_relaxed);
        s.bytes.store(bytes, std::memory_order_relaxed);
        s.kernel.store(kernel, std::memory_order_release);
        break;
    }
    return cudaSuccess;
}

cudaError_t launch_attention_join(const AttnParams& p, int dtype, const AttnPlan& plan, cudaStream_t st) {
    return dtype == 0 ? launch_join<float>(p, plan, st) : launch_join<bf16_t>(p, plan, st);
}

int attention_simt_rows() { return kRows; }

int attention_simt_kv(int dtype, int D) { return dtype == 0 && D > 128 ? 32 : 64; }

cudaError_t launch_attention_simt(const AttnParams& p, int dtype, const AttnPlan& plan, cudaStream_t st) {
    if (dtype != 0) return launch_simt<bf16_t, 64>(p, plan, st);
    return plan.kv == 64 ? launch_simt<float, 64>(p, plan, st) : launch_simt<float, 32>(p, plan, st);
}

// CTAs of an SM: what its shared memory holds, four at most.
int attention_simt_ctas(int dtype, int D) {
    const size_t smem = dtype != 0 ? simt_smem<bf16_t, 64>(D)
                        : attention_simt_kv(dtype, D) == 64 ? simt_smem<float, 64>(D) : simt_smem<float, 32>(D);
    return (int)std::max<size_t>(1, std::min<size_t>(4, (size_t)227 * 1024 / (smem + 2048)));
}

SV_DEBUG_READER(attention)

}  // namespace sv
