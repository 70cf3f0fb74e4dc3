// Attention weights of accepted rows, added up a position (weigh.cuh), on the
// CUDA cores: float32, and bf16 heads that the tensor-core kernel does not take.
//
// A block holds a tile of 64 keys in shared memory (fp32, whatever the type) and
// brings its rows 32 at a time; a thread has 4 keys and 2 rows of the products.
// The sums over rows stay in registers until the tile's end.
//
// Bound by latency where there are few tiles (keys, rows, products and sums follow
// one another; four blocks an SM overlap them: 8 chains of 8, 12 heads of 64,
// float32, 20-1500 positions 20.8 us, 26.5 with two; one token of 16 sequences, to
// 8000 positions, 8 x 4 heads of 128: 197 us, 1.3 TB/s), else by the products' reads
// of shared memory, 10 wavefronts for 32 multiplications of a warp (trees' paths of 1
// to 17 of 61 nodes, 16 sequences, 300-4000 positions, 8 x 4 heads of 96, bf16: 118).

#include <algorithm>

#include "attention.cuh"
#include "weigh.cuh"
#include "specverify.h"

namespace sv {
namespace {

constexpr int NT = 256;
constexpr int KV = 64;
constexpr int R = 32;

struct alignas(16) Ctl {
    WeighScan scan;
    float lse[R];       // of a block's rows, in octaves; +inf: no weight
    int see[R];         // first position that the row does not see
    int bad;
    float sums[NT / 32][KV];
};

size_t smem_bytes(int D) { return sizeof(Ctl) + (size_t)(KV + R) * (D + 4) * sizeof(float); }

// A word's elements, as 16-byte words of floats.
template <int VN>
SV_DEV void put(float* to, const float (&v)[VN]) {
#pragma unroll
    for (int e = 0; e < VN; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
}

template <typename E>
__global__ void __launch_bounds__(NT, 4) weigh_kernel(const __grid_constant__ WeighParams p) {
    constexpr int VN = VecTraits<E>::kN;
    extern __shared__ __align__(16) unsigned char smem[];
    Ctl* c = reinterpret_cast<Ctl*>(smem);
    float* ks = reinterpret_cast<float*>(smem + sizeof(Ctl));
    const int stride = p.D + 4, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float* qs = ks + KV * stride;
    const int words = p.D / VN, kx = tid & 15, ry = tid >> 4;
    weigh_statuses<false>(p, blockIdx.x * (NT / 32) + warp, gridDim.x * (NT / 32));
    WeighPart part = weigh_locate<KV, R, NT>(p, &c->scan);
    const E* q = reinterpret_cast<const E*>(p.q);
    const E* k = reinterpret_cast<const E*>(p.k);
    WeighStay s;
    int good = -1;  // the sequence whose path is known to be good
    while (weigh_next<KV, R>(p, &part, &s)) {
        const int rows = s.n * p.G, Hq = p.Hkv * p.G;
        const int32_t* path = p.path ? p.path + (long long)s.b * p.W : nullptr;
        if (path && good != s.b) {
            bool bad = false;
            for (int r = tid; r < s.n; r += NT) bad |= path[r] < 0 || path[r] >= p.N;
            if (__syncthreads_or(bad)) continue;
            good = s.b;
        }
        const int32_t* table = p.table + s.b * p.table_stride;
        const long long len = (long long)s.L + s.n;
        for (int tile = s.first; tile < s.last; ++tile) {
            const long long t0 = (long long)tile * KV;
            const int live = (int)min((long long)KV, len - t0);
            __syncthreads();  // (the last tile's keys and sums are done with)
            // four words of keys a thread on their way at a time (one after the other: 220
            // us for 16 float32 contexts to 8000, 8 heads of 128)
            constexpr int U = 4;
#pragma unroll 1
            for (int i0 = tid; i0 < KV * words; i0 += NT * U) {
                int id[U];
                uint4 x[U];
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int t = (i0 + j * NT) / words;
                    id[j] = t < live ? __ldg(table + ((t0 + t) >> p.page_shift)) : -1;
                }
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int i = i0 + j * NT, t = i / words, w = i - t * words;
                    x[j] = make_uint4(0u, 0u, 0u, 0u);
                    if (id[j] >= 0 && id[j] < p.num_pages)
                        x[j] = *reinterpret_cast<const uint4*>(k + id[j] * p.page_stride +
                                                               ((t0 + t) & ((1 << p.page_shift) - 1)) * p.token_stride +
                                                               s.h * p.head_stride + w * VN);
                }
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int i = i0 + j * NT, t = i / words, w = i - t * words;
                    if (t < KV) {
                        float v[VN];
                        VecTraits<E>::unpack(x[j], v);
                        put<VN>(ks + t * stride + w * VN, v);
                    }
                }
            }
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            for (int r0 = 0; r0 < rows; r0 += R) {
                __syncthreads();
                // (rows that are one chunk stay for the stay's other tiles)
                const bool fresh = rows > R || tile == s.first;
                for (int i = tid; fresh && i < R * words; i += NT) {
                    const int r = i / words, w = i - r * words;
                    float v[VN];
#pragma unroll
                    for (int e = 0; e < VN; ++e) v[e] = 0.f;
                    if (r0 + r < rows) {
                        const int row = (r0 + r) / p.G, g = r0 + r - row * p.G, node = path ? path[row] : row;
                        const long long at = (((long long)s.b * p.N + node) * Hq + s.h * p.G + g) * p.D + w * VN;
                        VecTraits<E>::unpack(*reinterpret_cast<const uint4*>(q + at), v);
                    }
                    put<VN>(qs + r * stride + w * VN, v);
                }
                if (tid < R) {
                    float z = INFINITY;
                    int see = 0;
                    if (r0 + tid < rows) {
                        const int row = (r0 + tid) / p.G, g = r0 + tid - row * p.G;
                        if (fresh) {
                            const int node = path ? path[row] : row;
                            z = __ldg(p.lse + ((long long)s.b * p.N + node) * Hq + s.h * p.G + g) * 1.4426950408889634f;
                        } else {
                            z = c->lse[tid];
                        }
                        // (a row that sees nothing has no weights)
                        see = z == -INFINITY ? 0 : (int)min((long long)KV, max(0LL, (long long)s.L + row + 1 - t0));
                    }
                    c->lse[tid] = z;
                    c->see[tid] = see;
                }
                __syncthreads();
                float d[4][2] = {};
                for (int e = 0; e < p.D; e += 4) {
                    float4 a[4], b[2];
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(ks + (kx + 16 * i) * stride + e);
#pragma unroll
                    for (int j = 0; j < 2; ++j) b[j] = *reinterpret_cast<const float4*>(qs + (ry + 16 * j) * stride + e);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            d[i][j] = fmaf(a[i].x, b[j].x, d[i][j]);
                            d[i][j] = fmaf(a[i].y, b[j].y, d[i][j]);
                            d[i][j] = fmaf(a[i].z, b[j].z, d[i][j]);
                            d[i][j] = fmaf(a[i].w, b[j].w, d[i][j]);
                        }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float z = c->lse[ry + 16 * j];
                    const int see = c->see[ry + 16 * j];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (kx + 16 * i < see) acc[i] += ex2(fmaf(d[i][j], p.c2, -z));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], 16);
                if (lane < 16) c->sums[warp][kx + 16 * i] = acc[i];
            }
            __syncthreads();
            if (tid < live) {
                const int id = __ldg(table + ((t0 + tid) >> p.page_shift));
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < NT / 32; ++w) sum += c->sums[w][tid];
                if (id >= 0 && id < p.num_pages && SV_IN(t0 + tid, p.capacity))
                    p.weights[((long long)s.b * p.Hkv + s.h) * p.capacity + t0 + tid] += sum;
            }
        }
    }
}

template <typename E>
cudaError_t launch(const WeighParams& p, cudaStream_t st) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(weigh_kernel<E>), smem_bytes(SPEC_MAX_HEAD_DIM));
    if (e != cudaSuccess) return e;
    const size_t bytes = smem_bytes(p.D);
    const int ctas = (int)std::min<size_t>(4, 220 * 1024 / (bytes + 1024));
    weigh_kernel<E><<<152 * ctas, NT, bytes, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_weigh_simt(const WeighParams& p, int dtype, cudaStream_t st) {
    return dtype == 0 ? launch<float>(p, st) : launch<bf16_t>(p, st);
}

SV_DEBUG_READER(weigh)

}  // namespace sv
