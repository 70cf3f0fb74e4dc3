// Attention weights of accepted rows, added up a position (weigh.cuh), on the
// tensor cores (bf16, heads of 64 and 128).
//
// The products are S^T = K Q^T: 128 keys are the lanes of tensor memory and the
// rows (nodes' query heads) its columns, so that a position's sum over the rows is
// a sum over one thread's columns and no thread needs another's. One CTA an SM,
// twelve warps:
//   producer  (warp 8) copies tiles of 128 keys page by page (tensor copies with
//             the 128-byte swizzle) into a ring of stages;
//   issuer    (warp 9) issues the products of up to two tiles with a chunk of up
//             to 128 rows (whole nodes);
//   loaders   (warps 10, 11) bring the chunks (a chain's by tensor copies; a path's
//             nodes lie anywhere: copies of 16 bytes) and their log-sums, three ahead;
//   two groups (warps 0-3, 4-7) of 128 threads, a key each: one of the two tiles.
// The second loader also checks the sequences' data, when its chunks are on their way.
// A stay's only chunk is brought once. Where there are more, they go by for every
// two tiles, from L2.
//
// What bounds it. Few rows: memory (one token of 64 sequences, contexts to 8192, 8
// key heads of 4 query heads: 103 us, 5.4 TB/s of keys and weights; 100 with five
// stages and two chunks). Accepted paths of 1 to 7 nodes, 16 sequences, 300-4000
// positions, 8 x 8 heads: 23.7 us, of which the keys at that rate would take 13; the
// rest are the first lookups of a launch and of each stay. Many rows: the latency
// of a chunk's way (wait, tensor memory, exponentials, release; tensor pipe and
// exponential unit are a quarter busy, the schedulers a third): a chunk of 500 nodes
// at 4000 positions, 8 x 4 heads 33.4 us, 0.52 PFLOP/s (0.8 more with two chunks of rows
// in shared memory; 44.9 with the chunks brought by 16-byte copies, whose addresses
// took two warps longer than the products; 0.7 more with scalar in the place of packed
// arithmetic; the second 32 columns fetched beside the first ones' sums or after them, the same).

#include <cuda.h>

#include <algorithm>

#include "attention.cuh"
#include "tcgen.cuh"
#include "weigh.cuh"

namespace sv {
namespace {

#ifdef SPEC_DEBUG
static __device__ int g_withhold = -1;  // spec_debug_withhold_tile
#endif

constexpr int NT = 384;
constexpr int kKv = 128;    // keys of a tile
constexpr int kRows = 128;  // rows of a chunk, at most
constexpr int kChunks = 3;  // chunks in shared memory
constexpr int kMaxStages = 10;
constexpr uint32_t kHalf = kKv * 128;  // bytes of 64 columns of a tile or a chunk

template <int D>
struct Shape {
    static constexpr uint32_t kTile = kKv * D * 2;
    static constexpr int kStages = D == 128 ? 4 : 10;
    static constexpr size_t kSmem = 1024 + 2048 + (size_t)(kChunks + kStages) * kTile;
};

struct Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t q_full[kChunks], q_empty[kChunks];
    uint64_t s_full[2][2], s_free[2][2];  // of a group's two places
    uint64_t drain;
    uint32_t tmem, loads, asked;  // ring entries and chunks that copies were issued for
    int abort;
    int odd[kChunks][2];  // a log-sum of -inf among a loader's rows
    union {
        WeighScan scan;  // (before the loop)
        alignas(16) float lse[kChunks][kRows];  // less the log-sums, in octaves; -inf: no weight
    };
};
static_assert(sizeof(Ctl) <= 2048 && offsetof(Ctl, lse) % 16 == 0, "control region");

// The way through the part that all warps go: stays, their tiles two at a time,
// and for each two the chunks. Everything in it is a function of the inputs.
struct Way {
    const WeighParams& p;
    WeighPart part;
    WeighStay s;
    int nodes, chunks;  // nodes of a chunk, chunks of the stay

    SV_DEV Way(const WeighParams& p, const WeighPart& w) : p(p), part(w), nodes(kRows / p.G), chunks(0) {}

    // The next stay whose path is good (whole warps).
    SV_DEV bool next() {
        const int lane = threadIdx.x & 31;
#pragma unroll 1
        while (weigh_next<kKv, kRows>(p, &part, &s)) {
            bool bad = false;
            if (p.path)
#pragma unroll 1
                for (int r = lane; r < s.n; r += 32) {
                    const int i = __ldg(p.path + (long long)s.b * p.W + r);
                    bad |= i < 0 || i >= p.N;
                }
            if (__any_sync(0xFFFFFFFFu, bad)) continue;
            chunks = (s.n + nodes - 1) / nodes;
            return true;
        }
        return false;
    }
    SV_DEV int cols(int c) const { return min(nodes, s.n - c * nodes) * p.G; }
    // Whether any row of chunk c sees anything of a tile (the last chunk's do).
    SV_DEV bool seen(int tile, int c) const {
        return (long long)tile * kKv <= (long long)s.L + min((c + 1) * nodes, s.n) - 1;
    }
    SV_DEV int first_chunk(int tile) const {
        int c = 0;
        while (!seen(tile, c)) ++c;
        return c;
    }
};

// ---- keys -----------------------------------------------------------------------

template <int D>
SV_DEV void produce(const WeighParams& p, Ctl* c, const CUtensorMap* map, uint32_t stages, Way way) {
    constexpr uint32_t NS = Shape<D>::kStages, halves = D / 64;
    const int lane = threadIdx.x & 31, ps1 = (1 << p.page_shift) - 1, ps = min(ps1 + 1, kKv), pages = kKv / ps;
    const int pg = lane / halves, half = lane % halves;
    const uint32_t to = half * kHalf + pg * ps * 128;
    uint32_t ring = 0, st = 0, free_phase = 1;  // (a first round's stages are free)
    bool ok = true;
    while (ok && way.next()) {
        const WeighStay& s = way.s;
        const long long len = (long long)s.L + s.n;
        const int32_t* table = p.table + s.b * p.table_stride;
        auto look = [&](int tile) {  // this lane's page of a tile
            const long long pos = (long long)tile * kKv + pg * ps;
            return pg < pages && tile < s.last && pos < len ? __ldg(table + (pos >> p.page_shift)) : -1;
        };
        int id = look(s.first), id1 = look(s.first + 1), id2 = look(s.first + 2);
#pragma unroll 1
        for (int tile = s.first; tile < s.last; ++tile) {
            const int id3 = look(tile + 3);
            const long long pos = (long long)tile * kKv + pg * ps;
            const bool there = id >= 0 && id < p.num_pages;
            const unsigned who = __ballot_sync(0xFFFFFFFFu, there);
            bool copy = there;
#ifdef SPEC_DEBUG
            copy = copy && !(blockIdx.x == 0 && (int)ring == g_withhold);  // the entry is never filled
#endif
            if (!(ok = warp_wait(&c->empty[st], free_phase, &c->abort))) break;
            if (lane == 0) mbar_expect_tx(&c->full[st], __popc(who) * (uint32_t)ps * 128);
            __syncwarp();
            if (copy)
                tma_load4(stages + st * Shape<D>::kTile + to, map, half * 64, (int)(pos & ps1), s.h, id, &c->full[st]);
            ++ring;
            if (++st == NS) {
                st = 0;
                free_phase ^= 1;
            }
            id = id1;
            id1 = id2;
            id2 = id3;
        }
    }
    if (lane == 0) c->loads = ring;
    if (!ok) c->abort = 1;
}

// ---- rows -----------------------------------------------------------------------

// One chunk by 64 threads: rows whose log-sum says that they see nothing, and
// those that fill the last 16 columns up, take no part (zeros; lse -inf).
template <int D>
struct Loader {
    static constexpr int kWords = D / 8, kPer = 32 / kWords;  // 16-byte words of a row, rows of a warp at a time
    const WeighParams& p;
    Ctl* c;
    const CUtensorMap* map;
    uint32_t qs;
    int w;  // 0, 1
    uint32_t buf = 0, phase = 1, count = 0;

    SV_DEV bool chunk(const Way& way, int k) {
        const int lane = threadIdx.x & 31, cols = way.cols(k), whole = (cols + 15) & ~15, Hq = p.Hkv * p.G;
        const WeighStay& s = way.s;
        long long at[kRows / 32];
        float z[kRows / 32];
        bool odd = false;
#pragma unroll
        for (int i = 0; i < kRows / 32; ++i) {
            const int row = 32 * i + lane, r = row / p.G, g = row - r * p.G;
            at[i] = -1;
            z[i] = -INFINITY;
            if (row < cols) {
                int node = k * way.nodes + r;
                if (p.path) node = __ldg(p.path + (long long)s.b * p.W + node);
                at[i] = ((long long)s.b * p.N + node) * Hq + s.h * p.G + g;
                if (i / 2 == w) {
                    z[i] = -__ldg(p.lse + at[i]) * 1.4426950408889634f;
                    if (z[i] == INFINITY) {
                        z[i] = -INFINITY;
                        odd = true;
                    }
                }
            }
        }
        if (!warp_wait(&c->q_empty[buf], phase, &c->abort)) return false;
        const uint32_t base = qs + buf * Shape<D>::kTile;
        if (!p.path) {
            if (w == 0 && lane == 0) {
                const int box = min(way.nodes, p.N);  // (nodes past the last one are zeros)
                mbar_expect_tx(&c->q_full[buf], (uint32_t)(box * p.G) * (D * 2));
#pragma unroll
                for (int i = 0; i < D / 64; ++i)
                    tma_load4(base + i * kHalf, map, i * 64, s.h * p.G, k * way.nodes, s.b, &c->q_full[buf]);
            }
            __syncwarp();
        } else {
            const int word = lane % kWords;
            const uint32_t col = (word >> 3) * kHalf;
#pragma unroll
            for (int i = 0; i < kRows / 32; ++i) {
                if (32 * i >= whole) break;
#pragma unroll
                for (int j = 0; j < 32 / kPer / 2; ++j) {
                    const int lr = (2 * j + w) * kPer + lane / kWords, row = 32 * i + lr;
                    const long long from = __shfl_sync(0xFFFFFFFFu, at[i], lr);
                    if (row < whole) {
                        const uint32_t dst = base + col + row * 128 + (((word & 7) ^ (row & 7)) << 4);
                        const char* src = reinterpret_cast<const char*>(p.q) + (from < 0 ? 0 : from * (D * 2) + word * 16);
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(from < 0 ? 0 : 16)
                                     : "memory");
                    }
                }
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&c->q_full[buf])) : "memory");
        }
#pragma unroll
        for (int i = 0; i < kRows / 32; ++i)
            if (i / 2 == w) c->lse[buf][32 * i + lane] = z[i];
        odd = __any_sync(0xFFFFFFFFu, odd);
        if (lane == 0) c->odd[buf][w] = odd;
        mbar_arrive(&c->q_full[buf]);
        ++count;
        if (++buf == kChunks) {
            buf = 0;
            phase ^= 1;
        }
        return true;
    }

    SV_DEV void run(Way way) {
        bool ok = true;
        while (ok && way.next()) {
            if (way.chunks == 1) {
                ok = chunk(way, 0);
                continue;
            }
#pragma unroll 1
            for (int tile = way.s.first; ok && tile < way.s.last; tile += 2)
#pragma unroll 1
                for (int k = way.first_chunk(tile); ok && k < way.chunks; ++k) ok = chunk(way, k);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (w == 0 && (threadIdx.x & 31) == 0) c->asked = count;
        if (!ok) c->abort = 1;
    }
};

// ---- products ---------------------------------------------------------------------

template <int D>
struct Issuer {
    static constexpr uint32_t NS = Shape<D>::kStages, kTile = Shape<D>::kTile;
    Ctl* c;
    uint32_t tmem, qs, stages;
    uint32_t st = 0, phase = 0, qb = 0, q_phase = 0, places = 0, free_phase = 0xF;
    // places: bit w: which of group w's two is next; free_phase: bit 2 w + place

    SV_DEV void run(Way way) {
        bool ok = true;
        while (ok && way.next()) {
            const WeighStay& s = way.s;
            const int chunks = (int)uni(way.chunks), last = (int)uni(s.last);
            bool have = false;  // the only chunk is there
#pragma unroll 1
            for (int tile = (int)uni(s.first); ok && tile < last; tile += 2) {
                const int nt = min(2, last - tile);
                uint32_t stage[2] = {st, st + 1 == NS ? 0 : st + 1};
                bool there[2] = {false, false};
#pragma unroll 1
                for (int k = chunks == 1 ? 0 : (int)uni(way.first_chunk(tile)); ok && k < chunks; ++k) {
                    if (!have && !(ok = warp_wait(&c->q_full[qb], q_phase, &c->abort))) break;
                    have = chunks == 1;
                    const uint32_t n = uni((way.cols(k) + 15) & ~15), q = qs + qb * kTile;
                    const bool last_k = k + 1 == chunks, done = chunks > 1 || tile + 2 >= last;
                    fence_proxy_async();  // (the chunk was written by ordinary copies)
#pragma unroll 1
                    for (int w = 0; w < nt; ++w) {
                        if (w > 0 && !way.seen(tile + w, k)) break;
                        if (!there[w]) {
                            if (!(ok = warp_wait(&c->full[st], phase, &c->abort))) break;
                            there[w] = true;
                            if (++st == NS) {
                                st = 0;
                                phase ^= 1;
                            }
                        }
                        const uint32_t place = places >> w & 1, bit = 2 * w + place;
                        if (!(ok = warp_wait(&c->s_free[w][place], free_phase >> bit & 1, &c->abort))) break;
                        free_phase ^= 1u << bit;
                        places ^= 1u << w;
                        tc_fence_after();
                        const uint32_t d = tmem + 256 * w + 128 * place, idesc = mma_idesc((int)n, false);
                        const uint32_t sk = uni(stage[w]);
                        const uint64_t a = mma_desc(stages + sk * kTile, 16, 1024), b = mma_desc(q, 16, 1024);
                        if (elected()) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                                mma_ss(d, a + off, b + off, idesc, kk > 0);
                            }
                            mma_commit(&c->s_full[w][place]);
                            if (last_k) mma_commit(&c->empty[sk]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (done) {
                        if (elected()) mma_commit(&c->q_empty[qb]);
                        __syncwarp();
                        if (++qb == kChunks) {
                            qb = 0;
                            q_phase ^= 1;
                        }
                    }
                }
            }
        }
        if (!ok) c->abort = 1;
    }
};

// ---- sums -------------------------------------------------------------------------

// 32 columns of the thread's key: sum of 2^(c2 s + z); HIDE: over the columns from
// `from` on whose z is not -inf.
template <bool HIDE>
SV_DEV float weigh32(const float (&x)[32], const float* z, float c2, int from) {
    const uint64_t cc = pack2(c2, c2);
    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const float4 l = *reinterpret_cast<const float4*>(z + i);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float l0 = j ? l.z : l.x, l1 = j ? l.w : l.y;
            float a, b;
            unpack2(fma2(pack2(x[i + 2 * j], x[i + 2 * j + 1]), cc, pack2(l0, l1)), &a, &b);
            a = ex2(a);
            b = ex2(b);
            if (HIDE) {
                a = i + 2 * j >= from && l0 != -INFINITY ? a : 0.f;
                b = i + 2 * j + 1 >= from && l1 != -INFINITY ? b : 0.f;
            }
            sum[j] = add2(sum[j], pack2(a, b));
        }
    }
    float a, b;
    unpack2(add2(sum[0], sum[1]), &a, &b);
    return a + b;
}

struct Group {
    const WeighParams& p;
    Ctl* c;
    int w;
    uint32_t tmem;  // its lanes and columns
    uint32_t place = 0, full_phase = 0, qb = 0, q_phase = 0;

    SV_DEV bool chunk_done() {  // (this warp's)
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&c->q_empty[qb]);
        if (++qb == kChunks) {
            qb = 0;
            q_phase ^= 1;
        }
        return true;
    }

    SV_DEV void run(Way way) {
        const int lane = threadIdx.x & 31, key = threadIdx.x & 127;
        bool ok = true;
        while (ok && way.next()) {
            const WeighStay& s = way.s;
            const long long len = (long long)s.L + s.n;
            const int32_t* table = p.table + s.b * p.table_stride;
            float* weights = p.weights + ((long long)s.b * p.Hkv + s.h) * p.capacity;
            bool have = false;
#pragma unroll 1
            for (int tile = s.first; ok && tile < s.last; tile += 2) {
                const int mine = tile + w;
                const long long t = (long long)mine * kKv + key;
                // (this position is no other thread's: what it holds is fetched early)
                bool store = mine < s.last && t < len;
                float before = 0.f;
                if (store) {
                    const int id = __ldg(table + (t >> p.page_shift));
                    store = id >= 0 && id < p.num_pages;
                    before = weights[t];
                }
                float acc = 0.f;
#pragma unroll 1
                for (int k = way.chunks == 1 ? 0 : way.first_chunk(tile); ok && k < way.chunks; ++k) {
                    if (!have && !(ok = warp_wait(&c->q_full[qb], q_phase, &c->abort))) break;
                    have = way.chunks == 1;
                    if (mine < s.last && way.seen(mine, k)) {
                        if (!(ok = warp_wait(&c->s_full[w][place], full_phase >> place & 1, &c->abort))) break;
                        full_phase ^= 1u << place;
                        tc_fence_after();
                        const int cols = way.cols(k), row0 = k * way.nodes;
                        const float* z = c->lse[qb];
                        const volatile int* odd = c->odd[qb];
                        const long long hidden = ((long long)t - s.L - row0) * p.G;  // columns that do not see this key
                        const bool all = (long long)mine * kKv + kKv - 1 <= (long long)s.L + row0 && !odd[0] && !odd[1];
                        const uint32_t from = tmem + 128 * place;
                        auto sum = [&](const float (&x)[32], int j) {
                            acc += all && j + 32 <= cols ? weigh32<false>(x, z + j, p.c2, 0)
                                                         : weigh32<true>(x, z + j, p.c2, (int)max(0LL, min(hidden - j, 32LL)));
                        };
                        // (the second 32 columns are on their way while the first are added
                        // up; a place has 128, what lies past the chunk's is not used)
#pragma unroll 1
                        for (int j = 0; j < cols; j += 64) {
                            float x[32], y[32];
                            tmem_ld32_start(from + j, x);
                            tmem_ld32_wait(x);
                            tmem_ld32_start(from + j + 32, y);
                            sum(x, j);
                            tmem_ld32_wait(y);
                            if (j + 32 < cols) sum(y, j + 32);
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&c->s_free[w][place]);
                        place ^= 1;
                    }
                    if (way.chunks > 1) chunk_done();
                }
                if (ok && store && SV_IN(t, p.capacity)) weights[t] = before + acc;
            }
            if (ok && way.chunks == 1) chunk_done();
        }
        if (!ok) c->abort = 1;
    }
};

// Clears the statuses, which the weighing's CTAs only raise: a plain store of a good one by a
// CTA that began late, behind another stream's work, would take back what one that gave up
// reported. The weighing's blocks are launched beside it. (Paths of 16 sequences: 23.7 us,
// 22.6 with the plain stores, 26.6 with a memset. With the checks in this kernel too, one
// token over 100003 positions in pages of 8 took 63.6 for 61.0, as its blocks keep the
// weighing's from their SMs, and of 4000 sequences 668 for 595.)
__global__ void __launch_bounds__(256) weigh_clear_kernel(int32_t* status, int B) {
    asm volatile("griddepcontrol.launch_dependents;");
    const int b = blockIdx.x * 256 + threadIdx.x;
    if (b < B) status[b] = kOk;
}

template <int D>
__global__ void __launch_bounds__(NT, 1)
    weigh_tc_kernel(const __grid_constant__ WeighParams p, const __grid_constant__ CUtensorMap map,
                    const __grid_constant__ CUtensorMap mq) {
    extern __shared__ unsigned char dyn[];
    unsigned char* mem = dyn + ((1024 - (smem_u32(dyn) & 1023)) & 1023);
    Ctl* c = reinterpret_cast<Ctl*>(mem);
    const uint32_t qs = smem_u32(mem) + 2048, stages = qs + kChunks * Shape<D>::kTile;
    const int tid = threadIdx.x, warp = tid >> 5;

    // (nothing is read before the kernel that clears the statuses is done: what another thread
    // has put on the stream between the two is done then too)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const WeighPart part = weigh_locate<kKv, kRows, NT>(p, &c->scan);
    if (tid == 0) {
        for (int i = 0; i < Shape<D>::kStages; ++i) {
            mbar_init(&c->full[i], 1);
            mbar_init(&c->empty[i], 1);
        }
        for (int i = 0; i < kChunks; ++i) {
            mbar_init(&c->q_full[i], p.path ? 2 * 64 : 1 + 64);  // the loaders' copies and their stores
            mbar_init(&c->q_empty[i], 1 + 8);  // the products and the groups' warps
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&c->s_full[i >> 1][i & 1], 1);
            mbar_init(&c->s_free[i >> 1][i & 1], 4);
        }
        mbar_init(&c->drain, 1);
        c->loads = c->asked = 0;
        c->abort = 0;
        mbar_init_fence();
    }
    if (tid == 8 * 32) tma_prefetch(&map);
    if (tid == 10 * 32 && !p.path) tma_prefetch(&mq);
    if (warp == 9) tmem_alloc512(&c->tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c->tmem;
    const Way way(p, part);

    if (warp < 8) {
        Group g{p, c, warp >> 2, tmem + ((uint32_t)(warp & 3) << 21) + 256 * (warp >> 2)};
        g.run(way);
    } else if (warp == 8) {
        produce<D>(p, c, &map, stages, way);
    } else if (warp == 9) {
        Issuer<D> is{c, uni(tmem), qs, stages};
        is.run(way);
    } else {
        Loader<D> l{p, c, &mq, qs, warp - 10};
        l.run(way);
        if (warp == 11) weigh_statuses<true>(p, blockIdx.x, gridDim.x);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (c->abort) {  // copies and products in flight end before the CTA does
        constexpr uint32_t NS = Shape<D>::kStages;
        if (tid == 10 * 32 && !p.path)
            for (uint32_t r = c->asked > kChunks ? c->asked - kChunks : 0; r < c->asked; ++r)
                tc_wait(&c->q_full[r % kChunks], (r / kChunks) & 1, nullptr);
        if (tid == 8 * 32)
            for (uint32_t r = c->loads > NS ? c->loads - NS : 0; r < c->loads; ++r)
                tc_wait(&c->full[r % NS], (r / NS) & 1, nullptr);
        if (warp == 9 && elected()) {  // (the lane that issued the products)
            mma_commit(&c->drain);
            tc_wait(&c->drain, 0, nullptr);
        }
        __syncthreads();
    }
    if (warp == 9) tmem_free512(tmem);
    if (warp == 0 && c->abort && p.status) {  // a wait gave up: the sequences of this part are not whole
        Way again(p, part);
        while (again.next())
            if (tid == 0) atomicMax(p.status + again.s.b, kETimeout);
    }
}

template <int D>
cudaError_t launch(const WeighParams& p, const CUtensorMap& map, const CUtensorMap& mq, cudaStream_t st) {
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(weigh_tc_kernel<D>), Shape<D>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(152);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = Shape<D>::kSmem;
    cfg.stream = st;
    if (p.status) {
        weigh_clear_kernel<<<(p.B + 255) / 256, 256, 0, st>>>(p.status, p.B);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, weigh_tc_kernel<D>, p, map, mq);
}

}  // namespace

cudaError_t launch_weigh_tc(const WeighParams& p, cudaStream_t st, bool* took) {
    AttnParams a = {};
    a.D = p.D;
    a.Hkv = p.Hkv;
    a.num_pages = p.num_pages;
    a.page_shift = p.page_shift;
    a.page_stride = p.page_stride;
    a.token_stride = p.token_stride;
    a.head_stride = p.head_stride;
    a.q = p.q;
    a.B = p.B;
    a.N = p.N;
    a.G = p.G;
    AttnMaps k, q;
    *took = cache_tc_map(a, p.k, &k) && query_tc_map(a, &q);
    if (!*took) return cudaSuccess;
    const CUtensorMap &mk = *reinterpret_cast<const CUtensorMap*>(&k), &mq = *reinterpret_cast<const CUtensorMap*>(&q);
    return p.D == 128 ? launch<128>(p, mk, mq, st) : launch<64>(p, mk, mq, st);
}

int debug_withhold_weigh_tile(int j) {
#ifdef SPEC_DEBUG
    return cudaMemcpyToSymbol(g_withhold, &j, sizeof(int)) == cudaSuccess ? 0 : -1;
#else
    (void)j;
    return -1;
#endif
}

SV_DEBUG_READER(weigh_tc)

}  // namespace sv
