// Tree attention over a paged cache on the tensor cores (bf16, heads of 64 and
// 128; attention.cuh: the mathematics and the division of the work).
//
// One CTA an SM, a persistent part of the range each, twelve warps:
//   producer   (warp 8) copies K and V tiles of 128 positions page by page
//              (tensor copies with the 128-byte swizzle) into a ring of stages;
//   issuers    (warps 9, 10; one a stream) issue the products: S = Q K^T into
//              tensor memory, and O += P V with P taken from tensor memory;
//   helper     (warp 11) walks the part and posts each stay in a unit (a
//              segment) for the others, brings its queries (while the last
//              one's results are still being written) and clears what V must
//              not contain (warp 10 first writes the rows that no unit covers);
//   two groups (warps 0-3, 4-7) of 128 threads, a row each: the softmax between
//              the two products, and the results.
// The groups are two streams that the tensor core serves in turn, one's
// products while the other computes its softmax:
//   more than 128 rows  both streams go over the same tiles, each for a half of
//                       the unit's 256 rows (a tile is read once for 256 rows;
//                       a half holds whole nodes, so fewer rows where G does
//                       not divide 128);
//   else                both have the same rows and take alternate tiles; group
//                       0 joins their sums at the end (both O lie in the lanes
//                       that it can read).
// A stream goes by halves of a tile, 64 positions: S of a half takes columns
// 128 w + 64 (half) of tensor memory, and P (bf16, two a column) its place 32
// positions at a time, 16 columns of the weights' first parts and 16 of the second; O_w columns
// 256 + 128 w. With two halves' places, a half's scores are there before the
// softmax of the half before is done, and the products run beside it (with one
// place of 128 positions a stream, scores, softmax and product came one after
// the other: 4450 cycles for two tiles of the two streams, whose products take
// 2048). A stream's products are issued by one thread and run in its order, so
// the scores of the next half in a place cannot overtake the product that reads it.
//
// Weights are formed against a whole-number reference that follows the running
// maximum with slack (Group::softmax), so O_w is rarely scaled. Statistics and
// sums are fp32. For the product with V a weight goes as two bf16 numbers, its
// upper 16 bits and what they leave, so that V is multiplied twice: 16 bits of
// a weight count (off by 2^-16 of it at the most). One bf16 weight would be off
// by 2^-9, as much as the output's own rounding, and that does not average out
// against the output: over values of mean zero both become smaller alike
// (error of the outputs, against that of their rounding alone, with one
// rounded weight where none is above a sixteenth of its row's sum: 1.38 times
// at 900 positions, 1.12 at 20000). Neither part is negative, and neither is
// zero unless the weight is, so that an infinity in V keeps its sign in every row.
//
// Tiles that reach past the context also hold nodes and the end: a thread forms
// its row's visibility bits, and the elements of V there that are not finite
// are zeroed in shared memory before the product (a zero weight times an
// infinity would be NaN in rows that do not see the node) and added to the rows
// that do see them when the results are written.

// What bounds it. One token of 64 sequences, contexts to 8192, 8 key heads of 4
// query heads, 128 columns: memory (176 us, 6.1 TB/s of K and V). With 64 or
// more rows the way of a half from its scores over the softmax and its products
// to the next scores in its place: a warp takes some 440 instructions, mostly of
// latency at one or two warps a scheduler (issue 23 to 39 %), and the tensor
// pipe is 34 to 61 % busy. 16 trees of 64 nodes, contexts
// to 1900, 32 heads of one query head (64 rows, half of the product's 128):
// 78.6 us (3.7 TB/s); contexts to 4000, 8 heads of 8 (512 rows): 107 us (0.63
// PFLOP/s); a tree of 61 nodes over 100003 positions, 8 heads of 4: 124 us
// (weights of one bf16 number, and a second only where it was heavy: 82.1, 103
// and 106).
// Around that a launch takes some 13000 cycles to its first scores (the cut,
// the first lookup, the first copies) and a unit 4000 to 6000 for its end.
// Small pages cost copies: an entry of pages of 16 is 16 of them, and heads of
// 64 columns (16 KB an entry) read 3.7 TB/s at pages of 16, 4.2 at 128. Code
// size counts too: the warps' paths together are larger than the instruction
// caches near them, and more unrolling anywhere slowed everything (loops are
// rolled and paths shared for it).

#include <cuda.h>

#include <algorithm>

#include "attention.cuh"
#include "tcgen.cuh"

namespace sv {
namespace {

#ifdef SPEC_DEBUG
static __device__ int g_withhold = -1;  // spec_debug_withhold_tile
#endif

constexpr int NT = 384;
// Registers: 384 x 168 at launch, handed over as 208 to the softmax groups and
// 88 to the third (2 x 208 + 88 = 3 x 168).
constexpr int kGroupRegs = 208, kOtherRegs = 88;
constexpr int kKv = 128;     // positions of a tile
constexpr int kMaxStages = 10;
constexpr int kExtra = 3, kExtraDual = 4;
constexpr int kWhole = 4;  // tiles of a unit that is not split
constexpr float kKeep = 1.f + 0x1p-20f;  // a weight's second part is kKeep of it less its first
constexpr float kSlack = 8.f;  // octaves of a score above the reference that raise it
constexpr uint32_t kHalf = kKv * 128;  // bytes of 64 columns of a tile
constexpr int kHalfKv = 64;            // positions of a half of a tile
constexpr uint32_t kHalfRows = kHalfKv * 128;  // bytes from its rows to the other half's, in 64 columns

template <int D>
struct Shape {
    static constexpr uint32_t kTile = kKv * D * 2;
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr size_t kSmem = 1024 + 2048 + (size_t)(2 + kStages) * kTile;
};

// A stay in a unit; dual: both streams go over its tiles.
struct Seg : AttnStay {
    bool dual;
    int steps;  // softmax tiles of both streams together
};
struct Walk : AttnWalk<kKv> {
    using AttnWalk<kKv>::AttnWalk;
    SV_DEV bool next(const AttnParams& p, Seg* s) {
        if (!AttnWalk<kKv>::next(p, s)) return false;
        s->dual = s->rows > p.tile_rows / 2;
        s->steps = (s->last - s->first) * (s->dual ? 2 : 1);
        return true;
    }
};

struct Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages], clean[kMaxStages];
    uint64_t q_full, q_empty, s_full[2][2], p_full[2][2], pv[2], o_full[2], ask[2], groups, drain;
    uint32_t loads;  // ring entries filled
    uint32_t asks;   // segments whose queries were asked for
    AttnScan scan;
    uint32_t tmem;
    int abort;
    uint64_t seg_full[4];
    Seg seg[4];    // the helper's post: segment number modulo 4; b = -1: no more
    int flags[4];  // of a segment: 1 V had elements that are not finite, 2 a bad page
    float2 ml[128];
};
static_assert(sizeof(Ctl) <= 2048, "control region");

// Order of a segment's tiles in the ring (cnt tiles): the order of their first
// use. Two streams on the same tiles: K0 V0 K1 V1 ..; on alternate tiles: K0
// K1 V0 K2 V1 K3 ..
SV_DEV int ring_v(const Seg& s, int i) { return s.dual ? 2 * i + 1 : i + min(i + 2, s.last - s.first); }

// Whether tile i of a segment reaches past the context; the stages that the V
// of such tiles i in [i0, i1) lie in, a bit each (no two in the same: they are
// neighbours).
SV_DEV bool tail_tile(const Seg& s, int i) { return (long long)(s.first + i + 1) * kKv > s.L; }
template <int D>
SV_DEV uint32_t clean_stages(const Seg& s, uint32_t ring0, int i0, int i1) {
    uint32_t bits = 0;
    for (int i = i0; i < i1; ++i)
        if (tail_tile(s, i)) bits ^= 1u << ((ring0 + ring_v(s, i)) % Shape<D>::kStages);
    return bits;
}

// Positions of a tile that hold anything; the product with V goes over whole
// steps of 16 of them.
SV_DEV int live_of(const Seg& s, int i) { return (int)min((long long)kKv, s.len - (long long)(s.first + i) * kKv); }

// Halves of stream w's tiles: two each, one where nothing of the last tile's
// second half is there.
SV_DEV int halves_of(const Seg& s, int w) {
    const int cnt = s.last - s.first, mine = s.dual ? cnt : (cnt + 1 - w) >> 1;
    const bool has_last = s.dual || ((cnt - 1) & 1) == w;
    return 2 * mine - (mine && has_last && live_of(s, cnt - 1) <= kHalfKv ? 1 : 0);
}

// Waits give up after some 2^18 polls (a poll that finds nothing takes up to
// 2 us: half a second; 2^22 took 8 seconds), or once `abort` is set. They poll
// without a suspension of their own: its wake-up costs more than these short
// waits last.
SV_DEV bool tc_wait(uint64_t* bar, uint32_t parity, const volatile int* abort) {
    uint32_t n = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity))
        if (!(++n & 0xFFu) && (n >> 18 || (abort && *abort))) return false;
    return true;
}
// By whole warps: every lane gets the same answer.
SV_DEV bool warp_wait(uint64_t* bar, uint32_t parity, const int* abort) {
    return __all_sync(0xFFFFFFFFu, tc_wait(bar, parity, abort)) != 0;
}

// The post of segment number `seg`, null after the last (or a timeout). It
// stays until segment seg + 3 begins.
SV_DEV const Seg* next_seg(Ctl* c, uint32_t seg, bool* ok) {
    *ok = warp_wait(&c->seg_full[seg & 3], (seg >> 2) & 1, &c->abort);
    return *ok && c->seg[seg & 3].b >= 0 ? &c->seg[seg & 3] : nullptr;
}

// ---- copies ----------------------------------------------------------------------

template <int D>
SV_DEV void produce(const AttnParams& p, Ctl* c, const CUtensorMap* mk, const CUtensorMap* mv, uint32_t stages) {
    constexpr uint32_t NS = Shape<D>::kStages, halves = D / 64;
    const int lane = threadIdx.x & 31, ps1 = (1 << p.page_shift) - 1, ps = min(ps1 + 1, kKv), pages = kKv / ps;
    const int pg = lane / halves, half = lane % halves;
    const uint32_t to = half * kHalf + pg * ps * 128;
    uint32_t ring = 0, seg = 0, st = 0, free_phase = 1;  // (a first round's stages are free)
    bool ok = true;
    while (const Seg* at = next_seg(c, seg, &ok)) {
        const Seg& s = *at;
        const int cnt = s.last - s.first, ahead = s.dual ? 1 : 2, h = s.h;
        const long long len = s.len, pos0 = (long long)s.first * kKv + pg * ps;
        const int32_t* table = p.table + s.b * p.table_stride;
        auto look = [&](int i) {  // this lane's page of tile i
            const long long pos = pos0 + (long long)i * kKv;
            return pg < pages && i >= 0 && i < cnt && pos < len ? __ldg(table + (pos >> p.page_shift)) : -1;
        };
        auto entry = [&](int id, int i, const CUtensorMap* map) {
            if (i < 0 || i >= cnt) return;
            const long long pos = pos0 + (long long)i * kKv;
            const bool there = pg < pages && pos < len;
            if (there && (uint32_t)id >= (uint32_t)p.num_pages) {
                id = -1;
                atomicOr(&c->flags[seg & 3], 2);
            }
            const unsigned who = __ballot_sync(0xFFFFFFFFu, there && id >= 0);
            bool copy = there && id >= 0;
#ifdef SPEC_DEBUG
            copy = copy && !(blockIdx.x == 0 && (int)ring == g_withhold);  // the entry is never filled
#endif
            if (!(ok = warp_wait(&c->empty[st], free_phase, &c->abort))) return;
            if (lane == 0) mbar_expect_tx(&c->full[st], __popc(who) * (uint32_t)ps * 128);
            __syncwarp();
            if (copy)
                tma_load4(stages + st * Shape<D>::kTile + to, map, half * 64, (int)(pos & ps1), h, id, &c->full[st]);
            ++ring;
            if (++st == NS) {
                st = 0;
                free_phase ^= 1;
            }
        };
        // V(i), then K(i + ahead); the pages of four tiles are known or on their way
        int id0 = -1, id1 = look(1 - ahead), id2 = look(2 - ahead), id3 = look(3 - ahead);
#pragma unroll 1
        for (int i = -ahead; ok && i < cnt; ++i) {
            const int next = look(i + 4);
#pragma unroll 1
            for (int k = 0; ok && k < 2; ++k)
                entry(k == 0 ? id0 : s.dual ? id1 : id2, k == 0 ? i : i + ahead, k == 0 ? mv : mk);
            id0 = id1;
            id1 = id2;
            id2 = id3;
            id3 = next;
        }
        if (!ok) break;
        ++seg;
    }
    if (lane == 0) c->loads = ring;
    if (!ok) c->abort = 1;
}

// ---- products ---------------------------------------------------------------------

// The whole warp goes through the steps and one elected lane issues: operands
// broadcast from lane 0 are known to be the same in every lane, so that they
// stay in uniform registers (issued by one thread from its own registers, a
// product of 16 positions took 80 to 160 cycles to issue and 64 to run).
SV_DEV uint32_t uni(uint32_t x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

SV_DEV bool elected() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// A stream's way along the ring. Both issuers wait for every entry in its
// order and both release it (one's products on it, or its having seen an entry
// that is the other's): a barrier's parity tells neighbouring rounds of a stage
// apart and no more, so none may skip one.
template <int D>
struct Issuer {
    static constexpr uint32_t NS = Shape<D>::kStages, kTile = Shape<D>::kTile;
    Ctl* c;
    uint32_t w, tmem, qs, stages;
    uint32_t st = 0, phase = 0, left = 0;               // the next entry's stage and round, entries left of the segment
    uint32_t p_phase = 0, q_phase = 0, clean = 0;       // clean: phase of each stage's barrier

    SV_DEV bool advance() {
        const bool ok = warp_wait(&c->full[st], phase, &c->abort);
        --left;
        if (++st == NS) {
            st = 0;
            phase ^= 1;
        }
        return ok;
    }
    // The next entry, this stream's: its stage.
    SV_DEV bool take(uint32_t* stage) {
        *stage = st;
        return advance();
    }
    // The next n entries, the other stream's.
    SV_DEV bool pass(int n) {
        bool ok = true;
        for (; ok && n > 0; --n) {
            const uint32_t at = st;
            ok = advance();
            if (elected()) mbar_arrive(&c->empty[at]);
            __syncwarp();
        }
        return ok;
    }

    // The products of one step: for each half, O += P V of this stream's tile in
    // stage_v (nv halves; `last` of the segment) and then, in the place that
    // this frees, the scores of its next tile in stage_k (nk halves). One lane
    // waits and issues: its few instructions between two products are what the
    // other stream's products have to cover.
    SV_DEV bool step(bool dual, uint32_t stage_v, int nv, bool first, bool last, bool tail, int live, uint32_t stage_k,
                     int nk, bool last_k) {
        constexpr uint32_t idesc_s = mma_idesc(kHalfKv, false), idesc_o = mma_idesc(D, true);
        const uint32_t sv = uni(stage_v), sk = uni(stage_k);
        const uint32_t ds = tmem + 128 * w, dp = tmem + 256 + 128 * w;
        const uint64_t q = mma_desc(qs + (dual ? w * kTile : 0u), 16, 1024);
        const uint64_t k = mma_desc(stages + sk * kTile, 16, 1024), v = mma_desc(stages + sv * kTile, kHalf, 1024);
        bool ok = true;
        if (elected()) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (half < nv) {
                    ok = tc_wait(&c->p_full[w][half], p_phase >> half & 1, &c->abort);
                    if (tail && half == 0) ok = ok && tc_wait(&c->clean[sv], clean >> sv & 1, &c->abort);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (64 * half + 16 * kk < live) {
                            const uint32_t a = ds + 64 * half + (kk >> 1) * 32 + (kk & 1) * 8;
                            const uint64_t b = v + (half * kHalfRows + kk * 2048 >> 4);
                            mma_ts(dp, a, b, idesc_o, !first || half > 0 || kk > 0);
                            mma_ts(dp, a + 16, b, idesc_o, true);
                        }
                    mma_commit(&c->pv[w]);
                    if (half + 1 == nv) {
                        mma_commit(&c->empty[sv]);
                        if (last) mma_commit(&c->o_full[w]);
                    }
                }
                if (half < nk) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                        mma_ss(ds + 64 * half, q + off, k + (half * kHalfRows >> 4) + off, idesc_s, kk > 0);
                    }
                    mma_commit(&c->s_full[w][half]);
                    if (half + 1 == nk) {
                        mma_commit(&c->empty[sk]);
                        if (last_k) mma_commit(&c->q_empty);
                    }
                }
            }
        }
        p_phase ^= (1u << nv) - 1u;  // (a bit a half)
        return __all_sync(0xFFFFFFFFu, ok) != 0;
    }

    SV_DEV void run() {
        uint32_t ring0 = 0, seg = 0;
        bool ok = true;
        while (const Seg* at = next_seg(c, seg, &ok)) {
            const Seg& s = *at;
            const bool dual = uni(s.dual);
            const int cnt = (int)uni(s.last - s.first), halves = (int)uni(halves_of(s, w));  // of this stream's tiles
            const int mine = (halves + 1) >> 1, tails = (int)uni(max(0, s.L / kKv - s.first));  // tiles from here on reach
            const int live = (int)uni(live_of(s, cnt - 1));                                     // past the context
            ok = warp_wait(&c->q_full, q_phase, &c->abort);
            q_phase ^= 1;
            if (halves == 0 && elected()) mbar_arrive(&c->q_empty);
            __syncwarp();
            left = 2 * cnt;
            uint32_t sv = 0, sk = 0;
            if (mine && !dual) ok = ok && pass(w);  // K0
#pragma unroll 1
            for (int j = -1; ok && j < mine; ++j) {
                if (!mine) continue;
                const int i = dual ? j : 2 * j + (int)w;
                const bool tail = j >= 0 && i >= tails;
                if (j >= 0) {
                    // between this stream's K(i) and V(i): V(i - 1) and K(i + 1)
                    if (!dual && !(ok = pass((i > 0) + (i + 1 < cnt)))) break;
                    if (!(ok = take(&sv))) break;
                    if (tail && (!dual || w == 0)) {  // V has to be cleaned first
                        if (elected()) mbar_arrive(&c->ask[w]);
                        __syncwarp();
                    }
                }
                if (j + 1 < mine && !(ok = take(&sk))) break;
                tc_fence_after();
                ok = step(dual, sv, j < 0 ? 0 : min(2, halves - 2 * j), j == 0, j + 1 == mine, tail,
                          i + 1 == cnt ? live : kKv, sk, min(2, halves - 2 * j - 2), j + 2 == mine);
                // (phases of the stages whose V these tiles have had cleaned, the other stream's too)
                const int i0 = dual ? j : 2 * j, i1 = dual ? j + 1 : min(2 * j + 2, cnt);
                if (j >= 0 && i1 > tails) clean ^= clean_stages<D>(s, ring0, i0, i1);
            }
            if (!dual && mine < (cnt + 1) >> 1) clean ^= clean_stages<D>(s, ring0, 2 * mine, cnt);
            ring0 += 2 * cnt;
            if (!ok || !(ok = pass((int)left))) break;
            ++seg;
        }
        if (!ok) c->abort = 1;
    }
};

// ---- softmax and results ------------------------------------------------------------

// The visibility of 64 positions for the rows of a warp (lanes in the order of
// their nodes), 32 a word: a node's mask bytes by the whole warp, a ballot a
// word. Node j of the rows' own sequence is at position L + j.
SV_DEV uint2 see_bits(const AttnParams& p, const Seg& s, int node, long long pos0) {
    const int lane = threadIdx.x & 31;
    const long long ctx = s.L - pos0, upto = s.len - pos0;  // context below ctx, nothing from upto on
    const int j0 = (int)max(-64LL, -ctx);                   // node of bit 0 (negative: context)
    uint32_t see[2];
    if (!p.mask) {
        const long long to = min(upto, ctx + node + 1);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int n = (int)min(32LL, max(0LL, to - 32 * k));
            see[k] = n == 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
        }
        return make_uint2(see[0], see[1]);
    }
    const int first = __shfl_sync(0xFFFFFFFFu, node, 0), last = __shfl_sync(0xFFFFFFFFu, node, 31);
    const uint8_t* row = p.mask + ((long long)s.b * p.N + first) * p.N + j0 + lane;
    const bool c0 = j0 + lane < 0, c1 = j0 + lane + 32 < 0;                       // context
    const bool n0 = !c0 && j0 + lane < s.n, n1 = !c1 && j0 + lane + 32 < s.n;  // a node
    see[0] = see[1] = 0u;
#pragma unroll 1
    for (int m0 = first; m0 <= last; m0 += 8) {
        uint8_t x[8], y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            x[u] = n0 && m0 + u <= last ? __ldg(row + u * p.N) : 0;
            y[u] = n1 && m0 + u <= last ? __ldg(row + u * p.N + 32) : 0;
        }
        row += 8 * (long long)p.N;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t a = __ballot_sync(0xFFFFFFFFu, c0 || x[u] != 0), b = __ballot_sync(0xFFFFFFFFu, c1 || y[u] != 0);
            if (node == m0 + u) {
                see[0] = a;
                see[1] = b;
            }
        }
    }
    return make_uint2(see[0], see[1]);
}

// What clean_v took out, added to a row's written results (columns [col, col +
// cols)); rare, so it is kept small.
SV_DEV void add_unclean(const AttnParams& p, const Seg& s, int node, char* out, int col, int cols) {
    const int j0 = (int)max(0LL, (long long)s.first * kKv - s.L);
    const int j1 = (int)min((long long)s.n, (long long)s.last * kKv - s.L);
    const uint16_t* v = reinterpret_cast<const uint16_t*>(p.v) + s.h * p.head_stride + col;
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
        const bool see = p.mask ? __ldg(p.mask + ((long long)s.b * p.N + node) * p.N + j) != 0 : j <= node;
        const long long pos = (long long)s.L + j;
        const int id = __ldg(p.table + s.b * p.table_stride + (pos >> p.page_shift));
        if (!see || id < 0 || id >= p.num_pages) continue;
        const uint16_t* row = v + id * p.page_stride + (pos & ((1 << p.page_shift) - 1)) * p.token_stride;
#pragma unroll 1
        for (int e = 0; e < cols; ++e) {
            const uint32_t x = row[e];
            if ((x & 0x7F80u) != 0x7F80u) continue;
            if (s.whole) {
                uint16_t* o = reinterpret_cast<uint16_t*>(out) + e;
                *o = (uint16_t)pack_bf16(__uint_as_float((uint32_t)*o << 16) + __uint_as_float(x << 16), 0.f);
            } else {
                reinterpret_cast<float*>(out)[e] += __uint_as_float(x << 16);
            }
        }
    }
}

SV_DEV uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

constexpr float kNegInf = -__builtin_inff();

SV_DEV float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

SV_DEV void st32(char* dst, const uint32_t* x) {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(x[4], x[5], x[6], x[7]);
}

// ---- queries, pages, edges -----------------------------------------------------------

// Rows of a V tile past the context (one warp): elements that are not finite
// become zero (flag 1), and so do the rows past the end that the product's last
// step covers.
template <int D>
SV_DEV void clean_v(Ctl* c, const Seg& s, uint32_t tile_addr, int i, int slot) {
    constexpr int C = D / 8, R = 32 / C, U = 8;  // 16-byte words of a row, rows at a time, words in flight
    const int lane = threadIdx.x & 31, ch = lane % C, live = live_of(s, i);
    const long long ctx = s.L - (long long)(s.first + i) * kKv;
    const uint32_t col = tile_addr + (ch >> 3) * kHalf;
    auto word = [&](int r) { return col + r * 128 + (((ch & 7) ^ (r & 7)) * 16); };
    bool found = false;
    for (int r0 = (int)max(0LL, ctx) + lane / C; r0 < live; r0 += R * U) {
        uint32_t y[U][4], zero[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = min(r0 + u * R, live - 1);
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(y[u][0]), "=r"(y[u][1]), "=r"(y[u][2]), "=r"(y[u][3])
                         : "r"(word(r)));
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e)  // 0 + 0 x stays 0 unless x is not finite
                asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(zero[e]) : "r"(y[u][e]), "r"(0u));
        if ((zero[0] | zero[1]) | (zero[2] | zero[3])) {
            found = true;
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int e = 0; e < 4; ++e) y[u][e] &= ~__vcmpeq2(y[u][e] & 0x7F807F80u, 0x7F807F80u);
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(word(min(r0 + u * R, live - 1))), "r"(y[u][0]),
                             "r"(y[u][1]), "r"(y[u][2]), "r"(y[u][3])
                             : "memory");
            }
        }
    }
    for (int r = live + lane / C; r < ((live + 15) & ~15); r += R)
        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(word(r)), "r"(0u) : "memory");
    if (found) atomicOr(&c->flags[slot], 1);
}

template <int D>
SV_DEV void help(const AttnParams& p, Ctl* c, const CUtensorMap* mq, uint32_t qs, uint32_t stages, Walk walk) {
    constexpr uint32_t NS = Shape<D>::kStages;
    const int lane = threadIdx.x & 31, nodes = 128 / p.G;  // nodes of a half
    const uint32_t box = 128u * min(nodes, p.N) * p.G;     // bytes of 64 columns of them
    uint32_t seg = 0, ring0 = 0, asked = 0, asks = 0;
    auto ask_q = [&](const Seg& s) {  // a segment's queries
        ++asks;
        if (lane == 0) mbar_expect_tx(&c->q_full, box * (D / 64) * (s.dual ? 2 : 1));
        __syncwarp();
        if (lane < D / 64 * (s.dual ? 2 : 1)) {
            const int w = lane / (D / 64), half = lane - w * (D / 64);
            tma_load4(qs + w * Shape<D>::kTile + half * kHalf, mq, half * 64, s.h * p.G, s.row0 / p.G + w * nodes, s.b,
                      &c->q_full);
        }
    };
    bool ok = true, more = true;
#pragma unroll 1
    for (;; ++seg) {
        // Post `seg`. With segment seg - 2's queries free (below), the groups have
        // begun segment seg - 3, the issuers and the producer seg - 2: it takes the
        // place of one that nobody needs.
        Seg next;
        const bool again = more && walk.next(p, &next);
        if (!ok) {  // what is left of the part will not be done
            if (!again) break;
            if (lane == 0 && p.status) atomicMax(p.status + next.b, kETimeout);
            continue;
        }
        if (lane == 0) {
            c->flags[seg & 3] = 0;
            if (!again) next.b = -1;
            c->seg[seg & 3] = next;
            mbar_arrive(&c->seg_full[seg & 3]);
        }
        __syncwarp();
        more = again;
        if (seg == 0) {
            if (!more) break;
            ask_q(c->seg[0]);
            continue;
        }
        // the segment before it, whose queries are on their way: its V
        const Seg& s = c->seg[(seg - 1) & 3];
        const int cnt = s.last - s.first;
#pragma unroll 1
        for (int i = max(0, s.L / kKv - s.first); ok && i < cnt; ++i) {
            if (!tail_tile(s, i)) continue;
            const uint32_t st = (ring0 + ring_v(s, i)) % NS, w = s.dual ? 0u : i & 1;
            if (!(ok = warp_wait(&c->ask[w], asked >> w & 1, &c->abort))) break;  // (the tile is there)
            asked ^= 1u << w;
            clean_v<D>(c, s, stages + st * Shape<D>::kTile, i, (seg - 1) & 3);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->clean[st]);
        }
        ring0 += 2 * cnt;
        if (ok && !more) break;
        if (ok && (ok = warp_wait(&c->q_empty, (seg - 1) & 1, &c->abort))) ask_q(c->seg[seg & 3]);
        if (!ok) c->abort = 1;
    }
    if (lane == 0) c->asks = asks;
}

template <int D>
struct Group {
    const AttnParams& p;
    Ctl* c;
    int w, warp, lane, t;       // group, warp of the group, lane, thread of the group = row of its tile
    uint32_t tm_s, tm_o;        // this warp's lanes of S_w and O_w
    uint32_t s_phase = 0, o_phase = 0, g_phase = 0, pv_count = 0;

    // Both groups; false after a timeout.
    SV_DEV bool meet() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->groups);
        const bool ok = warp_wait(&c->groups, g_phase, &c->abort);
        g_phase ^= 1;
        return ok;
    }

    SV_DEV static void hide(float (&x)[64], const uint2& see) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (!(see.x >> i & 1)) x[i] = kNegInf;
            if (!(see.y >> i & 1)) x[32 + i] = kNegInf;
        }
    }

    // O_w and l by a power of two, once the product of the half before (the
    // pv_count-th of this stream) is done: the one before that is, as its place
    // holds this half's scores.
    SV_DEV bool rescale(float f, float& l) {
        if (!warp_wait(&c->pv[w], (pv_count - 1) & 1, &c->abort)) return false;
        tc_fence_after();
        l *= f;
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
            float o[32];
            uint32_t r[32];
            tmem_ld32(tm_o + k, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(o[e] * f);
            tmem_st32(tm_o + k, r);
        }
        return true;
    }

    // A row's weights are 2^(s - ref) with a whole number for ref, at first the
    // maximum of the first positions that it sees, rounded up. Weights may
    // exceed 1: fp32 sums and bf16 weights scale without loss. ref is raised to
    // the running maximum m where a score of the half lies more than 8 octaves
    // above it, so a weight is 2^8 at the most, and sums stay in range for values
    // up to 2^119 / T (with weights to 2^64 before ref followed, values above 2^56
    // could overflow).
    //
    // One half: S -> P.
    SV_DEV bool softmax(int half, const uint2 see, bool tail, bool first, bool on, float c2, float& m, float& ref, float& l) {
        const uint32_t at = tm_s + 64 * half;
        float x[64], mx[4];
        tmem_ld64(at, x);
        if (tail) hide(x, see);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a = max3(x[16 * i], x[16 * i + 1], x[16 * i + 2]), b = max3(x[16 * i + 3], x[16 * i + 4], x[16 * i + 5]);
            a = max3(a, x[16 * i + 6], x[16 * i + 7]);
            b = max3(b, x[16 * i + 8], x[16 * i + 9]);
            a = max3(a, x[16 * i + 10], x[16 * i + 11]);
            b = max3(b, x[16 * i + 12], x[16 * i + 13]);
            mx[i] = max3(fmaxf(a, b), x[16 * i + 14], x[16 * i + 15]);
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
        if (ref == kNegInf) ref = ceilf(top);  // (nothing seen so far: all sums are zero)
        // (a lane without a row may hold anything)
        if (!first && __any_sync(0xFFFFFFFFu, on && top - kSlack > ref)) {
            const float to = fmaxf(ref, ceilf(fmaxf(m, top)));
            if (!rescale(ref == to ? 1.f : ex2(ref - to), l)) return false;
            ref = to;
        }
        m = fmaxf(m, top);
        const float r = ref == kNegInf ? 0.f : ref;
        const uint64_t cc = pack2(c2, c2), rr = pack2(-r, -r), keep = pack2(kKeep, kKeep);
        uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t parts[32];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float a, b, c, d;
                unpack2(fma2(pack2(x[32 * j + 2 * e], x[32 * j + 2 * e + 1]), cc, rr), &a, &b);
                a = ex2(a);
                b = ex2(b);
                const uint64_t w = pack2(a, b);
                sum[e & 3] = add2(sum[e & 3], w);
                const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
                parts[e] = __byte_perm(ua, ub, 0x7632);  // the upper halves
                const uint64_t upper = pack2(__uint_as_float((ua & 0xFFFF0000u) | 0x80000000u),
                                             __uint_as_float((ub & 0xFFFF0000u) | 0x80000000u));
                unpack2(fma2(w, keep, upper), &c, &d);
                parts[16 + e] = pack_bf16(c, d);
            }
            tmem_st32(at + 32 * j, parts);
        }
        float a, b;
        unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), &a, &b);
        l += a + b;
        tmem_wait_st();
        return true;
    }

    // A row's place in the result: bf16, or fp32 among the pieces.
    SV_DEV char* place(const Seg& s, int rr) {
        if (!s.whole) return reinterpret_cast<char*>(p.part_o + ((long long)s.slot * p.tile_rows + rr) * D);
        const int node = (s.row0 + rr) / p.G, g = (s.row0 + rr) - node * p.G;
        const long long row = ((long long)s.b * p.N + node) * (p.Hkv * p.G) + s.h * p.G + g;
        return SV_IN(row, (long long)p.B * p.N * p.Hkv * p.G) ? reinterpret_cast<char*>(p.out) + row * (D * 2) : nullptr;
    }
    // 32 columns of it.
    SV_DEV static void put(bool whole, char* dst, const float (&o)[32], float inv) {
        uint32_t x[32];
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (whole) x[k] = pack_bf16(o[2 * k] * inv, o[2 * k + 1] * inv);
            else {
                x[2 * k] = __float_as_uint(o[2 * k]);
                x[2 * k + 1] = __float_as_uint(o[2 * k + 1]);
            }
        st32(dst, x);
        st32(dst + 32, x + 8);
        if (whole) return;
        st32(dst + 64, x + 16);
        st32(dst + 96, x + 24);
    }
    SV_DEV void put_ml(const Seg& s, int rr, float m, float l) {
        if (!s.whole) {
            p.part_ml[(long long)s.slot * p.tile_rows + rr] = make_float2(m, l);
        } else if (p.lse) {
            const int node = (s.row0 + rr) / p.G, g = (s.row0 + rr) - node * p.G;
            p.lse[((long long)s.b * p.N + node) * (p.Hkv * p.G) + s.h * p.G + g] = lse_of(m, l);
        }
    }

    // A segment's result: each group its own rows, or group 0 both groups' sums.
    SV_DEV bool finish(const Seg& s, int slot, float m, float l) {
        const bool joined = !s.dual && s.steps > 1;
        const int half = p.tile_rows / 2, rr = s.dual ? half * w + t : t;
        const bool mine = t < half && rr < s.rows;
        const bool warp_on = warp * 32 < half && (s.dual ? half * w : 0) + warp * 32 < s.rows && s.steps > w;
        if (s.steps > w) {
            if (!warp_wait(&c->o_full[w], o_phase >> w & 1, &c->abort)) return false;
            o_phase ^= 1 << w;
        }
        if (joined && w == 0 && !warp_wait(&c->o_full[1], o_phase >> 1 & 1, &c->abort)) return false;
        if (w == 0 && s.steps > 1) o_phase ^= 2;  // a phase passed, waited for or not (the groups meet in between)
        tc_fence_after();
        if (!warp_on || (joined && w == 1)) return true;
        const int fl = *reinterpret_cast<volatile int*>(&c->flags[slot]);
        const int node = (s.row0 + min(rr, s.rows - 1)) / p.G;
        float w0 = 1.f, w1 = 0.f;
        if (joined) {
            const volatile float2* z = &c->ml[t];
            const float zm = z->x, zl = z->y;
            const float mn = fmaxf(m, zm), ref = mn == kNegInf ? 0.f : mn;
            w0 = ex2(m - ref);
            w1 = ex2(zm - ref);
            m = mn;
            l = l * w0 + zl * w1;
        }
        if (fl & 2) l = __uint_as_float(0x7FC00000u);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const bool whole = s.whole;
        char* dst = mine ? place(s, rr) : nullptr;
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
            float o[32];
            tmem_ld32(tm_o + k, o);
            if (joined) {
                float z[32];
                tmem_ld32(tm_o + 128 + k, z);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = o[e] * w0 + z[e] * w1;
            }
            if (dst) put(whole, dst + k * (whole ? 2 : 4), o, inv);
        }
        if (dst && fl & 1) add_unclean(p, s, node, dst, 0, D);
        if (mine) put_ml(s, rr, m, l);
        return true;
    }

    SV_DEV void run() {
        const float c2 = p.c2;
        uint32_t seg = 0;
        bool ok = true;
        while (const Seg* at = next_seg(c, seg, &ok)) {
            const Seg& s = *at;
            const int slot = seg & 3;
            // (group 0 has read the last segment's O_1)
            if (!(ok = meet())) break;

            float m = kNegInf, ref = kNegInf, l = 0.f;
            const int half = p.tile_rows / 2, rr = s.dual ? half * w + t : t;
            const bool warp_on = warp * 32 < half && (s.dual ? half * w : 0) + warp * 32 < s.rows;
            const bool on = t < half && rr < s.rows;
            const int node = (s.row0 + min(rr, s.rows - 1)) / p.G;
            const int halves = halves_of(s, w);
            // where a half begins, and the context ends, from the start of the stream's first tile
            const int step = s.dual ? kKv : 2 * kKv, reach = s.L - (s.first + (s.dual ? 0 : w)) * kKv;
#pragma unroll 1
            for (int u = 0; u < halves; ++u) {
                const int half = u & 1, off = kHalfKv * half + step * (u >> 1);
                const bool tail = off + kHalfKv > reach;
                uint2 see = make_uint2(0u, 0u);
                if (tail && warp_on) see = see_bits(p, s, node, (long long)s.L - reach + off);
                if (!(ok = warp_wait(&c->s_full[w][half], s_phase >> half & 1, &c->abort))) break;
                s_phase ^= 1u << half;
                tc_fence_after();
                if (warp_on && !(ok = softmax(half, see, tail, u == 0, on, c2, m, ref, l))) break;
                ++pv_count;
                if (w == 1 && u + 1 == halves) c->ml[t] = make_float2(ref, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c->p_full[w][half]);
            }
            if (!ok) break;
            __syncwarp();
            if (!(ok = finish(s, slot, ref, l))) break;
            tc_fence_before();
            ++seg;
        }
        if (!ok) c->abort = 1;
    }
};

template <int D>
__global__ void __launch_bounds__(NT, 1)
    attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mq) {
    extern __shared__ unsigned char dyn[];
    unsigned char* mem = dyn + ((1024 - (smem_u32(dyn) & 1023)) & 1023);
    Ctl* c = reinterpret_cast<Ctl*>(mem);
    const uint32_t qs = smem_u32(mem) + 2048, stages = qs + 2 * Shape<D>::kTile;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    asm volatile("griddepcontrol.launch_dependents;");
    const AttnCut cut = attn_locate<kKv, NT>(p, &c->scan);
    Walk walk(c->scan, cut);

    if (tid == 0) {
        for (int i = 0; i < Shape<D>::kStages; ++i) {
            mbar_init(&c->full[i], 1);
            mbar_init(&c->empty[i], 2);
            mbar_init(&c->clean[i], 1);
        }
        mbar_init(&c->q_full, 1);
        mbar_init(&c->q_empty, 2);
        for (int i = 0; i < 2; ++i) {
            for (int h = 0; h < 2; ++h) {
                mbar_init(&c->s_full[i][h], 1);
                mbar_init(&c->p_full[i][h], 4);
            }
            mbar_init(&c->pv[i], 1);
            mbar_init(&c->o_full[i], 1);
            mbar_init(&c->ask[i], 1);
            c->flags[2 * i] = c->flags[2 * i + 1] = 0;
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&c->seg_full[i], 1);
            c->seg[i].b = -1;
        }
        mbar_init(&c->groups, 8);
        mbar_init(&c->drain, 2);
        c->abort = 0;
        mbar_init_fence();
    }
    if (tid == 8 * 32) {
        tma_prefetch(&mk);
        tma_prefetch(&mv);
        tma_prefetch(&mq);
    }
    if (warp == 9) tmem_alloc512(&c->tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c->tmem;

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGroupRegs));
        const int w = warp >> 2, lanes = (warp & 3) * 32;
        Group<D> g{p, c, w, warp & 3, lane, tid & 127, tmem + ((uint32_t)lanes << 16) + 128 * w,
                   tmem + ((uint32_t)lanes << 16) + 256 + 128 * w};
        g.run();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) produce<D>(p, c, &mk, &mv, stages);
        if (warp == 10) {
            if (lane == 0) attn_join<kKv>(p, c->scan, cut);
            __syncwarp();
            attn_edges<bf16_t>(p, blockIdx.x, gridDim.x);
        }
        if (warp == 9 || warp == 10) {
            Issuer<D> is{c, uni(warp - 9), uni(tmem), qs, stages};
            is.run();
        }
        if (warp == 11) help<D>(p, c, &mq, qs, stages, walk);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (c->abort) {  // copies and products in flight end before the CTA does
        constexpr uint32_t NS = Shape<D>::kStages;
        if (tid == 8 * 32)
            for (uint32_t r = c->loads > NS ? c->loads - NS : 0; r < c->loads; ++r)
                tc_wait(&c->full[r % NS], (r / NS) & 1, nullptr);
        if (tid == 11 * 32 && c->asks) tc_wait(&c->q_full, (c->asks - 1) & 1, nullptr);
        if ((warp == 9 || warp == 10) && elected()) {  // (the lane that issued the products)
            mma_commit(&c->drain);
            tc_wait(&c->drain, 0, nullptr);
        }
        __syncthreads();
    }
    if (warp == 9) tmem_free512(tmem);
    if (tid < 4 && c->abort && p.status && c->seg[tid].b >= 0)  // a wait gave up: these segments are not whole
        atomicMax(p.status + c->seg[tid].b, kETimeout);
}

using Encode = decltype(&cuTensorMapEncodeTiled);
Encode encoder() {
    static const Encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
                cudaSuccess || found != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<Encode>(fn);
    }();
    return encode;
}

// A rank-4 bf16 tensor, copied in boxes of 64 elements x box1 x box2 with the
// 128-byte swizzle; strides in elements.
bool encode_map(CUtensorMap* map, const void* base, const cuuint64_t (&dims)[4], const long long (&strides)[3],
                cuuint32_t box1, cuuint32_t box2) {
    cuuint64_t st[3];
    for (int i = 0; i < 3; ++i) {
        // the stride of an index that only takes 0 may be anything that the encoding accepts
        st[i] = dims[i + 1] > 1 ? (cuuint64_t)strides[i] * 2 : 16;
        if (st[i] == 0 || st[i] % 16 != 0 || st[i] >= (1ull << 40)) return false;
    }
    const cuuint32_t box[4] = {64, box1, box2, 1}, step[4] = {1, 1, 1, 1};
    const Encode encode = encoder();
    auto make = [&] {
        return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, st, box, step,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    if (!encode) return false;
    CUresult r = make();
    // a thread that has not called the runtime yet has no context (without this,
    // its first call went to the CUDA cores)
    int dev = 0;
    if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = make();
    return r == CUDA_SUCCESS;
}

// k or v: boxes of (page_size, at most 128) slots of one head of one page.
bool make_map(CUtensorMap* map, const AttnParams& p, const void* base) {
    const int ps = 1 << p.page_shift;
    return encode_map(map, base, {(cuuint64_t)p.D, (cuuint64_t)ps, (cuuint64_t)p.Hkv, (cuuint64_t)p.num_pages},
                      {p.token_stride, p.head_stride, p.page_stride}, (cuuint32_t)std::min(ps, kKv), 1);
}

template <int D>
cudaError_t launch_tc(const AttnParams& p, const AttnPlan& plan, const CUtensorMap* maps, cudaStream_t st) {
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(attn_tc_kernel<D>), Shape<D>::kSmem);
    if (e != cudaSuccess) return e;
    attn_tc_kernel<D><<<plan.grid, NT, Shape<D>::kSmem, st>>>(p, maps[0], maps[1], maps[2]);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_attention_join(p, 1, plan, st);
}

}  // namespace

// What a unit's start and end cost, in tiles: more where both streams go over
// the same tiles. Measured with 2, 3 and 5 (alternate tiles): 16 trees of 64
// rows, 32 heads 89.0, 78.5, 81.5 us; 48 of 48 rows, 12 heads 70.2, 72.8, 77.8; 8
// of 100 rows, 16 heads of 64 columns 65.3, 53.2, 43.0; 200 single tokens, 4 x 6
// heads 112.9, 114.3, 116.9. With 4, 6 and 8 (same tiles): 16 trees of 512 rows
// 107.0, 109.3, 112.5; 10 of 450 rows 54.5, 55.8, 57.1; 3 of 600 rows, 64 columns
// 149, 151, 155; one of 4000 rows 168, 173, 175; 30 of 150 rows 31.5, 33.0, 34.6;
// one of 244 rows over 100003 positions 124 each.
int attention_tc_extra(int group, int N) { return N * group > attention_tc_rows(group) / 2 ? kExtraDual : kExtra; }

// Two halves of whole nodes, 128 rows at most each.
int attention_tc_rows(int group) { return 2 * (128 / group) * group; }
int attention_tc_kv() { return kKv; }
int attention_tc_whole() { return kWhole; }

bool attention_tc_maps(const AttnParams& p, AttnMaps* m) {
    static_assert(sizeof(AttnMaps) >= 3 * sizeof(CUtensorMap), "three maps");
    CUtensorMap* maps = reinterpret_cast<CUtensorMap*>(m);
    const long long Hq = (long long)p.Hkv * p.G;
    // queries: boxes of the nodes of a half, the heads of one group
    return make_map(maps, p, p.k) && make_map(maps + 1, p, p.v) &&
           encode_map(maps + 2, p.q, {(cuuint64_t)p.D, (cuuint64_t)Hq, (cuuint64_t)p.N, (cuuint64_t)p.B},
                      {p.D, Hq * p.D, p.N * Hq * p.D}, (cuuint32_t)p.G, (cuuint32_t)std::min(128 / p.G, p.N));
}

cudaError_t launch_attention_tc(const AttnParams& p, const AttnPlan& plan, const AttnMaps& m, cudaStream_t st) {
    const CUtensorMap* maps = reinterpret_cast<const CUtensorMap*>(&m);
    return p.D == 128 ? launch_tc<128>(p, plan, maps, st) : launch_tc<64>(p, plan, maps, st);
}

SV_DEBUG_READER(attention_tc)

}  // namespace sv

extern "C" int spec_debug_withhold_tile(int j) {
#ifdef SPEC_DEBUG
    return cudaMemcpyToSymbol(sv::g_withhold, &j, sizeof(int)) == cudaSuccess ? 0 : -1;
#else
    (void)j;
    return -1;
#endif
}
