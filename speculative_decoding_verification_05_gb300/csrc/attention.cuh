// Shared parts of the tree-attention kernels: parameters, the division of the
// work over the CTAs, and the record layout of partial results.
//
// One step's drafted nodes (N per sequence, node 0 the last context token)
// attend to their sequence's committed context and to their ancestors:
//   o_i = sum_t p_it v_t,  p_it = exp(s_it - lse_i),  s_it = scale q_i . k_t,
//   lse_i = log sum_t exp(s_it),
// t over the positions < L = cache_len[b] and the nodes' positions L + j with
// mask[i][j] = 1 (no mask: j <= i). The rows of one key / value head are its
// nodes' query heads, row r = node r / G, head r % G of the group of G that
// shares it, so a key is read once for all of them.
//
// Division. A unit is (sequence, key / value head, row tile); its tiles are
// the kKv-position tiles of L + n positions. All units' tiles in order form
// one range that is cut into equal parts, one a CTA, whatever the lengths
// are (they are known on the device only). In the range a unit counts a few
// tiles more than it has (`extra`, before its tiles), for what its start and end
// cost; a cut that falls among these is moved to the unit's start. A unit inside one part is finished
// by its CTA; the others leave partial results (unnormalised sums with their
// running maximum and sum) that the join kernel adds up in range order, so
// results depend on the lengths and the grid alone, never on timing. Where there
// are no more units than parts and a sequence can only have a few tiles (the
// page table's width), a unit is one part's: nothing is left to join then.
#pragma once

#include "common.cuh"

namespace sv {

// A unit that several CTAs' parts share, written by the second of them.
struct AttnJoin {
    int b, h, row0, rows;  // rows = 0: nothing to join here
    int slot0;             // the first piece's slot; the others' are 2 * part
    int first, last;       // parts of the other pieces
    int pad;
};

struct AttnParams {
    const void* q;    // [B, N, Hkv * G, D]
    const void* k;    // page p, slot s, head h at p * page_stride + s * token_stride + h * head_stride
    const void* v;
    long long page_stride, token_stride, head_stride;  // elements
    const int32_t* table;  // [B] rows of table_stride entries
    long long table_stride;
    const int32_t* cache_len;  // [B]
    const uint8_t* mask;       // [B, N, N] or null (j <= i)
    const int32_t* n_nodes;    // [B] or null (N)
    int B, N, Hkv, G, D, num_pages, max_pages, page_shift;
    int tile_rows;       // rows of a row tile
    int extra;           // tiles that a unit's start and end count for
    int whole;           // a unit is its first part's, all of it
    float c2;            // scale * log2(e): scores in octaves
    void* out;           // [B, N, Hkv * G, D]
    float* lse;          // [B, N, Hkv * G] or null
    int32_t* status;     // [B] or null
    float* part_o;       // [2 * grid][rows of a tile][D] partial sums
    float2* part_ml;     // [2 * grid][rows of a tile] running maximum (octaves) and sum
    AttnJoin* joins;     // [grid] the units to join
};

// A sequence's nodes and context; n = -1: bad data.
struct AttnSeq {
    int n, L;
};

SV_DEV AttnSeq attn_seq(const AttnParams& p, int b) {
    AttnSeq s;
    s.L = __ldg(p.cache_len + b);
    s.n = p.n_nodes ? __ldg(p.n_nodes + b) : p.N;
    if (s.L < 0 || s.n < 0 || s.n > p.N || (long long)s.L + s.n > ((long long)p.max_pages << p.page_shift)) s.n = -1;
    return s;
}

template <int KV>
SV_DEV int attn_kv_tiles(const AttnSeq& s) {
    return s.n > 0 ? (int)(((long long)s.L + s.n + KV - 1) / KV) : 0;
}

SV_DEV int attn_row_tiles(const AttnParams& p, const AttnSeq& s) {
    return s.n > 0 ? (s.n * p.G + p.tile_rows - 1) / p.tile_rows : 0;
}

template <int KV>
SV_DEV long long attn_seq_work(const AttnParams& p, int b) {
    const AttnSeq s = attn_seq(p, b);
    return s.n > 0 ? (long long)(attn_kv_tiles<KV>(s) + p.extra) * attn_row_tiles(p, s) * p.Hkv : 0;
}

// Where tile `at` of the whole range lies: its sequence and that sequence's
// first tile in the range; total: all tiles.
struct AttnPlace {
    int b;
    long long base;
};

// Scratch of attn_locate in shared memory.
struct AttnScan {
    long long warp_sum[32];
    AttnPlace place;
};

// The range cut into parts, one a CTA (the first `extra` one tile longer).
struct AttnCut {
    long long each;
    int extra, parts;
    SV_DEV long long at(int c) const { return each * c + min(c, extra); }
};

// Called by all NT threads of a block: the cut range, and in sc->place where
// this CTA's part begins (if it has one). Each thread sums a run of sequences,
// one scan orders the runs.
template <int KV, int NT>
SV_DEV AttnCut attn_locate(const AttnParams& p, AttnScan* sc) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int run = (p.B + NT - 1) / NT;
    const int b0 = min(tid * run, p.B), b1 = min(b0 + run, p.B);
    long long mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += attn_seq_work<KV>(p, b);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) sc->warp_sum[warp] = inc;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const long long u = sc->warp_sum[w];
        if (w < warp) before += u;
        total += u;
    }
    long long lo = before + inc - mine;
    AttnCut cut;
    cut.parts = (int)min(total, (long long)gridDim.x);
    cut.each = cut.parts ? total / cut.parts : 0;
    cut.extra = (int)(total - cut.each * cut.parts);
    const long long at = (int)blockIdx.x < cut.parts ? cut.at(blockIdx.x) : -1;
    if (at >= lo && at < lo + mine) {
        long long base = lo;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const long long w = attn_seq_work<KV>(p, b);
            if (at < base + w) {
                sc->place = AttnPlace{b, base};
                break;
            }
            base += w;
        }
    }
    __syncthreads();
    return cut;
}

// One CTA's stay in a unit: tiles [first, last) of its kt.
struct AttnStay {
    int b, h, row0, rows, first, last, kt, L, n, slot;
    long long len;
    bool whole;
};

// Walks this CTA's part of the range.
template <int KV>
struct AttnWalk {
    long long t, end, base;
    int b, stays;
    SV_DEV AttnWalk(const AttnScan& sc, const AttnCut& cut) : t(0), end(0), base(0), b(0), stays(0) {
        if ((int)blockIdx.x >= cut.parts) return;
        t = cut.at(blockIdx.x);
        end = cut.at(blockIdx.x + 1);
        base = sc.place.base;
        b = sc.place.b;
    }

    // (a sequence's own part of the range is below 2^31)
    SV_DEV bool next(const AttnParams& p, AttnStay* s) {
#pragma unroll 1
        while (t < end) {
            AttnSeq q = attn_seq(p, b);
            int kt = attn_kv_tiles<KV>(q), rt = attn_row_tiles(p, q);
#pragma unroll 1
            while (q.n <= 0 || t >= base + (long long)(kt + p.extra) * rt * p.Hkv) {
                if (q.n > 0) base += (long long)(kt + p.extra) * rt * p.Hkv;
                q = attn_seq(p, ++b);
                kt = attn_kv_tiles<KV>(q);
                rt = attn_row_tiles(p, q);
            }
            const uint32_t in = (uint32_t)(t - base), unit = in / (uint32_t)(kt + p.extra);
            const int from = (int)(in - unit * (uint32_t)(kt + p.extra));
            const int to = (int)min((long long)(kt + p.extra), from + (end - t));
            t += to - from;
            s->first = p.whole ? 0 : max(0, from - p.extra);
            s->last = p.whole ? (from == 0 ? kt : 0) : max(0, to - p.extra);
            if (s->first == s->last) continue;
            s->b = b;
            s->kt = kt;
            s->h = (int)(unit / (uint32_t)rt);
            s->row0 = (int)(unit - (uint32_t)s->h * rt) * p.tile_rows;
            s->rows = min(p.tile_rows, q.n * p.G - s->row0);
            s->L = q.L;
            s->n = q.n;
            s->len = (long long)q.L + q.n;
            s->whole = s->first == 0 && s->last == kt;
            s->slot = 2 * blockIdx.x + (stays > 0);
            ++stays;
            return true;
        }
        return false;
    }
};

// This CTA's entry of p.joins (one thread): its part begins inside a unit that
// the part before it has the first piece of.
template <int KV>
SV_DEV void attn_join(const AttnParams& p, const AttnScan& sc, const AttnCut& cut) {
    AttnJoin j = {};
    const int c = blockIdx.x;
    if (c > 0 && c < cut.parts) {
        const AttnSeq q = attn_seq(p, sc.place.b);
        const int kt = attn_kv_tiles<KV>(q), rt = attn_row_tiles(p, q);
        const long long at = cut.at(c), before = cut.at(c - 1);
        const uint32_t unit = (uint32_t)(at - sc.place.base) / (uint32_t)(kt + p.extra);
        const long long start = sc.place.base + (long long)unit * (kt + p.extra), stop = start + kt + p.extra;
        if (at > start + p.extra && before <= start + p.extra) {
            j.b = sc.place.b;
            j.h = (int)(unit / (uint32_t)rt);
            j.row0 = (int)(unit - (uint32_t)j.h * rt) * p.tile_rows;
            j.rows = min(p.tile_rows, q.n * p.G - j.row0);
            j.slot0 = 2 * (c - 1) + (before < start);
            j.first = j.last = c;
#pragma unroll 1
            while (j.last + 1 < cut.parts && cut.at(j.last + 1) < stop) ++j.last;
        }
    }
    p.joins[c] = j;
}

// The sequences' own checks and edges, shared out over `warps` warps of the
// grid (this is warp `gw`; as many warps a sequence as there are): status, and
// the rows that no unit writes, zeros (lse -inf) from the node count on and NaN
// everywhere for a sequence with bad data. A bad page id is reported here; the
// units that meet it make their rows NaN.
template <typename E>
SV_DEV void attn_edges(const AttnParams& p, int gw, int warps) {
    const int lane = threadIdx.x & 31, team = max(1, warps / p.B), member = gw % team;
#pragma unroll 1
    for (int b = gw / team; b < p.B; b += (warps + team - 1) / team) {
        const AttnSeq s = attn_seq(p, b);
        if (p.status && member == 0) {
            bool bad = s.n < 0;
            if (s.n > 0) {
                const int pages = (int)(((long long)s.L + s.n + (1 << p.page_shift) - 1) >> p.page_shift);
#pragma unroll 1
                for (int i = lane; i < pages; i += 32) {
                    const int id = __ldg(p.table + b * p.table_stride + i);
                    bad |= id < 0 || id >= p.num_pages;
                }
            }
            bad = __any_sync(0xFFFFFFFFu, bad) != 0;
            if (lane == 0) p.status[b] = bad ? kEData : kOk;
        }
        const int Hq = p.Hkv * p.G, n = max(s.n, 0);
        const long long row0 = ((long long)b * p.N + n) * Hq, rows = (long long)(p.N - n) * Hq;
        const long long words = rows * p.D * (long long)sizeof(E) / 16;
        const uint32_t fill = s.n < 0 ? (sizeof(E) == 4 ? 0x7FC00000u : 0x7FC07FC0u) : 0u;
        uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<E*>(p.out) + row0 * p.D);
#pragma unroll 1
        for (long long i = member * 32 + lane; i < words; i += team * 32) o[i] = make_uint4(fill, fill, fill, fill);
        if (p.lse)
#pragma unroll 1
            for (long long i = member * 32 + lane; i < rows; i += team * 32)
                p.lse[row0 + i] = __uint_as_float(s.n < 0 ? 0x7FC00000u : 0xFF800000u);
    }
}

SV_DEV float lse_of(float m2, float l) {
    return l > 0.f ? (m2 + log2f(l)) * 0.6931471805599453f : (l == 0.f ? __uint_as_float(0xFF800000u) : l + m2);
}

// Two floats as one operand of the packed instructions.
SV_DEV uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
SV_DEV void unpack2(uint64_t r, float* x, float* y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*x), "=f"(*y) : "l"(r)); }
SV_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

template <typename E>
SV_DEV void store4(E* dst, float4 x);
template <>
SV_DEV void store4<float>(float* dst, float4 x) {
    *reinterpret_cast<float4*>(dst) = x;
}
SV_DEV uint32_t pack_bf16(float lo, float hi) {  // round to nearest even
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
SV_DEV void store4<bf16_t>(bf16_t* dst, float4 x) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}

// Host side.
struct AttnPlan {
    int grid, rows, kv;   // CTAs of the main kernel, rows of a tile, positions of a tile
    int extra, whole;     // AttnParams::extra, whole
    size_t part_o, part_ml, joins, total;  // workspace layout
};

// Lets a kernel have its most dynamic shared memory, the same for every call
// (set once a device: it takes about a microsecond).
cudaError_t allow_smem(const void* kernel, size_t most);
cudaError_t launch_attention_simt(const AttnParams& p, int dtype, const AttnPlan& plan, cudaStream_t st);
bool attention_simt_many(int rows, int D);
int attention_simt_rows(bool many);
int attention_simt_kv(int dtype, int D, bool many);
int attention_simt_ctas(int dtype, int D, bool many);
int attention_simt_extra();
int attention_simt_whole();
// The tensor-core kernel (bf16, D 64 or 128) reads K, V and Q through tensor
// maps; attention_tc_maps: false where the cache's strides have none.
struct alignas(64) AttnMaps {
    unsigned char bytes[384];
};
int attention_tc_rows(int group);
int attention_tc_kv();
int attention_tc_extra(int group, int N);
int attention_tc_whole();
bool attention_tc_maps(const AttnParams& p, AttnMaps* m);
cudaError_t launch_attention_tc(const AttnParams& p, const AttnPlan& plan, const AttnMaps& m, cudaStream_t st);
cudaError_t launch_attention_join(const AttnParams& p, int dtype, const AttnPlan& plan, cudaStream_t st);
cudaError_t debug_read_attention_tc(unsigned int* count, unsigned int* line);
cudaError_t debug_read_attention(unsigned int* count, unsigned int* line);

}  // namespace sv
