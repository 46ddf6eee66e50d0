// attn_common.cuh -- what the multi-query attention kernels share (prompt
// attention and drafted-tree attention over the paged cache): the launch
// parameters, the division of the work among CTAs, the rule that says which
// keys a row sees, and the merge of split items.
//
// Rows.  The queries of a sequence that read one kv head are stacked
// token-major, head-minor: row r of a tile is token r / G of the tile and
// query head g * G + r % G.  One tile then holds ROWS / G consecutive tokens
// for all G query heads, every K and V row loaded serves G heads, and a
// causal tile of the scores is as narrow as the tokens it holds.
//
// Work.  An item is (query tile, kv head): its cost is the keys it has to
// visit plus a constant for its start and end.  Lengths are known on the
// device only, and a planning launch would cost small calls more than their
// work does, so every CTA sums the sequences' costs itself (closed forms,
// one block scan) and takes the b-th of gridDim.x equal intervals of the
// whole, walking sequence, tile, kv head.  An item that an interval's end
// cuts is split there; the parts' results are merged by the part that comes
// last.  Every CTA then has the same work up to one cut's rounding, a CTA
// leaves at most two partial results, and the cuts, hence the order of every
// sum, depend on the lengths alone.
#pragma once

#include <math.h>

#include "common.cuh"

namespace pkv {

struct AttnParams {
    void* out;
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* query_start;
    const int32_t* parents;  // tree attention: parent of each draft in its sequence, or -1; else null
    const float* k_scales;   // fp8 caches, else null
    const float* v_scales;
    int* counters;           // [gridDim.x][8] parts finished of the item whose first part the CTA owns (of all
                             // its rows, or of each warp's); zero between launches
    float2* ws_ml;           // [2 gridDim.x][part_rows] (maximum in log2 units, sum)
    float4* ws_o;            // [2 gridDim.x][D / 4][part_rows]: neighbouring rows side by side
    int* err;
    long long q_stride;      // elements between two tokens of q
    int num_seqs;
    int num_tokens;
    int num_heads;
    int num_kv_heads;
    int group_log2;          // log2(num_heads / num_kv_heads)
    int block_size;
    int max_blocks_per_seq;
    int num_blocks;
    int part_rows;           // rows of the largest tile of the call
    float qscale;            // scale * log2(e)
    unsigned long long wait_ns;
};

// ------------------------------------------------------------ the division
// ROWS: rows of a tile.  A key is LESS work for a tile of at most HALF rows
// and MORE for a larger one.  An item whose share of a CTA is at least COARSE
// keys is cut at multiples of FINE keys (balance), in smaller calls items are
// cut at multiples of COARSE only (a part shorter than that costs more in its
// merge than it saves).  ITEM: work of an item besides its keys.
template <int ROWS_, int HALF_, int LESS_, int MORE_, int FINE_, int COARSE_, int ITEM_>
struct AttnDivision {
    static constexpr int ROWS = ROWS_, HALF = HALF_, LESS = LESS_, MORE = MORE_, FINE = FINE_, COARSE = COARSE_,
                         ITEM = ITEM_;
    static_assert(COARSE % FINE == 0 && (FINE & (FINE - 1)) == 0 && (COARSE & (COARSE - 1)) == 0, "");
    static constexpr int FULL = ROWS > HALF ? MORE : LESS;  // work per key of a full tile
    __host__ __device__ static constexpr int per_key(int rows) { return rows > HALF ? MORE : LESS; }
};

// Sequence s of a launch: its rows, and what its tiles cost.
struct AttnSeq {
    int q0, n, first;  // first row, queries, position of the first query
    bool valid;        // false: no valid context; its rows are written as zeros

    __host__ __device__ __forceinline__ void load(const AttnParams& p, int s, bool report) {
        q0 = p.query_start[s];
        const int q1 = p.query_start[s + 1], ctx = p.context_lens[s];
        const bool rows_ok = q0 >= 0 && q1 >= q0 && q1 <= p.num_tokens;
        n = rows_ok ? q1 - q0 : 0;
        valid = rows_ok && ctx >= n && ctx <= (long long)p.max_blocks_per_seq * p.block_size;
        first = valid ? ctx - n : 0;
#ifdef __CUDA_ARCH__
        if (report && !valid) set_error(p.err, PKV_ERR_DEVICE_BOUNDS);
#endif
    }
    __host__ __device__ __forceinline__ int tiles(int tt) const { return (n + tt - 1) / tt; }
    // keys tile t visits: those up to its last query's own position
    __host__ __device__ __forceinline__ int keys(int t, int tt) const {
        if (!valid) return 0;
        const long long end = (long long)(t + 1) * tt;
        return first + (end < n ? (int)end : n);
    }
    // work per key of tile t
    template <class Div>
    __host__ __device__ __forceinline__ int per_key(int t, int tt, int group_log2) const {
        return Div::per_key((n - t * tt < tt ? n - t * tt : tt) << group_log2);
    }
    // work of the tiles before tile t, for one kv head
    template <class Div>
    __host__ __device__ __forceinline__ long long before(int t, int tt, int group_log2) const {
        const int last = tiles(tt) - 1;
        const int full = t <= last ? t : last;  // tiles that are surely full
        if (full < 0) return 0;
        long long c = (long long)full * Div::ITEM;
        if (valid) c += Div::FULL * ((long long)full * first + (long long)tt * full * (full + 1) / 2);
        if (t > last) c += (long long)keys(last, tt) * per_key<Div>(last, tt, group_log2) + Div::ITEM;
        return c;
    }
};

struct AttnItem {
    int seq;
    int row;       // row of q / out of the tile's first token
    int ntok;      // tokens in the tile
    int pos;       // absolute position of the tile's first token
    int first;     // position of the sequence's first query (tree: the committed tokens)
    int kv0, kv1;  // keys of this part
    int g;         // kv head
    int part, nparts;
    int keys;      // keys of the whole item
    int per_key;   // work of each
    long long at;  // start of the item in the launch's work
};

template <class Div>
struct AttnWalk {
    long long begin, end, at, share;
    int tt, s, t, g;
    AttnSeq q;

    // key at which a boundary `o` past the start of an item of K keys, f each, cuts it
    __host__ __device__ __forceinline__ static int cut(long long o, int K, int f, long long share) {
        if (o <= 0) return 0;
        if (o >= (long long)K * f) return K;
        // o passes 31 bits: up to 2^31 keys times f
        const int k = (int)(f == Div::MORE ? (unsigned long long)o / Div::MORE : (unsigned long long)o / Div::LESS);
        if (share >= Div::COARSE * f) return k & ~(Div::FINE - 1);
        const int most = K > Div::COARSE ? K - Div::COARSE : 0;  // no part shorter than COARSE
        return (k < most ? k : most) & ~(Div::COARSE - 1);
    }
    // CTA that owns part i of the item (at, K, f).  With a share of at least
    // COARSE keys every boundary but one short of FINE keys makes a cut; with a
    // smaller one every multiple of COARSE up to K - COARSE is cut, and a part
    // belongs to the last CTA that starts before the part's end.
    __host__ __device__ __forceinline__ static int owner(const AttnItem& it, long long share, int i) {
        const int b0 = (int)(it.at / share), f = it.per_key, K = it.keys;
        const long long o1 = (b0 + 1) * share - it.at;
        if (share >= Div::COARSE * f) return b0 + i + (o1 < Div::FINE * f && o1 < (long long)K * f ? 1 : 0);
        const long long e = i + 1 < parts(it, share) ? (long long)(i + 1) * Div::COARSE * f : (long long)K * f;
        return b0 + (int)((it.at - b0 * share + e - 1) / share);
    }
    __host__ __device__ __forceinline__ static int parts(const AttnItem& it, long long share) {
        const int f = it.per_key, K = it.keys;
        if (share >= Div::COARSE * f) {
            const long long o1 = (it.at / share + 1) * share - it.at, all = (long long)K * f;
            if (o1 >= all) return 1;
            return (o1 >= Div::FINE * f ? 2 : 1) + (int)((all - 1 - o1) / share);
        }
        return K < Div::COARSE ? 1 : K / Div::COARSE;
    }

    // The next item with work for CTA `cta`.
    __host__ __device__ bool next(const AttnParams& p, int cta, AttnItem& it) {
        while (at < end) {
            const int K = q.keys(t, tt), f = q.template per_key<Div>(t, tt, p.group_log2);
            const long long c = (long long)K * f + Div::ITEM, a = begin - at;
            const int k0 = cut(a, K, f, share);
            const int k1 = at + c <= end ? K : cut(end - at, K, f, share);
            const bool mine = K == 0 ? a <= 0 : k0 < k1;
            if (mine) {
                it.seq = s;
                it.row = q.q0 + t * tt;
                it.ntok = q.n - t * tt < tt ? q.n - t * tt : tt;
                it.first = q.first;
                it.pos = q.first + t * tt;
                it.kv0 = k0;
                it.kv1 = k1;
                it.g = g;
                it.keys = K;
                it.per_key = f;
                it.at = at;
                it.nparts = 1;
                it.part = 0;
                if (k0 > 0 || k1 < K) {
                    it.nparts = parts(it, share);
                    // with large shares the parts' owners follow one another
                    it.part = share >= Div::COARSE * f ? cta - owner(it, share, 0) : k0 / Div::COARSE;
                }
            }
            at += c;
            if (++g == p.num_kv_heads) {
                g = 0;
                if (++t >= q.tiles(tt)) {
                    t = 0;
                    while (++s < p.num_seqs) {
                        q.load(p, s, false);
                        if (q.n > 0) break;
                    }
                    if (s >= p.num_seqs) at = end;
                }
            }
            if (mine) return true;
        }
        return false;
    }
};

// The item of a sequence that the work `o` past the sequence's start falls in:
// tile, kv head and the item's own start.
template <class Div>
__host__ __device__ __forceinline__ void attn_place(const AttnSeq& q, int tt, int group_log2, int kv_heads, long long o,
                                                    int& tile, int& g, long long& at) {
    int lo = 0, hi = q.tiles(tt) - 1;  // the last tile that starts at or before o
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (q.before<Div>(mid, tt, group_log2) * kv_heads <= o) lo = mid; else hi = mid - 1;
    }
    const long long start = q.before<Div>(lo, tt, group_log2) * kv_heads;
    const long long each_head = (long long)q.keys(lo, tt) * q.per_key<Div>(lo, tt, group_log2) + Div::ITEM;
    tile = lo;
    g = (int)((o - start) / each_head);
    at = start + g * each_head;
}

// All NT threads of a CTA: sum the costs and place the walk at the CTA's
// share.  `scratch` holds NT / 32 + 8 long longs of shared memory; the walk
// that the threads get is the same for all.  Ends with a barrier.
template <class Div, int NT>
__device__ __forceinline__ AttnWalk<Div> attn_walk_start(const AttnParams& p, long long* scratch) {
    constexpr int NW = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    AttnWalk<Div> w;
    w.tt = Div::ROWS >> p.group_log2;
    const int each = (p.num_seqs + NT - 1) / NT;
    const int s0 = tid * each < p.num_seqs ? tid * each : p.num_seqs;
    const int s1 = s0 + each < p.num_seqs ? s0 + each : p.num_seqs;
    long long mine = 0;
    for (int s = s0; s < s1; ++s) {
        AttnSeq q;
        q.load(p, s, blockIdx.x == 0);
        mine += q.before<Div>(q.tiles(w.tt), w.tt, p.group_log2) * p.num_kv_heads;
    }
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 31) scratch[warp] = incl;
    if (tid == 0) scratch[NW + 1] = -1;
    __syncthreads();
    long long pre = incl - mine, total = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        if (i < warp) pre += scratch[i];
        total += scratch[i];
    }
    long long share = (total + gridDim.x - 1) / gridDim.x;
    if (share < 1) share = 1;
    w.share = share;
    w.begin = share * blockIdx.x;
    w.end = w.begin + share < total ? w.begin + share : total;
    if (w.begin < total && pre <= w.begin && w.begin < pre + mine) {
        for (int s = s0; s < s1; ++s) {
            AttnSeq q;
            q.load(p, s, false);
            const long long c = q.before<Div>(q.tiles(w.tt), w.tt, p.group_log2) * p.num_kv_heads;
            if (w.begin < pre + c) {
                int tile, g;
                long long at;
                attn_place<Div>(q, w.tt, p.group_log2, p.num_kv_heads, w.begin - pre, tile, g, at);
                scratch[NW + 1] = s;
                scratch[NW + 2] = tile;
                scratch[NW + 3] = g;
                scratch[NW + 4] = pre + at;
                scratch[NW + 5] = q.q0;
                scratch[NW + 6] = q.n;
                scratch[NW + 7] = q.valid ? q.first : -1;
                break;
            }
            pre += c;
        }
    }
    __syncthreads();
    w.s = (int)scratch[NW + 1];
    if (w.s < 0) {
        w.at = w.end = w.begin;  // nothing to do
        w.s = w.t = w.g = 0;
        return w;
    }
    w.t = (int)scratch[NW + 2];
    w.g = (int)scratch[NW + 3];
    w.at = scratch[NW + 4];
    w.q.q0 = (int)scratch[NW + 5];
    w.q.n = (int)scratch[NW + 6];
    w.q.valid = scratch[NW + 7] >= 0;
    w.q.first = w.q.valid ? (int)scratch[NW + 7] : 0;
    return w;
}

// The same start on the host, for CTA `cta` of `grid`; p's arrays are host ones.
template <class Div>
inline AttnWalk<Div> attn_walk_start_host(const AttnParams& p, int cta, int grid) {
    AttnWalk<Div> w;
    w.tt = Div::ROWS >> p.group_log2;
    long long total = 0;
    for (int s = 0; s < p.num_seqs; ++s) {
        AttnSeq q;
        q.load(p, s, false);
        total += q.before<Div>(q.tiles(w.tt), w.tt, p.group_log2) * p.num_kv_heads;
    }
    w.share = (total + grid - 1) / grid;
    if (w.share < 1) w.share = 1;
    w.begin = w.share * cta;
    w.end = w.begin + w.share < total ? w.begin + w.share : total;
    long long pre = 0;
    for (int s = 0; s < p.num_seqs; ++s) {
        w.q.load(p, s, false);
        const long long c = w.q.template before<Div>(w.q.tiles(w.tt), w.tt, p.group_log2) * p.num_kv_heads;
        if (w.begin < pre + c) {
            w.s = s;
            attn_place<Div>(w.q, w.tt, p.group_log2, p.num_kv_heads, w.begin - pre, w.t, w.g, w.at);
            w.at += pre;
            return w;
        }
        pre += c;
    }
    w.at = w.end = w.begin;  // nothing to do
    w.s = w.t = w.g = 0;
    return w;
}

// ------------------------------------------------------------------- masks
// Whether the query at index `i` of its sequence (position first + i) sees
// key position `key`: the keys up to its own position, or, with a tree, the
// committed tokens (key < first), itself and its ancestors.  The walk goes
// from parent to parent while the index stays above the key's; a parent that
// is not smaller than its child ends it (and is reported, attn_check_parents).
__device__ __forceinline__ bool sees(const int32_t* parents_of_seq, int first, int i, int key) {
    if (parents_of_seq == nullptr) return key <= first + i;
    const int d = key - first;
    if (d < 0) return true;
    while (i > d) {
        const int up = parents_of_seq[i];
        if (up >= i) return false;
        i = up;
    }
    return i == d;
}

// A draft's parent is -1 or comes before it in its sequence.
__device__ __forceinline__ void attn_check_parents(const AttnParams& p, const AttnItem& it, int tid, int nt) {
    for (int i = tid; i < it.ntok; i += nt) {
        const int up = p.parents[it.row + i];
        if (up < -1 || up >= it.pos - it.first + i) set_error(p.err, PKV_ERR_DEVICE_BOUNDS);
    }
}

// ------------------------------------------------------------------- merge
// Partial result of part i of an item that CTA b owns: a CTA's first item may
// go on from the CTA before (part > 0), its last may go on in the next.
__host__ __device__ __forceinline__ int attn_partial(int b, int part) { return 2 * b + (part == 0 ? 1 : 0); }
// Place in ws_o of dims d .. d + 3 of a partial result's row.
__device__ __forceinline__ long long attn_partial_at(const AttnParams& p, int partial, int D, int d, int row) {
    return ((long long)partial * (D / 4) + d / 4) * p.part_rows + row;
}

// End of one part of a split item, called by NT threads (tid, sync() a
// barrier over them) once they have written the part's rows to ws_o / ws_ml.
// The last part to arrive merges all of them in their order,
//     M = max m_i,  out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,
// so the result does not depend on which part came last, and zeroes the
// counter for the next launch.  `turns` counts the parts this CTA has
// reported.  False when a barrier gave up.
template <class Div, typename T, int D, int NT, class Sync>
__device__ __forceinline__ bool attn_merge(const AttnParams& p, const AttnItem& it, long long share, int* flag,
                                           int* turns, int tid, Sync&& sync) {
    using Walk = AttnWalk<Div>;
    const int G = 1 << p.group_log2;
    const int rows = it.ntok << p.group_log2;
    __threadfence();
    if (!sync()) return false;
    if (tid == 0) {
        int* count = p.counters + Walk::owner(it, share, 0) * 8;
        const int last = atomicAdd(count, 1) == it.nparts - 1;
        if (last) *count = 0;
        *flag = last;
        *turns += 1;
    }
    if (!sync()) return false;
    if (!*flag) return true;
    __threadfence();
    // a thread takes 16 dims of a row; threads side by side take neighbouring rows
    const int units = rows * (D / 16);
    for (int unit = tid; unit < units; unit += NT) {
        const int c = unit / rows, r = unit - c * rows;
        float M = -INFINITY, L = 0.f, acc[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = 0.f;
        for (int i0 = 0; i0 < it.nparts; i0 += 2) {
            float2 ml[2];
            float4 v[2][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int i = i0 + b;
                ml[b] = make_float2(-INFINITY, 0.f);
                if (i < it.nparts) {
                    const int slot = attn_partial(Walk::owner(it, share, i), i);
                    ml[b] = __ldcg(&p.ws_ml[(long long)slot * p.part_rows + r]);
                    const float4* o = p.ws_o + attn_partial_at(p, slot, D, 16 * c, r);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[b][e] = __ldcg(o + e * (long long)p.part_rows);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[b][e] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            const float Mn = fmaxf(M, fmaxf(ml[0].x, ml[1].x));
            // no key seen in any part so far: the sums are 0 (or NaN), taken as they are
            const bool none = Mn == -INFINITY;
            const float a = none ? 1.f : exp2f(M - Mn);
            M = Mn;
            L *= a;
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] *= a;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float w = none ? 1.f : exp2f(ml[b].x - Mn);
                L = fmaf(w, ml[b].y, L);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[4 * e] = fmaf(w, v[b][e].x, acc[4 * e]);
                    acc[4 * e + 1] = fmaf(w, v[b][e].y, acc[4 * e + 1]);
                    acc[4 * e + 2] = fmaf(w, v[b][e].z, acc[4 * e + 2]);
                    acc[4 * e + 3] = fmaf(w, v[b][e].w, acc[4 * e + 3]);
                }
            }
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;  // no key seen: a zero row
        T* dst = static_cast<T*>(p.out) +
                 ((long long)(it.row + (r >> p.group_log2)) * p.num_heads + it.g * G + (r & (G - 1))) * D + 16 * c;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[8 * h + 2 * e] * inv, acc[8 * h + 2 * e + 1] * inv);
                    w[e] = *reinterpret_cast<const uint32_t*>(&b);
                }
                reinterpret_cast<uint4*>(dst)[h] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                reinterpret_cast<float4*>(dst)[e] = make_float4(acc[4 * e] * inv, acc[4 * e + 1] * inv,
                                                                acc[4 * e + 2] * inv, acc[4 * e + 3] * inv);
        }
    }
    return true;
}

}  // namespace pkv
