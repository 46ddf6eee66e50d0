// attn_tc.cuh -- multi-query attention over the paged cache on the tensor
// cores (tcgen05 + TMEM): prompt attention and drafted-tree attention over
// bf16 and fp8 caches, head_dim 64 and 128.
//
//   out_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = 2^(x_rj - m_r),  x = scale log2(e) q . k
// in one pass over the keys, 128 at a time, with the running maximum m and sum
// of a softmax in fp32.
//
// One CTA per SM walks its share of the items (attn_common.cuh): up to 256
// rows of one kv head, as two pipelines of 128 rows that share every K and V
// tile.  An item of at most 128 rows runs its even steps on one pipeline and
// its odd steps on the other and adds the two at its end, so that both are busy
// either way.  Each pipeline alternates
//     S = Q K^T (128 x 128, both operands in shared memory, S in TMEM),
//     softmax (one warpgroup, one row per thread: TMEM -> registers -> P in
//              TMEM, over the columns of S it came from),
//     O += P V (P from TMEM, V from shared memory, O in TMEM),
// and while one is in its softmax the tensor cores work for the other.  O
// stays in TMEM for the whole item: it is scaled down only when a row's
// maximum has grown by more than 2^8 since the last time (a stale maximum
// cancels in the quotient; P stays below 2^8), which after the first steps
// hardly ever happens.
//
// Warps: 0-3 and 4-7 softmax, 8 producer (TMA: one 5-D copy brings a whole
// block of K or V in the layout the MMA wants), 9 MMA issue, 10 the walk;
// fp8 caches: 12-15 widen each K and V tile to f16.  e4m3 values are exact in
// f16, q is scaled per row by a power of two so that its bf16 values fit f16
// (exact for all within 2^31 of the row's largest), and P is rounded to f16.
//
// Rounding: P to bf16 (f16 over fp8 caches) before the product with V, as the
// tensor cores take it; sums, maxima and O are fp32.
//
// A masked key's weight is 0, and 0 * inf or 0 * nan would reach the row all
// the same: rows whose result is not finite are computed again, key by key,
// from the keys they see (slow_row).  Every wait is bounded.
#pragma once

#include <cuda.h>

#include "attn_common.cuh"
#include "decode_tc.cuh"

namespace pkv {
namespace atc {

using tc::fence_proxy_async_smem;
using tc::sw128_desc;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tma_load_5d;

using TcDivision = AttnDivision<256, 128, 512, 192>;

// ------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
        : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}

// 16-bit MMAs with fp32 accumulators, by the lane with `one`: the whole warp
// comes here with the same operands, which then stay in uniform registers (one
// lane alone in a branch took 70 to 120 clocks for each instruction's
// operands, longer than the 64 that the product itself takes).
// D[tmem] (+)= A[smem desc] . B[smem desc]
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
// D[tmem] (+)= A[tmem] . B[smem desc]
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
// Arrive on `bar` when every MMA of the electing lane so far has completed.
__device__ __forceinline__ void commit_one(uint64_t* bar, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
        "r"(one)
        : "memory");
}

// 32 consecutive fp32 columns of this thread's TMEM lane (no wait).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int REGS>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// 2^x, within 2^-22 relative; 2^-inf = 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---------------------------------------------------------------- geometry
template <int D_, bool FP8_>
struct Cfg {
    static constexpr int D = D_;
    static constexpr bool FP8 = FP8_;
    static constexpr int KEYS = 128;                // per step
    static constexpr int HALVES = D / 64;           // 128-byte spans of a row
    static constexpr int TILE = KEYS * D * 2;       // one 16-bit K or V tile
    static constexpr int GSTRIDE = HALVES * 1024;   // 8 rows of it: [half][8][64]
    static constexpr int HSTEP = 1024;
    static constexpr int QHALF = 128 * 128;         // 128 rows of one span of Q
    static constexpr int QTILE = HALVES * QHALF;
    static constexpr int RAW = KEYS * D;            // one fp8 tile
    // slots of 16-bit tiles (fp8: the widened ones) and of raw fp8 tiles: what
    // 227 KB hold next to two tiles of Q
    static constexpr int NSLOT = FP8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 10);
    static constexpr int NRAW = FP8 ? (D == 128 ? 4 : 8) : 0;
    static constexpr int NLOAD = FP8 ? NRAW : NSLOT;  // slots that TMA fills
    static constexpr int THREADS = FP8 ? 512 : 384;
    static constexpr int ITEMS = 4;                 // items the walk is ahead
    // registers: what the launch gives all threads, and its split among roles
    static constexpr int REGS_SOFTMAX = FP8 ? 176 : 216;
    static constexpr int REGS_ISSUE = FP8 ? 64 : 72;
    static constexpr int REGS_WIDEN = 96;
    static constexpr int REGS_LAUNCH = 65536 / THREADS / 8 * 8;
    static_assert(256 * REGS_SOFTMAX + 128 * REGS_ISSUE + (FP8 ? 128 * REGS_WIDEN : 0) <= THREADS * REGS_LAUNCH,
                  "the roles' registers come out of the launch's");
    // P is held 2^SHIFT times larger where it is f16, whose smallest step is 2^-24: its
    // largest value then stays below 2^15, and a weight loses less than 2^-32 of the largest
    static constexpr float SHIFT = FP8 ? 7.f : 0.f;
    static constexpr uint32_t TMEM_COLS = 512;      // S / P of both pipelines, then O of both
    static constexpr uint32_t O_COL = 256;
    static constexpr uint32_t FORMAT = FP8 ? 0u : 1u;  // f16 or bf16
    static constexpr uint32_t IDESC_QK = tc::idesc_make(128, 128, FORMAT, false, false);
    static constexpr uint32_t IDESC_PV = tc::idesc_make(128, D, FORMAT, false, true);

    static constexpr int Q_OFF = 0;
    static constexpr int SLOT_OFF = 2 * QTILE;
    static constexpr int RAW_OFF = SLOT_OFF + NSLOT * TILE;
    static constexpr int BAR_OFF = RAW_OFF + NRAW * RAW;
    // full/empty of the load ring, of the widened ring, q_full q_empty q_wide,
    // s_full[2] p_full[2] o_full[2], x_full x_empty, item full/empty, sync, mma_done
    static constexpr int NBARS = 2 * NLOAD + (FP8 ? 2 * NSLOT : 0) + 3 + 6 + 2 + 2 * ITEMS + 2;
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;  // tmem address, abort, flag, turns
    static constexpr int ITEM_OFF = (MISC_OFF + 16 + 15) / 16 * 16;
    static constexpr int WALK_OFF = ITEM_OFF + ITEMS * 64;
    static constexpr int ML_OFF = WALK_OFF + (THREADS / 32 + 8) * 8;  // float2[128]
    static constexpr int QS_OFF = ML_OFF + 128 * 8;                    // 256 exponents, fp8
    static constexpr int SMEM_BYTES = QS_OFF + (FP8 ? 256 : 0) + 1024;
    static_assert(SMEM_BYTES <= 232448, "227 KB of shared memory");
    static_assert(sizeof(AttnItem) <= 64, "");
};

// What an item asks of the two pipelines.
struct Plan {
    bool wide;      // both tiles of rows; else even and odd steps of one tile
    int steps;
    int n0, n1;     // steps of each pipeline
    __device__ __forceinline__ void set(const AttnItem& u, int group_log2) {
        steps = (u.kv1 - u.kv0 + 127) >> 7;
        wide = (u.ntok << group_log2) > 128;
        if (wide) {
            n1 = steps;
            // the first 128 rows see nothing past their last token
            const int end = u.pos + (128 >> group_log2);
            const int k = ((end < u.kv1 ? end : u.kv1) - u.kv0 + 127) >> 7;
            n0 = k < 0 ? 0 : k;
        } else {
            n0 = (steps + 1) >> 1;
            n1 = steps >> 1;
        }
    }
    __device__ __forceinline__ int n(int i) const { return i == 0 ? n0 : n1; }
    __device__ __forceinline__ int step(int i, int t) const { return wide ? t : 2 * t + i; }
    // Place of a step's K and V among the item's 2 * steps loads: the order in
    // which the MMA warp wants them.  wide: K0 V0 K1 V1 ..; else K0 K1 V0 K2 V1 K3 ..
    __device__ __forceinline__ int k_load(int j) const { return wide ? 2 * j : j == 0 ? 0 : 2 * j - 1; }
    __device__ __forceinline__ int v_load(int j) const {
        return wide ? 2 * j + 1 : (j == steps - 1 ? 2 * steps - 1 : 2 * j + 2);
    }
    // the step and kind of load l
    __device__ __forceinline__ int load_step(int l, bool& v) const {
        if (wide) {
            v = l & 1;
            return l >> 1;
        }
        if (l == 2 * steps - 1) {
            v = true;
            return steps - 1;
        }
        if (l == 0) {
            v = false;
            return 0;
        }
        v = (l & 1) == 0;
        return v ? (l >> 1) - 1 : (l + 1) >> 1;
    }
};

// Keys k0 .. k0 + 127 that the query at index i of its sequence sees, as bits.
__device__ __forceinline__ void seen_words(const int32_t* parents_of_seq, int first, int i, int k0, uint32_t (&w)[4]) {
    const int n = (parents_of_seq ? first : first + i + 1) - k0;  // keys seen from k0 on, without ancestors
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int x = n - 32 * j;
        w[j] = x >= 32 ? 0xffffffffu : x <= 0 ? 0u : (1u << x) - 1u;
    }
    if (parents_of_seq == nullptr) return;
    const int d0 = k0 - first;
    while (i >= 0 && i >= d0) {
        const int at = i - d0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if ((at >> 5) == j) w[j] |= 1u << (at & 31);
        const int up = __ldg(parents_of_seq + i);
        if (up >= i) break;
        i = up;
    }
}

// Keys of a step that are there: below kv1 (count: kv1 - k0) and in a block
// of the pool (bad: bits of blocks that are not).
__device__ __forceinline__ void there_words(int count, uint32_t bad, int bs, uint32_t (&w)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int x = count - 32 * j;
        w[j] = x >= 32 ? 0xffffffffu : x <= 0 ? 0u : (1u << x) - 1u;
        if (bad) {
            const int per = 32 / bs;  // blocks of the word
            for (int b = 0; b < per; ++b)
                if (bad >> (j * per + b) & 1) w[j] &= ~((bs == 32 ? 0xffffffffu : ((1u << bs) - 1u)) << (b * bs));
        }
    }
}

// One row again, by one warp, from the keys it sees alone: what a row whose
// result is not finite gets (a value of v outside the row's mask may have
// reached it as 0 * inf).  Lanes hold D / 32 dims each; acc is not divided by l.
template <int D, bool FP8>
__device__ __noinline__ void slow_row(const AttnParams& p, const AttnItem& u, int r, float& m, float& l, float* acc) {
    constexpr int VE = D / 32;
    using TKV = typename std::conditional<FP8, __nv_fp8_e4m3, __nv_bfloat16>::type;
    const int lane = threadIdx.x & 31;
    const int G = 1 << p.group_log2, bs = p.block_size;
    const int i = u.pos - u.first + (r >> p.group_log2);
    const int32_t* par = p.parents ? p.parents + (u.row - (u.pos - u.first)) : nullptr;
    const int32_t* bt = p.block_tables + (long long)u.seq * p.max_blocks_per_seq;
    const float qs = FP8 ? p.qscale * p.k_scales[u.g] : p.qscale;
    const float vs = FP8 ? p.v_scales[u.g] : 1.f;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) +
                             (long long)(u.row + (r >> p.group_log2)) * p.q_stride + (u.g * G + (r & (G - 1))) * D +
                             lane * VE;
    float qv[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) qv[e] = __bfloat162float(q[e]), acc[e] = 0.f;
    m = -INFINITY;
    l = 0.f;
    for (int key = u.kv0; key < u.kv1; ++key) {
        if (!sees(par, u.first, i, key)) continue;
        const int e = bt[key / bs];
        if (e < 0 || e >= p.num_blocks) continue;
        const long long at = (((long long)e * p.num_kv_heads + u.g) * bs + key % bs) * D + lane * VE;
        const TKV* k = static_cast<const TKV*>(p.k_cache) + at;
        const TKV* v = static_cast<const TKV*>(p.v_cache) + at;
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < VE; ++x) s = fmaf(qv[x], static_cast<float>(k[x]), s);
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= qs;
        const float mn = fmaxf(m, s);
        const float a = mn == -INFINITY ? 1.f : exp2f(m - mn);
        const float w = s == -INFINITY ? 0.f : exp2f(s - mn);
        m = mn;
        l = fmaf(l, a, w);
#pragma unroll
        for (int x = 0; x < VE; ++x) acc[x] = fmaf(acc[x], a, w * static_cast<float>(v[x]) * vs);
    }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::THREADS, 1)
    attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap tmq,
                   const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using C = Cfg<D, FP8>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t* load_full = bars;
    uint64_t* load_empty = load_full + C::NLOAD;
    uint64_t* slot_full = FP8 ? load_empty + C::NLOAD : load_full;  // what the MMA waits for
    uint64_t* slot_empty = FP8 ? slot_full + C::NSLOT : load_empty;
    uint64_t* q_full = slot_empty + C::NSLOT;
    uint64_t* q_empty = q_full + 1;
    uint64_t* q_wide = q_full + 2;
    uint64_t* s_full = q_full + 3;
    uint64_t* p_full = s_full + 2;
    uint64_t* o_full = s_full + 4;
    uint64_t* x_full = s_full + 6;
    uint64_t* x_empty = s_full + 7;
    uint64_t* item_full = s_full + 8;
    uint64_t* item_empty = item_full + C::ITEMS;
    uint64_t* sync_bar = item_empty + C::ITEMS;
    uint64_t* mma_done = sync_bar + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
    int* merge_flag = reinterpret_cast<int*>(smem + C::MISC_OFF + 8);
    int* turns = reinterpret_cast<int*>(smem + C::MISC_OFF + 12);  // split items this CTA has counted
    float2* ml_x = reinterpret_cast<float2*>(smem + C::ML_OFF);
    unsigned char* q_row_scale = smem + C::QS_OFF;  // biased exponents

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < C::NLOAD; ++i) {
            mbar_init(&load_full[i], 1);
            mbar_init(&load_empty[i], FP8 ? 4 : 1);
        }
        if constexpr (FP8) {
            for (int i = 0; i < C::NSLOT; ++i) {
                mbar_init(&slot_full[i], 4);
                mbar_init(&slot_empty[i], 1);
            }
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, FP8 ? 9 : 1);  // the last QK^T, fp8: and the softmax warps have the rows' scales
        mbar_init(q_wide, 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
        }
        mbar_init(x_full, 4);
        mbar_init(x_empty, 4);
        for (int i = 0; i < C::ITEMS; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], 10 + (FP8 ? 4 : 0));  // producer, MMA, softmax and widening warps
        }
        mbar_init(sync_bar, 8);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        *turns = 0;
        fence_mbarrier_init();
    }
    if (warp == 9) {
        tc::tmem_alloc(tmem_slot, C::TMEM_COLS);
        tc::tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const AttnWalk<TcDivision> walk0 =
        attn_walk_start<TcDivision, C::THREADS>(p, reinterpret_cast<long long*>(smem + C::WALK_OFF));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int gl = p.group_log2, G = 1 << gl, bs = p.block_size, Hkv = p.num_kv_heads;
    const int bpt = C::KEYS / bs;  // blocks of a step
    const int bl = 31 - __clz(bs);

    // A wait by the whole warp (or by the one lane that is there); false: wind down.
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (mbar_wait_bounded(bar, parity, abort_flag, p.wait_ns)) return true;
        set_error(p.err, PKV_ERR_TIMEOUT);
        *abort_flag = 1;
        return false;
    };
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool ok = mbar_wait_bounded(bar, parity, abort_flag, p.wait_ns);
        if (__all_sync(0xffffffffu, ok)) return true;
        if (lane == 0) {
            set_error(p.err, PKV_ERR_TIMEOUT);
            *abort_flag = 1;
        }
        return false;
    };
    // Item n of the CTA, as the walk put it into the ring (seq < 0: no more).
    auto item_slot = [&](int n) { return reinterpret_cast<AttnItem*>(smem + C::ITEM_OFF + (n % C::ITEMS) * 64); };

    int loads = 0;  // producer: copies issued; of Q: items
    int q_loads = 0;
    bool mma_any = false;

    if (warp >= 8 && warp < 12) {
        regs_dec<C::REGS_ISSUE>();
        if (warp == 10) {
            // ------------------------------------------------------- the walk
            if (lane == 0) {
                AttnWalk<TcDivision> walk = walk0;
                for (int n = 0;; ++n) {
                    if (n >= C::ITEMS && !wait(&item_empty[n % C::ITEMS], (n / C::ITEMS - 1) & 1)) break;
                    AttnItem u;
                    const bool more = walk.next(p, u);
                    if (!more) u.seq = -1;
                    *item_slot(n) = u;
                    mbar_arrive(&item_full[n % C::ITEMS]);
                    if (!more) break;
                }
            }
        } else if (warp == 8) {
            // ------------------------------------------------------- producer
            for (int n = 0;; ++n) {
                if (!wait_warp(&item_full[n % C::ITEMS], (n / C::ITEMS) & 1)) break;
                const AttnItem u = *item_slot(n);
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[n % C::ITEMS]);
                if (u.seq < 0) break;
                Plan plan;
                plan.set(u, gl);
                if (plan.steps == 0) continue;
                if (q_loads > 0 && !wait_warp(q_empty, (q_loads - 1) & 1)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, (plan.wide ? 2 : 1) * C::QTILE);
                    for (int t = 0; t < (plan.wide ? 2 : 1); ++t)
                        for (int h = 0; h < C::HALVES; ++h)
                            tma_load_3d(smem + C::Q_OFF + t * C::QTILE + h * C::QHALF, &tmq, h * 64, u.g * G,
                                        u.row + t * (128 >> gl), q_full);
                }
                ++q_loads;
                const int32_t* bt = p.block_tables + (long long)u.seq * p.max_blocks_per_seq;
                auto entry = [&](int l) {  // lane j: block j of load l
                    bool v;
                    if (l >= 2 * plan.steps) return -1;
                    const int key = u.kv0 + plan.load_step(l, v) * C::KEYS + lane * bs;
                    if (lane >= bpt || key >= u.kv1) return -1;
                    const int e = __ldg(bt + (key >> bl));
                    if (e >= 0 && e < p.num_blocks) return e;
                    set_error(p.err, PKV_ERR_DEVICE_BOUNDS);
                    return -1;
                };
                int e = entry(0), e1 = entry(1);
                bool ok = true;
                for (int l = 0; l < 2 * plan.steps; ++l) {
                    const int e2 = entry(l + 2);  // two loads ahead of its use
                    const int st = loads % C::NLOAD;
                    if (loads >= C::NLOAD && !wait_warp(&load_empty[st], (loads / C::NLOAD - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    bool v;
                    plan.load_step(l, v);
                    const int count = __popc(__ballot_sync(0xffffffffu, e >= 0));
                    if (lane == 0) {
                        if (count > 0)
                            mbar_arrive_expect_tx(&load_full[st], (uint32_t)(count * bs * D * (FP8 ? 1 : 2)));
                        else
                            mbar_arrive(&load_full[st]);
                    }
                    __syncwarp();  // the expected byte count is registered before any copy lands
                    if (e >= 0) {
                        const CUtensorMap* map = v ? &tmv : &tmk;
                        if constexpr (FP8)
                            tma_load_3d(smem + C::RAW_OFF + st * C::RAW + lane * bs * D, map, 0, 0, e * Hkv + u.g,
                                        &load_full[st]);
                        else
                            tma_load_5d(smem + C::SLOT_OFF + st * C::TILE + lane * bs * D * 2, map, 0, 0, 0, 0,
                                        e * Hkv + u.g, &load_full[st]);
                    }
                    ++loads;
                    e = e1;
                    e1 = e2;
                }
                if (!ok) break;
            }
        } else if (warp == 9) {
            // ------------------------------------------------------ MMA issue
            const uint32_t one = elect_one();
            const uint32_t q_base = smem_addr(smem + C::Q_OFF), s_base = smem_addr(smem + C::SLOT_OFF);
            // descriptors of the first tile; others differ in the address field (16-byte units)
            const uint64_t q_desc = sw128_desc(q_base, 16, 1024), k_desc = sw128_desc(s_base, 16, C::GSTRIDE),
                           v_desc = sw128_desc(s_base, C::HSTEP, C::GSTRIDE);
            int base = 0;  // loads of the items before
            int items_with_q = 0;
            uint32_t p_phase[2] = {0, 0};
            for (int n = 0;; ++n) {
                if (!wait_warp(&item_full[n % C::ITEMS], (n / C::ITEMS) & 1)) break;
                const AttnItem u = *item_slot(n);
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[n % C::ITEMS]);
                if (u.seq < 0) break;
                Plan plan;
                plan.set(u, gl);
                if (plan.steps == 0) continue;
                if (!wait_warp(FP8 ? q_wide : q_full, items_with_q & 1)) break;
                ++items_with_q;
                mma_any = true;
                auto qk = [&](int i, int t) -> bool {
                    const int j = plan.step(i, t), li = base + plan.k_load(j), st = li % C::NSLOT;
                    if (!wait_warp(&slot_full[st], (li / C::NSLOT) & 1)) return false;
                    tc_fence_after();
                    const uint64_t a0 = q_desc + (plan.wide ? i : 0) * (C::QTILE >> 4),
                                   b0 = k_desc + st * (C::TILE >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ss(tmem + i * 128, a0 + (((kk >> 2) * C::QHALF + (kk & 3) * 32) >> 4),
                               b0 + (((kk >> 2) * C::HSTEP + (kk & 3) * 32) >> 4), C::IDESC_QK, kk > 0, one);
                    commit_one(&s_full[i], one);
                    if (!plan.wide || i == 1) {
                        commit_one(&slot_empty[st], one);
                        if (j == plan.steps - 1) commit_one(q_empty, one);
                    }
                    return true;
                };
                auto pv = [&](int i, int t) -> bool {
                    const int j = plan.step(i, t), li = base + plan.v_load(j), st = li % C::NSLOT;
                    if (!wait_warp(&slot_full[st], (li / C::NSLOT) & 1)) return false;
                    if (!wait_warp(&p_full[i], p_phase[i])) return false;
                    p_phase[i] ^= 1;
                    tc_fence_after();
                    const uint64_t b0 = v_desc + st * (C::TILE >> 4);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(tmem + C::O_COL + i * 128, tmem + i * 128 + kk * 8, b0 + ((kk * 2 * C::GSTRIDE) >> 4),
                               C::IDESC_PV, kk > 0 || t > 0, one);
                    if (t == plan.n(i) - 1) commit_one(&o_full[i], one);
                    if (!plan.wide || i == 1) commit_one(&slot_empty[st], one);
                    return true;
                };
                bool ok = true;
                for (int i = 0; i < 2 && ok; ++i)
                    if (plan.n(i) > 0) ok = qk(i, 0);
                const int nmax = plan.n0 > plan.n1 ? plan.n0 : plan.n1;
                for (int t = 0; t < nmax && ok; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (!ok || t >= plan.n(i)) continue;
                        ok = pv(i, t);
                        if (ok && t + 1 < plan.n(i)) ok = qk(i, t + 1);
                    }
                if (!ok) break;
                base += 2 * plan.steps;
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------ softmax
        regs_inc<C::REGS_SOFTMAX>();
        const int wg = warp >> 2;
        const int lane_row = (warp & 3) * 32 + lane;   // TMEM lane
        const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_s = t_lane + wg * 128, t_o = t_lane + C::O_COL + wg * 128;
        int base = 0;                  // loads of the items before
        uint32_t s_phase = 0, o_phase[2] = {0, 0}, x_phase = 0, sync_phase = 0;
        bool x_pending = false;        // WG 1: its O has not been read yet
        int q_items = 0;
        bool ok = true;
        auto sync = [&]() -> bool {    // all 256 threads
            __syncwarp();
            if (lane == 0) mbar_arrive(sync_bar);
            const bool s = wait_warp(sync_bar, sync_phase);
            sync_phase ^= 1;
            return s;
        };
        for (int n = 0; ok; ++n) {
            if (!(ok = wait_warp(&item_full[n % C::ITEMS], (n / C::ITEMS) & 1))) break;
            const AttnItem u = *item_slot(n);
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[n % C::ITEMS]);
            if (u.seq < 0) break;
            Plan plan;
            plan.set(u, gl);
            const int rows = u.ntok << gl;
            const int row = (plan.wide ? wg * 128 : 0) + lane_row;  // of the item
            const int nt = plan.n(wg);
            const int32_t* bt = p.block_tables + (long long)u.seq * p.max_blocks_per_seq;
            const int32_t* par = p.parents ? p.parents + (u.row - (u.pos - u.first)) : nullptr;
            if (par != nullptr && u.part == 0 && u.g == 0) attn_check_parents(p, u, tid, 256);
            const int tok = (row >> gl) < u.ntok ? row >> gl : u.ntok - 1;
            const int qi = u.pos - u.first + tok;  // index in its sequence
            float qs = p.qscale;
            if constexpr (FP8) {
                qs *= p.k_scales[u.g];
                if (plan.steps > 0) {
                    if (!(ok = wait_warp(q_wide, q_items & 1))) break;
                    ++q_items;
                    qs *= __uint_as_float((uint32_t)q_row_scale[row] << 23);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(q_empty);
                }
            }
            const bool negate = qs < 0.f;  // a negative scale turns the order of the scores
            // keys that every row of the warp sees
            const int row0 = (plan.wide ? wg * 128 : 0) + (warp & 3) * 32;
            const int clear = par ? u.first : u.pos + (row0 >> gl) + 1;
            float m = -INFINITY, l = 0.f;
            auto entry = [&](int t) {  // lane j: whether block j of step t is not in the pool
                const int key = u.kv0 + plan.step(wg, t) * C::KEYS + lane * bs;
                if (t >= nt || lane >= bpt || key >= u.kv1) return 0;
                return __ldg(bt + (key >> bl));
            };
            int e_next = entry(0);
            for (int t = 0; t < nt; ++t) {
                const int j = plan.step(wg, t), k0 = u.kv0 + j * C::KEYS;
                const uint32_t bad = __ballot_sync(0xffffffffu, e_next < 0 || e_next >= p.num_blocks);
                e_next = entry(t + 1);
                if (!(ok = wait_warp(&s_full[wg], s_phase))) break;
                s_phase ^= 1;
                tc_fence_after();
                float x[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, x + 32 * c);
                tmem_wait_ld();
                if (negate) {
#pragma unroll
                    for (int c = 0; c < 128; ++c) x[c] = -x[c];
                }
                const bool short_step = k0 + C::KEYS > u.kv1 || bad != 0;
                if (short_step || k0 + C::KEYS > clear) {
                    uint32_t w[4], there[4];
                    seen_words(par, u.first, qi, k0, w);
                    there_words(u.kv1 - k0, bad, bs, there);
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (!(w[c >> 5] & there[c >> 5] & (1u << (c & 31)))) x[c] = -INFINITY;
                    if (!FP8 && short_step && (!plan.wide || wg == 0 || j >= plan.n0)) {
                        // keys that are not there: their rows of V may hold anything
                        const int li = base + plan.v_load(j), st = li % C::NSLOT;
                        if (!(ok = wait_warp(&slot_full[st], (li / C::NSLOT) & 1))) break;
                        const uint32_t word = lane_row < 32 ? there[0] : lane_row < 64 ? there[1]
                                              : lane_row < 96 ? there[2] : there[3];
                        if (!(word >> (lane_row & 31) & 1)) {
                            unsigned char* v = smem + C::SLOT_OFF + st * C::TILE + (lane_row >> 3) * C::GSTRIDE +
                                               (lane_row & 7) * 128;
#pragma unroll
                            for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    reinterpret_cast<uint4*>(v + h * C::HSTEP)[c] = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                }
                // a scale of 0 weighs what is seen alike, and -inf * 0 is not -inf
                const float qa = fmaxf(fabsf(qs), __uint_as_float(1u));
                float mx0 = x[0], mx1 = x[1], mx2 = x[2], mx3 = x[3];
#pragma unroll
                for (int c = 4; c < 124; c += 8) {
                    mx0 = fmaxf(fmaxf(mx0, x[c]), x[c + 1]);
                    mx1 = fmaxf(fmaxf(mx1, x[c + 2]), x[c + 3]);
                    mx2 = fmaxf(fmaxf(mx2, x[c + 4]), x[c + 5]);
                    mx3 = fmaxf(fmaxf(mx3, x[c + 6]), x[c + 7]);
                }
                mx0 = fmaxf(fmaxf(mx0, x[124]), x[125]);
                mx1 = fmaxf(fmaxf(mx1, x[126]), x[127]);
                const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * qa;
                if (__any_sync(0xffffffffu, mx > m + (8.f + C::SHIFT))) {
                    const float mn = fmaxf(m, mx - C::SHIFT);
                    const float alpha = mn == -INFINITY ? 1.f : ex2(m - mn);
                    m = mn;
                    l *= alpha;
                    if (t > 0) {  // s_full: the product before this step's scores is complete
#pragma unroll
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            tmem_ld32(t_o + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= alpha;
                            tmem_st32(t_o + c, reinterpret_cast<const uint32_t*>(o));
                        }
                    }
                }
                const float mm = m == -INFINITY ? 0.f : -m;
                const float2 q2 = make_float2(qa, qa), m2 = make_float2(mm, mm);
                float2 sum0 = make_float2(l, 0.f), sum1 = make_float2(0.f, 0.f);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        float2 y = fma2(make_float2(x[64 * half + 2 * c], x[64 * half + 2 * c + 1]), q2, m2);
                        y.x = ex2(y.x);
                        y.y = ex2(y.y);
                        if (c & 1) sum1 = add2(sum1, y); else sum0 = add2(sum0, y);
                        pk[c] = FP8 ? pack_f16(y.x, y.y) : pack_bf16(y.x, y.y);
                    }
                    tmem_st32(t_s + 32 * half, pk);
                }
                sum0 = add2(sum0, sum1);
                l = sum0.x + sum0.y;
                tmem_wait_st();
                if (x_pending) {  // the item before: O of this pipeline is still being read
                    if (!(ok = wait_warp(x_empty, x_phase))) break;
                    x_phase ^= 1;
                    x_pending = false;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[wg]);
            }
            if (!ok) break;
            base += 2 * plan.steps;
            // ------------------------------------------------ end of the item
            const float vs = FP8 ? p.v_scales[u.g] : 1.f;
            const bool two = !plan.wide && plan.n1 > 0;  // both pipelines hold parts of the same rows
            float w0 = 1.f, w1 = 0.f;
            if (wg == 1 && !plan.wide) {
                if (two) {
                    if (x_pending) {
                        if (!(ok = wait_warp(x_empty, x_phase))) break;
                        x_phase ^= 1;
                        x_pending = false;
                    }
                    ml_x[lane_row] = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(x_full);
                    o_phase[1] ^= 1;
                    x_pending = true;
                }
            } else {
                if (nt > 0) {
                    if (!(ok = wait_warp(&o_full[wg], o_phase[wg]))) break;
                    o_phase[wg] ^= 1;
                }
                if (two) {
                    if (!(ok = wait_warp(x_full, x_phase))) break;
                    x_phase ^= 1;
                    if (!(ok = wait_warp(&o_full[1], o_phase[1]))) break;
                    o_phase[1] ^= 1;
                    const float2 o = ml_x[lane_row];
                    const float M = fmaxf(m, o.x);
                    w0 = M == -INFINITY ? 1.f : ex2(m - M);
                    w1 = M == -INFINITY ? 1.f : ex2(o.x - M);
                    l = fmaf(w0, l, w1 * o.y);
                    m = M;
                } else if (wg == 0 && plan.wide) {
                    if (plan.n1 > 0) o_phase[1] ^= 1;
                }
                tc_fence_after();
                const bool whole = u.nparts == 1;
                const float inv = whole ? (l == 0.f ? 0.f : vs / l) : vs;  // no key seen: a zero row
                w0 *= inv;
                w1 *= inv;
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                                     ((long long)(u.row + (row >> gl)) * p.num_heads + u.g * G + (row & (G - 1))) * D;
                const long long pr = attn_partial_row(p, blockIdx.x, u.part) + row;
                float odd = 0.f;  // becomes NaN with the first value that is not finite
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float o[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                    if (nt > 0) {
                        tmem_ld32(t_o + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= w0;
                    }
                    if (two) {
                        float o1[32];
                        tmem_ld32(t_lane + C::O_COL + 128 + c, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = fmaf(o1[e], w1, o[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) odd = fmaf(o[e], 0.f, odd);
                    if (row < rows) {
                        if (whole) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                *reinterpret_cast<uint4*>(dst + c + e) =
                                    make_uint4(pack_bf16(o[e], o[e + 1]), pack_bf16(o[e + 2], o[e + 3]),
                                               pack_bf16(o[e + 4], o[e + 5]), pack_bf16(o[e + 6], o[e + 7]));
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                *reinterpret_cast<float4*>(p.ws_o + pr * D + c + e) =
                                    make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        }
                    }
                }
                if (!whole && row < rows) p.ws_ml[pr] = make_float2(m, l);
                if (two) {  // the other pipeline's O may be written again
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(x_empty);
                }
                uint32_t again = __ballot_sync(0xffffffffu, row < rows && nt > 0 && !(odd == 0.f && l == l));
                __syncwarp();
                while (again) {
                    const int r = __ffs(again) - 1;
                    again &= again - 1;
                    float ms, ls, acc[D / 32];
                    slow_row<D, FP8>(p, u, row0 + r, ms, ls, acc);
                    const long long at = __shfl_sync(0xffffffffu, pr, r);
                    const int rr = row0 + r;
                    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) +
                                        ((long long)(u.row + (rr >> gl)) * p.num_heads + u.g * G + (rr & (G - 1))) * D;
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) {
                        if (whole)
                            to[lane * (D / 32) + e] = __float2bfloat16_rn(ls == 0.f ? 0.f : acc[e] / ls);
                        else
                            p.ws_o[at * D + lane * (D / 32) + e] = acc[e];
                    }
                    if (!whole && lane == 0) p.ws_ml[at] = make_float2(ms, ls);
                }
            }
            if (u.nparts > 1) {
                if (!(ok = attn_merge<TcDivision, __nv_bfloat16, D, 256>(p, u, walk0.share, merge_flag, turns, tid, sync)))
                    break;
            }
        }
    } else {
        // ----------------------------------------------------------- widening
        if constexpr (FP8) {
            regs_dec<C::REGS_WIDEN>();
            const int t128 = tid - 384;
            int count = 0;  // loads so far
            int q_items = 0;
            bool ok = true;
            for (int n = 0; ok; ++n) {
                if (!(ok = wait_warp(&item_full[n % C::ITEMS], (n / C::ITEMS) & 1))) break;
                const AttnItem u = *item_slot(n);
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[n % C::ITEMS]);
                if (u.seq < 0) break;
                Plan plan;
                plan.set(u, gl);
                if (plan.steps == 0) continue;
                const int32_t* bt = p.block_tables + (long long)u.seq * p.max_blocks_per_seq;
                // q: bf16 -> f16 in place, each row times a power of two that brings
                // its largest value to [2^14, 2^15)
                if (!(ok = wait_warp(q_full, q_items & 1))) break;
                ++q_items;
                for (int t = 0; t < (plan.wide ? 2 : 1); ++t) {
                    unsigned char* qr = smem + C::Q_OFF + t * C::QTILE + t128 * 128;
                    uint32_t top = 0;
#pragma unroll
                    for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
                        for (int c0 = 0; c0 < 8; ++c0) {
                            const int c = c0 ^ (t128 & 7);  // neighbouring rows: other banks
                            const uint4 w = *reinterpret_cast<const uint4*>(qr + h * C::QHALF + c * 16);
                            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t lo = (x[e] & 0x7fffu) << 16, hi = x[e] & 0x7fff0000u;
                                top = top > lo ? top : lo;
                                top = top > hi ? top : hi;
                            }
                        }
                    // exponent of the largest |q| (as bits, they order like integers); infinities
                    // and NaN stay what they are under any scale
                    int ex = (int)(top >> 23);
                    ex = ex == 0 ? 127 + 14 : ex > 254 ? 254 : ex;
                    int up = 127 + 14 - ex + 127;  // biased exponent of the scale
                    up = up < 1 ? 1 : up > 253 ? 253 : up;
                    const float f = __uint_as_float((uint32_t)up << 23);
                    q_row_scale[t * 128 + t128] = (unsigned char)(254 - up);
#pragma unroll
                    for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
                        for (int c0 = 0; c0 < 8; ++c0) {
                            const int c = c0 ^ (t128 & 7);
                            uint4* at = reinterpret_cast<uint4*>(qr + h * C::QHALF + c * 16);
                            const uint4 w = *at;
                            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                y[e] = pack_f16(__uint_as_float(x[e] << 16) * f,
                                                __uint_as_float(x[e] & 0xffff0000u) * f);
                            *at = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_wide);
                for (int lo = 0; lo < 2 * plan.steps; ++lo, ++count) {
                    bool v;
                    const int k0 = u.kv0 + plan.load_step(lo, v) * C::KEYS;
                    const int key = k0 + lane * bs;
                    const int e = lane < bpt && key < u.kv1 ? __ldg(bt + (key >> bl)) : 0;
                    const uint32_t bad = __ballot_sync(0xffffffffu, e < 0 || e >= p.num_blocks);
                    const bool short_step = k0 + C::KEYS > u.kv1 || bad != 0;
                    uint32_t there[4];
                    there_words(u.kv1 - k0, bad, bs, there);
                    const int rs = count % C::NRAW, st = count % C::NSLOT;
                    if (!(ok = wait_warp(&load_full[rs], (count / C::NRAW) & 1))) break;
                    if (count >= C::NSLOT && !(ok = wait_warp(&slot_empty[st], (count / C::NSLOT - 1) & 1))) break;
                    const unsigned char* raw = smem + C::RAW_OFF + rs * C::RAW;
                    unsigned char* wide = smem + C::SLOT_OFF + st * C::TILE;
                    constexpr int CPR = D / 16;  // 16-byte chunks of a raw row
#pragma unroll
                    for (int i = 0; i < C::KEYS * CPR / 128; ++i) {
                        const int x = t128 + 128 * i, r = x / CPR, c = x % CPR;
                        uint4 w = *reinterpret_cast<const uint4*>(raw + x * 16);
                        if (short_step) {
                            const uint32_t word = r < 32 ? there[0] : r < 64 ? there[1] : r < 96 ? there[2] : there[3];
                            if (!(word >> (r & 31) & 1)) w = make_uint4(0u, 0u, 0u, 0u);
                        }
                        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
                        uint32_t y[8];
#pragma unroll
                        for (int e2 = 0; e2 < 4; ++e2) {
                            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                                "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                                : "=r"(y[2 * e2]), "=r"(y[2 * e2 + 1])
                                : "r"(in[e2]));
                        }
                        unsigned char* to = wide + (r >> 3) * C::GSTRIDE + (c >> 2) * C::HSTEP + (r & 7) * 128;
                        // lanes of the second half store their chunks in the other order: no bank conflicts
                        const int first = (c >> 2) & 1, cc = 2 * (c & 3);
                        const uint4 a = make_uint4(y[0], y[1], y[2], y[3]), b = make_uint4(y[4], y[5], y[6], y[7]);
                        *reinterpret_cast<uint4*>(to + (((cc + first) ^ (r & 7)) << 4)) = first ? b : a;
                        *reinterpret_cast<uint4*>(to + (((cc + 1 - first) ^ (r & 7)) << 4)) = first ? a : b;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&slot_full[st]);
                        mbar_arrive(&load_empty[rs]);
                    }
                }
            }
        }
    }

    // ------------------------------------------------------------- wind down
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // copies and products in flight land before the CTA leaves; each wait is bounded
        auto land = [&](uint64_t* bar, uint32_t parity) {
            const unsigned long long t0 = globaltimer_ns();
            while (!mbar_try_wait(bar, parity))
                if (globaltimer_ns() - t0 > kWaitTimeoutNs) break;
        };
        if (warp == 8 && lane == 0) {
            for (int li = loads > C::NLOAD ? loads - C::NLOAD : 0; li < loads; ++li)
                land(&load_full[li % C::NLOAD], (li / C::NLOAD) & 1);
            if (q_loads > 0) land(q_full, (q_loads - 1) & 1);
        }
        if (warp == 9 && mma_any) {
            commit_one(mma_done, elect_one());
            land(mma_done, 0);
        }
        // parts that were not counted: empty ones, so that the counters end at zero
        AttnWalk<TcDivision> walk =
            attn_walk_start<TcDivision, C::THREADS>(p, reinterpret_cast<long long*>(smem + C::WALK_OFF));
        if (tid == 0) {
            AttnItem u;
            int k = 0;
            while (walk.next(p, u)) {
                if (u.nparts == 1 || k++ < *turns) continue;
                for (int r = 0; r < (u.ntok << gl); ++r)
                    p.ws_ml[attn_partial_row(p, blockIdx.x, u.part) + r] = make_float2(-INFINITY, 0.f);
                __threadfence();
                int* c = p.counters + AttnWalk<TcDivision>::owner(u.at, u.keys, walk.share, 0);
                if (atomicAdd(c, 1) == u.nparts - 1) *c = 0;
            }
        }
        tc_fence_before();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 9) tc::tmem_dealloc(tmem, C::TMEM_COLS);
}

}  // namespace atc
}  // namespace pkv
