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
// stays in TMEM for the whole item.
//
// The reference m of a row's weights need not be its maximum, it cancels in
// the quotient, and bf16 weights are as wide in range as fp32: m is the largest
// of the first 32 scores that the row sees, and no other maximum is taken.
// When weights take the sum past 2^40, m is raised past their scores, the sum
// and O are moved by that, and the weights are taken again (hardly ever).
//
// Warps: 0-3 and 4-7 softmax, 8 producer (TMA: one 5-D copy brings a whole
// block of K or V in the layout the MMA wants), 9 MMA issue, 10 the walk;
// fp8 caches: 12-19 widen each K and V tile to
// bf16, which holds every e4m3 value.
//
// Rounding: P to bf16 before the product with V, as the tensor cores take it;
// sums and O are fp32.
//
// A masked key's weight is 0, and 0 * inf or 0 * nan would reach the row all
// the same, as would sums past fp32 of values near the largest: rows whose
// result is not finite are computed again from the keys they see alone
// (slow_rows: 148 tiles of 256 rows over 4096 keys take 21 ms of bf16 cache and
// 37 ms of fp8 if every row goes that way, 0.11 and 0.12 ms if none does).
// Every wait is bounded, by its own time and that of rows computed again.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "attn_common.cuh"
#include "decode_tc.cuh"
#include "f32x2.cuh"

namespace pkv {
namespace atc {

using tc::fence_proxy_async_smem;
using tc::sw128_desc;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tma_load_5d;

// Fitted over 1 to 6 items a CTA of 4 to 32 steps, caches cold, head_dim 128: a step
// of 128 keys takes a full tile 2.05 us (fp8 2.5), a tile of at most 128 rows, two steps
// at a time, 1.6 us (1.8) where K and V come from HBM; an item takes 5.4 us (5.0) or
// 3.0 us (3.8) besides, a launch 14 us.  3 : 2 and three full steps an item are what
// the calls gain by: 8192 tokens of 32 heads 567 -> 508 us, drafted trees over 128K
// contexts 778 -> 672 us.
using TcDivision = AttnDivision<256, 128, 2, 3, 128, 512, 1152>;

// ------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
        : "memory");
}

// Barriers by their shared-memory address.
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}
// Whether the phase is complete: at a look, or after a sleep of at most `ns`.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity, uint32_t ns) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(ns)
        : "memory");
    return ok != 0;
}
// Two of the CTA's words behind a shared-memory address: whether it has given
// up, and when it last did work that others have to wait for (slow_rows; at
// first its start).
constexpr uint32_t ABORT = 8, BUSY_AT = 12;
__device__ __forceinline__ void store_word(uint32_t at, uint32_t x) {
    asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}
__device__ __forceinline__ uint2 load_words(uint32_t words) {
    uint2 x;
    asm volatile("ld.volatile.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(words + ABORT) : "memory");
    return x;
}
__device__ __forceinline__ int short_time(unsigned long long ns) { return (int)(ns >> 10); }
constexpr unsigned long long UNHURRIED = 1ull << 40;  // 18 minutes
// Rest of a warp's wait whose first look was in vain: false when it ran out
// of time or another warp has given up.  The time (in 1024 ns) runs from the
// wait's start or from BUSY_AT, which rows that are computed again keep moving:
// their loops end with the row's keys.
__device__ __forceinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, uint32_t words, unsigned long long wait_ns,
                                              int* err) {
    const int t0 = short_time(globaltimer_ns());
    for (;;) {
        if (__all_sync(0xffffffffu, bar_try(bar, parity, 500u))) return true;
        const int now = short_time(globaltimer_ns());
        const uint2 w = load_words(words);
        // differences are signed: another warp may have moved BUSY_AT past `now`
        if (__any_sync(0xffffffffu, min(now - t0, now - (int)w.y) > short_time(wait_ns) || w.x != 0u)) {
            if ((threadIdx.x & 31) == 0) {
                set_error(err, PKV_ERR_TIMEOUT);
                store_word(words + ABORT, 1u);
            }
            return false;
        }
    }
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
// operands, longer than the 64 that the product itself takes).  Descriptors
// come as their two words: only the low one, with the address, varies.
// D[tmem] (+)= A[smem desc] . B[smem desc]
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t accumulate, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
// D[tmem] (+)= A[tmem] . B[smem desc]
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t accumulate, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
// Arrive on `bar` when every MMA of the electing lane so far has completed.
__device__ __forceinline__ void commit_one(uint32_t bar, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
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

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

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

// max(a, b, c), NaN if any of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 2^x of two values on the FMA pipe: x = n + f with n the nearest integer and
// |f| <= 1/2, 2^f by the polynomial of degree 3 with the least relative error
// there (an exchange algorithm's; 7.5e-5, a thirtieth of bf16's half step), n
// added to the exponent.  Below -125 it gives 2^-125 (of a value, next to the largest
// weight of at least 2^-1: nothing that bf16 keeps), above 127 and for NaN 2^127.
__device__ __forceinline__ float2 ex2_poly(float2 x) {
    x.x = fmaxf(fminf(x.x, 127.f), -125.f);
    x.y = fmaxf(fminf(x.y, 127.f), -125.f);
    const float2 big = make_float2(12582912.f, 12582912.f), neg = make_float2(-12582912.f, -12582912.f);
    const float2 t = add2(x, big);  // 1.5 2^23 + n: n in the low bits
    const float2 n = add2(t, neg);
    const float2 f = fma2(n, make_float2(-1.f, -1.f), x);
    float2 y = fma2(f, make_float2(0.0551716685295105f, 0.0551716685295105f),
                    make_float2(0.2426111251115799f, 0.2426111251115799f));
    y = fma2(y, f, make_float2(0.6932609677314758f, 0.6932609677314758f));
    y = fma2(y, f, make_float2(0.9999280571937561f, 0.9999280571937561f));
    y.x = __uint_as_float(__float_as_uint(y.x) + (__float_as_uint(t.x) << 23));
    y.y = __uint_as_float(__float_as_uint(y.y) + (__float_as_uint(t.y) << 23));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// 32 bytes of a lane's own, both halves of one sector at once.
__device__ __forceinline__ void store_sector(void* to, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Weights 2^(x q + m) of N scores of a row, packed for the MMA; sum gets their
// total.  One pair in POLY_OF goes by ex2_poly, so that the special-function
// unit (a quarter of the lanes a clock) and the FMA pipe share the work; not
// over fp8 caches (952 us with it, 931 without, on 1024-token chunks over 15K
// contexts), where widening is what keeps the pipes busy.  (4, 8, 16 and none
// differ by less than runs do: 521, 522, 518, 515 us on 8192 tokens of 32 heads, and
// 152 to 170 us each at head_dim 64 on 4096 tokens.)
constexpr int POLY_OF = 8;
template <int N, bool POLY>
__device__ __forceinline__ void weights(const float* x, float2 q, float2 m, uint32_t* pk, float2& sum) {
    float2 sum1 = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < N / 2; ++c) {
        float2 y = fma2(make_float2(x[2 * c], x[2 * c + 1]), q, m);
        if (POLY && c % POLY_OF == POLY_OF - 1) {
            y = ex2_poly(y);
        } else {
            y.x = ex2(y.x);
            y.y = ex2(y.y);
        }
        if (c & 1) sum1 = add2(sum1, y); else sum = add2(sum, y);
        pk[c] = pack_bf16(y.x, y.y);
    }
    sum = add2(sum, sum1);
}

// Largest of m and 32 scores; NaN if any of them is.
__device__ __forceinline__ float largest32(const float* x, float m) {
    float m0 = max3_nan(m, x[0], x[1]), m1 = max3_nan(x[2], x[3], x[4]);
#pragma unroll
    for (int c = 5; c < 29; c += 4) {
        m0 = max3_nan(m0, x[c], x[c + 1]);
        m1 = max3_nan(m1, x[c + 2], x[c + 3]);
    }
    m0 = max3_nan(m0, x[29], x[30]);
    return max3_nan(m0, m1, x[31]);
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
    static constexpr int WIDEN = FP8 ? 256 : 0;      // threads that widen
    static constexpr int THREADS = 384 + WIDEN;
    static constexpr int ITEMS = FP8 ? 2 : 4;       // items the walk is ahead
    // registers: what the launch gives all threads, and its split among roles
    static constexpr int REGS_SOFTMAX = FP8 ? 152 : 216;
    static constexpr int REGS_ISSUE = FP8 ? 64 : 72;
    static constexpr int REGS_WIDEN = 56;
    static constexpr int REGS_LAUNCH = 65536 / THREADS / 8 * 8;
    static_assert(256 * REGS_SOFTMAX + 128 * REGS_ISSUE + WIDEN * REGS_WIDEN <= THREADS * REGS_LAUNCH,
                  "the roles' registers come out of the launch's");
    static constexpr uint32_t TMEM_COLS = 512;      // S / P of both pipelines, then O of both
    static constexpr uint32_t O_COL = 256;
    static constexpr uint32_t IDESC_QK = tc::idesc_bf16(128, 128, false, false);
    static constexpr uint32_t IDESC_PV = tc::idesc_bf16(128, D, false, true);

    static constexpr int Q_OFF = 0;
    static constexpr int SLOT_OFF = 2 * QTILE;
    static constexpr int RAW_OFF = SLOT_OFF + NSLOT * TILE;
    static constexpr int BAR_OFF = RAW_OFF + NRAW * RAW;
    // full/empty of the load ring, of the widened ring, q_full q_empty,
    // s_full[2] p_full[2] p_rest[2] o_full[2] o_half[2], x_full x_empty, item full/empty, sync, mma_done
    static constexpr int NBARS = 2 * NLOAD + (FP8 ? 2 * NSLOT : 0) + 2 + 10 + 2 + 2 * ITEMS + 2;
    static constexpr int LOAD_FULL = BAR_OFF, LOAD_EMPTY = LOAD_FULL + 8 * NLOAD;
    static constexpr int SLOT_FULL = FP8 ? LOAD_EMPTY + 8 * NLOAD : LOAD_FULL;  // what the MMA waits for
    static constexpr int SLOT_EMPTY = FP8 ? SLOT_FULL + 8 * NSLOT : LOAD_EMPTY;
    static constexpr int Q_FULL = SLOT_EMPTY + 8 * NSLOT, Q_EMPTY = Q_FULL + 8;
    static constexpr int S_FULL = Q_FULL + 16, P_FULL = S_FULL + 16, P_REST = S_FULL + 32, O_FULL = S_FULL + 48;
    static constexpr int O_HALF = S_FULL + 64, X_FULL = S_FULL + 80, X_EMPTY = X_FULL + 8;
    static constexpr int ITEM_FULL = X_EMPTY + 8, ITEM_EMPTY = ITEM_FULL + 8 * ITEMS;
    static constexpr int SYNC_BAR = ITEM_EMPTY + 8 * ITEMS, MMA_DONE = SYNC_BAR + 8;
    static_assert(MMA_DONE + 8 == BAR_OFF + NBARS * 8, "");
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;  // tmem address, flag, abort, busy at, turns
    static constexpr int ITEM_OFF = (MISC_OFF + 48 + 15) / 16 * 16;
    static constexpr int WALK_OFF = ITEM_OFF + ITEMS * 64;  // the CTA's walk, as it starts
    static constexpr int ML_OFF = WALK_OFF + 64;            // float2[128]; first the scratch of the walk's start
    static_assert((THREADS / 32 + 8) * 8 <= 128 * 8 && sizeof(AttnWalk<TcDivision>) <= 64, "");
    static constexpr int SMEM_BYTES = ML_OFF + 128 * 8 + 1024;
    static_assert(SMEM_BYTES <= 232448, "227 KB of shared memory");
    static_assert(sizeof(AttnItem) <= 64, "");
};

// An item of at most this many parts is joined by the warps that have its
// rows; more go over all threads (attn_merge).  With 2: 50 against 46 us on prompts
// behind a prefix (head_dim 64), 54 against 39 us on one prompt of 2048 tokens of 8 heads;
// with 8: 79.5 against 77.5 us on packed prompts, 75 against 72 us on a batch of 64
// drafted trees, though 49 against 65 us on two sequences of 64 queries over 3000 keys.
constexpr int FEW_PARTS = 4;

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

// Eight values of a cache row.
template <bool FP8>
__device__ __forceinline__ void load8(const void* cache, long long at, float* v) {
    if constexpr (FP8) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const unsigned char*>(cache) + at));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2_raw h =
                __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1))), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
        Elem<__nv_bfloat16>::unpack(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(cache) + at)), v);
    }
}

// Rows again, SLOW at a time by one warp, from the keys they see alone: what
// rows whose result is not finite get (a value of v outside a row's mask may
// have reached it as 0 * inf).  32 keys at a time; a lane holds eight dims of
// the rows, so D / 8 lanes read a key and the warp reads 2 or 4 keys at once;
// sums of values stay apart by those until the end.  acc is not divided by l.
// Meanwhile the CTA's other waits are put off (BUSY_AT).  One row at a time with a
// key a lane took 70 and 61 ms where this takes 21 and 37.
template <int SLOW>
struct SlowRows {
    int r[SLOW];  // rows of the item
    float m[SLOW], l[SLOW], acc[SLOW][8];
};
template <int D, bool FP8, int SLOW>
__device__ __noinline__ void slow_rows(const AttnParams& p, const AttnItem& u, uint32_t words, SlowRows<SLOW>& z) {
    constexpr int LPR = D / 8;  // lanes that read a key
    const int lane = threadIdx.x & 31, d0 = (lane & (LPR - 1)) * 8, group = lane & ~(LPR - 1);
    const int G = 1 << p.group_log2, bs = p.block_size;
    const int32_t* par = p.parents ? p.parents + (u.row - (u.pos - u.first)) : nullptr;
    const int32_t* bt = p.block_tables + (long long)u.seq * p.max_blocks_per_seq;
    const float qs = FP8 ? p.qscale * p.k_scales[u.g] : p.qscale;
    const float vs = FP8 ? p.v_scales[u.g] : 1.f;
    float q[SLOW][8], acc[SLOW][8], m[SLOW], l[SLOW];
#pragma unroll
    for (int b = 0; b < SLOW; ++b) {
        const int r = z.r[b];
        load8<false>(p.q, (long long)(u.row + (r >> p.group_log2)) * p.q_stride + (u.g * G + (r & (G - 1))) * D + d0, q[b]);
        m[b] = -INFINITY;
        l[b] = 0.f;
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[b][x] = 0.f;
    }
#pragma unroll 1
    for (int k0 = u.kv0; k0 < u.kv1; k0 += 32) {
        if (lane == 0) store_word(words + BUSY_AT, short_time(globaltimer_ns()));
        const int key = k0 + lane;
        uint32_t seen[SLOW], any = 0u;
        long long at = 0;  // the lane's key in the pools
        bool there = false;
        if (key < u.kv1) {
            const int e = __ldg(bt + key / bs);
            there = e >= 0 && e < p.num_blocks;
            if (there) at = (((long long)e * p.num_kv_heads + u.g) * bs + key % bs) * D;
        }
#pragma unroll
        for (int b = 0; b < SLOW; ++b) {
            seen[b] = __ballot_sync(0xffffffffu, there && sees(par, u.first, u.pos - u.first + (z.r[b] >> p.group_log2), key));
            any |= seen[b];
        }
        if (any == 0u) continue;
        float s[SLOW];
#pragma unroll
        for (int b = 0; b < SLOW; ++b) s[b] = -INFINITY;
#pragma unroll 4
        for (int i = 0; i < LPR; ++i) {  // keys i, LPR + i, ..
            const long long a = __shfl_sync(0xffffffffu, at, group + i);
            float k[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (any >> (group + i) & 1u) load8<FP8>(p.k_cache, a + d0, k);
#pragma unroll
            for (int b = 0; b < SLOW; ++b) {
                float dot = 0.f;
#pragma unroll
                for (int x = 0; x < 8; ++x) dot = fmaf(q[b][x], k[x], dot);
#pragma unroll
                for (int d = LPR / 2; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
                if (lane == group + i && (seen[b] >> lane & 1u)) s[b] = dot * qs;
            }
        }
#pragma unroll
        for (int b = 0; b < SLOW; ++b) {
            float mx = s[b];
#pragma unroll
            for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(m[b], mx);
            const float a = mn == -INFINITY ? 1.f : exp2f(m[b] - mn);
            s[b] = s[b] == -INFINITY ? 0.f : exp2f(s[b] - mn);
            float sum = s[b];
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            m[b] = mn;
            l[b] = fmaf(l[b], a, sum);
            s[b] *= vs;
#pragma unroll
            for (int x = 0; x < 8; ++x) acc[b][x] *= a;
        }
#pragma unroll 4
        for (int i = 0; i < LPR; ++i) {
            const long long a = __shfl_sync(0xffffffffu, at, group + i);
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (any >> (group + i) & 1u) load8<FP8>(p.v_cache, a + d0, v);
#pragma unroll
            for (int b = 0; b < SLOW; ++b) {
                const float w = __shfl_sync(0xffffffffu, s[b], group + i);
                if (seen[b] >> (group + i) & 1u) {
#pragma unroll
                    for (int x = 0; x < 8; ++x) acc[b][x] = fmaf(w, v[x], acc[b][x]);
                }
            }
        }
        bool done = true;  // NaN from here on
#pragma unroll
        for (int b = 0; b < SLOW; ++b) done = done && l[b] != l[b];
        if (done) break;
    }
#pragma unroll
    for (int b = 0; b < SLOW; ++b) {
        z.m[b] = m[b];
        z.l[b] = l[b];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            float o = acc[b][x];
#pragma unroll
            for (int d = LPR; d < 32; d <<= 1) o += __shfl_xor_sync(0xffffffffu, o, d);
            z.acc[b][x] = l[b] == l[b] ? o : l[b];
        }
    }
}

// Rows whose sum l_now with the weights of n more keys (32 or 64 scores at
// t_x, `word` the seen ones of 32) has passed 2^40: a new reference at least as
// large as those scores, moved by a power of two where that is within range, and what the
// row has so far scaled to it: its sum l, O (t_o; ~0: nothing there yet) and, with
// `scale_p`, the 16 columns of weights at t_p that no product has taken yet.
// half: the barrier of the step's first product, which is waited for (0: none
// in flight).  A row that sees an infinite score gets NaN as its sum.
struct Raised {
    float m, l;
    bool ok;
};
template <int D>
__device__ __noinline__ Raised raise(const AttnParams& p, uint32_t t_x, int n, uint32_t word, bool scale_p, uint32_t t_p,
                                     uint32_t t_o, uint32_t half, uint32_t parity, uint32_t words, float qa,
                                                                         float m, float l, float l_now) {
    tmem_wait_st();  // weights of the chunk before
    float mx = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < n; c += 32) {
        float x[32];
        tmem_ld32(t_x + c, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = word & (1u << e) ? x[e] : -INFINITY;
        mx = largest32(x, mx);
    }
    mx *= qa;
    Raised r = {m, l, true};
    float alpha = 1.f;
    if (l > 0x1p40f) {
        r.l = __uint_as_float(0x7fffffffu);  // raised in vain before
    } else if (l_now > 0x1p40f) {
        const float e = fmaxf(ceilf(mx - m), l > 1.f ? (float)((int)(__float_as_uint(l) >> 23) - 127) : 0.f);
        if (e <= 126.f) {
            alpha = __uint_as_float((uint32_t)(127 - (int)e) << 23);
            r.m = m + e;
        } else {  // nothing of the old sums is left
            alpha = 0.f;
            r.m = mx;
        }
        r.l = mx < INFINITY ? l * alpha : __uint_as_float(0x7fffffffu);
    }
    __syncwarp();
    if (half != 0u && !(__all_sync(0xffffffffu, bar_test(half, parity)) ||
                        bar_wait_slow(half, parity, words, p.wait_ns, p.err))) {
        r.ok = false;
        return r;
    }
    tc_fence_after();
    if (t_o != ~0u) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(t_o + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tmem_st32(t_o + c, reinterpret_cast<const uint32_t*>(o));
        }
    }
    if (scale_p) {
        float x[32];
        uint32_t* pk = reinterpret_cast<uint32_t*>(x);
        tmem_ld32(t_p, x);
        tmem_wait_ld();
        const __nv_bfloat162 a = __float2bfloat162_rn(alpha);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&pk[e]), a);
            pk[e] = *reinterpret_cast<const uint32_t*>(&y);
        }
        tmem_st16(t_p, pk);
    }
    tmem_wait_st();
    return r;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::THREADS, 1)
    attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap tmq,
                   const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using C = Cfg<D, FP8>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_addr(smem);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    int* merge_flag = reinterpret_cast<int*>(smem + C::MISC_OFF + 4);
    int* turns = reinterpret_cast<int*>(smem + C::MISC_OFF + 16);  // [8] split items each softmax warp has counted
    float2* ml_x = reinterpret_cast<float2*>(smem + C::ML_OFF);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < C::NBARS; i += C::THREADS) {
        const int off = C::BAR_OFF + 8 * i;
        int count = 1;
        if (off >= C::LOAD_EMPTY && off < C::LOAD_EMPTY + 8 * C::NLOAD && FP8) count = C::WIDEN / 32;
        if (FP8 && off >= C::SLOT_FULL && off < C::SLOT_FULL + 8 * C::NSLOT) count = C::WIDEN / 32;
        if (off >= C::P_FULL && off < C::O_FULL) count = 4;    // P_FULL, P_REST: a pipeline's softmax warps
        if (off == C::X_FULL || off == C::X_EMPTY) count = 4;  // those of one pipeline
        if (off >= C::ITEM_EMPTY && off < C::SYNC_BAR) count = 10 + C::WIDEN / 32;  // all warps that read items
        if (off == C::SYNC_BAR) count = 8;                     // all softmax warps
        mbar_init(reinterpret_cast<uint64_t*>(smem + off), count);
    }
    if (tid < 8) turns[tid] = 0;
    if (tid == 0) {
        store_word(sb + C::MISC_OFF + ABORT, 0u);
        store_word(sb + C::MISC_OFF + BUSY_AT, short_time(globaltimer_ns()));
        for (const CUtensorMap* m : {&tmq, &tmk, &tmv})
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    }
    fence_mbarrier_init();
    if (warp == 9) {
        tc::tmem_alloc(tmem_slot, C::TMEM_COLS);
        tc::tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const AttnWalk<TcDivision> walk0 =
        attn_walk_start<TcDivision, C::THREADS>(p, reinterpret_cast<long long*>(smem + C::ML_OFF));
    if (tid == 0) *reinterpret_cast<AttnWalk<TcDivision>*>(smem + C::WALK_OFF) = walk0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int gl = p.group_log2, G = 1 << gl, bs = p.block_size, Hkv = p.num_kv_heads;
    const int bpt = C::KEYS / bs;  // blocks of a step
    const int bl = 31 - __clz(bs);

    // A wait by a converged warp; false: wind down.
    auto wait = [&](uint32_t off, uint32_t parity, unsigned long long at_least = 0) -> bool {
        if (__all_sync(0xffffffffu, bar_test(sb + off, parity))) return true;
        return bar_wait_slow(sb + off, parity, sb + C::MISC_OFF, at_least > p.wait_ns ? at_least : p.wait_ns, p.err);
    };
    auto arrive = [&](uint32_t off) {  // once for the warp, after what its lanes did
        __syncwarp();
        if (lane == 0) bar_arrive(sb + off);
    };
    // Items in the order in which the walk puts them into the ring; false: no more, or wind down.
    static_assert((C::ITEMS & (C::ITEMS - 1)) == 0, "");
    auto take_item = [&](int n, AttnItem& u, bool& ok) -> bool {
        const uint32_t i = n & (C::ITEMS - 1);
        if (!(ok = wait(C::ITEM_FULL + 8 * i, (n / C::ITEMS) & 1))) return false;
        u = *reinterpret_cast<const AttnItem*>(smem + C::ITEM_OFF + i * 64);
        arrive(C::ITEM_EMPTY + 8 * i);
        return u.seq >= 0;
    };

    int loads = 0;  // producer: copies issued; of Q: items
    int q_loads = 0;
    bool mma_any = false;

    if (warp >= 8 && warp < 12) {
        regs_dec<C::REGS_ISSUE>();
        if (warp == 10) {
            // ------------------------------------------------------- the walk
            AttnWalk<TcDivision> walk = walk0;
            for (int n = 0;; ++n) {
                const uint32_t i = n & (C::ITEMS - 1);
                // (as long as an item takes, which may be any time: the other warps' waits end this one)
                if (n >= C::ITEMS && !wait(C::ITEM_EMPTY + 8 * i, (n / C::ITEMS - 1) & 1, UNHURRIED)) break;
                AttnItem u;
                const bool more = walk.next(p, (int)blockIdx.x, u);
                if (!more) u.seq = -1;
                if (lane == 0) *reinterpret_cast<AttnItem*>(smem + C::ITEM_OFF + i * 64) = u;
                arrive(C::ITEM_FULL + 8 * i);
                if (!more) break;
            }
        } else if (warp == 8) {
            // ------------------------------------------------------- producer
            uint32_t st = 0, phase = 1;  // slot, parity of its emptying (the first round finds them empty)
            AttnItem u;
            bool ok = true;
            for (int n = 0; ok && take_item(n, u, ok); ++n) {
                Plan plan;
                plan.set(u, gl);
                if (plan.steps == 0) continue;
                const int32_t* bt = p.block_tables + (long long)u.seq * p.max_blocks_per_seq;
                const int n_loads = 2 * plan.steps;
                auto entry = [&](int l) {  // lane j: block j of load l
                    bool v;
                    if (l >= n_loads || lane >= bpt) return -1;
                    const int key = u.kv0 + plan.load_step(l, v) * C::KEYS + lane * bs;
                    if (key >= u.kv1) return -1;
                    const int e = __ldg(bt + (key >> bl));
                    if (e >= 0 && e < p.num_blocks) return e;
                    set_error(p.err, PKV_ERR_DEVICE_BOUNDS);
                    return -1;
                };
                int e = entry(0), e1 = entry(1);
                for (int l = 0; l < n_loads; ++l) {
                    const int e2 = entry(l + 2);  // two loads ahead of its use
                    if (!(ok = wait(C::LOAD_EMPTY + 8 * st, phase))) break;
                    bool v;
                    plan.load_step(l, v);
                    const uint32_t full = sb + C::LOAD_FULL + 8 * st;
                    const int count = __popc(__ballot_sync(0xffffffffu, e >= 0));
                    if (lane == 0) {
                        if (count > 0)
                            bar_expect(full, (uint32_t)(count * bs * D * (FP8 ? 1 : 2)));
                        else
                            bar_arrive(full);
                    }
                    __syncwarp();  // the expected byte count is registered before any copy lands
                    if (e >= 0 && PKV_DCHECK(p.err, e < p.num_blocks && u.g < Hkv && lane < bpt)) {
                        const CUtensorMap* map = v ? &tmv : &tmk;
                        uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::LOAD_FULL + 8 * st);
                        if constexpr (FP8)
                            tma_load_3d(smem + C::RAW_OFF + st * C::RAW + lane * bs * D, map, 0, 0, e * Hkv + u.g, bar);
                        else
                            tma_load_5d(smem + C::SLOT_OFF + st * C::TILE + lane * bs * D * 2, map, 0, 0, 0, 0,
                                        e * Hkv + u.g, bar);
                    }
                    ++loads;
                    if (++st == C::NLOAD) st = 0, phase ^= 1;
                    e = e1;
                    e1 = e2;
                    if (l == 1) {
                        // Q after the first K and V: its space is free only after the item before
                        if (q_loads > 0 && !(ok = wait(C::Q_EMPTY, (q_loads - 1) & 1))) break;
                        if (lane == 0) {
                            bar_expect(sb + C::Q_FULL, (plan.wide ? 2 : 1) * C::QTILE);
                            for (int t = 0; t < (plan.wide ? 2 : 1); ++t)
                                for (int h = 0; h < C::HALVES; ++h)
                                    tma_load_3d(smem + C::Q_OFF + t * C::QTILE + h * C::QHALF, &tmq, h * 64, u.g * G,
                                                u.row + t * (128 >> gl), reinterpret_cast<uint64_t*>(smem + C::Q_FULL));
                        }
                        ++q_loads;
                    }
                }
                if (!ok) break;
            }
        } else if (warp == 9) {
            // ------------------------------------------------------ MMA issue
            // The tensor cores hold a few instructions in advance, some 250 clocks of work.
            // What this warp does between two of them has to fit into that, so waits and
            // bookkeeping are spread: after four of a product's eight, between two products
            // and in the middle of QK^T.
            const uint32_t one = elect_one();
            // descriptors of the first tile; others differ in the address field (16-byte units)
            const uint64_t q_desc = sw128_desc(sb + C::Q_OFF, 16, 1024),
                           k_desc = sw128_desc(sb + C::SLOT_OFF, 16, C::GSTRIDE),
                           v_desc = sw128_desc(sb + C::SLOT_OFF, C::HSTEP, C::GSTRIDE);
            const uint32_t q_lo = (uint32_t)q_desc, q_hi = (uint32_t)(q_desc >> 32), k_lo = (uint32_t)k_desc,
                           k_hi = (uint32_t)(k_desc >> 32), v_lo = (uint32_t)v_desc, v_hi = (uint32_t)(v_desc >> 32);
            uint32_t idesc_qk = 0;
            uint32_t slot = 0, slot_phase = 0;  // loads are used in their order
            uint32_t q_phase = 0, p_phases = 0;  // a bit for each pipeline
            bool ok = true;
            auto next_load = [&]() -> uint32_t {
                const uint32_t st = slot;
                ok = ok && wait(C::SLOT_FULL + 8 * st, slot_phase);
                if (++slot == C::NSLOT) slot = 0, slot_phase ^= 1;
                return st;
            };
            auto release = [&](uint32_t st) { commit_one(sb + C::SLOT_EMPTY + 8 * st, one); };
            // half 0 and half 1 of S_i = Q K^T
            auto qk = [&](int i, uint32_t q_tile, uint32_t st, int half) {
                const uint32_t a = q_lo + q_tile * (C::QTILE >> 4), b = k_lo + st * (C::TILE >> 4);
                constexpr int N = D / 32;
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int kk = half * N + k;
                    mma_ss(tmem + i * 128, a + (((kk >> 2) * C::QHALF + (kk & 3) * 32) >> 4), q_hi,
                           b + (((kk >> 2) * C::HSTEP + (kk & 3) * 32) >> 4), k_hi, idesc_qk, kk > 0, one);
                }
                if (half == 1) commit_one(sb + C::S_FULL + 8 * i, one);
            };
            // keys 0 .. 63 and 64 .. 127 of O_i += P V
            auto pv = [&](int i, uint32_t st, uint32_t phase, uint32_t accumulate, int part) {
                const uint32_t b = v_lo + st * (C::TILE >> 4);
                ok = ok && wait((part == 0 ? C::P_FULL : C::P_REST) + 8 * i, phase);
                if (!ok) return;
                tc_fence_after();
#pragma unroll
                for (int kk = 4 * part; kk < 4 * part + 4; ++kk)
                    mma_ts(tmem + C::O_COL + i * 128, tmem + i * 128 + kk * 8, b + ((kk * 2 * C::GSTRIDE) >> 4), v_hi,
                           C::IDESC_PV, kk > 0 ? 1u : accumulate, one);
                if (part == 0) commit_one(sb + C::O_HALF + 8 * i, one);  // for raise()
            };
            AttnItem u;
            for (int n = 0; ok && take_item(n, u, ok); ++n) {
                Plan plan;
                plan.set(u, gl);
                if (plan.steps == 0) continue;
                const bool wide = plan.wide;
                const int n0 = plan.n0, n1 = plan.n1;
                // a negative scale turns the order of the scores: they are taken with A negated
                idesc_qk = C::IDESC_QK | ((FP8 ? p.qscale * p.k_scales[u.g] : p.qscale) < 0.f ? 1u << 13 : 0u);
                if (!(ok = wait(C::Q_FULL, q_phase))) break;
                q_phase ^= 1;
                mma_any = true;
                int left = plan.steps;  // K tiles not used up yet
                uint32_t ks = next_load(), vs = 0;
                if (!ok) break;
                tc_fence_after();
#pragma unroll (FP8 ? 1 : 2)
                for (int i = 0; i < 2; ++i) {
                    if (i == 1 && !wide) {  // its own K tile
                        release(ks);
                        --left;
                        if (n1 > 0) ks = next_load();
                    }
                    if (!ok || (i ? n1 : n0) == 0) continue;
                    qk(i, wide ? i : 0, ks, 0);
                    qk(i, wide ? i : 0, ks, 1);
                    if (i == 1) {
                        release(ks);
                        --left;
                    }
                }
                if (!ok) break;
                if (left == 0) commit_one(sb + C::Q_EMPTY, one);
                vs = next_load();
                const int nmax = n0 > n1 ? n0 : n1;
                // Steps of the pipelines by turns.  Code that serves both is shorter, code for each
                // has its addresses ready: fp8 kernels, with one role more to hold in the
                // instruction caches, gain by the first (156 -> 147 us on the drafted trees of 24
                // sequences), bf16 kernels by the second (82 against 84 us on packed prompts).
#pragma unroll (FP8 ? 1 : 2)
                for (int x = 0; x < 2 * nmax; ++x) {
                    const int i = x & 1, t = x >> 1, mine = i ? n1 : n0, other = i ? n0 : n1;
                    if (t >= mine) continue;
                    const bool more = t + 1 < mine;
                    const bool lone = !wide || i == 1;             // this pipeline is the last to want its tiles
                    const uint32_t phase = p_phases >> i & 1;
                    pv(i, vs, phase, t > 0, 0);
                    // wide: pipeline 0 brings the next K for both, while it goes on
                    if (more && (!wide || i == 0 || t + 1 >= n0)) ks = next_load();
                    pv(i, vs, phase, t > 0, 1);
                    if (!ok) break;
                    p_phases ^= 1u << i;
                    if (more) qk(i, wide ? i : 0, ks, 0);
                    else commit_one(sb + C::O_FULL + 8 * i, one);
                    if (lone) {
                        release(vs);
                        // the V of what comes next: the other pipeline's step, or this one's
                        if (i == 0 ? t < other : more || t + 1 < other) vs = next_load();
                    }
                    if (more) {
                        qk(i, wide ? i : 0, ks, 1);
                        if (lone) {
                            release(ks);
                            if (--left == 0) commit_one(sb + C::Q_EMPTY, one);
                        }
                    }
                }
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
        bool ok = true;
        auto sync = [&]() -> bool {    // all 256 threads
            arrive(C::SYNC_BAR);
            const bool s = wait(C::SYNC_BAR, sync_phase);
            sync_phase ^= 1;
            return s;
        };
        auto o_readable = [&]() -> bool {  // the item before: O of this pipeline has been read
            if (!x_pending) return true;
            x_pending = false;
            const bool r = wait(C::X_EMPTY, x_phase);
            x_phase ^= 1;
            return r;
        };
        AttnItem u;
        for (int n = 0; ok && take_item(n, u, ok); ++n) {
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
            if constexpr (FP8) qs *= p.k_scales[u.g];
            // (a negative scale: the scores come negated.)  A scale of 0 weighs what is
            // seen alike, and -inf * 0 is not -inf; a scale of NaN stays one
            const float qa = qs == 0.f ? __uint_as_float(1u) : fabsf(qs);
            const float2 q2 = make_float2(qa, qa);
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
                if (!(ok = wait(C::S_FULL + 8 * wg, s_phase))) break;
                s_phase ^= 1;
                tc_fence_after();
                const bool short_step = k0 + C::KEYS > u.kv1 || bad != 0;
                bool masked = short_step || k0 + C::KEYS > clear;
                uint32_t w[4];
                if (masked) {
                    uint32_t there[4];
                    seen_words(par, u.first, qi, k0, w);
                    there_words(u.kv1 - k0, bad, bs, there);
#pragma unroll
                    for (int c = 0; c < 4; ++c) w[c] &= there[c];
                    masked = __any_sync(0xffffffffu, (w[0] & w[1] & w[2] & w[3]) != 0xffffffffu);
                    if (!FP8 && short_step && (!plan.wide || wg == 0 || j >= plan.n0)) {
                        // keys that are not there: their rows of V may hold anything
                        const int li = base + plan.v_load(j), st = li % C::NSLOT;
                        if (!(ok = wait(C::SLOT_FULL + 8 * st, (li / C::NSLOT) & 1))) break;
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
                auto mask32 = [&](float* x, uint32_t word) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = word & (1u << e) ? x[e] : -INFINITY;
                };
                // Weights that take the sum past 2^40 are not used: the row's reference is raised first
                // and they are taken again.  Once: where the reference's own rounding is that large
                // (scores of 2^24 and more) the sum stays as it is, and the row is left to slow_rows.
                bool raised = false;
                auto past = [&](float l_now) -> bool { return __any_sync(0xffffffffu, l_now > 0x1p40f) && !raised; };
                auto lift = [&](float l_now, int c, int n, uint32_t word) {  // scores n c .. n c + n - 1 are in place
                    const bool second = c * n >= 64;
                    const Raised r = raise<D>(p, t_s + n * c, n, word, n == 32 && (c & 1), t_s + 16 * (c - 1),
                                              t > 0 || second ? t_o : ~0u, second ? sb + C::O_HALF + 8 * wg : 0u,
                                              s_phase ^ 1, sb + C::MISC_OFF, qa, m, l, l_now);
                    m = r.m;
                    l = r.l;
                    raised = true;
                    return r.ok;
                };
                if (masked || (t > 0 && __any_sync(0xffffffffu, m == -INFINITY))) {
                    // steps with masks, in a short loop; of its 32 keys a warp's rows mostly see
                    // all or none
#pragma unroll 1
                    for (int c = 0; c < 4;) {
                        uint32_t pk[16];
                        const uint32_t word = !masked ? 0xffffffffu : c == 0 ? w[0] : c == 1 ? w[1] : c == 2 ? w[2] : w[3];
                        if (__any_sync(0xffffffffu, word != 0u)) {
                            float x[32];
                            tmem_ld32(t_s + 32 * c, x);
                            tmem_wait_ld();
                            if (!__all_sync(0xffffffffu, word == 0xffffffffu)) mask32(x, word);
                            // the first keys that a row sees give its reference
                            if (__any_sync(0xffffffffu, m == -INFINITY)) {
                                const float mx = largest32(x, -INFINITY) * qa;
                                m = m == -INFINITY ? mx : m;
                            }
                            const float mm = m == -INFINITY ? 0.f : -m;
                            float2 sum = make_float2(0.f, 0.f);
                            weights<32, false>(x, q2, make_float2(mm, mm), pk, sum);  // exactly 0 where masked
                            const float l_now = l + (sum.x + sum.y);
                            if (past(l_now)) {
                                if (!(ok = lift(l_now, c, 32, word))) break;
                                continue;
                            }
                            l = l_now;
                            raised = false;
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) pk[e] = 0u;
                        }
                        tmem_st16(t_s + 16 * c, pk);  // over scores that have been read
                        if (c & 1) {
                            tmem_wait_st();
                            if (!(ok = o_readable())) break;
                            tc_fence_before();
                            arrive((c == 1 ? C::P_FULL : C::P_REST) + 8 * wg);
                        }
                        ++c;
                    }
                } else {
                    // 64 keys at a time, in a loop: shorter code than the 128 in a row, which kept
                    // the roles waiting for instructions (4096 tokens of 16 heads: 102 us in a row,
                    // 97 in a loop)
                    bool first = t == 0;
#pragma unroll 1
                    for (int c = 0; c < 2;) {
                        float x[64];
                        uint32_t pk[32];
                        tmem_ld32(t_s + 64 * c, x);
                        tmem_ld32(t_s + 64 * c + 32, x + 32);
                        tmem_wait_ld();
                        if (first) {
                            first = false;
                            m = largest32(x, -INFINITY) * qa;  // the row's reference
                            if (!(ok = o_readable())) break;
                        }
                        const float2 m2 = make_float2(-m, -m);
                        float2 sum = make_float2(0.f, 0.f);
                        weights<32, !FP8>(x, q2, m2, pk, sum);
                        weights<32, !FP8>(x + 32, q2, m2, pk + 16, sum);
                        tmem_st32(t_s + 32 * c, pk);
                        const float l_now = l + (sum.x + sum.y);
                        tmem_wait_st();
                        tc_fence_before();
                        // (before the store, this look took 2 % more of a long prompt; scores that the
                        // store went over have to go back)
                        if (past(l_now)) {
                            tmem_st32(t_s + 64 * c, reinterpret_cast<const uint32_t*>(x));
                            tmem_st32(t_s + 64 * c + 32, reinterpret_cast<const uint32_t*>(x) + 32);
                            tmem_wait_st();
                            if (!(ok = lift(l_now, c, 64, 0xffffffffu))) break;
                            continue;
                        }
                        l = l_now;
                        raised = false;
                        // every lane's store is complete: each has waited for it before the vote
                        if (lane == 0) bar_arrive(sb + (c == 0 ? C::P_FULL : C::P_REST) + 8 * wg);
                        ++c;
                    }
                }
                if (!ok) break;
            }
            if (!ok) break;
            base += 2 * plan.steps;
            if (m == -INFINITY) l = 0.f;  // no key seen
            // The reference is a score that the row sees, or at most a power of two above one, and
            // its weight in the sum: less (or more than 2^40) comes of scores whose rounding is
            // larger than a weight's range.  For slow_rows, which rounds a score once.
            else if (!(l >= 0.25f && l <= 0x1p40f)) l = __uint_as_float(0x7fffffffu);
            // ------------------------------------------------ end of the item
            const float vs = FP8 ? p.v_scales[u.g] : 1.f;
            const bool two = !plan.wide && plan.n1 > 0;  // both pipelines hold parts of the same rows
            float w0 = 1.f, w1 = 0.f;
            if (wg == 1 && !plan.wide) {
                if (two) {
                    if (!(ok = o_readable())) break;
                    ml_x[lane_row] = make_float2(m, l);
                    arrive(C::X_FULL);
                    o_phase[1] ^= 1;
                    x_pending = true;
                }
            } else {
                if (nt > 0) {
                    if (!(ok = wait(C::O_FULL + 8 * wg, o_phase[wg]))) break;
                    o_phase[wg] ^= 1;
                }
                if (two) {
                    if (!(ok = wait(C::X_FULL, x_phase))) break;
                    x_phase ^= 1;
                    if (!(ok = wait(C::O_FULL + 8, o_phase[1]))) break;
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
                const int rows_left = rows - row0;  // of this warp
                const bool here = row < rows && PKV_DCHECK(p.err, u.row + (row >> gl) < p.num_tokens && row < p.part_rows);
                const bool split = u.nparts > 1, few = u.nparts <= FEW_PARTS;
                const int slot = attn_partial(blockIdx.x, u.part);
                int* count = split ? p.counters + AttnWalk<TcDivision>::owner(u, walk0.share, 0) * 8 + (warp & 7)
                                   : nullptr;
                // A whole item: o / l.  Part of a split one: o, with its m and l.
                w0 *= split ? vs : l == 0.f ? 0.f : vs / l;  // no key seen: a zero row
                w1 *= split ? vs : l == 0.f ? 0.f : vs / l;
                auto own = [&](int c, float* o) {  // 32 dims of this part
                    if (nt == 0) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.f;
                        return;
                    }
                    tmem_ld32(t_o + c, o);
                    if (two) {
                        float o1[32];
                        tmem_ld32(t_lane + C::O_COL + 128 + c, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = fmaf(o1[e], w1, o[e] * w0);
                    } else {
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= w0;
                    }
                };
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                                     ((long long)(u.row + (row >> gl)) * p.num_heads + u.g * G + (row & (G - 1))) * D;
                const bool sectors = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
                auto store32 = [&](__nv_bfloat16* to, const float* o) {
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        uint32_t r[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) r[i] = pack_bf16(o[e + 2 * i], o[e + 2 * i + 1]);
                        if (sectors) {
                            store_sector(to + e, r);
                        } else {
                            *reinterpret_cast<uint4*>(to + e) = make_uint4(r[0], r[1], r[2], r[3]);
                            *reinterpret_cast<uint4*>(to + e + 8) = make_uint4(r[4], r[5], r[6], r[7]);
                        }
                    }
                };
                float2 odd = make_float2(0.f, 0.f);  // becomes NaN with the first value that is not finite
                auto look = [&](const float* o) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        odd = fma2(make_float2(o[e], o[e + 1]), make_float2(0.f, 0.f), odd);
                };
                auto odd_rows = [&]() {
                    return __ballot_sync(0xffffffffu, here && nt > 0 && !(odd.x + odd.y == 0.f && l == l));
                };
                // Rows of this warp (bits) again; put(rows, which of them) by D / 8 lanes, with eight dims each.
                constexpr int SLOW = FP8 ? 2 : 4;  // what the fp8 kernel's registers hold without spills
                auto redo = [&](uint32_t again, auto&& put) {
                    __syncwarp();
                    while (again) {
                        SlowRows<SLOW> z;
#pragma unroll
                        for (int b = 0; b < SLOW; ++b) {  // fewer rows than SLOW: the last one more than once
                            z.r[b] = again ? row0 + __ffs(again) - 1 : z.r[b ? b - 1 : 0];
                            again &= again - 1;
                        }
                        slow_rows<D, FP8, SLOW>(p, u, sb + C::MISC_OFF, z);
                        if (lane < D / 8) {
#pragma unroll 1
                            for (int b = 0; b < SLOW; ++b) put(z, b);
                        }
                    }
                    __syncwarp();
                };
                if (rows_left <= 0) {
                    // no rows of this warp
                } else if (!split) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float o[32];
                        own(c, o);
                        look(o);
                        if (here) store32(dst + c, o);
                    }
                    redo(odd_rows(), [&](const auto& z, int b) {
                        const int r = z.r[b];
                        __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) +
                                            ((long long)(u.row + (r >> gl)) * p.num_heads + u.g * G + (r & (G - 1))) * D;
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[e] = z.l[b] == 0.f ? 0u : pack_bf16(z.acc[b][2 * e] / z.l[b], z.acc[b][2 * e + 1] / z.l[b]);
                        reinterpret_cast<uint4*>(to)[lane] = make_uint4(y[0], y[1], y[2], y[3]);
                    });
                } else {
                    // With few parts each warp joins its own rows: the last of an item's parts to
                    // come has the others' results at hand and needs not write its own.
                    float4* to = p.ws_o + attn_partial_at(p, slot, D, 0, row);
                    float2* to_ml = p.ws_ml + (long long)slot * p.part_rows + row;
                    auto to_ws = [&](const auto& z, int b) {
                        const int r = z.r[b];
                        float4* to4 = p.ws_o + attn_partial_at(p, slot, D, 8 * lane, r);
                        to4[0] = make_float4(z.acc[b][0], z.acc[b][1], z.acc[b][2], z.acc[b][3]);
                        to4[p.part_rows] = make_float4(z.acc[b][4], z.acc[b][5], z.acc[b][6], z.acc[b][7]);
                        if (lane == 0) p.ws_ml[(long long)slot * p.part_rows + r] = make_float2(z.m[b], z.l[b]);
                    };
                    int seen = 0;
                    if (few && lane == 0) asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(seen) : "l"(count) : "memory");
                    seen = __shfl_sync(0xffffffffu, seen, 0);
                    bool last = few && seen == u.nparts - 1;
                    bool from_ws = !last;  // this row's own part
                    if (!last) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            own(c, o);
                            look(o);
                            if (here) {
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    to[(c / 4 + e) * (long long)p.part_rows] =
                                        make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                            }
                        }
                        if (here) *to_ml = make_float2(m, l);
                        const uint32_t again = odd_rows();
                        redo(again, to_ws);
                    }
                    if (few) {
                        if (!last) {
                            __threadfence();
                            __syncwarp();
                            if (lane == 0) seen = atomicAdd(count, 1);
                            last = __shfl_sync(0xffffffffu, seen, 0) == u.nparts - 1;
                        }
                        if (lane == 0) {
                            if (last) *count = 0;
                            turns[warp] += 1;
                        }
                        if (last) __threadfence();
                        // M = max m_i, out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i, in the parts' order
                        while (last) {
                            float wi[FEW_PARTS], li[FEW_PARTS], M = -INFINITY, L = 0.f;
                            const float4* from[FEW_PARTS];
#pragma unroll
                            for (int i = 0; i < FEW_PARTS; ++i) {
                                wi[i] = -INFINITY;
                                li[i] = 0.f;
                                from[i] = nullptr;
                                if (i >= u.nparts || !here) continue;
                                float2 ml = make_float2(m, l);
                                if (i != u.part || from_ws) {
                                    const int si = attn_partial(AttnWalk<TcDivision>::owner(u, walk0.share, i), i);
                                    ml = __ldcg(&p.ws_ml[(long long)si * p.part_rows + row]);
                                    from[i] = p.ws_o + attn_partial_at(p, si, D, 0, row);
                                }
                                wi[i] = ml.x;
                                li[i] = ml.y;
                                M = fmaxf(M, ml.x);
                            }
#pragma unroll
                            for (int i = 0; i < FEW_PARTS; ++i) {
                                // no key seen in any part: all sums are 0 (or NaN), taken as they are
                                wi[i] = M == -INFINITY ? 1.f : ex2(wi[i] - M);
                                L = fmaf(wi[i], li[i], L);
                            }
                            const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                float o[32], x[32];
                                own(c, x);
                                look(x);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = 0.f;
#pragma unroll
                                for (int i = 0; i < FEW_PARTS; ++i) {
                                    if (i >= u.nparts) continue;
                                    float4 v[8];
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        v[e] = from[i] != nullptr
                                                   ? __ldcg(from[i] + (c / 4 + e) * (long long)p.part_rows)
                                                   : make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
#pragma unroll
                                    for (int e = 0; e < 8; ++e) {
                                        o[4 * e] = fmaf(wi[i], v[e].x, o[4 * e]);
                                        o[4 * e + 1] = fmaf(wi[i], v[e].y, o[4 * e + 1]);
                                        o[4 * e + 2] = fmaf(wi[i], v[e].z, o[4 * e + 2]);
                                        o[4 * e + 3] = fmaf(wi[i], v[e].w, o[4 * e + 3]);
                                    }
                                }
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= inv;
                                if (here) store32(dst + c, o);
                            }
                            // rows of this part, not written so far, that are not finite: once more
                            const bool mine = !from_ws && nt > 0 && here && !(odd.x + odd.y == 0.f && l == l);
                            const uint32_t again = __ballot_sync(0xffffffffu, mine);
                            if (again == 0) break;
                            redo(again, to_ws);
                            from_ws = from_ws || mine;
                        }
                    }
                }
                if (two) {  // the other pipeline's O may be written again
                    tc_fence_before();
                    arrive(C::X_EMPTY);
                }
            }
            if (u.nparts > FEW_PARTS) {
                if (!(ok = attn_merge<TcDivision, __nv_bfloat16, D, 256>(p, u, walk0.share, merge_flag, turns, tid, sync)))
                    break;
            }
        }
        if (!ok && lane == 0) {
            // given up: parts that this warp has not counted become empty ones, so that the
            // counters end at zero and the others' results meet nothing stale
            AttnWalk<TcDivision> walk = *reinterpret_cast<const AttnWalk<TcDivision>*>(smem + C::WALK_OFF);
            int k = 0;
            while (walk.next(p, (int)blockIdx.x, u)) {
                const int n_rows = u.ntok << gl, first_row = n_rows > 128 ? warp * 32 : (warp & 3) * 32;
                const bool few = u.nparts <= FEW_PARTS;
                if (u.nparts == 1 || (few ? first_row >= n_rows || (n_rows <= 128 && warp >= 4) : warp > 0)) continue;
                if (k++ < turns[warp]) continue;
                const int n = few && n_rows > first_row + 32 ? first_row + 32 : n_rows;
                for (int r = few ? first_row : 0; r < n; ++r)
                    p.ws_ml[(long long)attn_partial(blockIdx.x, u.part) * p.part_rows + r] = make_float2(-INFINITY, 0.f);
                __threadfence();
                int* c = p.counters + AttnWalk<TcDivision>::owner(u, walk.share, 0) * 8 + warp;
                if (atomicAdd(c, 1) == u.nparts - 1) *c = 0;
            }
        }
    } else {
        // ----------------------------------------------------------- widening
        if constexpr (FP8) {
            regs_dec<C::REGS_WIDEN>();
            // A thread's 16-byte chunks of a raw tile: the same place c of rows r0, r0 + RSTEP, ..;
            // widened they are two chunks.  Threads with the second half of a row store them in the
            // other order: no bank conflicts.
            constexpr int CPR = D / 16, RSTEP = C::WIDEN / CPR;
            static_assert(RSTEP % 8 == 0, "rows of a thread have the same place in the swizzle");
            const int tw = tid - 384, c = tw % CPR, r0 = tw / CPR, second = (c >> 2) & 1;
            const int to0 = (r0 >> 3) * C::GSTRIDE + (c >> 2) * C::HSTEP + (r0 & 7) * 128;
            const int to_a = to0 + (((2 * (c & 3) + second) ^ (r0 & 7)) << 4);
            const int to_b = to0 + (((2 * (c & 3) + 1 - second) ^ (r0 & 7)) << 4);
            uint32_t rs = 0, raw_phase = 0, st = 0, empty_phase = 1;
            bool ok = true;
            AttnItem u;
            for (int n = 0; ok && take_item(n, u, ok); ++n) {
                Plan plan;
                plan.set(u, gl);
                if (plan.steps == 0) continue;
                const int32_t* bt = p.block_tables + (long long)u.seq * p.max_blocks_per_seq;
                for (int lo = 0; lo < 2 * plan.steps; ++lo) {
                    bool v;
                    const int k0 = u.kv0 + plan.load_step(lo, v) * C::KEYS;
                    const int key = k0 + lane * bs;
                    const int e = lane < bpt && key < u.kv1 ? __ldg(bt + (key >> bl)) : 0;
                    const uint32_t bad = __ballot_sync(0xffffffffu, e < 0 || e >= p.num_blocks);
                    const bool short_step = k0 + C::KEYS > u.kv1 || bad != 0;
                    uint32_t there[4];
                    if (short_step) there_words(u.kv1 - k0, bad, bs, there);
                    if (!(ok = wait(C::LOAD_FULL + 8 * rs, raw_phase))) break;
                    if (!(ok = wait(C::SLOT_EMPTY + 8 * st, empty_phase))) break;
                    const unsigned char* raw = smem + C::RAW_OFF + rs * C::RAW + tw * 16;
                    unsigned char* wide = smem + C::SLOT_OFF + st * C::TILE;
                    // (in full unrolled, this loop made the whole kernel a tenth slower, by two 3 %: the
                    // instruction caches hold its code beside the softmax's)
#pragma unroll 1
                    for (int r = r0; r < C::KEYS; r += RSTEP) {
                        uint4 w = *reinterpret_cast<const uint4*>(raw);
                        if (short_step) {
                            const uint32_t word = r < 32 ? there[0] : r < 64 ? there[1] : r < 96 ? there[2] : there[3];
                            if (!(word >> (r & 31) & 1)) w = make_uint4(0u, 0u, 0u, 0u);
                        }
                        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
                        uint32_t y[8];
#pragma unroll
                        for (int e2 = 0; e2 < 4; ++e2) {
                            uint32_t h[2];  // f16 pairs
                            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                                "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                                : "=r"(h[0]), "=r"(h[1])
                                : "r"(in[e2]));
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
                                y[2 * e2 + k] = pack_bf16(f.x, f.y);
                            }
                        }
                        const uint4 a = make_uint4(y[0], y[1], y[2], y[3]), b = make_uint4(y[4], y[5], y[6], y[7]);
                        *reinterpret_cast<uint4*>(wide + to_a) = second ? b : a;
                        *reinterpret_cast<uint4*>(wide + to_b) = second ? a : b;
                        raw += C::WIDEN * 16;
                        wide += RSTEP / 8 * C::GSTRIDE;
                    }
                    fence_proxy_async_smem();
                    arrive(C::SLOT_FULL + 8 * st);
                    if (lane == 0) bar_arrive(sb + C::LOAD_EMPTY + 8 * rs);
                    if (++rs == C::NRAW) rs = 0, raw_phase ^= 1;
                    if (++st == C::NSLOT) st = 0, empty_phase ^= 1;
                }
            }
        }
    }

    // ------------------------------------------------------------- wind down
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (load_words(sb + C::MISC_OFF).x != 0u) {
        // copies and products in flight land before the CTA leaves; each wait is bounded
        auto land = [&](uint32_t off, uint32_t parity) {
            const unsigned long long t0 = globaltimer_ns();
            while (!bar_try(sb + off, parity, 1000u))
                if (globaltimer_ns() - t0 > kWaitTimeoutNs) break;
        };
        if (warp == 8 && lane == 0) {
            for (int li = loads > C::NLOAD ? loads - C::NLOAD : 0; li < loads; ++li)
                land(C::LOAD_FULL + 8 * (li % C::NLOAD), (li / C::NLOAD) & 1);
            if (q_loads > 0) land(C::Q_FULL, (q_loads - 1) & 1);
        }
        if (warp == 9 && mma_any) {
            commit_one(sb + C::MMA_DONE, elect_one());
            land(C::MMA_DONE, 0);
        }
        tc_fence_before();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 9) tc::tmem_dealloc(tmem, C::TMEM_COLS);
}

}  // namespace atc
}  // namespace pkv
