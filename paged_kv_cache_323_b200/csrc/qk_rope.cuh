// qk_rope.cuh -- what lies between the q/k/v projection and the attention:
// per-head RMS norm of q and k, the position rotation, and the store of k and
// v into their slots of the paged cache, in one pass.
//
//   x' = x * rsqrt(mean(x^2) + eps) * w          (per head; no norm when w is null)
//   a_i = position[axis(i)] * inv_freq[i]        (i < R / 2; R = rotary dims)
//   (x'_p, x'_r) -> (x'_p cos a_i - x'_r sin a_i, x'_r cos a_i + x'_p sin a_i)
// with the pair (p, r) = (i, i + R/2), or (2i, 2i + 1) when interleaved; dims
// from R on stay.  v is stored as it is.  Everything is fp32 until the one
// rounding to the output's type (for an fp8 cache: of value / scale to e4m3).
//
// Angles.  fp32 has no room for them (at position 10^6 its spacing is 0.06), so
// the product is taken in fp64, brought into [-pi, pi] there and only then
// rounded; the sine and cosine of a token's pairs are computed once and serve
// all its heads.  (The product is exact for positions below 2^29.  From there on
// a 24-bit by a 31-bit number may need 55 bits where fp64 has 53: the farthest
// angles are within 2^-22 radians at frequencies up to 1.)  With bf16 rows sine
// and cosine come from the special-function unit, within 2^-21: a thousandth of
// a bf16 step.
//
// Bound: HBM in bytes (one read of q, k, v and one write), and close behind it
// the instructions of some 80 rows of 128 values a token.  A lane holds both
// values of its pairs: it owns two 16-byte pieces of a row, R/2 dims apart
// where pairs are, so that only the sum of squares crosses lanes (a row is 4
// to 16 of them).  A CTA takes up to eight tokens, computes their angles side
// by side, and runs through their q rows, k rows and v rows, so that one
// kind's weights are in registers at a time; the cosines and sines of a row
// come from shared memory.
#pragma once

#include "common.cuh"
#include "f32x2.cuh"

namespace pkv {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxAxes = 4;
constexpr int kRopeMaxTokens = 8;  // of a CTA

struct RopeParams {
    void* q_out;
    const void* q;
    const void* k;
    const void* v;
    void* k_cache;
    void* v_cache;
    const float* k_scales;  // fp8 caches, else null
    const float* v_scales;
    const int64_t* slot_mapping;
    const int32_t* positions;  // [axes][num_tokens]
    const float* inv_freq;     // [pairs]
    const void* q_weight;      // [D] or null
    const void* k_weight;
    int* err;
    long long q_out_stride, q_stride, k_stride, v_stride;  // elements between two tokens
    long long num_slots;
    int num_tokens;
    int num_heads;
    int num_kv_heads;
    int block_size;
    int pairs;                       // R / 2
    int axis_end[kRopeMaxAxes];      // first pair past each axis; INT_MAX from the last axis on
    int tokens_per_cta;
    int head_splits;                 // CTAs that share a token's heads
    int kinds_apart;                 // 1: q, k and v rows of a token go to three CTAs
    float eps;
};

// Cosine and sine of position `pos` at frequency f; the angle within [-pi, pi].
template <bool EXACT>
__device__ __forceinline__ float2 rope_turn(int pos, float f) {
    const double a = (double)pos * (double)f;
    const double k = rint(a * 0.15915494309189535);  // 1 / (2 pi)
    // 2 pi as two doubles, the first of them subtracted with one rounding
    const double r = fma(-k, 2.4492935982947064e-16, fma(-k, 6.283185307179586, a));
    float s, c;
    if constexpr (EXACT) {
        sincosf((float)r, &s, &c);
    } else {
        s = __sinf((float)r);
        c = __cosf((float)r);
    }
    return make_float2(c, s);
}

// A lane's piece of a row: 16 bytes, as pairs of values.
template <typename T>
struct RopePiece;
template <>
struct RopePiece<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 r, float2* x) {
        x[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
        x[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
    }
    static __device__ __forceinline__ uint4 pack(const float2* x) {
        return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                          __float_as_uint(x[1].y));
    }
};
template <>
struct RopePiece<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 r, float2* x) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    static __device__ __forceinline__ uint4 pack(const float2* x) {  // nearest even
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __float22bfloat162_rn(x[i]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// x / scale, correctly rounded, given r = 1 / scale correctly rounded: the
// quotient's residual is exact in one fma, and one more rounds it (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000", 1990).
// Infinities and NaN are those of x r, and a zero keeps its sign with the
// residual taken this way round.  Holds for scales from 2^-90 to 2^100: r is a
// normal number there, and where the residual is not exact (|x| below 2^-103)
// the quotient is below 2^-13, the smallest code's half 2^-10.
__device__ __forceinline__ float rope_quotient(float x, float scale, float r) {
    const float q = x * r;
    const float y = fmaf(-fmaf(q, scale, -x), r, q);
    return fabsf(q) < INFINITY ? y : q;
}
// Any other scale: values and scale times a power of two (or minus one) that
// brings it there.  Values that overflow or lose bits by it have codes of 448
// and 0 all the same.
__device__ __forceinline__ float rope_factor(float scale) {
    const float a = fabsf(scale);
    return copysignf(a < 0x1p-90f ? 0x1p64f : a > 0x1p100f ? 0x1p-64f : 1.f, scale);
}

// Eight codes of value / scale, rounded to nearest even, saturated at 448.
__device__ __forceinline__ uint2 rope_codes(const float2* x, float scale, float r) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            w[i] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(rope_quotient(x[2 * i + j].x, scale, r),
                                                                   rope_quotient(x[2 * i + j].y, scale, r)),
                                                       __NV_SATFINITE, __NV_E4M3)
                    << (16 * j);
    }
    return make_uint2(w[0], w[1]);
}

template <typename T, int D, bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, 4) qk_rope_kernel(const RopeParams p) {
    // a decode launched next as a programmatic dependent may start now; it
    // waits for this grid to finish before it reads the pools
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    using Piece = RopePiece<T>;
    constexpr int N = Piece::N;              // values of a piece
    constexpr int M = N / 2;                 // as pairs
    constexpr int LPR = D / (2 * N);         // lanes per row
    constexpr int RPI = kRopeThreads / LPR;  // rows per pass of the CTA
    __shared__ __align__(16) float2 cs[kRopeMaxTokens][D / 2];  // (cos, sin) of the tokens' pairs
    __shared__ long long rows_at[kRopeMaxTokens];  // row of the token's slot, kv head 0, in the pools; -1: none
    const int tid = threadIdx.x;
    const int c = tid % LPR, rg = tid / LPR;
    const int H = p.num_heads, Hkv = p.num_kv_heads;
    const int block = p.kinds_apart ? blockIdx.x / 3 : blockIdx.x;
    const int kind = p.kinds_apart ? blockIdx.x % 3 : -1;  // 0 q, 1 k, 2 v; -1: all
    const int split = block % p.head_splits;
    const int t0 = (block / p.head_splits) * p.tokens_per_cta;
    const int tokens = p.num_tokens - t0 < p.tokens_per_cta ? p.num_tokens - t0 : p.tokens_per_cta;

    // the lane's two pieces: of its N pairs, or the next 2 N dims in a row (adjacent
    // pairs; dims past the rotary ones)
    const bool turns = c * N < p.pairs;
    const int d0 = INTERLEAVED || !turns ? 2 * N * c : N * c;
    const int d1 = INTERLEAVED || !turns ? d0 + N : d0 + p.pairs;

    // Rows (token j, head h) of one kind, j-major, RPI a pass; each(j, h, live, pieces),
    // the next ones on their way.  The first ones are loaded before ready().
    auto rows = [&](const void* base, long long stride, int count, auto&& ready, auto&& each) {
        const int total = tokens * count, step = p.head_splits * RPI;
        int j = (split * RPI + rg) / count, h = split * RPI + rg - j * count;
        uint4 next[2];
        auto load = [&] {
            next[0] = next[1] = make_uint4(0u, 0u, 0u, 0u);
            if (j < tokens) {
                const T* src = static_cast<const T*>(base) + (long long)(t0 + j) * stride + h * D;
                next[0] = *reinterpret_cast<const uint4*>(src + d0);
                next[1] = *reinterpret_cast<const uint4*>(src + d1);
            }
        };
        load();
        ready();
        // whole warps stay in the loop, so the shuffles see every lane
        for (int r0 = split * RPI; r0 < total; r0 += step) {
            const uint4 r[2] = {next[0], next[1]};
            const int j_now = j, h_now = h;
            h += step;
            if (h >= count) {
                const int more = h / count;
                j += more;
                h -= more * count;
            }
            if (r0 + step < total) load();
            each(j_now, h_now, j_now < tokens, r);
        }
    };
    // norm and rotation of a lane's 2 N values
    auto turn = [&](float2* x, int j, bool norm, const float2* w) {
        if (norm) {
            float2 sq = mul2(x[0], x[0]);
#pragma unroll
            for (int e = 1; e < 2 * M; ++e) sq = fma2(x[e], x[e], sq);
            float ss = sq.x + sq.y;
#pragma unroll
            for (int d = LPR / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            const float inv = rsqrtf(fmaf(ss, 1.f / D, p.eps));  // within 2 ulp
#pragma unroll
            for (int e = 0; e < 2 * M; ++e) x[e] = mul2(x[e], mul2(w[e], make_float2(inv, inv)));
        }
        if (!turns || j >= tokens) return;
#pragma unroll
        for (int e = 0; e < M; ++e) {
            const float4 z = *reinterpret_cast<const float4*>(&cs[j][N * c + 2 * e]);  // cos, sin of two pairs
            const float2 co = make_float2(z.x, z.z), si = make_float2(z.y, z.w);
            float2 u = x[e], v = x[M + e];
            if constexpr (INTERLEAVED) {  // two pairs in a row
                u = make_float2(x[2 * e].x, x[2 * e + 1].x);
                v = make_float2(x[2 * e].y, x[2 * e + 1].y);
            }
            const float2 a = fma2(u, co, mul2(v, make_float2(-si.x, -si.y)));
            const float2 b = fma2(v, co, mul2(u, si));
            if constexpr (INTERLEAVED) {
                x[2 * e] = make_float2(a.x, b.x);
                x[2 * e + 1] = make_float2(a.y, b.y);
            } else {
                x[e] = a;
                x[M + e] = b;
            }
        }
    };
    auto weights = [&](const void* w, float2* to) {
        Piece::unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(w) + d0), to);
        Piece::unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(w) + d1), to + M);
    };
    // a row of a pool
    auto store = [&](void* cache, const float* scales, int j, int g, float2* x) {
        const long long row = rows_at[j];
        if (row < 0 || !PKV_DCHECK(p.err, row + (long long)g * p.block_size < p.num_slots * Hkv && j < tokens)) return;
        const long long at = (row + (long long)g * p.block_size) * D;
        if constexpr (FP8) {
            uint8_t* to = static_cast<uint8_t*>(cache) + at;
            float scale = scales[g];
            if (!(scale >= 0x1p-90f && scale <= 0x1p100f)) {
                const float f = rope_factor(scale);
                scale *= f;
#pragma unroll
                for (int e = 0; e < 2 * M; ++e) x[e] = mul2(x[e], make_float2(f, f));
            }
            const float r = __frcp_rn(scale);
            if (scale == INFINITY) scale = 1.f;  // (r = 0)
            *reinterpret_cast<uint2*>(to + d0) = rope_codes(x, scale, r);
            *reinterpret_cast<uint2*>(to + d1) = rope_codes(x + M, scale, r);
        } else {
            T* to = static_cast<T*>(cache) + at;
            *reinterpret_cast<uint4*>(to + d0) = Piece::pack(x);
            *reinterpret_cast<uint4*>(to + d1) = Piece::pack(x + M);
        }
    };

    float2 w[2 * M];
    const bool norm_q = p.q_weight != nullptr, norm_k = p.k_weight != nullptr;
    auto angles = [&] {
        for (int n = tid; n < tokens * p.pairs; n += kRopeThreads) {
            const int j = n / p.pairs, i = n - j * p.pairs;
            int axis = 0;
#pragma unroll
            for (int x = 0; x < kRopeMaxAxes - 1; ++x) axis += i >= p.axis_end[x];
            cs[j][i] = rope_turn<sizeof(T) == 4>(p.positions[(long long)axis * p.num_tokens + t0 + j], p.inv_freq[i]);
        }
    };
    auto places = [&] {
        if (tid >= tokens) return;
        const long long slot = p.slot_mapping[t0 + tid];
        if (slot >= p.num_slots && split == 0) set_error(p.err, PKV_ERR_DEVICE_BOUNDS);
        const long long blk = slot / p.block_size;
        rows_at[tid] =
            slot >= 0 && slot < p.num_slots ? blk * Hkv * p.block_size + (slot - blk * p.block_size) : -1;
    };
    if (kind <= 0)
        rows(p.q, p.q_stride, H,
             [&] {
                 if (norm_q) weights(p.q_weight, w);
                 angles();
                 if (kind < 0) places();
                 __syncthreads();
             },
             [&](int j, int h, bool live, const uint4* r) {
                 float2 x[2 * M];
                 Piece::unpack(r[0], x);
                 Piece::unpack(r[1], x + M);
                 turn(x, j, norm_q, w);
                 if (!live) return;
                 T* to = static_cast<T*>(p.q_out) + (long long)(t0 + j) * p.q_out_stride + h * D;
                 *reinterpret_cast<uint4*>(to + d0) = Piece::pack(x);
                 *reinterpret_cast<uint4*>(to + d1) = Piece::pack(x + M);
             });
    if (kind < 0 || kind == 1)
        rows(p.k, p.k_stride, Hkv,
             [&] {
                 if (norm_k) weights(p.k_weight, w);
                 if (kind == 1) {
                     angles();
                     places();
                     __syncthreads();
                 }
             },
             [&](int j, int g, bool live, const uint4* r) {
                 float2 x[2 * M];
                 Piece::unpack(r[0], x);
                 Piece::unpack(r[1], x + M);
                 turn(x, j, norm_k, w);
                 if (live) store(p.k_cache, p.k_scales, j, g, x);
             });
    if (kind < 0 || kind == 2)
        rows(p.v, p.v_stride, Hkv,
             [&] {
                 if (kind == 2) {
                     places();
                     __syncthreads();
                 }
             },
             [&](int j, int g, bool live, const uint4* r) {
                 if (!live) return;
                 float2 x[2 * M];
                 Piece::unpack(r[0], x);
                 Piece::unpack(r[1], x + M);
                 store(p.v_cache, p.v_scales, j, g, x);  // bf16 and fp32: the same bits
             });
}

}  // namespace pkv
