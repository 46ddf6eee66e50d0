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
// Angles.  fp32 has no room for them (position 10^6 times 1 has half a radian
// of spacing 0.06), so the product, exact in fp64 (a 24-bit by a 31-bit
// number), is brought into [-pi, pi] there and only then rounded; the sine and cosine of
// a token's pairs are computed once and serve all its heads.
//
// Bound: HBM.  One read of q, k, v and one write; a lane owns 16 bytes of a
// row, so a row is 8 to 32 lanes, sums of squares and the partner of a pair
// come from lane shuffles, and a lane keeps the sines, cosines and weights of
// its dims in registers for all heads of a token.
#pragma once

#include "common.cuh"

namespace pkv {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxAxes = 4;

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
    float eps;
};

// Angle of position `pos` at frequency f, reduced to [-pi, pi].
__device__ __forceinline__ float rope_angle(int pos, float f) {
    const double a = (double)pos * (double)f;
    const double k = rint(a * 0.15915494309189535);  // 1 / (2 pi)
    // 2 pi as two doubles, the first of them subtracted with one rounding
    const double r = fma(-k, 2.4492935982947064e-16, fma(-k, 6.283185307179586, a));
    return (float)r;
}

// 16 bytes of a row, each value rounded to the row's type (nearest even).
__device__ __forceinline__ void store_row16(float* dst, const float (&x)[4]) {
    *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_row16(__nv_bfloat16* dst, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int D, bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const RopeParams p) {
    // a decode launched next as a programmatic dependent may start now; it
    // waits for this grid to finish before it reads the pools
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int VE = Elem<T>::kPer16B;  // values per lane
    constexpr int LPR = D / VE;           // lanes per row
    constexpr int RPI = kRopeThreads / LPR;  // rows per pass of the CTA
    __shared__ float2 cs[D / 2];          // (cos, sin) of the token's pairs
    const int tid = threadIdx.x;
    const int c = tid % LPR, rg = tid / LPR;
    const int H = p.num_heads, Hkv = p.num_kv_heads, NH = H + 2 * Hkv;
    const int half = p.pairs / VE;        // lanes of half the rotary dims (pairs split in halves)
    const int split = blockIdx.x % p.head_splits;
    const int t0 = (blockIdx.x / p.head_splits) * p.tokens_per_cta;
    const int t1 = t0 + p.tokens_per_cta < p.num_tokens ? t0 + p.tokens_per_cta : p.num_tokens;

    float wq[VE], wk[VE];
    const bool norm_q = p.q_weight != nullptr, norm_k = p.k_weight != nullptr;
    if (norm_q) Elem<T>::unpack(static_cast<const uint4*>(p.q_weight)[c], wq);
    if (norm_k) Elem<T>::unpack(static_cast<const uint4*>(p.k_weight)[c], wk);

    for (int t = t0; t < t1; ++t) {
        if (t > t0) __syncthreads();
        for (int i = tid; i < p.pairs; i += kRopeThreads) {
            int axis = 0;
#pragma unroll
            for (int x = 0; x < kRopeMaxAxes - 1; ++x) axis += i >= p.axis_end[x];
            float s, co;
            sincosf(rope_angle(p.positions[(long long)axis * p.num_tokens + t], p.inv_freq[i]), &s, &co);
            cs[i] = make_float2(co, s);
        }
        const long long slot = p.slot_mapping[t];
        if (slot >= p.num_slots && tid == 0) set_error(p.err, PKV_ERR_DEVICE_BOUNDS);
        const bool keep = slot >= 0 && slot < p.num_slots;
        const long long blk = keep ? slot / p.block_size : 0;
        const long long off = keep ? slot - blk * p.block_size : 0;
        __syncthreads();
        // the lane's pairs: with halves, dims 8c + e pair with lane c +- half's
        float co[INTERLEAVED ? VE / 2 : VE], si[INTERLEAVED ? VE / 2 : VE];
        const bool turns = INTERLEAVED ? c * VE < 2 * p.pairs : c < 2 * half;
        const int partner = INTERLEAVED ? 0 : (c < half ? c + half : c - half);
        if (turns) {
            constexpr int N = INTERLEAVED ? VE / 2 : VE;
            const int i0 = INTERLEAVED ? c * VE / 2 : (c < half ? c : c - half) * VE;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float2 z = cs[i0 + e];
                co[e] = z.x;
                si[e] = !INTERLEAVED && c < half ? -z.y : z.y;
            }
        }
        // rows of the token: q heads, k heads, v heads.  Whole warps stay in
        // the loop, so the shuffles see every lane
        for (int h0 = split * RPI; h0 < NH; h0 += p.head_splits * RPI) {
            const int h = h0 + rg;
            const bool live = h < NH && (h < H || keep);
            const bool is_q = h < H, is_k = !is_q && h < H + Hkv;
            const T* src = static_cast<const T*>(is_q ? p.q : is_k ? p.k : p.v) +
                           (is_q   ? (long long)t * p.q_stride + h * D
                            : is_k ? (long long)t * p.k_stride + (h - H) * D
                                   : (long long)t * p.v_stride + (h - H - Hkv) * D);
            uint4 raw = make_uint4(0u, 0u, 0u, 0u);
            if (live) raw = *reinterpret_cast<const uint4*>(src + c * VE);
            float x[VE];
            Elem<T>::unpack(raw, x);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < VE; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int d = LPR / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            if (is_q ? norm_q : is_k && norm_k) {
                // 1 / sqrt(mean + eps), correctly rounded steps: once per row
                const float inv = 1.f / sqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
                for (int e = 0; e < VE; ++e) x[e] *= inv * (is_q ? wq[e] : wk[e]);
            }
            const bool turn = turns && (is_q || is_k);
            if constexpr (INTERLEAVED) {
                if (turn) {
#pragma unroll
                    for (int e = 0; e < VE / 2; ++e) {
                        const float a = x[2 * e], b = x[2 * e + 1];
                        x[2 * e] = a * co[e] - b * si[e];
                        x[2 * e + 1] = b * co[e] + a * si[e];
                    }
                }
            } else {
                const int from = (tid & 31 & ~(LPR - 1)) + (turns ? partner : c);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float y = __shfl_sync(0xffffffffu, x[e], from);
                    if (turn) x[e] = x[e] * co[e] + y * si[e];
                }
            }
            if (!live) continue;
            if (is_q) {
                store_row16(static_cast<T*>(p.q_out) + (long long)t * p.q_out_stride + h * D + c * VE, x);
            } else {
                const int g = is_k ? h - H : h - H - Hkv;
                const long long at = ((blk * Hkv + g) * p.block_size + off) * D + c * VE;
                if constexpr (FP8) {
                    const float scale = (is_k ? p.k_scales : p.v_scales)[g];
                    uint8_t* dst = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) + at;
                    uint32_t w[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        w[i] = 0;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            w[i] |= (uint32_t)__nv_cvt_float2_to_fp8x2(
                                        make_float2(__fdiv_rn(x[4 * i + 2 * j], scale),
                                                    __fdiv_rn(x[4 * i + 2 * j + 1], scale)),
                                        __NV_SATFINITE, __NV_E4M3)
                                    << (16 * j);
                    }
                    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
                } else if (is_k) {
                    store_row16(static_cast<T*>(p.k_cache) + at, x);
                } else {
                    *reinterpret_cast<uint4*>(static_cast<T*>(p.v_cache) + at) = raw;
                }
            }
        }
    }
}

}  // namespace pkv
