// attn_simt.cuh -- multi-query attention over the paged cache on the CUDA
// cores, in fp32 throughout: prompt attention and drafted-tree attention over
// fp32 caches.
//
//   out_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = 2^(x_rj - m_r),  x = scale log2(e) q . k
// over the keys row r sees, with the running maximum m and sum of a softmax in
// one pass over the keys.
//
// A CTA of 256 threads (a 16 x 16 grid) takes items of ROWS = 64 rows in 64-key
// steps, or of 16 rows in calls of few rows a sequence.  Q, K and V are staged
// in shared memory; a thread holds an R x 4 piece of the scores (rows R ty + i,
// keys tx + 16 j; R = ROWS / 16) and an R x D/16 piece of the output.  Per 4
// dims of the head it reads R + 4 float4 for 16 R FMAs, which with R = 4 puts
// the kernel near what shared memory can feed; padded rows keep those reads
// free of bank conflicts.  The scores go from one thread to the others of its
// row through K's space, so two CTAs fit an SM and one's loads overlap the
// other's products.
#pragma once

#include "attn_common.cuh"

namespace pkv {

// A 64-key step is long enough to be a part of its own in calls that do not
// fill the SMs otherwise.
template <int ROWS>
using SimtDivision = AttnDivision<ROWS, ROWS, 1, 1, 64, 64, 16>;

template <int D, int ROWS_>
struct SimtCfg {
    static constexpr int ROWS = ROWS_, KEYS = 64, THREADS = 256;
    static constexpr int R = ROWS / 16;  // rows per thread
    static constexpr int CTAS_PER_SM = 2;
    static constexpr int LD = D + 4;  // padded row of Q and K
    static constexpr int LP = KEYS + 4;
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = ROWS * LD;
    static constexpr int V_OFF = K_OFF + KEYS * LD;
    static constexpr int FLOATS = V_OFF + KEYS * D;
    static constexpr int SMEM_BYTES = FLOATS * 4;
    static_assert(ROWS * LP <= KEYS * LD, "the probabilities reuse K's space");
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <int D, int ROWS>
__global__ void __launch_bounds__(256, 2) attn_simt_kernel(const AttnParams p) {
    using C = SimtCfg<D, ROWS>;
    using Div = SimtDivision<ROWS>;
    constexpr int R = C::R;
    extern __shared__ __align__(16) float simt_smem[];
    float* sq = simt_smem + C::Q_OFF;
    float* sk = simt_smem + C::K_OFF;
    float* sp = sk;
    float* sv = simt_smem + C::V_OFF;
    __shared__ int flag, turns;
    __shared__ AttnItem item[2];
    __shared__ long long walk_scratch[C::THREADS / 32 + 8];
    const int tid = threadIdx.x;
    const int tx = tid & 15, ty = tid >> 4;
    const int G = 1 << p.group_log2, Hkv = p.num_kv_heads, bs = p.block_size;
    constexpr int OJ = D / 64;  // float4 columns of the output per thread
    constexpr int C4 = D / 4;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    AttnWalk<Div> walk = attn_walk_start<Div, C::THREADS>(p, walk_scratch);
    for (int n = 0;; ++n) {
        // the walk, by thread 0; a slot is written again only after the barrier of the item between
        if (tid == 0 && !walk.next(p, (int)blockIdx.x, item[n & 1])) item[n & 1].seq = -1;
        __syncwarp();
        __syncthreads();
        const AttnItem u = item[n & 1];
        if (u.seq < 0) break;
        const int g = u.g;
        const int rows = u.ntok << p.group_log2;
        const float qscale = p.qscale;
        const int32_t* bt = p.block_tables + (long long)u.seq * p.max_blocks_per_seq;
        const int32_t* par = p.parents ? p.parents + (u.row - (u.pos - u.first)) : nullptr;
        if (par != nullptr && u.part == 0 && g == 0) attn_check_parents(p, u, tid, C::THREADS);
        for (int i = tid; i < C::ROWS * C4; i += C::THREADS) {
            const int r = i / C4, c = i % C4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows)
                v = load4(static_cast<const float*>(p.q) + (long long)(u.row + (r >> p.group_log2)) * p.q_stride +
                          (g * G + (r & (G - 1))) * D + 4 * c);
            *reinterpret_cast<float4*>(sq + r * C::LD + c * 4) = v;
        }
        float m[R], l[R], o[R][4 * OJ];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 4 * OJ; ++j) o[i][j] = 0.f;
        }
        for (int k0 = u.kv0; k0 < u.kv1; k0 += C::KEYS) {
            __syncthreads();
            // K and V rows of the step; rows past the part's end, and of blocks outside the
            // pool, are zeros that no row sees (and that nothing is multiplied into)
            int bad = 0;
            constexpr int N = C::KEYS * C4 / C::THREADS;  // float4 of K, and of V, per thread
            int e[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int key = k0 + (tid + n * C::THREADS) / C4;
                e[n] = key < u.kv1 ? bt[key / bs] : -1;
                if (key < u.kv1 && (e[n] < 0 || e[n] >= p.num_blocks)) {
                    bad = 1;
                    e[n] = -1;
                }
            }
#pragma unroll
            for (int n0 = 0; n0 < N; n0 += 4) {
                float4 kv[4], vv[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int i = tid + (n0 + n) * C::THREADS, r = i / C4, c = i % C4;
                    kv[n] = vv[n] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (e[n0 + n] >= 0 && PKV_DCHECK(p.err, e[n0 + n] < p.num_blocks && g < Hkv)) {
                        const long long at = (((long long)e[n0 + n] * Hkv + g) * bs + (k0 + r) % bs) * D + 4 * c;
                        kv[n] = load4(static_cast<const float*>(p.k_cache) + at);
                        vv[n] = load4(static_cast<const float*>(p.v_cache) + at);
                    }
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int i = tid + (n0 + n) * C::THREADS, r = i / C4, c = i % C4;
                    *reinterpret_cast<float4*>(sk + r * C::LD + c * 4) = kv[n];
                    *reinterpret_cast<float4*>(sv + r * D + c * 4) = vv[n];
                }
            }
            if (bad) set_error(p.err, PKV_ERR_DEVICE_BOUNDS);
            bad = __syncthreads_or(bad);
            float s[R][4];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
            for (int c = 0; c < C4; ++c) {
                float4 a[R], b[4];
#pragma unroll
                for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4*>(sq + (R * ty + i) * C::LD + 4 * c);
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * C::LD + 4 * c);
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
                        s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
                        s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
                        s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
                    }
            }
            // keys every row of the tile sees need no test
            const int seen_by_all = p.parents ? u.first : u.pos + 1;
            const bool masked = bad || k0 + C::KEYS > (seen_by_all < u.kv1 ? seen_by_all : u.kv1);
            float alpha[R];
            uint32_t unseen = 0u;  // a bit for each of the thread's scores
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int r = R * ty + i;
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] *= qscale;
                    if (masked) {
                        const int key = k0 + tx + 16 * j;
                        bool ok = r < rows && key < u.kv1;
                        if (ok) ok = sees(par, u.first, u.pos - u.first + (r >> p.group_log2), key);
                        if (ok && bad) {
                            const int e = bt[key / bs];
                            ok = e >= 0 && e < p.num_blocks;
                        }
                        if (!ok) {
                            s[i][j] = -INFINITY;
                            unseen |= 1u << (4 * i + j);
                        }
                    }
                    mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int d = 8; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float mn = fmaxf(m[i], mx);
                alpha[i] = mn == -INFINITY ? 1.f : exp2f(m[i] - mn);
                m[i] = mn;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // -inf scores weigh zero whatever the maximum is
                    s[i][j] = s[i][j] == -INFINITY ? 0.f : exp2f(s[i][j] - mn);
                    sum += s[i][j];
                }
                l[i] = fmaf(l[i], alpha[i], sum);
            }
            __syncthreads();  // every thread is done with K
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sp[(R * ty + i) * C::LP + tx + 16 * j] = unseen >> (4 * i + j) & 1u ? -1.f : s[i][j];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4 * OJ; ++j) o[i][j] *= alpha[i];
            __syncwarp();  // a row's 16 threads are one half of a warp
#pragma unroll 2
            for (int c = 0; c < C::KEYS / 4; ++c) {
                float4 a[R];
#pragma unroll
                for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4*>(sp + (R * ty + i) * C::LP + 4 * c);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int j = 0; j < OJ; ++j) {
                        const float4 b = *reinterpret_cast<const float4*>(sv + (4 * c + k) * D + 64 * j + 4 * tx);
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            const float w = k == 0 ? a[i].x : k == 1 ? a[i].y : k == 2 ? a[i].z : a[i].w;
                            if (masked && w < 0.f) continue;  // 0 * inf: an unseen key's V stays out, a seen one's does not
                            o[i][4 * j + 0] = fmaf(w, b.x, o[i][4 * j + 0]);
                            o[i][4 * j + 1] = fmaf(w, b.y, o[i][4 * j + 1]);
                            o[i][4 * j + 2] = fmaf(w, b.z, o[i][4 * j + 2]);
                            o[i][4 * j + 3] = fmaf(w, b.w, o[i][4 * j + 3]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int d = 8; d; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = R * ty + i;
            if (r >= rows || !PKV_DCHECK(p.err, u.row + (r >> p.group_log2) < p.num_tokens && r < p.part_rows)) continue;
            if (u.nparts == 1) {
                const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // no key seen: a zero row
                float* dst = static_cast<float*>(p.out) +
                         ((long long)(u.row + (r >> p.group_log2)) * p.num_heads + g * G + (r & (G - 1))) * D;
#pragma unroll
                for (int j = 0; j < OJ; ++j)
                    *reinterpret_cast<float4*>(dst + 64 * j + 4 * tx) = make_float4(
                        o[i][4 * j] * inv, o[i][4 * j + 1] * inv, o[i][4 * j + 2] * inv, o[i][4 * j + 3] * inv);
            } else {
                const int slot = attn_partial(blockIdx.x, u.part);
                if (tx == 0) p.ws_ml[(long long)slot * p.part_rows + r] = make_float2(m[i], l[i]);
#pragma unroll
                for (int j = 0; j < OJ; ++j)
                    p.ws_o[attn_partial_at(p, slot, D, 64 * j + 4 * tx, r)] =
                        make_float4(o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]);
            }
        }
        if (u.nparts > 1)
            attn_merge<Div, float, D, C::THREADS>(p, u, walk.share, &flag, &turns, tid, [] {
                __syncthreads();
                return true;
            });
    }
}

}  // namespace pkv
