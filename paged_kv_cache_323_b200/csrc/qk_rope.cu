// qk_rope.cu -- launch of the q/k norm, rotation and append.
#include "attn_launch.h"

namespace pkv {
namespace {

template <typename T, int D, bool FP8>
cudaError_t launch_inst(const RopeParams& p, bool interleaved, unsigned grid, cudaStream_t st) {
    if (interleaved)
        qk_rope_kernel<T, D, FP8, true><<<grid, kRopeThreads, 0, st>>>(p);
    else
        qk_rope_kernel<T, D, FP8, false><<<grid, kRopeThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_rope(const RopeParams& p0, int dtype, bool fp8, bool interleaved, int D, cudaStream_t st) {
    RopeParams p = p0;
    const int rows_per_pass = kRopeThreads / (D * (dtype == PKV_F32 ? 4 : 2) / 32);
    // several tokens to a CTA while every SM has four CTAs; few tokens: q, k and v apart
    // (their loads one behind the other are what such a call waits for), and a token's
    // heads over several CTAs until every SM has one
    p.tokens_per_cta = 1;
    while (p.tokens_per_cta < kRopeMaxTokens && p.num_tokens >= 8 * kAttnSms * p.tokens_per_cta) p.tokens_per_cta *= 2;
    p.kinds_apart = p.num_tokens <= 8 * kAttnSms;
    const int passes = (p.tokens_per_cta * p.num_heads + rows_per_pass - 1) / rows_per_pass;
    p.head_splits = 1;
    while (p.head_splits < passes && (long long)p.num_tokens * p.head_splits < kAttnSms) ++p.head_splits;
    const long long ctas = ((long long)p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta * p.head_splits *
                           (p.kinds_apart ? 3 : 1);
    const unsigned grid = (unsigned)ctas;
    if (dtype == PKV_F32)
        return D == 64 ? launch_inst<float, 64, false>(p, interleaved, grid, st)
                       : launch_inst<float, 128, false>(p, interleaved, grid, st);
    if (fp8)
        return D == 64 ? launch_inst<__nv_bfloat16, 64, true>(p, interleaved, grid, st)
                       : launch_inst<__nv_bfloat16, 128, true>(p, interleaved, grid, st);
    return D == 64 ? launch_inst<__nv_bfloat16, 64, false>(p, interleaved, grid, st)
                   : launch_inst<__nv_bfloat16, 128, false>(p, interleaved, grid, st);
}

}  // namespace pkv
