// attn_launch.h -- host-side entry points of the multi-query attention and
// q/k rotation translation units.
#pragma once

#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "qk_rope.cuh"

namespace pkv {

constexpr int kAttnSms = 148;

// What a launch asks of its workspace: CTAs of the grid (two partial results
// each) and rows of a full tile.
struct AttnShape {
    int grid;
    int rows;
};
// fp32 caches on the CUDA cores; bf16 and fp8 ones (bf16 q) on the tensor cores
AttnShape attn_simt_shape();
cudaError_t launch_attn_simt(const AttnParams& p, int D, cudaStream_t st);
AttnShape attn_tc_shape();
cudaError_t launch_attn_tc(const AttnParams& p, bool fp8, int D, cudaStream_t st);

cudaError_t launch_qk_rope(const RopeParams& p, int dtype, bool fp8, bool interleaved, int D, cudaStream_t st);

}  // namespace pkv
