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
AttnShape attn_shape(int kv_dtype);

// dtype: q and out; kv_dtype: the caches (dtype, or PKV_FP8_E4M3 with bf16 q).
cudaError_t launch_attn(const AttnParams& p, int dtype, int kv_dtype, int D, cudaStream_t st);

cudaError_t launch_qk_rope(const RopeParams& p, int dtype, bool fp8, bool interleaved, int D, cudaStream_t st);

}  // namespace pkv
