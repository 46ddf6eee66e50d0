// attn_tc.cu -- host side of the tensor-core multi-query attention: tensor
// maps over q and the pools, and the launch.
#include <atomic>

#include "attn_launch.h"
#include "attn_tc.cuh"

namespace pkv {

void* tc_tensor_map_encoder();  // cuTensorMapEncodeTiled, or null

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                   const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
    EncodeTiledFn fn = reinterpret_cast<EncodeTiledFn>(tc_tensor_map_encoder());
    if (fn == nullptr) return cudaErrorNotSupported;
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const CUresult r = fn(map, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// q as (dim, head, token): a box is 64 dims of G heads of 128 / G tokens, the
// rows of a tile one after the other.
cudaError_t make_q_map(CUtensorMap* map, const AttnParams& p, int D) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.num_heads, (cuuint64_t)p.num_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.q_stride * 2};
    const cuuint32_t G = 1u << p.group_log2;
    const cuuint32_t box[3] = {64, G, 128 / G};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// A pool with one (block, kv head) slice per last coordinate.  bf16: the slice
// as (dim of a 64-dim span, slot of 8, span, 8-slot group), so that one box is
// the whole slice and lands as [group][span][8][64] with 128-byte rows
// swizzled: what the matrix descriptors walk.  fp8: the slice as it is.
cudaError_t make_pool_map(CUtensorMap* map, const AttnParams& p, const void* pool, int D, bool fp8) {
    const cuuint64_t slices = (cuuint64_t)p.num_blocks * p.num_kv_heads, bs = p.block_size;
    if (fp8) {
        const cuuint64_t dims[3] = {(cuuint64_t)D, bs, slices};
        const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)D * bs};
        const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)bs, 1};
        return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, pool, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
    }
    const cuuint64_t row = (cuuint64_t)D * 2;
    const cuuint64_t dims[5] = {64, 8, (cuuint64_t)D / 64, bs / 8, slices};
    const cuuint64_t strides[4] = {row, 128, 8 * row, bs * row};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)D / 64, (cuuint32_t)bs / 8, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, pool, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, bool FP8>
cudaError_t launch_inst(const AttnParams& p, cudaStream_t st) {
    using C = atc::Cfg<D, FP8>;
    auto kern = atc::attn_tc_kernel<D, FP8>;
    static std::atomic<unsigned long long> configured{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    CUtensorMap mq, mk, mv;
    if ((e = make_q_map(&mq, p, D)) != cudaSuccess) return e;
    if ((e = make_pool_map(&mk, p, p.k_cache, D, FP8)) != cudaSuccess) return e;
    if ((e = make_pool_map(&mv, p, p.v_cache, D, FP8)) != cudaSuccess) return e;
    // a programmatic dependent of the append or rotation before it
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)kAttnSms);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p, mq, mk, mv);
}

}  // namespace

AttnShape attn_tc_shape() { return AttnShape{kAttnSms, atc::TcDivision::ROWS}; }

cudaError_t launch_attn_tc(const AttnParams& p, bool fp8, int D, cudaStream_t st) {
    if (fp8) return D == 64 ? launch_inst<64, true>(p, st) : launch_inst<128, true>(p, st);
    return D == 64 ? launch_inst<64, false>(p, st) : launch_inst<128, false>(p, st);
}

}  // namespace pkv
