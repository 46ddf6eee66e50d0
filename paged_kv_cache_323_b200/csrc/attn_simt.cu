// attn_simt.cu -- launch of the CUDA-core multi-query attention.
#include <atomic>

#include "attn_launch.h"
#include "attn_simt.cuh"

namespace pkv {
namespace {

template <int D, int ROWS>
cudaError_t launch_inst(const AttnParams& p, cudaStream_t st) {
    using C = SimtCfg<D, ROWS>;
    auto kern = attn_simt_kernel<D, ROWS>;
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
    // a programmatic dependent of the append or rotation before it
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(kAttnSms * C::CTAS_PER_SM));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

AttnShape attn_simt_shape() { return AttnShape{kAttnSms * SimtCfg<64, 64>::CTAS_PER_SM, SimtCfg<64, 64>::ROWS}; }

cudaError_t launch_attn_simt(const AttnParams& p, int D, cudaStream_t st) {
    // few rows a sequence on average: small tiles, a quarter of the products each.  64 sequences
    // over 500 keys, small tiles against large: 65 against 98 us and 115 against 183 us at 16
    // rows (2 and 4 kv heads), 213 against 184 us at 17, 105 against 101 us at 32.  (Two sequences
    // over 300 keys leave most SMs idle and gain further up: 27 against 44 us at 32 rows.)
    if (((long long)p.num_tokens << p.group_log2) <= 16LL * p.num_seqs)
        return D == 64 ? launch_inst<64, 16>(p, st) : launch_inst<128, 16>(p, st);
    return D == 64 ? launch_inst<64, 64>(p, st) : launch_inst<128, 64>(p, st);
}

}  // namespace pkv
