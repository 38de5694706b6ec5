// Instantiations of the decode attention kernels for the bf16 cache
// (attn_decode.cuh), one file per format so that they compile in parallel.
#include "attn_decode.cuh"

namespace nvfp4 {
namespace attn {

int run_bf16(const Args& a, const Shape& sh, int y_dtype, cudaStream_t st) {
    return y_dtype == NVFP4_DTYPE_BF16 ? run_fmt<NVFP4_KV_BF16, __nv_bfloat16>(a, sh, st) : run_fmt<NVFP4_KV_BF16, float>(a, sh, st);
}

}  // namespace attn
}  // namespace nvfp4
