// qmv_attn_bf16.cu -- attn_decode_kernel for the BF16 cache.
#include "qmv_attn.cuh"
#include "qmv_attn_launch.h"
#include "qmv_launch.cuh"

namespace qmv {

cudaError_t launch_attn_bf16(const AttnParams &p, int grid, cudaStream_t st)
{
    return launch_attn<KV_BF16>(p, grid, st);
}

}  // namespace qmv
