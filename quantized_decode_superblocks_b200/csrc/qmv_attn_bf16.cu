// qmv_attn_bf16.cu -- attn_decode_kernel for the BF16 cache.
#include "qmv_attn.cuh"
#include "qmv_attn_launch.h"
#include "qmv_launch.cuh"

namespace qmv {

cudaError_t launch_attn_bf16(const AttnParams &p, int sms, int64_t steps, cudaStream_t st)
{
    return launch_attn<KV_BF16>(p, sms, steps, st);
}

}  // namespace qmv
