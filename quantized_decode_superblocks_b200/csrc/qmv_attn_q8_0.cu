// qmv_attn_q8_0.cu -- attn_decode_kernel for the Q8_0 cache.
#include "qmv_attn.cuh"
#include "qmv_attn_launch.h"
#include "qmv_launch.cuh"

namespace qmv {

cudaError_t launch_attn_q8_0(const AttnParams &p, int sms, int64_t steps, cudaStream_t st)
{
    return launch_attn<KV_Q8_0>(p, sms, steps, st);
}

}  // namespace qmv
