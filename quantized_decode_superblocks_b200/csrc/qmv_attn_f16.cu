// qmv_attn_f16.cu -- attn_decode_kernel for the F16 cache.
#include "qmv_attn.cuh"
#include "qmv_attn_launch.h"
#include "qmv_launch.cuh"

namespace qmv {

cudaError_t launch_attn_f16(const AttnParams &p, int sms, int64_t steps, cudaStream_t st)
{
    return launch_attn<KV_F16>(p, sms, steps, st);
}

}  // namespace qmv
