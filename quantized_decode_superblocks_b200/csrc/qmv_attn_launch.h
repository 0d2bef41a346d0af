// qmv_attn_launch.h -- the launches of attn_decode_kernel, one translation
// unit per cache type so that they compile in parallel.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace qmv {

struct AttnParams;
__attribute__((visibility("hidden"))) cudaError_t launch_attn_f16(const AttnParams &p, int sms, int64_t steps, cudaStream_t st);
__attribute__((visibility("hidden"))) cudaError_t launch_attn_bf16(const AttnParams &p, int sms, int64_t steps, cudaStream_t st);
__attribute__((visibility("hidden"))) cudaError_t launch_attn_q8_0(const AttnParams &p, int sms, int64_t steps, cudaStream_t st);

}  // namespace qmv
