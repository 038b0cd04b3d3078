// moe_attn_f16.cu -- one-token attention kernels for fp16 queries over an fp16 cache.
#include "moe_attn_core.cuh"

int moe_launch_attn_f16(const AttnParams &p, int num_sms, cudaStream_t s) {
  return moe_attn::dispatch<__half, 2, false>(p, num_sms, s);
}
