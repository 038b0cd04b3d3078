// moe_attn_bf16.cu -- one-token attention kernels for bf16 queries over a bf16 cache.
#include "moe_attn_core.cuh"

int moe_launch_attn_bf16(const AttnParams &p, int num_sms, cudaStream_t s) {
  return moe_attn::dispatch<__nv_bfloat16, 2, false>(p, num_sms, s);
}
