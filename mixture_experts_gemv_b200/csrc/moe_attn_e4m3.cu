// moe_attn_e4m3.cu -- one-token attention kernels over an e4m3 cache: its codes become fp16 in
// registers (exactly) and the products run in fp16.
#include "moe_attn_core.cuh"

int moe_launch_attn_e4m3(const AttnParams &p, int num_sms, bool q_bf16, cudaStream_t s) {
  return q_bf16 ? moe_attn::dispatch<__half, 1, true>(p, num_sms, s) : moe_attn::dispatch<__half, 1, false>(p, num_sms, s);
}
