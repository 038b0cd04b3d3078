// moe_attn.cuh -- what the attention operators share: the cache as the kernels see it, the
// launch parameters, and the host prototypes of their launchers.
#pragma once

#include "moe_common.cuh"

// Device error codes of the cache operators (their error word belongs to moe_attn_api.cu).
#define MOE_DEV_ERR_BAD_PAGE 3u     // a block-table entry inside a sequence is outside [0, num_pages)
#define MOE_DEV_ERR_BAD_LENGTH 4u   // a sequence length is negative or longer than its block table
#define MOE_DEV_ERR_BAD_SLOT 5u     // a slot is past the cache's last row

// Most warps of the one-token attention kernel: its workspace holds two pieces for each.
constexpr int MOE_ATTN_MAX_WORKERS = 1792;

// Head width the kernel is compiled for that holds D, and the most head rows it takes at once.
__host__ __device__ inline int moe_attn_width(int D) { return D <= 64 ? 64 : (D <= 128 ? 128 : (D <= 256 ? 256 : 512)); }
// Query heads of one KV head that a CTA takes together (8 per MMA column tile): the fewest
// column tiles that hold the group, up to the registers' limit of 512 / width tiles.
__host__ __device__ inline int moe_attn_tiles(int D, int group) {
  const int most = 512 / moe_attn_width(D);
  int nt = 1;
  while (nt < most && 8 * nt < group) nt *= 2;
  return nt;
}

struct AttnParams {
  const void *q;
  long long q_tok, q_head;               // elements
  const char *k, *v;
  long long page_b, tok_b, head_b;       // bytes
  const int32_t *tables;
  long long table_stride;
  int max_tokens;                        // that a block table can hold
  const int32_t *lens;
  int B, nq, nkv, D, group, n_groups;    // group = nq / nkv; n_groups: CTA passes over a KV head's group
  int page_size, page_shift, num_pages, window;   // page_shift: log2 of a power of two, else -1
  int groups_of_8;                       // 8 tokens from a multiple of 8 on always lie in one page
  float scale_log2;                      // scale * log2(e) * k_scale
  float v_scale;
  void *out;
  long long out_tok, out_head;
  float *lse;                            // [B, nq] or null
  float *ws_o;                           // [2 workers][D / 16][column tiles][32 lanes][4] unnormalised sums
  float2 *ws_ml;                         // [2 workers][rows] base (log2) and sum
  int4 *ws_cut;                          // [workers] cut segments: first worker and (bit 16) whether blocks join, last worker, sequence, number there
  int noted, by_segment;                 // whether they are noted; by segment, not by the worker in which one starts
  uint32_t *err;
};

struct RopeParams {
  const void *q, *k, *v;
  long long q_tok, q_head, k_tok, k_head, v_tok, v_head;   // elements
  void *q_out, *k_out;
  long long qo_tok, qo_head, ko_tok, ko_head;
  const int32_t *positions;
  const double *inv_freq;
  const float *q_gain, *k_gain;
  float eps, rope_scale, inv_d;                             // inv_d: 1 / D
  int T, nq, nkv, D, rot;
  char *ck, *cv;                           // cache, or null
  long long page_b, tok_b, head_b;         // bytes
  long long n_slots;
  int page_size;
  float inv_k_scale, inv_v_scale;
  const int64_t *slots;
  uint32_t *err;
};

// dtype / cache_dtype: MOE_DT_*. All return 0, or -1 after a CUDA error.
int moe_launch_attn_bf16(const AttnParams &p, int num_sms, cudaStream_t s);   // bf16 q and cache
int moe_launch_attn_f16(const AttnParams &p, int num_sms, cudaStream_t s);    // fp16 q and cache
int moe_launch_attn_e4m3(const AttnParams &p, int num_sms, bool q_bf16, cudaStream_t s);   // e4m3 cache
int moe_launch_rope(const RopeParams &p, int dtype, bool interleaved, bool cache_e4m3, int num_sms, cudaStream_t s);
