// moe_rope.cu -- per-head norms of q and k, their rotation, and the append of k and v to a paged
// cache, one pass over the rows:
//   u = x / sqrt(mean x^2 + eps) * gain;  (u_a, u_b) turned by position * inv_freq;  k, v -> cache
//
// Bound: HBM (each row read and written once; 16 bytes of bf16 in and out a head element pair and
// about 10 flops). A warp works on one token: 32 / L heads at a time, L = head_dim / 16 lanes a
// head (rounded up to a power of two), each lane holding two 16-byte pieces of its head that are
// each other's rotation partners (half layout: elements i.. and i + R/2..; interleaved: 16
// neighbours), so the rotation needs no exchange between lanes. A lane holds the same elements of
// every head it meets: gains, cosines and sines stay in registers. The next heads' loads are in
// flight while the current ones are computed. With few tokens a token's heads are spread over
// several warps so that the GPU is filled.
//
// Angles: position * inv_freq in 64 bits, reduced to a fraction of a turn there (at position 2^18
// a 32-bit product would be off by 2^-7 rad), then sincospif in 32 bits; a warp's lanes share the
// work through shared memory.
#include <cuda_fp8.h>

#include <type_traits>

#include "moe_attn.cuh"

namespace {

constexpr int kThreads = 256, kWarpsPerCta = kThreads / 32;

template <typename T> __device__ __forceinline__ void unpack2(uint32_t w, float &x, float &y);
template <> __device__ __forceinline__ void unpack2<__nv_bfloat16>(uint32_t w, float &x, float &y) {
  x = __uint_as_float(w << 16);
  y = __uint_as_float(w & 0xffff0000u);
}
template <> __device__ __forceinline__ void unpack2<__half>(uint32_t w, float &x, float &y) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
  x = f.x;
  y = f.y;
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float x, float y);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float x, float y) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <typename T> __device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8]) {
  unpack2<T>(w.x, v[0], v[1]);
  unpack2<T>(w.y, v[2], v[3]);
  unpack2<T>(w.z, v[4], v[5]);
  unpack2<T>(w.w, v[6], v[7]);
}
template <typename T> __device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}
// value / scale, saturated, one rounding (the quotient itself is rounded to FP32 first)
__device__ __forceinline__ uint2 pack8_e4m3(const float (&v)[8], float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v[2 * i], scale), __fdiv_rn(v[2 * i + 1], scale)),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// lanes: lanes of a head (a power of two); split: warps that share a token's heads.
template <typename T, bool INTER, bool F8>
__global__ void __launch_bounds__(kThreads, 3) k_qk_norm_rope(const __grid_constant__ RopeParams p, int lanes, int split) {
  extern __shared__ float2 sh_turn[];   // [warps][rot / 2] cos, sin
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned work = blockIdx.x * kWarpsPerCta + warp;   // below T + 16 SMs: fits
  const unsigned t = work / (unsigned)split;
  const int part = (int)(work - t * (unsigned)split);
  if (t >= (unsigned)p.T) return;
  const int per = 32 / lanes, sub = lane & (lanes - 1), grp = lane / lanes;
  const int pq = (p.nq + per - 1) / per, pk = (p.nkv + per - 1) / per;
  const int passes = pq + pk + (p.ck ? pk : 0);
  const int i0 = (int)((long long)passes * part / split), i1 = (int)((long long)passes * (part + 1) / split);

  // the lane's two pieces of a head, and whether they turn
  const int half = p.rot / 2;
  int ea = 16 * sub, eb = ea + 8;
  const bool turns = ea < p.rot;
  if (!INTER && turns) {
    ea = 8 * sub;
    eb = ea + half;
  }
  const bool in = 16 * sub < p.D;

  // cosines and sines of the lane's 8 pairs
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cs[j] = 1.f, sn[j] = 0.f;
  auto angles = [&]() {
    float2 *turn = sh_turn + warp * half;
    const double pos = (double)p.positions[t];
    for (int i = lane; i < half; i += 32) {
      const double rev = pos * p.inv_freq[i] * 0.15915494309189533577;   // / (2 pi)
      const float part_turn = (float)(rev - rint(rev));
      float s, c;
      sincospif(2.f * part_turn, &s, &c);
      turn[i] = make_float2(c * p.rope_scale, s * p.rope_scale);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = (INTER ? ea / 2 : ea) + j;
      if (turns && i < half) {
        const float2 v = turn[i];
        cs[j] = v.x;
        sn[j] = v.y;
      }
    }
  };

  long long row = -1;   // the token's place in the cache, bytes
  if (p.ck && i1 > pq) {
    const long long slot = p.slots[t];
    if (slot >= p.n_slots) {
      report_error(p.err, MOE_DEV_ERR_BAD_SLOT, 0);
    } else if (slot >= 0) {
      const long long page = slot >> 32 ? slot / p.page_size : (long long)((unsigned)slot / (unsigned)p.page_size);
      row = page * p.page_b + (slot - page * p.page_size) * p.tok_b;
    }
  }

  // Passes [from, to) of one kind of heads (kind 0: q, 1: k, 2: v). The next pass's loads are in
  // flight while one is computed; the first ones while the angles are.
  bool have_angles = false;
  auto heads_of = [&](auto kind_c, int from, int to, const T *src, long long src_head, int n, const float *gain, T *out,
                      long long out_head, char *cache, float scale) {
    constexpr int kind = decltype(kind_c)::value;
    if (from >= to) return;
    int h = from * per + grp;
    src += (long long)h * src_head;
    out += (long long)h * out_head;
    cache += (long long)h * p.head_b;
    uint4 ra = make_uint4(0, 0, 0, 0), rb = ra;
    auto load = [&]() {
      if (in && h < n) {
        ra = *reinterpret_cast<const uint4 *>(src + ea);
        rb = *reinterpret_cast<const uint4 *>(src + eb);
      }
    };
    load();
    float ga[8], gb[8];
    if (kind < 2 && gain) {
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (in) {
          x = *reinterpret_cast<const float4 *>(gain + ea + j);
          y = *reinterpret_cast<const float4 *>(gain + eb + j);
        }
        ga[j] = x.x, ga[j + 1] = x.y, ga[j + 2] = x.z, ga[j + 3] = x.w;
        gb[j] = y.x, gb[j + 1] = y.y, gb[j + 2] = y.z, gb[j + 3] = y.w;
      }
    }
    if (kind < 2 && p.rot && !have_angles) {
      angles();
      have_angles = true;
    }
#pragma unroll 1
    for (int i = from; i < to; ++i) {
      const bool ok = in && h < n;
      float a[8], b[8];
      unpack8<T>(ra, a);
      unpack8<T>(rb, b);
      h += per;
      src += per * src_head;
      if (i + 1 < to) load();
      if (kind < 2 && gain) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s0 = fmaf(a[j], a[j], s0);
          s1 = fmaf(b[j], b[j], s1);
        }
        float ss = s0 + s1;
        for (int o = lanes >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = 1.0f / sqrtf(ss / (float)p.D + p.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j] = a[j] * inv * ga[j];
          b[j] = b[j] * inv * gb[j];
        }
      }
      if (kind < 2 && turns) {
        if constexpr (INTER) {
          // pairs past rotary_dim keep their values (not 1 x + 0 y: y may be infinite)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (ea / 2 + j < half) {
              const float x = a[2 * j], y = a[2 * j + 1];
              a[2 * j] = x * cs[j] - y * sn[j];
              a[2 * j + 1] = y * cs[j] + x * sn[j];
            }
            if (ea / 2 + 4 + j < half) {
              const float x = b[2 * j], y = b[2 * j + 1];
              b[2 * j] = x * cs[4 + j] - y * sn[4 + j];
              b[2 * j + 1] = y * cs[4 + j] + x * sn[4 + j];
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = a[j], y = b[j];
            a[j] = x * cs[j] - y * sn[j];
            b[j] = y * cs[j] + x * sn[j];
          }
        }
      }
      if (ok) {
        if (kind == 0 || (kind == 1 && p.k_out)) {
          *reinterpret_cast<uint4 *>(out + ea) = pack8<T>(a);
          *reinterpret_cast<uint4 *>(out + eb) = pack8<T>(b);
        }
        if (kind > 0 && row >= 0) {
          if constexpr (F8) {
            *reinterpret_cast<uint2 *>(cache + ea) = pack8_e4m3(a, scale);
            *reinterpret_cast<uint2 *>(cache + eb) = pack8_e4m3(b, scale);
          } else {
            *reinterpret_cast<uint4 *>(cache + 2 * ea) = pack8<T>(a);
            *reinterpret_cast<uint4 *>(cache + 2 * eb) = pack8<T>(b);
          }
        }
      }
      out += per * out_head;
      cache += per * p.head_b;
    }
  };
  const long long tt = t, at = row < 0 ? 0 : row;
  heads_of(std::integral_constant<int, 0>{}, i0, min(i1, pq), static_cast<const T *>(p.q) + tt * p.q_tok, p.q_head, p.nq,
           p.q_gain, static_cast<T *>(p.q_out) + tt * p.qo_tok, p.qo_head, p.ck, 1.f);
  heads_of(std::integral_constant<int, 1>{}, max(i0 - pq, 0), min(i1 - pq, pk), static_cast<const T *>(p.k) + tt * p.k_tok,
           p.k_head, p.nkv, p.k_gain, static_cast<T *>(p.k_out) + tt * p.ko_tok, p.ko_head, p.ck + at, p.k_scale);
  heads_of(std::integral_constant<int, 2>{}, max(i0 - pq - pk, 0), i1 - pq - pk, static_cast<const T *>(p.v) + tt * p.v_tok,
           p.v_head, p.nkv, nullptr, static_cast<T *>(nullptr), 0, p.cv + at, p.v_scale);
}

template <typename T> int launch_rope(const RopeParams &p, bool inter, bool f8, int num_sms, cudaStream_t s) {
  int lanes = 1;
  while (lanes * 16 < p.D) lanes *= 2;
  const int per = 32 / lanes;
  const int pq = (p.nq + per - 1) / per, pk = (p.nkv + per - 1) / per, passes = pq + pk + (p.ck ? pk : 0);
  // warps a token: one where the tokens alone give 16 warps an SM, else as many as reach that
  const long long want = 16ll * num_sms;
  int split = (int)((want + p.T - 1) / p.T);
  if (split > passes) split = passes;
  if (split < 1) split = 1;
  const long long ctas = ((long long)p.T * split + kWarpsPerCta - 1) / kWarpsPerCta;
  const size_t smem = (size_t)kWarpsPerCta * (p.rot / 2) * sizeof(float2);
  const unsigned grid = (unsigned)ctas;
  if (inter) {
    if (f8) k_qk_norm_rope<T, true, true><<<grid, kThreads, smem, s>>>(p, lanes, split);
    else k_qk_norm_rope<T, true, false><<<grid, kThreads, smem, s>>>(p, lanes, split);
  } else {
    if (f8) k_qk_norm_rope<T, false, true><<<grid, kThreads, smem, s>>>(p, lanes, split);
    else k_qk_norm_rope<T, false, false><<<grid, kThreads, smem, s>>>(p, lanes, split);
  }
  if (cudaGetLastError() != cudaSuccess) return -1;
  moe_prof_count(1);
  return 0;
}

}  // namespace

int moe_launch_rope(const RopeParams &p, int dtype, bool interleaved, bool cache_e4m3, int num_sms, cudaStream_t s) {
  return dtype == MOE_DT_BF16 ? launch_rope<__nv_bfloat16>(p, interleaved, cache_e4m3, num_sms, s)
                              : launch_rope<__half>(p, interleaved, cache_e4m3, num_sms, s);
}
