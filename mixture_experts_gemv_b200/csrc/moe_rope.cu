// moe_rope.cu -- per-head norms of q and k, their rotation, and the append of k and v to a paged
// cache, one pass over the rows:
//   u = x / sqrt(mean x^2 + eps) * gain;  (u_a, u_b) turned by position * inv_freq;  k, v -> cache
//
// Bound: HBM (each row read and written once, about 10 flops an element). What the kernel waits
// for is latency: see the figures below.
//
// A warp works on one token: 32 / L heads at a time, L = head_dim / (2 V) lanes a head (rounded up
// to a power of two), each lane holding two pieces of V elements that are each other's rotation
// partners (half layout: elements i.. and i + R/2..; interleaved: 2 V neighbours), so the rotation
// needs no exchange between lanes. A lane holds the same elements of every head it meets: gains
// and angles are folded into four factors a pair that stay in registers. With few tokens a token's
// heads are spread over several warps so that the GPU is filled. V = 4 up to head_dim 256 (8-byte
// pieces, 64 registers, 32 warps an SM, the next two passes' loads in flight), V = 8 above (a head
// would not fit a warp; 80 registers, 24 warps). Both bounds cost 24 to 80 bytes of spills a thread.
//
// Measured (4,096 tokens of 32 + 8 + 8 heads of 128, bf16, 101 MB; 10,000 of 16 + 2 + 2 heads of
// 512 into an 8-bit cache, 389 MB): 25.4 and 83.4 us = 4.0 and 4.7 TB/s; without norm and rotation
// the first takes 22.9 us, a plain copy of the bytes 17.4. Tried: V = 8 with 24 warps 30.9 us, one
// load ahead 28.0, three 26.3; rows through shared memory by cp.async rings four or eight deep
// 30.8 and 39.7 (more instructions); by bulk copies with a warp of their own and three stages 24.5 to
// 25.8, but 127 us for the second.
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
// V values of 16 bits as one register vector.
template <int V> struct Piece;
template <> struct Piece<4> {
  using type = uint2;
  static __device__ __forceinline__ uint2 zero() { return make_uint2(0, 0); }
};
template <> struct Piece<8> {
  using type = uint4;
  static __device__ __forceinline__ uint4 zero() { return make_uint4(0, 0, 0, 0); }
};
template <typename T> __device__ __forceinline__ void unpack(const uint2 &w, float (&v)[4]) {
  unpack2<T>(w.x, v[0], v[1]);
  unpack2<T>(w.y, v[2], v[3]);
}
template <typename T> __device__ __forceinline__ void unpack(const uint4 &w, float (&v)[8]) {
  unpack2<T>(w.x, v[0], v[1]);
  unpack2<T>(w.y, v[2], v[3]);
  unpack2<T>(w.z, v[4], v[5]);
  unpack2<T>(w.w, v[6], v[7]);
}
template <typename T> __device__ __forceinline__ uint2 pack(const float (&v)[4]) { return make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])); }
template <typename T> __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
  return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}
// Values times inv_scale, saturated, as e4m3.
__device__ __forceinline__ uint32_t e4m3x4(const float *v, float inv_scale) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv_scale, v[1] * inv_scale), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv_scale, v[3] * inv_scale), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ void store_e4m3(char *to, const float (&v)[4], float inv_scale) { *reinterpret_cast<uint32_t *>(to) = e4m3x4(v, inv_scale); }
__device__ __forceinline__ void store_e4m3(char *to, const float (&v)[8], float inv_scale) {
  *reinterpret_cast<uint2 *>(to) = make_uint2(e4m3x4(v, inv_scale), e4m3x4(v + 4, inv_scale));
}

// Two FP32 values in a register pair, and the packed arithmetic on them.
struct F2 {
  unsigned long long v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
  __device__ __forceinline__ void get(float &x, float &y) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
};
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// V: elements of a piece. lanes: lanes of a head (a power of two). split: warps that share a token.
template <typename T, int V, bool INTER, bool F8>
__global__ void __launch_bounds__(kThreads, V == 4 ? 4 : 3) k_qk_norm_rope(const __grid_constant__ RopeParams p, int lanes, int split) {
  extern __shared__ float2 sh_turn[];   // [warps][rot / 2] cos, sin
  constexpr int kAhead = V == 4 ? 2 : 1;   // passes whose loads are in flight
  using P = Piece<V>;
  using Raw = typename P::type;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const unsigned work = blockIdx.x * kWarpsPerCta + warp;   // below T + the warps of a full GPU: fits
  const unsigned t = work / (unsigned)split;
  if (t >= (unsigned)p.T) return;
  const int part = (int)(work - t * (unsigned)split);
  const int per = 32 / lanes, sub = lane & (lanes - 1), grp = lane / lanes;
  const int pq = (p.nq + per - 1) / per, pk = (p.nkv + per - 1) / per;
  const int passes = pq + pk + (p.ck ? pk : 0);
  const int i0 = (int)((unsigned)passes * part / split), i1 = (int)((unsigned)passes * (part + 1) / split);

  // the lane's two pieces of a head, and whether they turn
  const int half = p.rot / 2;
  int ea = 2 * V * sub, eb = ea + V;
  const bool turns = ea < p.rot;
  if (!INTER && turns) {
    ea = V * sub;
    eb = ea + half;
  }
  const bool in = 2 * V * sub < p.D, even16 = p.rot % 16 == 0;

  long long row = -1;   // the token's place in the cache, bytes
  if (p.ck && i1 > pq) {
    const long long slot = p.slots[t];
    if (slot >= p.n_slots) {
      atomicCAS(p.err, 0u, MOE_DEV_ERR_BAD_SLOT);
    } else if (slot >= 0) {
      const long long page = slot >> 32 ? slot / p.page_size : (long long)((unsigned)slot / (unsigned)p.page_size);
      row = page * p.page_b + (slot - page * p.page_size) * p.tok_b;
    }
  }

  // Passes [from, to) of one kind of heads (kind 0: q, 1: k, 2: v), 32 / lanes heads each. The next
  // pass's loads are in flight while one is computed; the first ones while the angles are.
  float2 *turn = sh_turn + warp * half;
  bool have_angles = p.rot == 0;
  auto heads_of = [&](auto kind_c, int from, int to, int n, const void *in_rows, long long src_head, const float *gain, char *out,
                      long long out_head, char *cache, float inv_scale) {
    constexpr int kind = decltype(kind_c)::value;
    if (from >= to) return;
    int left = in ? n - (from * per + grp) : 0;   // heads from this lane's on; none for idle lanes
    const T *src = static_cast<const T *>(in_rows) + (from * per + grp) * src_head + ea;
    const int gap = eb - ea;
    out += 2 * ((from * per + grp) * out_head + ea);
    cache += (from * per + grp) * p.head_b + (F8 ? 1 : 2) * ea;
    const long long src_step = per * src_head, out_step = 2 * per * out_head, cache_step = per * p.head_b;
    // the loads of the next kAhead passes, in registers of their own (moving them along would wait for them)
    Raw ra[kAhead], rb[kAhead];
    auto load = [&](int x, int ahead) {
      ra[x] = rb[x] = P::zero();
      if (left > ahead * per) {
        ra[x] = *reinterpret_cast<const Raw *>(src + ahead * src_step);
        rb[x] = *reinterpret_cast<const Raw *>(src + ahead * src_step + gap);
      }
    };
    const int last = (to - from) * per;   // heads of the passes here
    if (left > last) left = last;
#pragma unroll
    for (int x = 0; x < kAhead; ++x) load(x, x);

    // What the lane multiplies with, the same for every head of the kind. With gains g and the
    // angle's c and s, out_a = inv (a ac - b bs), out_b = inv (b bc + a as): ac = g_a c,
    // bs = g_b s, bc = g_b c, as = g_a s (c = 1, s = 0 for elements that do not turn). Pair j of
    // the half layout is (a_j, b_j); interleaved, (a_2j, a_2j+1) and (b_2j, b_2j+1).
    F2 ac[V / 2], as[V / 2], bc[V / 2], bs[V / 2];
    if (kind < 2) {
      if (!have_angles) {
        const double pos = (double)p.positions[t];
        for (int i = lane; i < half; i += 32) {
          const double rev = pos * p.inv_freq[i] * 0.15915494309189533577;   // / (2 pi)
          const float part_turn = (float)(rev - rint(rev));
          float s, c;
          sincospif(2.f * part_turn, &s, &c);
          turn[i] = make_float2(c * p.rope_scale, s * p.rope_scale);
        }
        __syncwarp();
        have_angles = true;
      }
      float ga[V], gb[V], cs[V], sn[V];
#pragma unroll
      for (int j = 0; j < V; ++j) ga[j] = gb[j] = cs[j] = 1.f, sn[j] = 0.f;
      if (gain && in) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          const float4 x = *reinterpret_cast<const float4 *>(gain + ea + j), y = *reinterpret_cast<const float4 *>(gain + eb + j);
          ga[j] = x.x, ga[j + 1] = x.y, ga[j + 2] = x.z, ga[j + 3] = x.w;
          gb[j] = y.x, gb[j + 1] = y.y, gb[j + 2] = y.z, gb[j + 3] = y.w;
        }
      }
      if (turns) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int i = (INTER ? ea / 2 : ea) + j;
          if (i < half) cs[j] = turn[i].x, sn[j] = turn[i].y;
        }
      }
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        if constexpr (INTER) {   // angle j belongs to pair j of a, angle V / 2 + j to pair j of b
          ac[j] = F2(ga[2 * j] * cs[j], ga[2 * j + 1] * cs[j]);
          as[j] = F2(ga[2 * j] * sn[j], ga[2 * j + 1] * sn[j]);
          bc[j] = F2(gb[2 * j] * cs[V / 2 + j], gb[2 * j + 1] * cs[V / 2 + j]);
          bs[j] = F2(gb[2 * j] * sn[V / 2 + j], gb[2 * j + 1] * sn[V / 2 + j]);
        } else {
          ac[j] = F2(ga[2 * j] * cs[2 * j], ga[2 * j + 1] * cs[2 * j + 1]);
          as[j] = F2(ga[2 * j] * sn[2 * j], ga[2 * j + 1] * sn[2 * j + 1]);
          bc[j] = F2(gb[2 * j] * cs[2 * j], gb[2 * j + 1] * cs[2 * j + 1]);
          bs[j] = F2(-gb[2 * j] * sn[2 * j], -gb[2 * j + 1] * sn[2 * j + 1]);
        }
      }
    }
#pragma unroll 1
    for (int i = from; i < to; i += kAhead) {
#pragma unroll
      for (int buf = 0; buf < kAhead; ++buf) {
        if (i + buf >= to) break;
        const bool ok = left > 0;
        Raw ya = ra[buf], yb = rb[buf];   // v in its own type goes through as it is
        float a[V], b[V];
        if (kind < 2 || F8) {
          unpack<T>(ya, a);
          unpack<T>(yb, b);
        }
        load(buf, kAhead);
        left -= per;
        src += src_step;
        if (kind < 2) {
          F2 x[V / 2], y[V / 2];
#pragma unroll
          for (int j = 0; j < V / 2; ++j) x[j] = F2(a[2 * j], a[2 * j + 1]), y[j] = F2(b[2 * j], b[2 * j + 1]);
          float inv = 1.f;
          if (gain) {
            F2 s2 = mul2(x[0], x[0]), t2 = mul2(y[0], y[0]);
#pragma unroll
            for (int j = 1; j < V / 2; ++j) s2 = fma2(x[j], x[j], s2), t2 = fma2(y[j], y[j], t2);
            float s0, s1, t0, t1;
            s2.get(s0, s1);
            t2.get(t0, t1);
            float ss = (s0 + s1) + (t0 + t1);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
              if (o < lanes) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            inv = rsqrtf(fmaf(ss, p.inv_d, p.eps));
          }
          if (turns) {
            if constexpr (INTER) {
              // the two of a pair are neighbours: cross terms in single arithmetic. Pairs past
              // rotary_dim keep their values (not 1 x - 0 y: y may be infinite).
#pragma unroll
              for (int j = 0; j < V / 2; ++j) {
                float c0, c1, d0, d1;
                ac[j].get(c0, c1);
                as[j].get(d0, d1);
                const float a0 = a[2 * j], a1 = a[2 * j + 1], b0 = b[2 * j], b1 = b[2 * j + 1];
                const bool ta = even16 || ea / 2 + j < half, tb = even16 || eb / 2 + j < half;
                a[2 * j] = a0 * c0;
                a[2 * j + 1] = a1 * c1;
                if (ta) {
                  a[2 * j] -= a1 * d1;
                  a[2 * j + 1] += a0 * d0;
                }
                bc[j].get(c0, c1);
                bs[j].get(d0, d1);
                b[2 * j] = b0 * c0;
                b[2 * j + 1] = b1 * c1;
                if (tb) {
                  b[2 * j] -= b1 * d1;
                  b[2 * j + 1] += b0 * d0;
                }
                x[j] = F2(a[2 * j], a[2 * j + 1]);
                y[j] = F2(b[2 * j], b[2 * j + 1]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < V / 2; ++j) {
                const F2 u = fma2(y[j], bs[j], mul2(x[j], ac[j]));
                y[j] = fma2(x[j], as[j], mul2(y[j], bc[j]));
                x[j] = u;
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < V / 2; ++j) x[j] = mul2(x[j], ac[j]), y[j] = mul2(y[j], bc[j]);
          }
          const F2 inv2(inv, inv);
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            mul2(x[j], inv2).get(a[2 * j], a[2 * j + 1]);
            mul2(y[j], inv2).get(b[2 * j], b[2 * j + 1]);
          }
          ya = pack<T>(a);
          yb = pack<T>(b);
        }
        if (ok) {
          if (kind == 0 || (kind == 1 && p.k_out)) {
            *reinterpret_cast<Raw *>(out) = ya;
            *reinterpret_cast<Raw *>(out + 2 * gap) = yb;
          }
          if (kind > 0 && row >= 0) {
            if constexpr (F8) {
              store_e4m3(cache, a, inv_scale);
              store_e4m3(cache + gap, b, inv_scale);
            } else {
              *reinterpret_cast<Raw *>(cache) = ya;
              *reinterpret_cast<Raw *>(cache + 2 * gap) = yb;
            }
          }
        }
        out += out_step;
        cache += cache_step;
      }
    }
  };
  const long long tt = t, at = row < 0 ? 0 : row;
  heads_of(std::integral_constant<int, 0>{}, i0, min(i1, pq), p.nq, static_cast<const T *>(p.q) + tt * p.q_tok, p.q_head, p.q_gain,
           static_cast<char *>(p.q_out) + 2 * tt * p.qo_tok, p.qo_head, p.ck, 1.f);
  heads_of(std::integral_constant<int, 1>{}, max(i0 - pq, 0), min(i1 - pq, pk), p.nkv, static_cast<const T *>(p.k) + tt * p.k_tok, p.k_head,
           p.k_gain, static_cast<char *>(p.k_out) + 2 * tt * p.ko_tok, p.ko_head, p.ck + at, p.inv_k_scale);
  heads_of(std::integral_constant<int, 2>{}, max(i0 - pq - pk, 0), i1 - pq - pk, p.nkv, static_cast<const T *>(p.v) + tt * p.v_tok, p.v_head,
           nullptr, static_cast<char *>(nullptr), 0, p.cv + at, p.inv_v_scale);
}

template <typename T, int V> int launch_rope(const RopeParams &p, bool inter, bool f8, int num_sms, cudaStream_t s) {
  int lanes = 1;
  while (lanes * 2 * V < p.D) lanes *= 2;
  const int per = 32 / lanes;
  const int pq = (p.nq + per - 1) / per, pk = (p.nkv + per - 1) / per, passes = pq + pk + (p.ck ? pk : 0);
  // warps a token: one where the tokens alone give 16 warps an SM, else as many as reach that
  const long long want = 16ll * num_sms;
  int split = (int)((want + p.T - 1) / p.T);
  if (split > passes) split = passes;
  if (split < 1) split = 1;
  const unsigned grid = (unsigned)(((long long)p.T * split + kWarpsPerCta - 1) / kWarpsPerCta);
  const size_t smem = (size_t)kWarpsPerCta * (p.rot / 2) * sizeof(float2);
  const auto fn = inter ? (f8 ? k_qk_norm_rope<T, V, true, true> : k_qk_norm_rope<T, V, true, false>)
                        : (f8 ? k_qk_norm_rope<T, V, false, true> : k_qk_norm_rope<T, V, false, false>);
  PdlLaunch l(dim3(grid), kThreads, smem, s);
  if (cudaLaunchKernelEx(&l.cfg, fn, p, lanes, split) != cudaSuccess) return -1;
  moe_prof_count(1);
  return 0;
}

}  // namespace

int moe_launch_rope(const RopeParams &p, int dtype, bool interleaved, bool cache_e4m3, int num_sms, cudaStream_t s) {
  if (p.D <= 256)
    return dtype == MOE_DT_BF16 ? launch_rope<__nv_bfloat16, 4>(p, interleaved, cache_e4m3, num_sms, s)
                                : launch_rope<__half, 4>(p, interleaved, cache_e4m3, num_sms, s);
  return dtype == MOE_DT_BF16 ? launch_rope<__nv_bfloat16, 8>(p, interleaved, cache_e4m3, num_sms, s)
                              : launch_rope<__half, 8>(p, interleaved, cache_e4m3, num_sms, s);
}
