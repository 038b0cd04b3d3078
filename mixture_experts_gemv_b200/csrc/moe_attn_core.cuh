// moe_attn_core.cuh -- attention of one new token per sequence over a paged cache.
//
//   s_j = scale q . k_j for the keys j in [max(0, len - window), len);  p = softmax(s);
//   out = sum_j p_j v_j;  lse = log sum_j exp(s_j)
//
// Bound: HBM. Every K and V row in range is read once (2 D elements a token and KV head) for
// 4 D flops a query head: 8 query heads on a KV head are 8 flops a byte, so the work is kept
// off the CUDA cores but far from any tensor limit.
//
// Both products are taken transposed, S^T = K Q^T and O^T = V^T P^T, with tokens (then head
// elements) as the 16 rows of an mma.sync.m16n8k16 and the query heads that share the KV head
// as its 8 columns: a group of 8 heads fills the tile, K and V fragments come from shared
// memory once, and O takes D / 4 registers a thread for 8 heads. (With heads as rows, half the
// tile would be empty and O would not fit at D = 512.)
//
// Each warp takes 16 tokens at a time through its own ring of cp.async copies (K rows, then V
// rows), so the loop has no block barrier. A block takes 64 tokens at a time (16 per warp) and
// joins its four warps' (maximum, sum, O) through shared memory at the end of a segment = the
// tokens of one (sequence, KV head, head group).
//
// Work split: the 64-token chunks of all segments are numbered through and cut into equal
// ranges, one per CTA of a grid that fills the GPU once, whatever the lengths are. A segment
// cut by a range's end leaves unnormalised pieces in the workspace (at most two per CTA); the
// join kernel, launched behind with programmatic dependent launch, sums them in CTA order. No
// atomics: outputs repeat bit for bit.
//
// Precision: K Q^T products are exact, summed in FP32; the softmax runs in FP32 (base 2); P is
// rounded to the 16-bit type of the V product (half a step, 2^-9 or 2^-12 of each p, the sum l
// keeps the unrounded p); O is FP32 and rounded once. fp16: p is taken times 2^15, so that
// what fp16 cannot hold lies below 2^-39 of the largest p.
#pragma once

#include <type_traits>

#include "moe_attn.cuh"

namespace moe_attn {

constexpr int kWarps = 4;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T> struct Mma;
template <> struct Mma<__nv_bfloat16> {
  static __device__ __forceinline__ void run(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
  }
  static constexpr float kOff = 0.f;   // log2 of the factor on p
};
template <> struct Mma<__half> {
  static __device__ __forceinline__ void run(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
  }
  static constexpr float kOff = 15.f;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transposed8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {   // the low two bytes
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(v));
  return r;
}
// 16-byte asynchronous copy; with ok false nothing is read and zeros are written.
__device__ __forceinline__ void copy16(uint32_t dst, const char *src, bool ok) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Compile-time shape: W padded head width, NT column tiles of 8 heads, ES bytes an element.
template <int W, int NT, int ES> struct Shape {
  static constexpr int kRow = W * ES;             // bytes of a staged row
  static constexpr int kUnit = 16 * kRow;         // 16 tokens of K or of V
  // Units in a warp's ring. 96 KB a CTA (two CTAs an SM) up to W = 128, 192 KB above.
  static constexpr int kUnits = kUnit <= 2048 ? 12 : (kUnit <= 8192 ? 6 : 3);
  static constexpr int kRows = 8 * NT;
  static constexpr int kPitch = W + 4;            // floats; conflict-free C-fragment stores
  static constexpr int kJoin = kWarps * kRows * kPitch * 4;
  static constexpr int kRing = kWarps * kUnits * kUnit;
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
  static constexpr int kChunks = kRow / 16;       // 16-byte pieces of a row
  // XOR on a row's 16-byte pieces that spreads 8 consecutive rows over the banks
  static __device__ __forceinline__ int swz(int r) { return kChunks >= 8 ? (r & 7) : ((r >> 1) & 3); }
};

// Chunks of a sequence and its first key. A bad length is cut to what the table can hold.
struct Span {
  int len, lo, first, n;
};
__device__ __forceinline__ Span span_of(const AttnParams &p, int b) {
  Span s;
  int len = p.lens[b];
  const long long cap = (long long)p.max_pages * p.page_size;
  if (len < 0 || len > cap) {
    report_error(p.err, MOE_DEV_ERR_BAD_LENGTH, 0);
    len = len < 0 ? 0 : (int)cap;
  }
  s.len = len;
  s.lo = p.window > 0 && len > p.window ? len - p.window : 0;
  s.first = s.lo / MOE_ATTN_CHUNK;
  s.n = len > 0 ? (len - 1) / MOE_ATTN_CHUNK + 1 - s.first : 0;
  return s;
}

__device__ __forceinline__ long long shfl_up64(long long v, int d) { return __shfl_up_sync(0xffffffffu, v, d); }

// T: type of the products. QB: q is bf16 (only read with ES == 1; else q has type T).
template <typename T, int W, int NT, int ES, bool QB>
__global__ void __launch_bounds__(kWarps * 32) k_attn_decode(const AttnParams p) {
  using S = Shape<W, NT, ES>;
  using M = Mma<T>;
  extern __shared__ __align__(128) char smem[];
  __shared__ long long sh_scan[kWarps];
  __shared__ long long sh_found[2];
  __shared__ float sh_m[kWarps][S::kRows], sh_l[kWarps][S::kRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  pdl_launch_dependents();

  // ---- the CTA's range of chunks
  const int hs = p.nkv * p.n_groups;
  long long total = 0;
  for (int b = tid; b < p.B; b += kWarps * 32) total += span_of(p, b).n;
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) sh_scan[warp] = total;
  if (tid == 0) sh_found[0] = -1;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += sh_scan[w];
  __syncthreads();
  total *= hs;
  const long long ctas = total < (long long)gridDim.x ? total : (long long)gridDim.x;
  const long long cta = blockIdx.x;
  long long u = 0, u_end = 0;
  if (cta < ctas) {
    u = cta * total / ctas;
    u_end = (cta + 1) * total / ctas;
  }
  // sequences without a key: rows of zeros, lse = -inf
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (span_of(p, b).n) continue;
    for (int i = tid; i < p.nq * p.D; i += kWarps * 32) {
      const int h = i / p.D, d = i - h * p.D;
      const long long at = (long long)b * p.out_tok + (long long)h * p.out_head + d;
      if constexpr (ES == 1 && QB) static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(0.f);
      else static_cast<T *>(p.out)[at] = T(0.f);
      if (p.lse && d == 0) p.lse[(long long)b * p.nq + h] = __int_as_float(0xff800000);
    }
  }
  if (u >= u_end) {
    if (tid == 0) p.rec[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  // ---- the sequence that holds chunk u
  long long before = 0;   // chunks of the earlier sequences (for one head)
  for (int base = 0; base < p.B; base += kWarps * 32) {
    const int b = base + tid;
    const long long n = b < p.B ? span_of(p, b).n : 0;
    long long inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = shfl_up64(inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31) sh_scan[warp] = inc;
    __syncthreads();
    long long add = before, strip = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) add += sh_scan[w];
      strip += sh_scan[w];
    }
    const long long lo = (add + inc - n) * hs, hi = (add + inc) * hs;
    if (u >= lo && u < hi) {
      sh_found[0] = b;
      sh_found[1] = add + inc - n;
    }
    before += strip;
    __syncthreads();
    if (sh_found[0] >= 0) break;
  }
  int b = (int)sh_found[0];
  long long seq_first = sh_found[1];
  Span sp = span_of(p, b);

  const uint32_t ring = smem_u32(smem) + warp * (S::kUnits * S::kUnit);
  int4 rec = make_int4(0, 0, 0, 0);

  while (u < u_end) {
    const long long rel = u - seq_first * hs;
    const int seg = (int)(rel / sp.n), i0 = (int)(rel - (long long)seg * sp.n);
    const int cnt = (int)(u_end - u < (long long)(sp.n - i0) ? u_end - u : (long long)(sp.n - i0));
    const int kvh = seg / p.n_groups, h0 = kvh * p.group + (seg - kvh * p.n_groups) * S::kRows;
    const int heads = min(S::kRows, (kvh + 1) * p.group - h0);

    // ---- loader state: this lane looks up row (lane & 15) of each 16-token unit
    const int row = lane & 15;
    const int t_first = (sp.first + i0) * MOE_ATTN_CHUNK + warp * 16;   // of the warp's first unit
    const int32_t *table = p.tables + (long long)b * p.table_stride;
    const char *kb = p.k + (long long)kvh * p.head_b, *vb = p.v + (long long)kvh * p.head_b;
    int page = 0;
    auto look_up = [&](int i) {   // block-table entry of this lane's row of the warp's i-th unit
      const int t = t_first + i * MOE_ATTN_CHUNK + row;
      page = 0;
      if (i < cnt && t >= sp.lo && t < sp.len) page = __ldg(table + t / p.page_size);
    };
    long long off = 0;
    bool ok = false;
    auto locate = [&](int i) {
      const int t = t_first + i * MOE_ATTN_CHUNK + row;
      ok = i < cnt && t >= sp.lo && t < sp.len;
      if (ok && (page < 0 || page >= p.num_pages)) {
        report_error(p.err, MOE_DEV_ERR_BAD_PAGE, 0);
        ok = false;
      }
      off = ok ? (long long)page * p.page_b + (long long)(t % p.page_size) * p.tok_b : 0;
    };
    auto issue = [&](const char *base, int slot) {
      const uint32_t dst = ring + slot * S::kUnit;
#pragma unroll
      for (int j = 0; j < S::kUnit / 512; ++j) {
        const int idx = j * 32 + lane, r = idx / S::kChunks, ch = idx % S::kChunks;
        const long long ro = __shfl_sync(0xffffffffu, off, r);
        const bool rok = __shfl_sync(0xffffffffu, (int)ok, r) && ch * (16 / ES) < p.D;
        copy16(dst + r * S::kRow + ((ch ^ S::swz(r)) << 4), rok ? base + ro + ch * 16 : base, rok);
      }
      copy_commit();
    };
    const int units = 2 * cnt;   // K, V, K, V, ...
    int next = 0, slot_in = 0;   // next unit to issue
    auto issue_next = [&]() {
      if (next < units) {
        if (!(next & 1)) {
          locate(next >> 1);
          look_up((next >> 1) + 1);
          issue(kb, slot_in);
        } else {
          issue(vb, slot_in);
        }
      } else {
        copy_commit();
      }
      ++next;
      slot_in = slot_in + 1 == S::kUnits ? 0 : slot_in + 1;
    };
    look_up(0);
    for (int i = 0; i < S::kUnits - 1; ++i) issue_next();

    // ---- q as B fragments: columns = heads, k = head elements
    uint32_t qf[W / 16][NT][2];
    float sc[NT][2];   // score scale of the lane's two columns
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int hh = 8 * n + g;
      const long long at = (long long)b * p.q_tok + (long long)(h0 + hh) * p.q_head;
      if constexpr (ES == 2) {
        const T *q = static_cast<const T *>(p.q) + at;
#pragma unroll
        for (int s = 0; s < W / 16; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int d = 16 * s + 8 * e + 2 * c;
            qf[s][n][e] = hh < heads && d < p.D ? *reinterpret_cast<const uint32_t *>(q + d) : 0u;
          }
        sc[n][0] = sc[n][1] = p.scale_log2;
      } else {
        // k index of the e4m3 fragments: b0 holds elements 4c, 4c + 1 of the 16, b1 4c + 2, 4c + 3.
        // q is scaled by a power of two that puts the head's largest value in [1, 2), so that
        // fp16 holds a bf16 q; the scores are multiplied back.
        float top = 0.f;
        uint2 raw[W / 16];
#pragma unroll
        for (int s = 0; s < W / 16; ++s) {
          const int d = 16 * s + 4 * c;
          raw[s] = make_uint2(0u, 0u);
          if (hh < heads && d < p.D) raw[s] = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.q) + at + d);
        }
        auto up = [&](uint32_t w, float &x, float &y) {
          if constexpr (QB) {
            x = __uint_as_float(w << 16);
            y = __uint_as_float(w & 0xffff0000u);
          } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
            x = f.x;
            y = f.y;
          }
        };
#pragma unroll
        for (int s = 0; s < W / 16; ++s) {
          float x, y;
          up(raw[s].x, x, y);
          top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
          up(raw[s].y, x, y);
          top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int eb = (int)(__float_as_uint(top) >> 23);          // biased exponent
        eb = eb < 1 ? 127 : (eb > 253 ? 253 : eb);
        const float down = __uint_as_float((uint32_t)(254 - eb) << 23), back = __uint_as_float((uint32_t)eb << 23);
#pragma unroll
        for (int s = 0; s < W / 16; ++s) {
          float x, y;
          up(raw[s].x, x, y);
          qf[s][n][0] = M::pack(x * down, y * down);
          up(raw[s].y, x, y);
          qf[s][n][1] = M::pack(x * down, y * down);
        }
        sc[n][0] = p.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * c);
        sc[n][1] = p.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * c + 4);
      }
    }

    float o[W / 16][NT][4];
#pragma unroll
    for (int s = 0; s < W / 16; ++s)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[s][n][e] = 0.f;
    float mx[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = __int_as_float(0xff800000), l[n][0] = l[n][1] = 0.f;

    int slot = 0;
    for (int i = 0; i < cnt; ++i) {
      // ---- S^T = K Q^T
      copy_wait<S::kUnits - 2>();
      __syncwarp();
      float s[NT][2][4];   // two accumulators shorten the chain
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][0][e] = s[n][1][e] = 0.f;
      {
        const uint32_t ku = ring + slot * S::kUnit;
        const int r = (lane & 7) + (lane & 8), hi = lane >> 4;
        const uint32_t base = ku + r * S::kRow;
        const int x = S::swz(r);
        if constexpr (ES == 2) {
#pragma unroll
          for (int k = 0; k < W / 16; ++k) {
            uint32_t a[4];
            ldsm4(a, base + (((2 * k + hi) ^ x) << 4));
#pragma unroll
            for (int n = 0; n < NT; ++n) M::run(s[n][k & 1], a, qf[k][n][0], qf[k][n][1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < W / 32; ++k) {
            uint32_t w[4];
            ldsm4(w, base + (((2 * k + hi) ^ x) << 4));
            uint32_t a[4];
            a[0] = e4m3x2_to_f16x2(w[0]);
            a[1] = e4m3x2_to_f16x2(w[1]);
            a[2] = e4m3x2_to_f16x2(w[0] >> 16);
            a[3] = e4m3x2_to_f16x2(w[1] >> 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) M::run(s[n][0], a, qf[2 * k][n][0], qf[2 * k][n][1]);
            a[0] = e4m3x2_to_f16x2(w[2]);
            a[1] = e4m3x2_to_f16x2(w[3]);
            a[2] = e4m3x2_to_f16x2(w[2] >> 16);
            a[3] = e4m3x2_to_f16x2(w[3] >> 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) M::run(s[n][1], a, qf[2 * k + 1][n][0], qf[2 * k + 1][n][1]);
          }
        }
      }
      slot = slot + 1 == S::kUnits ? 0 : slot + 1;
      __syncwarp();
      issue_next();

      // ---- softmax over the unit's tokens, in base 2
      const int t0 = t_first + i * MOE_ATTN_CHUNK + g;
      const bool in0 = t0 >= sp.lo && t0 < sp.len, in1 = t0 + 8 >= sp.lo && t0 + 8 < sp.len;
      uint32_t pf[NT][2];
      bool scale_o = false;
      float al[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float ninf = __int_as_float(0xff800000);
        const float v0 = in0 ? (s[n][0][0] + s[n][1][0]) * sc[n][0] : ninf, v1 = in0 ? (s[n][0][1] + s[n][1][1]) * sc[n][1] : ninf;
        const float v2 = in1 ? (s[n][0][2] + s[n][1][2]) * sc[n][0] : ninf, v3 = in1 ? (s[n][0][3] + s[n][1][3]) * sc[n][1] : ninf;
        float m0 = fmaxf(v0, v2), m1 = fmaxf(v1, v3);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, x));
          m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, x));
        }
        m0 = fmaxf(m0, mx[n][0]);
        m1 = fmaxf(m1, mx[n][1]);
        // a maximum of -inf (no key yet) must not meet itself in a difference
        const float b0 = (m0 == ninf ? 0.f : m0) - M::kOff, b1 = (m1 == ninf ? 0.f : m1) - M::kOff;
        al[n][0] = exp2_fast(mx[n][0] - M::kOff - b0);
        al[n][1] = exp2_fast(mx[n][1] - M::kOff - b1);
        scale_o |= m0 != mx[n][0] || m1 != mx[n][1];
        mx[n][0] = m0;
        mx[n][1] = m1;
        const float p0 = exp2_fast(v0 - b0), p1 = exp2_fast(v1 - b1), p2 = exp2_fast(v2 - b0), p3 = exp2_fast(v3 - b1);
        l[n][0] = l[n][0] * al[n][0] + (p0 + p2);
        l[n][1] = l[n][1] * al[n][1] + (p1 + p3);
        pf[n][0] = transposed8x8(M::pack(p0, p1));
        pf[n][1] = transposed8x8(M::pack(p2, p3));
      }
      if (__any_sync(0xffffffffu, scale_o)) {
#pragma unroll
        for (int k = 0; k < W / 16; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[k][n][0] *= al[n][0];
            o[k][n][1] *= al[n][1];
            o[k][n][2] *= al[n][0];
            o[k][n][3] *= al[n][1];
          }
      }

      // ---- O^T += V^T P^T
      copy_wait<S::kUnits - 2>();
      __syncwarp();
      {
        const uint32_t vu = ring + slot * S::kUnit;
        if constexpr (ES == 2) {
          const int r = (lane & 7) + ((lane >> 4) << 3), hi = (lane >> 3) & 1;
          const uint32_t base = vu + r * S::kRow;
          const int x = S::swz(r);
#pragma unroll
          for (int k = 0; k < W / 16; ++k) {
            uint32_t a[4];
            ldsm4t(a, base + (((2 * k + hi) ^ x) << 4));
#pragma unroll
            for (int n = 0; n < NT; ++n) M::run(o[k][n], a, pf[n][0], pf[n][1]);
          }
        } else {
          const int r = (lane & 7) + (lane & 8), hi = lane >> 4;
          const uint32_t base = vu + r * S::kRow;
          const int x = S::swz(r);
#pragma unroll
          for (int k = 0; k < W / 32; ++k) {
            uint32_t w[4];
            ldsm4t(w, base + (((2 * k + hi) ^ x) << 4));
            // a word holds elements (2g, 2g + 1) of token 2c, then of token 2c + 1: row g of the
            // product's tile takes element 2g, row g + 8 element 2g + 1
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t lo = __byte_perm(w[2 * h], 0u, 0x3120), hi8 = __byte_perm(w[2 * h + 1], 0u, 0x3120);
              uint32_t a[4];
              a[0] = e4m3x2_to_f16x2(lo);
              a[1] = e4m3x2_to_f16x2(lo >> 16);
              a[2] = e4m3x2_to_f16x2(hi8);
              a[3] = e4m3x2_to_f16x2(hi8 >> 16);
#pragma unroll
              for (int n = 0; n < NT; ++n) M::run(o[2 * k + h][n], a, pf[n][0], pf[n][1]);
            }
          }
        }
      }
      slot = slot + 1 == S::kUnits ? 0 : slot + 1;
      __syncwarp();
      issue_next();
    }

    // ---- join the four warps
    copy_wait<0>();
    __syncthreads();
    float *jo = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        l[n][0] += __shfl_xor_sync(0xffffffffu, l[n][0], x);
        l[n][1] += __shfl_xor_sync(0xffffffffu, l[n][1], x);
      }
      if (g == 0) {
        sh_m[warp][8 * n + 2 * c] = mx[n][0];
        sh_m[warp][8 * n + 2 * c + 1] = mx[n][1];
        sh_l[warp][8 * n + 2 * c] = l[n][0];
        sh_l[warp][8 * n + 2 * c + 1] = l[n][1];
      }
      float *w0 = jo + (warp * S::kRows + 8 * n + 2 * c) * S::kPitch, *w1 = w0 + S::kPitch;
#pragma unroll
      for (int k = 0; k < W / 16; ++k) {
        const int d0 = ES == 2 ? 16 * k + g : 16 * k + 2 * g, d1 = ES == 2 ? d0 + 8 : d0 + 1;
        w0[d0] = o[k][n][0];
        w1[d0] = o[k][n][1];
        w0[d1] = o[k][n][2];
        w1[d1] = o[k][n][3];
      }
    }
    __syncthreads();
    const bool whole = cnt == sp.n;
    const int piece = 2 * (int)cta + (i0 == 0 ? 1 : 0);
    for (int i = tid; i < heads * (p.D / 2); i += kWarps * 32) {
      const int h = i / (p.D / 2), d = 2 * (i - h * (p.D / 2));
      float m = sh_m[0][h];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, sh_m[w][h]);
      const float base = m == __int_as_float(0xff800000) ? 0.f : m;
      float sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_fast(sh_m[w][h] - base);
        const float2 v = *reinterpret_cast<const float2 *>(jo + (w * S::kRows + h) * S::kPitch + d);
        sum = fmaf(f, sh_l[w][h], sum);
        x = fmaf(f, v.x, x);
        y = fmaf(f, v.y, y);
      }
      if (whole) {
        const float inv = sum == 0.f ? 0.f : p.v_scale / sum;
        const long long at = (long long)b * p.out_tok + (long long)(h0 + h) * p.out_head + d;
        if constexpr (ES == 1 && QB)
          *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.out) + at) = Mma<__nv_bfloat16>::pack(x * inv, y * inv);
        else
          *reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + at) = M::pack(x * inv, y * inv);
        if (p.lse && d == 0) p.lse[(long long)b * p.nq + h0 + h] = (m + (log2f(sum) - M::kOff)) * kLn2;
      } else {
        const long long at = (long long)piece * S::kRows + h;
        *reinterpret_cast<float2 *>(p.ws_o + at * p.D + d) = make_float2(x, y);
        if (d == 0) p.ws_ml[at] = make_float2(m, sum);
      }
    }
    __syncthreads();

    if (!whole && i0 == 0) {   // the segment starts here and goes on: its last chunk's CTA
      const long long e = seq_first * hs + (long long)(seg + 1) * sp.n;
      rec = make_int4(1, b, seg, (int)((e * ctas - 1) / total));
    }
    u += cnt;
    if (u < u_end && u >= (seq_first + sp.n) * hs) {
      seq_first += sp.n;
      do sp = span_of(p, ++b);
      while (sp.n == 0);
    }
  }
  if (tid == 0) p.rec[blockIdx.x] = rec;
}

// Sums the pieces of the segment that starts in CTA blockIdx.x and ends in a later one:
// row blockIdx.y of its heads. 256 threads: a float4 of the row each, several pieces at a time.
template <typename TO>
__global__ void __launch_bounds__(256) k_attn_join(const AttnParams p, int rows, float off) {
  __shared__ float sw[MOE_ATTN_MAX_CTAS];
  __shared__ float sred[8], ssum[8];
  __shared__ float4 sacc[256];
  pdl_wait();
  const int4 rec = p.rec[blockIdx.x];
  if (!rec.x) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = rec.y, kvh = rec.z / p.n_groups, h = kvh * p.group + (rec.z - kvh * p.n_groups) * rows + blockIdx.y;
  if (h >= (kvh + 1) * p.group) return;
  const int c0 = blockIdx.x, n = rec.w - c0 + 1;
  // piece j: the starting CTA's second slot, then the later CTAs' first slots
  auto at = [&](int j) { return (long long)(2 * (c0 + j) + (j == 0 ? 1 : 0)) * rows + blockIdx.y; };
  const float ninf = __int_as_float(0xff800000);
  float m = ninf;
  for (int j = tid; j < n; j += 256) m = fmaxf(m, p.ws_ml[at(j)].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) sred[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, sred[w]);
  const float base = m == ninf ? 0.f : m;
  float sum = 0.f;
  for (int j = tid; j < n; j += 256) {
    const float2 ml = p.ws_ml[at(j)];
    const float f = exp2_fast(ml.x - base);
    sw[j] = f;
    sum = fmaf(f, ml.y, sum);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) ssum[warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) sum += ssum[w];

  const int quads = p.D / 4, par = 256 / quads, j0 = tid / quads, q = tid - j0 * quads;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (j0 < par) {
#pragma unroll 4
    for (int j = j0; j < n; j += par) {
      const float4 v = *reinterpret_cast<const float4 *>(p.ws_o + at(j) * p.D + 4 * q);
      const float f = sw[j];
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
  }
  sacc[tid] = acc;
  __syncthreads();
  if (tid < quads) {
    for (int j = 1; j < par; ++j) {
      const float4 v = sacc[j * quads + tid];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
    const float inv = sum == 0.f ? 0.f : p.v_scale / sum;
    uint2 w;
    w.x = Mma<TO>::pack(acc.x * inv, acc.y * inv);
    w.y = Mma<TO>::pack(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2 *>(static_cast<TO *>(p.out) + (long long)b * p.out_tok + (long long)h * p.out_head + 4 * tid) = w;
    if (p.lse && tid == 0) p.lse[(long long)b * p.nq + h] = (m + (log2f(sum) - off)) * kLn2;
  }
}

template <typename T, int W, int NT, int ES, bool QB> int launch(const AttnParams &p, int num_sms, cudaStream_t s) {
  using S = Shape<W, NT, ES>;
  using TO = std::conditional_t<ES == 1 && QB, __nv_bfloat16, T>;
  static unsigned long long attr_done = 0;
  const auto fn = k_attn_decode<T, W, NT, ES, QB>;
  if (!moe_allow_dyn_smem(reinterpret_cast<const void *>(fn), &attr_done)) return -1;
  static int per_sm = 0;   // the same on every device this library runs on (sm_100)
  int occ = __atomic_load_n(&per_sm, __ATOMIC_RELAXED);
  if (!occ) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, kWarps * 32, S::kSmem) != cudaSuccess || occ < 1) return -1;
    __atomic_store_n(&per_sm, occ, __ATOMIC_RELAXED);
  }
  int grid = num_sms * occ;
  if (grid > MOE_ATTN_MAX_CTAS) grid = MOE_ATTN_MAX_CTAS;
  fn<<<grid, kWarps * 32, S::kSmem, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return -1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, S::kRows < p.group ? S::kRows : p.group);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, k_attn_join<TO>, p, S::kRows, Mma<T>::kOff) != cudaSuccess) return -1;
  moe_prof_count(2);
  return 0;
}

template <typename T, int ES, bool QB> int dispatch(const AttnParams &p, int num_sms, cudaStream_t s) {
  const int nt = moe_attn_tiles(p.D, p.group);
  switch (moe_attn_width(p.D)) {
    case 64:
      return nt == 1 ? launch<T, 64, 1, ES, QB>(p, num_sms, s) : nt == 2 ? launch<T, 64, 2, ES, QB>(p, num_sms, s)
           : nt == 4 ? launch<T, 64, 4, ES, QB>(p, num_sms, s) : launch<T, 64, 8, ES, QB>(p, num_sms, s);
    case 128:
      return nt == 1 ? launch<T, 128, 1, ES, QB>(p, num_sms, s) : nt == 2 ? launch<T, 128, 2, ES, QB>(p, num_sms, s)
                     : launch<T, 128, 4, ES, QB>(p, num_sms, s);
    case 256:
      return nt == 1 ? launch<T, 256, 1, ES, QB>(p, num_sms, s) : launch<T, 256, 2, ES, QB>(p, num_sms, s);
    default:
      return launch<T, 512, 1, ES, QB>(p, num_sms, s);
  }
}

}  // namespace moe_attn
