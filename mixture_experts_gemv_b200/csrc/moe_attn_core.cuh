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
// Warps are independent workers without a block barrier in their loop. A unit of work is 16 or 32
// tokens (one or two row tiles) of one (sequence, KV head, head group) = segment. The units of all
// segments are numbered through and cut into equal ranges, one per warp of a grid that fills the
// GPU once, whatever the lengths are. A warp streams its units' K and V rows through a ring of
// cp.async copies of its own, which runs ahead over the ends of segments. A segment that a range
// holds whole is written out by its warp; one cut by a range's end leaves unnormalised pieces in
// the workspace (at most two per warp, in fragment order; a block in the middle of a long segment
// joins its warps' first), and the join kernel, launched behind with programmatic dependent
// launch, sums them in order. No atomics: outputs repeat bit for bit.
//
// Precision: K Q^T products are exact (of a bf16 q over an 8-bit cache, for elements from 2^-31 of
// the head's largest on), summed in FP32; the softmax runs in FP32 (base 2); P is rounded to the
// 16-bit type of the V product (half a step, 2^-8 or 2^-11 of each p; the sum l keeps the unrounded
// p); O is FP32 and rounded once. p is 2^(score - base), the base being the largest score so far; for
// fp16 15 below it, rounded up, so that the largest p is at most 2^15 at any size of the scores, and
// what fp16 cannot hold lies below 2^-39 of it (2^-32 where the scores' own steps are 4 and more).
// Sums are kept with their base, so its rounding reaches no result.
//
// Measured (bytes of the keys in range, over the two launches replayed in a graph; a copy streams
// 6.5 TB/s): one sequence of 997 tokens, 8 KV heads of 128 8.7 us; of 10,000, 8 of 256 21.9 us =
// 3.7 TB/s; of 40,000, 2 of 512 41.8 us = 3.9; 8 sequences of up to 40,000, 8 of 128 43.8 us = 4.8;
// 128 of up to 4,096 in 8 bits, 4 of 128 48.6 us = 4.7; 64 of 16,384, 8 of 128 (4.3 GB) 626 us = 6.9.
// What does not grow with the lengths is about 9 us: 1.6 until a warp knows its range, 3 to 5 until
// the first K rows are there, 1 for the blocks' pieces, 3 for the join; and 0.01 us a sequence, for
// the numbering: 1,024 sequences of 64 tokens of one KV head take 15.6 us, out of L2. Over 8-bit
// caches neither memory (64 %) nor issue (41 %) is busy: 12 warps an SM wait for their own chain of
// conversions, products and softmax.
//
// Wide groups and wide heads hold more than 255 registers: heads of 512 spill 200 to 320 bytes a
// thread, 16 query heads of 256 260 to 600, 32 of 128 400 to 660, 64 of 64 810 to 1,200. Their time is
// the warp's own work: 8 sequences of 40,000 with 71 query heads on one KV head of 64 take 176 us, with
// 32 on one of 128 in 8 bits 80 us; the bytes are 12.5 us in both.
//
// Tried and left: K's 8-bit products as they are, q in two or three 8-bit terms (mma.sync with 8-bit
// operands is emulated: the 8-bit case went from 59 to 67 us); one bulk copy a row (a warp issues
// one per 70 clocks or so: 3.9 TB/s with rows of 256 bytes).
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
  static __device__ __forceinline__ float base(float top) { return top; }
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
  static __device__ __forceinline__ float base(float top) { return __fadd_ru(top, -15.f); }
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
// The low and the high two bytes of v as fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t v, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(v));
}
// 16-byte asynchronous copy; with ok false nothing is read and zeros are written.
__device__ __forceinline__ void copy16(uint32_t dst, const char *src, bool ok) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
// The same where `on` is not 0, without a branch; nothing is written otherwise.
__device__ __forceinline__ void copy16_if(uint32_t dst, const char *src, int on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\t"
               "@p cp.async.cg.shared.global.L2::128B [%0], [%1], 16;\n\t}" ::"r"(dst), "l"(src), "r"(on) : "memory");
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
  static constexpr int kRow = W * ES;               // bytes of a staged row
  // 16-token row tiles a warp takes per step: two where a row is short, which halves the share
  // of the softmax's shuffles and of the loop (not with 32 heads and more: registers)
  static constexpr int kTiles = kRow <= 256 && NT <= 2 ? 2 : 1;
  static constexpr int kTok = 16 * kTiles, kLog = kTiles == 1 ? 4 : 5;   // tokens of a unit, and log2
  static constexpr int kUnit = kTok * kRow;         // bytes of its K or V rows
  // FP32 rows of the tile's heads, which a warp stages in its ring when its block joins its pieces
  static constexpr int kStage = W * NT * 32;
  // Slots of kUnit in a warp's ring, which has to hold kStage too: of 16 KB 3 (192 KB a CTA), of
  // 8 KB 3 (96 KB), of 4 KB and less 4 (64 KB and 32 KB a CTA), or as many as kStage takes: wide
  // groups over short rows have 8 of 2 KB, 8 or 16 of 1 KB (32 or 64 KB a CTA)
  static constexpr int kCopySlots = kUnit >= 16384 ? 3 : kUnit <= 4096 ? 4 : 24576 / kUnit;
  static constexpr int kSlots = kCopySlots * kUnit >= kStage ? kCopySlots : (kStage + kUnit - 1) / kUnit;
  static_assert(kSlots * kUnit >= kStage, "a warp's ring holds its staged rows");
  static constexpr int kRows = 8 * NT;
  static constexpr int kSmem = kWarps * kSlots * kUnit;
  static constexpr int kPieces = kRow / 16;         // 16-byte pieces of a row
  // XOR on a row's 16-byte pieces that spreads 8 consecutive rows over the banks
  static __device__ __forceinline__ constexpr int swz(int r) { return kPieces >= 8 ? (r & 7) : ((r >> 1) & 3); }
  // Address of the k-th pair of pieces of the row whose first pair lies at base: the XOR touches
  // the low three bits of a piece's number, the rest is an offset
  static __device__ __forceinline__ constexpr uint32_t at(uint32_t base, int k) { return (base ^ (uint32_t)((k & 3) << 5)) + (k >> 2) * 128; }
};

// Keys [lo, len) of a sequence: n units of 2^LOG tokens from unit number lo >> LOG on. A bad length is
// cut to [0, what the table can hold] (Numbering reports it).
struct Span {
  int len, lo, n;
  __device__ __forceinline__ Span() : len(0), lo(0), n(0) {}
  __device__ __forceinline__ Span(const AttnParams &p, int length, int log) {
    len = min(max(length, 0), p.max_tokens);
    lo = p.window > 0 && len > p.window ? len - p.window : 0;
    n = len > 0 ? ((len - 1) >> log) + 1 - (lo >> log) : 0;
  }
};

static __device__ __noinline__ long long quotient64(long long a, int b) { return a / b; }
__device__ __forceinline__ long long quotient(long long a, int b) {   // a >= 0; 32-bit division where it fits
  return (a >> 32) ? quotient64(a, b) : (long long)((unsigned)a / (unsigned)b);
}

// Equal ranges of `total` costs for at most `most` workers, each at least one: the first
// `longer` workers have one more than `each`.
struct Split {
  int workers, longer;
  long long each;
  Split() = default;
  __device__ __forceinline__ Split(long long total, int most) {
    workers = total < most ? (int)total : most;
    each = workers ? quotient(total, workers) : 0;
    longer = (int)(total - each * workers);
  }
  __device__ __forceinline__ long long first(int worker) const { return worker * each + min(worker, longer); }
  __device__ __forceinline__ int owner(long long cost) const {
    const long long head = longer * (each + 1);
    return cost < head ? (int)quotient(cost, (int)each + 1) : longer + (int)quotient(cost - head, (int)each);
  }
};

// Pieces of a segment cut over the workers [w0, w1]: a block whose four workers all lie strictly
// inside (they then have nothing else) leaves one piece, as its first worker's.
struct Block {
  int at;
  __device__ __forceinline__ explicit Block(int b) : at(b * kWarps) {}
  __device__ __forceinline__ bool inside(int w0, int w1) const { return at > w0 && at + kWarps - 1 < w1; }
};
struct Pieces {
  int w0, head, blocks, tail, count;   // workers before the whole blocks, blocks, first worker behind them
  __device__ __forceinline__ Pieces(int first, int last, bool joined) {
    w0 = first;
    const int a = first / kWarps + 1, b = last / kWarps - 1;   // first and last whole block
    blocks = joined && b >= a ? b - a + 1 : 0;
    head = blocks ? a * kWarps - first : last - first + 1;
    tail = (b + 1) * kWarps;
    count = blocks ? head + blocks + last - tail + 1 : head;
  }
  __device__ __forceinline__ int worker(int i) const {
    return i < head ? w0 + i : i < head + blocks ? (w0 / kWarps + 1 + i - head) * kWarps : tail + i - head - blocks;
  }
};

// Two heads' bases and sums (m, l, m, l) and a fragment of their unnormalised rows, joined from pieces.
struct Joined {
  float4 ml, acc;
  __device__ __forceinline__ Joined() {
    const float ninf = __int_as_float(0xff800000);
    ml = make_float4(ninf, 0.f, ninf, 0.f);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void take(const float4 &pm, const float4 &v) {
    const float ninf = __int_as_float(0xff800000);
    const float m0 = fmaxf(ml.x, pm.x), m1 = fmaxf(ml.z, pm.z), b0 = m0 == ninf ? 0.f : m0, b1 = m1 == ninf ? 0.f : m1;
    const float a0 = exp2_fast(ml.x - b0), a1 = exp2_fast(ml.z - b1), f0 = exp2_fast(pm.x - b0), f1 = exp2_fast(pm.z - b1);
    ml = make_float4(m0, fmaf(ml.y, a0, f0 * pm.y), m1, fmaf(ml.w, a1, f1 * pm.w));
    acc.x = fmaf(acc.x, a0, f0 * v.x);
    acc.y = fmaf(acc.y, a1, f1 * v.y);
    acc.z = fmaf(acc.z, a0, f0 * v.z);
    acc.w = fmaf(acc.w, a1, f1 * v.w);
  }
};

// The numbering of the call's work. A segment (sequence, KV head, head group) costs its units and,
// where workers have several, one more that comes first: its q, its ends and its result (eight
// one-unit segments in one warp's range took 5 to 8 us beside a 36 us stream of 40,000 tokens).
// Every worker's range of costs still holds a unit: no two of the extra ones are neighbours.
// Held by a warp: lane l has sequences base + 4 l .. of the strip that was looked at last.
// COLD: lengths are read past L1.
template <bool COLD> struct Numbering {
  static constexpr unsigned kAll = 0xffffffffu;
  static constexpr int kOwn = 4, kStrip = 32 * kOwn;
  int segs, extra, log;
  long long units;      // of all sequences, for one segment each
  Split split;
  int base;             // the strip, and what comes before it
  long long before;     // units
  int before_filled;    // sequences with a key
  int n[kOwn], len[kOwn];   // the lane's units and lengths
  long long inc;        // units up to the lane's last sequence, inclusive
  int filled;           // sequences with a key up to there
  int next[kOwn];       // the next strip's lengths

  static __device__ __forceinline__ void load(const AttnParams &p, int at, int (&to)[kOwn]) {
    const int b = at + kOwn * (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      to[j] = 0;
      if (b + j < p.B) to[j] = COLD ? __ldcg(p.lens + b + j) : p.lens[b + j];
    }
  }
  __device__ __forceinline__ void strip(const AttnParams &p, int at) {   // `next` holds its lengths
    const int lane = threadIdx.x & 31;
    base = at;
    unsigned sum = 0, keyed = 0;   // a lane's sum: four lengths up to 2^30 over 16
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      len[j] = next[j];
      n[j] = Span(p, len[j], log).n;
      sum += n[j];
      keyed += n[j] > 0;
    }
    load(p, at + kStrip, next);
    // both in one scan: the strip's units stay below 2^34
    unsigned long long both = (unsigned long long)keyed << 40 | sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long t = __shfl_up_sync(kAll, both, o);
      if (lane >= o) both += t;
    }
    inc = before + (long long)(both & ((1ull << 40) - 1));
    filled = before_filled + (int)(both >> 40);
  }
  __device__ __forceinline__ void next_strip(const AttnParams &p) {
    before = __shfl_sync(kAll, inc, 31);
    before_filled = __shfl_sync(kAll, filled, 31);
    strip(p, base + kStrip);
  }
  __device__ __forceinline__ Numbering(const AttnParams &p, int log_, int all_workers) : segs(p.nkv * p.n_groups), extra(0), log(log_), before(0), before_filled(0) {
    load(p, 0, next);
    bool bad = false;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) bad |= (unsigned)next[j] > (unsigned)p.max_tokens;
    strip(p, 0);
    units = __shfl_sync(kAll, inc, 31);
    int with_key = __shfl_sync(kAll, filled, 31);
    if (p.B > kStrip) {
      long long more = 0;
      int more_keys = 0;
#pragma unroll 1
      for (int at = kStrip; at < p.B; at += 2 * kStrip) {
        int x[kOwn], y[kOwn];
        load(p, at, x);
        load(p, at + kStrip, y);   // zeros past the last sequence
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          const int m = Span(p, x[j], log).n, m2 = Span(p, y[j], log).n;
          more += m + (long long)m2;
          more_keys += (m > 0) + (m2 > 0);
          bad |= (unsigned)x[j] > (unsigned)p.max_tokens || (unsigned)y[j] > (unsigned)p.max_tokens;
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        more += __shfl_xor_sync(kAll, more, o);
        more_keys += __shfl_xor_sync(kAll, more_keys, o);
      }
      units += more;
      with_key += more_keys;
    }
    if (!COLD && bad) atomicCAS(p.err, 0u, MOE_DEV_ERR_BAD_LENGTH);
    extra = (units + with_key) * segs >= 2ll * all_workers ? 1 : 0;
    split = Split((units + extra * with_key) * segs, all_workers);
  }
  // A segment: its sequence, number there, units and first cost.
  struct Segment {
    int b, seg, n, len;
    long long first;
    long long units_before;   // units of all segments before it
  };
  __device__ __forceinline__ Segment segment(int src, int seg) const {   // of the strip's sequence src
    const int lane = src / kOwn, own = src % kOwn;
    int n_ = n[0], len_ = len[0], behind = 0, behind_keyed = 0;   // sequence `own` of the lane, and what follows it there
#pragma unroll
    for (int j = 1; j < kOwn; ++j) {
      if (own == j) n_ = n[j], len_ = len[j];
      if (own < j) behind += n[j], behind_keyed += n[j] > 0;
    }
    Segment s;
    s.b = base + src;
    s.seg = seg;
    s.n = __shfl_sync(kAll, n_, lane);
    s.len = __shfl_sync(kAll, len_, lane);
    const long long u = __shfl_sync(kAll, inc - behind - n_, lane);
    const int f = __shfl_sync(kAll, filled - behind_keyed, lane) - 1;
    s.first = (u + extra * f) * segs + (long long)seg * (s.n + extra);
    s.units_before = u * segs + (long long)seg * s.n;
    return s;
  }
  // The segment that holds a cost below the total, not before the last one asked for.
  __device__ __forceinline__ Segment holding(const AttnParams &p, long long cost) {
    unsigned hit;
#pragma unroll 1
    while (!(hit = __ballot_sync(kAll, cost < (inc + extra * filled) * segs))) next_strip(p);
    const int lane = __ffs(hit) - 1;
    // the first of the lane's sequences that ends behind the cost
    int own = 0, behind = 0, behind_keyed = 0;
#pragma unroll
    for (int j = kOwn - 1; j > 0; --j) {
      behind += n[j];
      behind_keyed += n[j] > 0;
      if (own == 0 && cost >= (inc - behind + extra * (filled - behind_keyed)) * segs) own = j;
    }
    Segment s = segment(lane * kOwn + __shfl_sync(kAll, own, lane), 0);
    s.seg = (int)quotient(cost - s.first, s.n + extra);
    s.first += (long long)s.seg * (s.n + extra);
    s.units_before += (long long)s.seg * s.n;
    return s;
  }
  __device__ __forceinline__ int unit(const Segment &s, long long cost) const { return max((int)(cost - s.first) - extra, 0); }
};

// A place in the numbering: unit i of segment seg of sequence b.
template <int LOG> struct Cursor {
  int b, seg, i;
  Span sp;
  __device__ __forceinline__ void next(const AttnParams &p, int segs) {   // not past the last unit
    if (++i < sp.n) return;
    i = 0;
    if (++seg < segs) return;
    seg = 0;
#pragma unroll 1
    do sp = Span(p, p.lens[++b], LOG);
    while (sp.n == 0);
  }
  __device__ __forceinline__ int token() const { return ((sp.lo >> LOG) + i) << LOG; }   // the unit's first
};
__device__ __forceinline__ int kv_head(const AttnParams &p, int seg) { return p.n_groups == 1 ? seg : seg / p.n_groups; }

// One accumulator fragment (two heads' values at two elements, over their sums l) into the rows of a
// KV head's group: out points at head 8 n, `heads` of them exist. 16 ES-dependent elements from 16 k
// on. An 8-bit cache's scale comes last: over l it could fall below the normal numbers.
template <typename TO, int ES>
__device__ __forceinline__ void store_fragment(TO *out, long long out_head, int k, int heads, int lane, float4 v, float l0, float l1, float v_scale) {
  const int g = lane >> 2, c = lane & 3;
  const float inv0 = l0 == 0.f ? 0.f : 1.f / l0, inv1 = l1 == 0.f ? 0.f : 1.f / l1;
  v = make_float4(v.x * inv0, v.y * inv1, v.z * inv0, v.w * inv1);
  if constexpr (ES == 1) v = make_float4(v.x * v_scale, v.y * v_scale, v.z * v_scale, v.w * v_scale);
  const uint32_t lo = transposed8x8(Mma<TO>::pack(v.x, v.y)), hi = transposed8x8(Mma<TO>::pack(v.z, v.w));
  if (g >= heads) return;
  TO *row = out + g * out_head + 16 * k;
  if constexpr (ES == 2) {   // rows g and g + 8 of the tile are elements g and g + 8
    *reinterpret_cast<uint32_t *>(row + 2 * c) = lo;
    *reinterpret_cast<uint32_t *>(row + 8 + 2 * c) = hi;
  } else {                   // elements 2 g and 2 g + 1
    *reinterpret_cast<uint2 *>(row + 4 * c) = make_uint2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
  }
}

// T: type of the products. QB: q is bf16 (only read with ES == 1; else q has type T).
template <typename T, int W, int NT, int ES, bool QB>
__global__ void __launch_bounds__(kWarps * 32) k_attn_decode(const __grid_constant__ AttnParams p) {
  using S = Shape<W, NT, ES>;
  using M = Mma<T>;
  using TO = std::conditional_t<ES == 1 && QB, __nv_bfloat16, T>;
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ __align__(1024) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const float ninf = __int_as_float(0xff800000);
  const uint32_t ring = smem_u32(smem) + warp * (S::kSlots * S::kUnit);
  if (p.D < W) {   // the pieces past head_dim are never copied: zeros
#pragma unroll 1
    for (int i = lane * 16; i < S::kSlots * S::kUnit; i += 512)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(ring + i), "r"(0) : "memory");
    __syncwarp();
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---- the warp's range of units
  const int all_workers = kWarps * gridDim.x;
  Numbering<false> num(p, S::kLog, all_workers);
  const int segs = num.segs, workers = num.split.workers;
  // Neighbours in the numbering are on different SMs where there is little to do, else in one
  // block, which can then join its warps' pieces
  const int worker = num.extra ? blockIdx.x * kWarps + warp : warp * gridDim.x + blockIdx.x;
  // sequences without a key: rows of zeros, lse = -inf
#pragma unroll 1
  for (int b = worker; b < p.B; b += all_workers) {
    if (Span(p, p.lens[b], S::kLog).n) continue;
#pragma unroll 1
    for (int h = 0; h < p.nq; ++h) {
#pragma unroll 1
      for (int d = lane; d < p.D; d += 32) static_cast<TO *>(p.out)[(long long)b * p.out_tok + (long long)h * p.out_head + d] = TO(0.f);
      if (p.lse && lane == 0) p.lse[(long long)b * p.nq + h] = ninf;
    }
    if (p.noted && p.by_segment) {   // nothing to join
#pragma unroll 1
      for (int x = lane; x < segs; x += 32) p.ws_cut[b * segs + x] = make_int4(0, 0, 0, 0);
    }
  }
  if (p.noted && !p.by_segment && lane == 0) p.ws_cut[worker] = make_int4(0, 0, 0, 0);   // for now
  if (worker >= workers) return;
  Cursor<S::kLog> at;        // the unit that is computed next
  long long seg_first;       // first cost of its segment
  int count;                 // the warp's units
  {
    long long begin = 0, end = num.units * segs;   // in units
#pragma unroll 1
    for (int x = 0; x < 2 && worker + x < workers; ++x) {   // where the range starts and where the next one does
      const long long cost = num.split.first(worker + x);
      const auto s = num.holding(p, cost);
      const int i = num.unit(s, cost);
      if (x == 0) {
        at.b = s.b;
        at.seg = s.seg;
        at.i = i;
        at.sp = Span(p, s.len, S::kLog);
        seg_first = s.first;
        begin = s.units_before + i;
      } else {
        end = s.units_before + i;
      }
    }
    count = (int)(end - begin);
  }
  const Split split = num.split;
  const int extra = num.extra;

  // ---- loader: runs ahead of the computation by the ring's slots, and its look-ups in the block
  // tables by two units more
  Cursor<S::kLog> ahead = at;   // the unit that is looked up next
  int to_look_up = count;
  struct Found {                // a looked-up unit, as lane r holds it for token r
    int page, in_page, kvh, first, last;   // tokens [first, last) of the unit are keys
  } now{}, then{};
  auto look_up = [&](Found &f) {
    if (to_look_up <= 0) return;
    const int t0 = ahead.token(), t = t0 + (lane & (S::kTok - 1));
    f.first = max(ahead.sp.lo - t0, 0);
    f.last = min(ahead.sp.len - t0, S::kTok);
    f.kvh = kv_head(p, ahead.seg);
    // with pages of whole 8-token groups, every lane of a group that holds a key has the group's page
    const int lo = p.groups_of_8 ? ahead.sp.lo & ~7 : ahead.sp.lo, hi = p.groups_of_8 ? (ahead.sp.len + 7) & ~7 : ahead.sp.len;
    if (t >= lo && t < hi) {
      const unsigned e = p.page_shift >= 0 ? (unsigned)t >> p.page_shift : (unsigned)t / (unsigned)p.page_size;
      f.in_page = t - (int)e * p.page_size;
      f.page = __ldcg(p.tables + (long long)ahead.b * p.table_stride + e);
    } else {
      f.page = f.in_page = 0;
    }
    if (--to_look_up > 0) {
      ahead.next(p, segs);
      if (ahead.i == 0) {   // a new segment: its q rows on their way to L1 (a lane per 128 bytes)
        const int kvh = kv_head(p, ahead.seg), h0 = kvh * p.group + (ahead.seg - kvh * p.n_groups) * S::kRows;
        const int lines = (p.D * 2 + 127) / 128, heads = min(S::kRows, (kvh + 1) * p.group - h0);
#pragma unroll 1
        for (int i = lane; i < heads * lines; i += 32) {
          const int h = i / lines;
          const char *q = static_cast<const char *>(p.q) + 2 * ((long long)ahead.b * p.q_tok + (long long)(h0 + h) * p.q_head) + (i - h * lines) * 128;
          asm volatile("prefetch.global.L1 [%0];" ::"l"(q));
        }
      }
    }
  };
  long long off = 0, group[S::kTok / 8];   // byte offsets in K and in V: this lane's row, each 8 rows
  bool ok = false, all = false;            // this lane's row is copied; every row is
  // A copy instruction moves 32 pieces: kPer rows, or a part of one.
  constexpr int kPer = S::kPieces <= 32 ? 32 / S::kPieces : 1, kParts = S::kPieces <= 32 ? 1 : S::kPieces / 32;
  const int my_row = S::kPieces <= 32 ? lane / S::kPieces : 0, my_piece = S::kPieces <= 32 ? lane % S::kPieces : lane;
  const uint32_t my_dst = my_row * S::kRow + ((my_piece ^ S::swz(my_row)) << 4);
  const uint32_t tok_b = (uint32_t)p.tok_b;
  const long long my_off = (long long)my_row * p.tok_b + my_piece * 16;
  int on[kParts];
#pragma unroll
  for (int x = 0; x < kParts; ++x) on[x] = x * 512 + my_piece * 16 < p.D * ES;
  int slot_in = 0, left_k = count, left_v = count;   // copies are made K, V, K, V, ...
  auto copy_unit = [&](const char *base) {
    const uint32_t dst = ring + slot_in * S::kUnit;
    const uint32_t to = dst + my_dst;   // its low bits hold the piece: slots are multiples of a row
    if (all) {
      // whole 8-token groups, each in one page: two additions and an XOR a copy
#pragma unroll
      for (int x = 0; x < S::kTok / 8; ++x) {
        const char *from = base + group[x] + my_off;
#pragma unroll
        for (int r = 0; r < 8; r += kPer) {
          const char *row = from + (unsigned long long)(tok_b * (uint32_t)r);
#pragma unroll
          for (int part = 0; part < kParts; ++part)
            copy16_if((to ^ (uint32_t)(S::swz(r) << 4)) + (x * 8 + r) * S::kRow + part * 512, row + part * 512, on[part]);
        }
      }
    } else if (p.groups_of_8) {
      // a sequence's or a window's end: rows that are no keys become zeros (0 x NaN in a page's
      // unused rows would reach the output)
      const unsigned rows = __ballot_sync(kAll, ok);
#pragma unroll 1
      for (int x = 0; x < S::kTok / 8; ++x) {
        const char *from = base + __shfl_sync(kAll, off, 8 * x) + my_off;
#pragma unroll
        for (int r = 0; r < 8; r += kPer) {
          const bool row_ok = rows >> (x * 8 + r + my_row) & 1;
          const char *row = row_ok ? from + (unsigned long long)(tok_b * (uint32_t)r) : base;
#pragma unroll
          for (int part = 0; part < kParts; ++part)
            copy16((to ^ (uint32_t)(S::swz(r) << 4)) + (x * 8 + r) * S::kRow + part * 512, row + part * 512, row_ok && on[part]);
        }
      }
    } else {
#pragma unroll 2
      for (int j = 0; j < S::kUnit / 512; ++j) {
        const int idx = j * 32 + lane, r = idx / S::kPieces, ch = idx % S::kPieces;
        const long long ro = __shfl_sync(kAll, off, r);
        const bool row_ok = __shfl_sync(kAll, (int)ok, r) && ch * 16 < p.D * ES;
        copy16(dst + r * S::kRow + ((ch ^ S::swz(r)) << 4), row_ok ? base + ro + ch * 16 : base, row_ok);
      }
    }
  };
  auto issue_k = [&]() {
    if (left_k > 0) {
      --left_k;
      const int r = lane & (S::kTok - 1);
      const bool good = (unsigned)now.page < (unsigned)p.num_pages;
      if (!good) atomicCAS(p.err, 0u, MOE_DEV_ERR_BAD_PAGE);
      off = (long long)now.kvh * p.head_b + (good ? (long long)now.page * p.page_b + (long long)now.in_page * p.tok_b : 0);
      ok = good && r >= now.first && r < now.last;
      all = p.groups_of_8 && __all_sync(kAll, ok);
      if (all) {
#pragma unroll
        for (int x = 0; x < S::kTok / 8; ++x) group[x] = __shfl_sync(kAll, off, 8 * x);
      }
      now = then;
      look_up(then);
      copy_unit(p.k);
    }
    copy_commit();
    slot_in = slot_in + 1 == S::kSlots ? 0 : slot_in + 1;
  };
  auto issue_v = [&]() {
    if (left_v > 0) {
      --left_v;
      copy_unit(p.v);
    }
    copy_commit();
    slot_in = slot_in + 1 == S::kSlots ? 0 : slot_in + 1;
  };
  look_up(now);
  then = now;
  look_up(then);
#pragma unroll 1
  for (int x = 0; x < (S::kSlots - 1) / 2; ++x) {
    issue_k();
    issue_v();
  }
  if (S::kSlots % 2 == 0) issue_k();

  int slot = 0, done = 0;
  while (true) {   // a piece: the units of one segment that are the warp's
    const int kvh = kv_head(p, at.seg), h0 = kvh * p.group + (at.seg - kvh * p.n_groups) * S::kRows;
    const int heads = min(S::kRows, (kvh + 1) * p.group - h0);
    const int i0 = at.i, cnt = min(at.sp.n - i0, count - done);
    const bool whole = cnt == at.sp.n;
    bool in_block = false;   // whether the block's four warps have nothing but parts of this segment
    if (!whole && (extra || p.noted)) {
      const int w0 = split.owner(seg_first + extra), w1 = split.owner(seg_first + extra + at.sp.n - 1);
      in_block = extra && Block(blockIdx.x).inside(w0, w1);
      if (p.noted && i0 == 0 && lane == 0) p.ws_cut[p.by_segment ? at.b * segs + at.seg : worker] = make_int4(w0 | extra << 16, w1, at.b, at.seg);
    } else if (whole && p.noted && p.by_segment && lane == 0) {
      p.ws_cut[at.b * segs + at.seg] = make_int4(0, 0, 0, 0);
    }

    uint32_t qf[W / 16][NT][2];
    float sc[NT][2];   // score scale of the lane's two columns
    auto load_q = [&]() {   // q as B fragments: columns = heads, k = head elements
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int hh = 8 * n + g;
        const long long q_at = (long long)at.b * p.q_tok + (long long)(h0 + hh) * p.q_head;
        if constexpr (ES == 2) {
          const T *q = static_cast<const T *>(p.q) + q_at;
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
          // An fp16 q is taken as it is. A bf16 one is multiplied by a power of two that puts the
          // head's largest value in [2^14, 2^15), so that fp16 holds it: exactly from 2^-31 of that
          // value on, smaller elements to 2^-39 of it. The scores are multiplied back.
          uint2 raw[W / 16];
#pragma unroll
          for (int s = 0; s < W / 16; ++s) {
            const int d = 16 * s + 4 * c;
            raw[s] = make_uint2(0u, 0u);
            if (hh < heads && d < p.D) raw[s] = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.q) + q_at + d);
          }
          if constexpr (QB) {
            auto up = [](uint32_t w, float &x, float &y) {
              x = __uint_as_float(w << 16);
              y = __uint_as_float(w & 0xffff0000u);
            };
            float top = 0.f;
#pragma unroll
            for (int s = 0; s < W / 16; ++s) {
              float x, y;
              up(raw[s].x, x, y);
              top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
              up(raw[s].y, x, y);
              top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
            }
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
            const int eb = max((int)(__float_as_uint(top) >> 23), 15);   // biased exponent; both factors are normal
            const float down = __uint_as_float((uint32_t)(268 - eb) << 23), back = __uint_as_float((uint32_t)(eb - 14) << 23);
#pragma unroll
            for (int s = 0; s < W / 16; ++s) {
              float x, y;
              up(raw[s].x, x, y);
              qf[s][n][0] = M::pack(x * down, y * down);
              up(raw[s].y, x, y);
              qf[s][n][1] = M::pack(x * down, y * down);
            }
            sc[n][0] = p.scale_log2 * __shfl_sync(kAll, back, 8 * c);
            sc[n][1] = p.scale_log2 * __shfl_sync(kAll, back, 8 * c + 4);
          } else {
#pragma unroll
            for (int s = 0; s < W / 16; ++s) {
              qf[s][n][0] = raw[s].x;
              qf[s][n][1] = raw[s].y;
            }
            sc[n][0] = sc[n][1] = p.scale_log2;
          }
        }
      }
    };
    float o[W / 16][NT][4];
#pragma unroll
    for (int s = 0; s < W / 16; ++s)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[s][n][e] = 0.f;
    float mx[NT][2], l[NT][2];   // bases (-inf: no key yet) and sums
#pragma unroll
    for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = ninf, l[n][0] = l[n][1] = 0.f;

    int t0 = at.token();
    uint32_t pf[S::kTiles][NT][2];   // P^T as B fragments
    load_q();
#pragma unroll 1
    for (int i = 0; i < cnt; ++i, t0 += S::kTok) {
      copy_wait<S::kSlots - 2>();
      __syncwarp();
      uint32_t unit = ring + slot * S::kUnit;
      // ---- S^T = K Q^T
      constexpr int kAcc = S::kTiles == 1 ? 2 : 1;   // a single row tile takes two accumulators, to shorten the chain
      float s[S::kTiles][NT][kAcc][4];
#pragma unroll
      for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int x = 0; x < kAcc; ++x) s[t][n][x][e] = 0.f;
      {
        const int r = (lane & 7) + (lane & 8), hi = lane >> 4;
        const uint32_t base = unit + r * S::kRow + ((hi ^ S::swz(r)) << 4);
        if constexpr (ES == 2) {
#pragma unroll
          for (int k = 0; k < W / 16; ++k)
#pragma unroll
            for (int t = 0; t < S::kTiles; ++t) {
              uint32_t a[4];
              ldsm4(a, S::at(base, k) + t * 16 * S::kRow);
#pragma unroll
              for (int n = 0; n < NT; ++n) M::run(s[t][n][k & (kAcc - 1)], a, qf[k][n][0], qf[k][n][1]);
            }
        } else {
#pragma unroll
          for (int k = 0; k < W / 32; ++k)
#pragma unroll
            for (int t = 0; t < S::kTiles; ++t) {
              uint32_t w[4];
              ldsm4(w, S::at(base, k) + t * 16 * S::kRow);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t a[4];
                e4m3x4_to_f16x2(w[2 * h], a[0], a[2]);
                e4m3x4_to_f16x2(w[2 * h + 1], a[1], a[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) M::run(s[t][n][h & (kAcc - 1)], a, qf[2 * k + h][n][0], qf[2 * k + h][n][1]);
              }
            }
        }
      }
      slot = slot + 1 == S::kSlots ? 0 : slot + 1;
      __syncwarp();
      // the freed slot takes the copy that is kSlots - 1 ahead
      if constexpr (S::kSlots % 2) issue_k();
      else issue_v();

      // ---- softmax over the unit's tokens, in base 2
      const bool full = t0 >= at.sp.lo && t0 + S::kTok <= at.sp.len;   // every token of the unit is a key
      bool scale_o = false;
      float al[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float v[S::kTiles][4];
#pragma unroll
        for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[t][e] = (kAcc == 2 ? s[t][n][0][e] + s[t][n][kAcc - 1][e] : s[t][n][0][e]) * sc[n][e & 1];
        if (!full) {
#pragma unroll
          for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tok = t0 + g + 16 * t + 8 * (e >> 1);
              if (tok < at.sp.lo || tok >= at.sp.len) v[t][e] = ninf;
            }
        }
        float m0 = fmaxf(v[0][0], v[0][2]), m1 = fmaxf(v[0][1], v[0][3]);
#pragma unroll
        for (int t = 1; t < S::kTiles; ++t) {
          m0 = fmaxf(m0, fmaxf(v[t][0], v[t][2]));
          m1 = fmaxf(m1, fmaxf(v[t][1], v[t][3]));
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, x));
          m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, x));
        }
        m0 = fmaxf(M::base(m0), mx[n][0]);
        m1 = fmaxf(M::base(m1), mx[n][1]);
        // a base of -inf must not meet itself in a difference
        const float b0 = m0 == ninf ? 0.f : m0, b1 = m1 == ninf ? 0.f : m1;
        al[n][0] = exp2_fast(mx[n][0] - b0);
        al[n][1] = exp2_fast(mx[n][1] - b1);
        scale_o |= m0 != mx[n][0] || m1 != mx[n][1];
        mx[n][0] = m0;
        mx[n][1] = m1;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int t = 0; t < S::kTiles; ++t) {
          const float p0 = exp2_fast(v[t][0] - b0), p1 = exp2_fast(v[t][1] - b1), p2 = exp2_fast(v[t][2] - b0), p3 = exp2_fast(v[t][3] - b1);
          s0 += p0 + p2;
          s1 += p1 + p3;
          pf[t][n][0] = transposed8x8(M::pack(p0, p1));
          pf[t][n][1] = transposed8x8(M::pack(p2, p3));
        }
        l[n][0] = fmaf(l[n][0], al[n][0], s0);
        l[n][1] = fmaf(l[n][1], al[n][1], s1);
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

      copy_wait<S::kSlots - 2>();
      __syncwarp();
      unit = ring + slot * S::kUnit;
      // ---- O^T += V^T P^T
      {
        if constexpr (ES == 2) {
          const int r = (lane & 7) + ((lane >> 4) << 3), hi = (lane >> 3) & 1;
          const uint32_t base = unit + r * S::kRow + ((hi ^ S::swz(r)) << 4);
#pragma unroll
          for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
            for (int k = 0; k < W / 16; ++k) {
              uint32_t a[4];
              ldsm4t(a, S::at(base, k) + t * 16 * S::kRow);
#pragma unroll
              for (int n = 0; n < NT; ++n) M::run(o[k][n], a, pf[t][n][0], pf[t][n][1]);
            }
        } else {
          const int r = (lane & 7) + (lane & 8), hi = lane >> 4;
          const uint32_t base = unit + r * S::kRow + ((hi ^ S::swz(r)) << 4);
#pragma unroll
          for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
            for (int k = 0; k < W / 32; ++k) {
              uint32_t w[4];
              ldsm4t(w, S::at(base, k) + t * 16 * S::kRow);
              // a word holds elements (2g, 2g + 1) of token 2c, then of token 2c + 1: row g of the
              // product's tile takes element 2g, row g + 8 element 2g + 1
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t lo = __byte_perm(w[2 * h], 0u, 0x3120), hi8 = __byte_perm(w[2 * h + 1], 0u, 0x3120);
                uint32_t a[4];
                e4m3x4_to_f16x2(lo, a[0], a[1]);
                e4m3x4_to_f16x2(hi8, a[2], a[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) M::run(o[2 * k + h][n], a, pf[t][n][0], pf[t][n][1]);
              }
            }
        }
      }
      slot = slot + 1 == S::kSlots ? 0 : slot + 1;
      __syncwarp();
      if constexpr (S::kSlots % 2) issue_v();
      else issue_k();
    }

    // ---- the piece's result
    done += cnt;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(kAll, l[n][e], x);
    if (whole) {
      TO *out = static_cast<TO *>(p.out) + (long long)at.b * p.out_tok + (long long)h0 * p.out_head;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < W / 16; ++k)
          if (16 * k < p.D)
            store_fragment<TO, ES>(out + 8 * n * p.out_head, p.out_head, k, heads - 8 * n, lane,
                                   make_float4(o[k][n][0], o[k][n][1], o[k][n][2], o[k][n][3]), l[n][0], l[n][1], p.v_scale);
        if (p.lse && g == 0) {
          float *lse = p.lse + (long long)at.b * p.nq + h0 + 8 * n + 2 * c;
          if (8 * n + 2 * c < heads) lse[0] = (mx[n][0] + log2f(l[n][0])) * kLn2;
          if (8 * n + 2 * c + 1 < heads) lse[1] = (mx[n][1] + log2f(l[n][1])) * kLn2;
        }
      }
    } else {
      float4 *ws = reinterpret_cast<float4 *>(p.ws_o), *ws_ml = reinterpret_cast<float4 *>(p.ws_ml);
      if (in_block) {   // one piece of the four
        __shared__ float4 sh_ml[kWarps][4 * NT];
        float4 *mine = reinterpret_cast<float4 *>(smem + warp * (S::kSlots * S::kUnit)) + lane;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < W / 16; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n) mine[(k * NT + n) * 32] = make_float4(o[k][n][0], o[k][n][1], o[k][n][2], o[k][n][3]);
        if (g == 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n) sh_ml[warp][4 * n + c] = make_float4(mx[n][0], l[n][0], mx[n][1], l[n][1]);
        }
        __syncthreads();
        const long long piece = 2ll * blockIdx.x * kWarps;
#pragma unroll 1
        for (int f = warp; f < p.D / 16 * NT; f += kWarps) {
          Joined j;
#pragma unroll
          for (int w = 0; w < kWarps; ++w)
            j.take(sh_ml[w][4 * (f % NT) + c], reinterpret_cast<const float4 *>(smem + w * (S::kSlots * S::kUnit))[f * 32 + lane]);
          ws[piece * (p.D / 16 * NT * 32) + f * 32 + lane] = j.acc;
          if (f < NT && g == 0) ws_ml[piece * (4 * NT) + 4 * f + c] = j.ml;
        }
      } else {
        // slot 0: a segment that came in from the worker before; slot 1: one that starts here
        const long long piece = 2ll * worker + (i0 == 0 ? 1 : 0);
#pragma unroll
        for (int k = 0; k < W / 16; ++k)
          if (16 * k < p.D) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
              ws[piece * (p.D / 16 * NT * 32) + (k * NT + n) * 32 + lane] = make_float4(o[k][n][0], o[k][n][1], o[k][n][2], o[k][n][3]);
          }
        if (g == 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n) ws_ml[piece * (4 * NT) + 4 * n + c] = make_float4(mx[n][0], l[n][0], mx[n][1], l[n][1]);
        }
      }
    }
    if (done == count) break;
    seg_first += at.sp.n + extra;
    at.i = at.sp.n - 1;
    at.next(p, segs);
  }
}

// Sums the pieces of one cut segment: segment blockIdx.x (by_segment), or the one that starts in
// worker blockIdx.x and goes on behind it. NOTED: which workers have its pieces is what the worker
// that starts it noted. Otherwise (few segments, by_segment) it follows from the lengths. They are
// read and numbered while the attention kernel still runs, then read again behind the wait for it,
// beside the pieces; only what is read there counts: where a length differs, all is done again.
// (Noted, calls of up to eight sequences took 0.3 to 1.7 us more, the check 0.3 at 997 tokens and
// nothing on longer ones; numbered here, 128 sequences of 4 KV heads took 4 us more and 1,024 short
// ones 12.) A thread takes one fragment of a piece (two heads at two elements: four values), of every
// par-th piece: the block's threads are par groups over the same threads / par fragments. Then the
// groups' sums are joined.
constexpr int kJoinMost = 512;   // threads
constexpr int kJoinPar = 16;     // groups
template <typename TO, int ES, bool NOTED>
__global__ void __launch_bounds__(kJoinMost) k_attn_join(const __grid_constant__ AttnParams p, int log, int all_workers, int nt, int par) {
  extern __shared__ __align__(16) float4 s_acc[];   // [threads] sums, [threads] (m, l): where par > 1
  float4 *s_ml = s_acc + blockDim.x;
  int w0, w1, b, h0, heads;   // heads: that exist from this column tile on
  const int tid = threadIdx.x, lane = tid & 31, per = blockDim.x / par, j0 = tid / per;   // per: a multiple of 32
  const int frags = p.D / 16 * nt * 32, f = blockIdx.y * per + (tid - j0 * per);
  const int k = f / (32 * nt), n = f / 32 - k * nt, c = lane & 3;
  const float4 *po = reinterpret_cast<const float4 *>(p.ws_o) + f, *pm = reinterpret_cast<const float4 *>(p.ws_ml) + (4 * n + c);
  auto rows_of = [&](int seg) {
    const int kvh = kv_head(p, seg);
    h0 = kvh * p.group + (seg - kvh * p.n_groups) * 8 * nt + 8 * n;
    heads = (kvh + 1) * p.group - h0;
  };
  Joined sum;
  auto take = [&](const Pieces &pieces) {
    if (f >= frags || w1 == w0) return;
    constexpr int kAhead = 4;
    for (int j = j0; j < pieces.count; j += kAhead * par) {
      float4 m[kAhead], v[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int i = min(j + x * par, pieces.count - 1);   // loads without a branch: all in flight together
        // piece 0: the starting worker's second slot; then the later workers' first slots
        const long long at = 2ll * pieces.worker(i) + (i == 0 ? 1 : 0);
        m[x] = pm[at * (4 * nt)];
        v[x] = po[at * frags];
      }
#pragma unroll
      for (int x = 0; x < kAhead; ++x)
        if (j + x * par < pieces.count) sum.take(m[x], v[x]);
    }
  };
  if constexpr (NOTED) {
    pdl_wait();
    const int4 cut = __ldcg(p.ws_cut + blockIdx.x);
    w0 = cut.x & 0xffff;
    w1 = cut.y;
    if (w1 == w0) return;   // nothing to join
    b = cut.z;
    rows_of(cut.w);
    take(Pieces(w0, w1, cut.x >> 16));
  } else {
    using Num = Numbering<true>;
    bool other;
    int turn = 0;
    do {
      const Num num(p, log, all_workers);   // its first strip has all sequences: segments are few
      b = blockIdx.x / num.segs;
      const int seg = blockIdx.x - b * num.segs;
      const typename Num::Segment s = num.segment(b, seg);
      w0 = w1 = 0;
      if (s.n) {
        w0 = num.split.owner(s.first + num.extra);
        w1 = num.split.owner(s.first + num.extra + s.n - 1);
      }
      rows_of(seg);
      Pieces pieces(w0, w1, num.extra);
      // worked out in front of the wait: the compiler would move some of it behind
      asm volatile("" : "+r"(pieces.w0), "+r"(pieces.head), "+r"(pieces.blocks), "+r"(pieces.tail), "+r"(pieces.count), "+l"(po), "+l"(pm),
                   "+r"(h0), "+r"(heads));
      pdl_wait();
      int now[Num::kOwn];
      Num::load(p, 0, now);
      sum = Joined();
      take(pieces);
      other = false;
#pragma unroll
      for (int j = 0; j < Num::kOwn; ++j) other |= now[j] != num.len[j];
    } while (__any_sync(Num::kAll, other) && ++turn < 2);   // the second time all is read behind the wait
    if (w1 == w0) return;   // nothing to join
  }
  // groups of up to four join at a time: 16 -> 4 -> 1
  for (int groups = par; groups > 1; groups = (groups + 3) / 4) {
    s_acc[tid] = sum.acc;
    s_ml[tid] = sum.ml;
    __syncthreads();
    const int keep = (groups + 3) / 4;
    if (j0 < keep) {
      for (int j = j0 + keep; j < groups; j += keep) sum.take(s_ml[tid + (j - j0) * per], s_acc[tid + (j - j0) * per]);
    }
    __syncthreads();
  }
  if (j0) return;
  if (f - lane >= frags) return;   // whole warps
  TO *out = static_cast<TO *>(p.out) + (long long)b * p.out_tok + (long long)h0 * p.out_head;
  store_fragment<TO, ES>(out, p.out_head, k, heads, lane, sum.acc, sum.ml.y, sum.ml.w, p.v_scale);
  if (p.lse && k == 0 && lane < 4) {
    float *lse = p.lse + (long long)b * p.nq + h0 + 2 * c;
    if (2 * c < heads) lse[0] = (sum.ml.x + log2f(sum.ml.y)) * kLn2;
    if (2 * c + 1 < heads) lse[1] = (sum.ml.z + log2f(sum.ml.w)) * kLn2;
  }
}

// static: what it keeps is this copy of the library's (a process may load several, each with its kernels)
template <typename T, int W, int NT, int ES, bool QB> static int launch(AttnParams p, int num_sms, cudaStream_t s) {
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
  if (grid * kWarps > MOE_ATTN_MAX_WORKERS) grid = MOE_ATTN_MAX_WORKERS / kWarps;
  const long long segments = (long long)p.B * p.nkv * p.n_groups;
  const int workers = grid * kWarps;
  p.by_segment = segments <= workers;   // a block of the join a segment, or one a worker
  // Threads that share a fragment in the join: as many as a quarter of the pieces that a segment
  // has when all are equally long and blocks join theirs, so that each one's loads are in flight
  // together
  int par = 1;
  while (par < kJoinPar && 4 * par * segments < grid) par *= 2;
  p.noted = par == 1;   // few segments: the join finds their workers itself
  PdlLaunch l(dim3(grid), kWarps * 32, S::kSmem, s);
  if (cudaLaunchKernelEx(&l.cfg, fn, p) != cudaSuccess) return -1;
  const int threads = par > 4 ? kJoinMost : kJoinMost / 2, frags = p.D / 16 * NT * 32, per = threads / par;
  PdlLaunch j(dim3(p.by_segment ? (unsigned)segments : workers, (frags + per - 1) / per), threads, par > 1 ? threads * 32 : 0, s);
  if (cudaLaunchKernelEx(&j.cfg, p.noted ? k_attn_join<TO, ES, true> : k_attn_join<TO, ES, false>, p, S::kLog, workers, NT, par) != cudaSuccess) return -1;
  moe_prof_count(2);
  return 0;
}

template <typename T, int ES, bool QB> static int dispatch(const AttnParams &p, int num_sms, cudaStream_t s) {
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
