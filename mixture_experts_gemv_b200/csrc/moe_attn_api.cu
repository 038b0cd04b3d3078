// moe_attn_api.cu -- the C entry points of the attention operators: argument checks, the device
// error word they share, and the launches.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <thread>

#include "moe_attn.cuh"
#include "moe_pages.cuh"

int moe_report_error(int code, const char *msg);   // moe_api.cu: sets moe_last_error()

namespace {

// Device error word of these operators: one per GPU, set by the first fault a kernel meets and
// kept until moe_cache_check reads it.
__device__ uint32_t g_cache_error;

// Takes the error word and clears it in one step: what is set behind it stays for the next check.
constexpr int kTaken = 32;   // checks at once
__device__ uint32_t g_cache_taken[kTaken];
__global__ void k_take_error(int slot) { g_cache_taken[slot] = atomicExch(&g_cache_error, 0u); }

struct Device {
  std::atomic<bool> ready{false};
  uint32_t *err = nullptr, *taken = nullptr;
  std::atomic<uint32_t> taking{0};   // slots of `taken` that checks hold
  int num_sms = 0;
};
constexpr int kMaxDevices = 64;
Device g_devices[kMaxDevices];
std::mutex g_device_setup;

int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char *fmt, ...) {
  char msg[384];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return moe_report_error(code, msg);
}

// The current device's record, set up on its first call.
int device(Device **out) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return fail(MOE_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  Device &d = g_devices[dev];
  if (!d.ready.load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(g_device_setup);
    if (!d.ready.load(std::memory_order_relaxed)) {
      int major = 0, minor = 0, sms = 0;
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
      if (major != 10 || minor != 0)
        return fail(MOE_ERR_UNSUPPORTED_DEVICE, "device %d is sm_%d%d; this library is built for sm_100a", dev, major, minor);
      void *p = nullptr;
      e = cudaGetSymbolAddress(&p, g_cache_error);
      if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "cudaGetSymbolAddress: %s", cudaGetErrorString(e));
      d.err = static_cast<uint32_t *>(p);
      e = cudaGetSymbolAddress(&p, g_cache_taken);
      if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "cudaGetSymbolAddress: %s", cudaGetErrorString(e));
      d.taken = static_cast<uint32_t *>(p);
      d.num_sms = sms;
      d.ready.store(true, std::memory_order_release);
    }
  }
  *out = &d;
  return MOE_OK;
}

bool mult16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int element_bytes(int dtype) { return dtype == MOE_DT_E4M3 ? 1 : 2; }

int check_head_dim(int D) {
  if (D < 16 || D > 512 || D % 16) return fail(MOE_ERR_BAD_ARG, "head_dim = %d must be a multiple of 16 in [16, 512]", D);
  return MOE_OK;
}

int check_cache(const moe_kv_cache *c, int layer, int dtype) {
  if (!c->k || !c->v) return fail(MOE_ERR_BAD_ARG, "null pointer in the cache");
  if (c->dtype != MOE_DT_BF16 && c->dtype != MOE_DT_F16 && c->dtype != MOE_DT_E4M3)
    return fail(MOE_ERR_BAD_ARG, "unknown cache dtype %d", c->dtype);
  if (dtype >= 0 && c->dtype != dtype && c->dtype != MOE_DT_E4M3)
    return fail(MOE_ERR_BAD_ARG, "cache dtype %d does not go with dtype %d", c->dtype, dtype);
  int rc = check_head_dim(c->head_dim);
  if (rc) return rc;
  if (c->n_layers < 1 || c->num_pages < 1 || c->page_size < 1 || c->n_kv < 1)
    return fail(MOE_ERR_BAD_ARG, "n_layers, num_pages, page_size and n_kv of the cache must be positive");
  if (layer < 0 || layer >= c->n_layers) return fail(MOE_ERR_BAD_ARG, "layer %d outside [0, %d)", layer, c->n_layers);
  const int es = element_bytes(c->dtype);
  if (c->layer_stride < 0 || c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0)
    return fail(MOE_ERR_BAD_ARG, "negative stride in the cache");
  if (!mult16(c->k) || !mult16(c->v) || c->layer_stride * es % 16 || c->page_stride * es % 16 ||
      c->token_stride * es % 16 || c->head_stride * es % 16)
    return fail(MOE_ERR_BAD_ALIGN, "the cache's bases and strides must be multiples of 16 bytes");
  // no two elements in one place: each dimension steps over the span of the smaller ones
  struct Dim { long long stride; long long n; } dims[] = {{c->layer_stride, c->n_layers}, {c->page_stride, c->num_pages},
                                                          {c->token_stride, c->page_size}, {c->head_stride, c->n_kv}};
  std::sort(dims, dims + 4, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
  long long span = c->head_dim;
  for (const Dim &d : dims) {
    if (d.n == 1) continue;
    if (d.stride < span) return fail(MOE_ERR_BAD_ARG, "the cache's strides overlap");
    span += (d.n - 1) * d.stride;
  }
  if (!std::isnormal(c->k_scale) || !std::isnormal(c->v_scale) || c->k_scale < 0 || c->v_scale < 0)   // 1 / scale is finite too
    return fail(MOE_ERR_BAD_ARG, "k_scale and v_scale must be positive, normal and finite");
  if (c->dtype != MOE_DT_E4M3 && (c->k_scale != 1.f || c->v_scale != 1.f))
    return fail(MOE_ERR_BAD_ARG, "k_scale and v_scale are for 8-bit caches: 1 otherwise");
  return MOE_OK;
}

int check_heads(const moe_heads *h, const char *name) {
  if (!h || !h->p) return fail(MOE_ERR_BAD_ARG, "%s: null pointer", name);
  if (h->token_stride < 0 || h->head_stride < 0) return fail(MOE_ERR_BAD_ARG, "%s: negative stride", name);
  if (!mult16(h->p) || h->token_stride % 8 || h->head_stride % 8)
    return fail(MOE_ERR_BAD_ALIGN, "%s: base and strides must be multiples of 16 bytes", name);
  return MOE_OK;
}

// An output's rows must lie apart (T tokens of n heads of D elements).
int check_apart(const moe_heads *h, const char *name, int T, int n, int D) {
  const long long a = std::min(h->token_stride, h->head_stride), b = std::max(h->token_stride, h->head_stride);
  const bool tokens_inner = h->token_stride < h->head_stride;
  const long long n_in = tokens_inner ? T : n, n_out = tokens_inner ? n : T;
  if ((n_in > 1 && a < D) || (n_out > 1 && b < (n_in > 1 ? (n_in - 1) * a + D : D)))
    return fail(MOE_ERR_BAD_ARG, "%s: rows overlap", name);
  return MOE_OK;
}

bool same(const moe_heads *a, const moe_heads *b) {
  return a->p == b->p && a->token_stride == b->token_stride && a->head_stride == b->head_stride;
}

// Whether rows of T tokens of nx and of ny heads (2-byte elements) share an address. Rows of unlike
// token strides, and more than 2^16 pairs of heads, count as sharing one where their extents do.
bool overlap(const moe_heads *x, int nx, const moe_heads *y, int ny, int T, int D) {
  const long long row = 2ll * D, hx = 2 * x->head_stride, hy = 2 * y->head_stride;   // bytes
  const long long wx = (nx - 1) * hx + row, wy = (ny - 1) * hy + row;                // a token's span
  const uintptr_t ax = reinterpret_cast<uintptr_t>(x->p), ay = reinterpret_cast<uintptr_t>(y->p);
  const uintptr_t bx = ax + 2 * (uintptr_t)(T - 1) * x->token_stride + wx, by = ay + 2 * (uintptr_t)(T - 1) * y->token_stride + wy;
  if (ax >= by || ay >= bx) return false;
  const long long step = T > 1 ? 2 * x->token_stride : 0, apart = (long long)(ay - ax);
  if (T > 1 && x->token_stride != y->token_stride) return true;
  if (step) {   // parts of the rows of one buffer: apart when the spans are, modulo a token
    const long long gap = (apart % step + step) % step;
    if (gap >= wx && gap + wy <= step) return false;
  }
  if ((long long)nx * ny > 1 << 16) return true;
  // heads between each other's heads: every pair, at the tokens that bring it closest
  for (int i = 0; i < nx; ++i)
    for (int j = 0; j < ny; ++j) {
      const long long d = apart + j * hy - i * hx;   // from x's row to y's, of one token
      const long long t = step ? std::min<long long>(std::max<long long>(-d / step, 1 - T), T - 1) : 0;
      for (long long u = std::max<long long>(t - 1, 1 - T); u <= std::min<long long>(t + 1, T - 1); ++u)
        if (std::llabs(d + u * step) < row) return true;
    }
  return false;
}

bool mult_of(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

extern "C" {

int moe_qk_norm_rope(const moe_heads *q, const moe_heads *k, const moe_heads *v, int dtype, int T, int n_q, int n_kv,
                     int head_dim, const int32_t *positions, const double *inv_freq, int rotary_dim, int interleaved,
                     float rope_scale, const float *q_gain, const float *k_gain, float eps, const moe_heads *q_out,
                     const moe_heads *k_out, const moe_kv_cache *cache, int layer, const int64_t *slots, void *stream) {
  if (dtype != MOE_DT_BF16 && dtype != MOE_DT_F16) return fail(MOE_ERR_BAD_ARG, "dtype %d is neither bf16 nor fp16", dtype);
  if (T < 0 || n_q < 0 || n_kv < 0 || n_q + n_kv == 0 || n_q > 4096 || n_kv > 4096)
    return fail(MOE_ERR_BAD_ARG, "bad shape T = %d, n_q = %d, n_kv = %d", T, n_q, n_kv);
  int rc = check_head_dim(head_dim);
  if (rc) return rc;
  if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % (interleaved ? 2 : 16))
    return fail(MOE_ERR_BAD_ARG, "rotary_dim = %d must be in [0, head_dim = %d], a multiple of 16 (of 2 when interleaved)",
                rotary_dim, head_dim);
  if (rotary_dim && (!positions || !inv_freq)) return fail(MOE_ERR_BAD_ARG, "null pointer argument");
  if (!std::isfinite(rope_scale) || !(eps >= 0) || !std::isfinite(eps))
    return fail(MOE_ERR_BAD_ARG, "rope_scale must be finite, eps finite and not negative");
  if (!mult_of(positions, 4) || !mult_of(inv_freq, 8) || !mult_of(slots, 8))
    return fail(MOE_ERR_BAD_ALIGN, "positions, inv_freq and slots must be aligned to their elements");
  if (!mult16(q_gain) || !mult16(k_gain)) return fail(MOE_ERR_BAD_ALIGN, "q_gain and k_gain must be 16-byte aligned");
  const int rows = T > 0 ? T : 1;
  if (n_q) {
    rc = check_heads(q, "q");
    if (!rc) rc = check_heads(q_out, "q_out");
    if (!rc) rc = check_apart(q_out, "q_out", rows, n_q, head_dim);
    if (rc) return rc;
  }
  if (n_kv) {
    rc = check_heads(k, "k");
    if (!rc && k_out) rc = check_heads(k_out, "k_out");
    if (!rc && k_out) rc = check_apart(k_out, "k_out", rows, n_kv, head_dim);
    if (rc) return rc;
    if (!k_out && !cache) return fail(MOE_ERR_BAD_ARG, "k goes nowhere: give k_out or a cache");
  } else {
    k_out = nullptr;
  }
  if (cache) {
    if (!n_kv) return fail(MOE_ERR_BAD_ARG, "a cache needs n_kv > 0");
    rc = check_heads(v, "v");
    if (!rc) rc = check_cache(cache, layer, dtype);
    if (rc) return rc;
    if (cache->n_kv != n_kv || cache->head_dim != head_dim)
      return fail(MOE_ERR_BAD_ARG, "the cache holds %d heads of %d, not %d of %d", cache->n_kv, cache->head_dim, n_kv, head_dim);
    if (!slots) return fail(MOE_ERR_BAD_ARG, "null pointer argument");
    if (cache->k == cache->v) return fail(MOE_ERR_BAD_ARG, "k and v of the cache are the same tensor");
  }
  // an output may be its own input and must not touch another
  const struct { const char *name; const moe_heads *h; int n; } ins[] = {
      {"q", n_q ? q : nullptr, n_q}, {"k", n_kv ? k : nullptr, n_kv}, {"v", cache ? v : nullptr, n_kv}};
  const struct { const char *name; const moe_heads *h; int n; } outs[] = {{"q_out", n_q ? q_out : nullptr, n_q}, {"k_out", k_out, n_kv}};
  for (int o = 0; o < 2; ++o) {
    if (!outs[o].h) continue;
    for (int i = 0; i < 3; ++i)
      if (ins[i].h && !(i == o && same(ins[i].h, outs[o].h)) && overlap(outs[o].h, outs[o].n, ins[i].h, ins[i].n, rows, head_dim))
        return fail(MOE_ERR_BAD_ARG, "%s overlaps %s", outs[o].name, ins[i].name);
  }
  if (outs[0].h && outs[1].h && overlap(outs[0].h, n_q, outs[1].h, n_kv, rows, head_dim))
    return fail(MOE_ERR_BAD_ARG, "q_out overlaps k_out");
  if (T == 0) return MOE_OK;
  Device *dev;
  rc = device(&dev);
  if (rc) return rc;
  RopeParams p{};
  if (n_q) {
    p.q = q->p, p.q_tok = q->token_stride, p.q_head = q->head_stride;
    p.q_out = q_out->p, p.qo_tok = q_out->token_stride, p.qo_head = q_out->head_stride;
  }
  if (n_kv) p.k = k->p, p.k_tok = k->token_stride, p.k_head = k->head_stride;
  if (k_out) p.k_out = k_out->p, p.ko_tok = k_out->token_stride, p.ko_head = k_out->head_stride;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.q_gain = q_gain;
  p.k_gain = k_gain;
  p.eps = eps;
  p.rope_scale = rope_scale;
  p.T = T;
  p.nq = n_q;
  p.nkv = n_kv;
  p.D = head_dim;
  p.rot = rotary_dim;
  p.inv_d = 1.f / (float)head_dim;
  bool f8 = false;
  if (cache) {
    const int es = element_bytes(cache->dtype);
    f8 = cache->dtype == MOE_DT_E4M3;
    p.v = v->p, p.v_tok = v->token_stride, p.v_head = v->head_stride;
    p.ck = static_cast<char *>(cache->k) + layer * cache->layer_stride * es;
    p.cv = static_cast<char *>(cache->v) + layer * cache->layer_stride * es;
    p.page_b = cache->page_stride * es;
    p.tok_b = cache->token_stride * es;
    p.head_b = cache->head_stride * es;
    p.n_slots = (long long)cache->num_pages * cache->page_size;
    p.page_size = cache->page_size;
    p.inv_k_scale = (float)(1.0 / cache->k_scale);
    p.inv_v_scale = (float)(1.0 / cache->v_scale);
    p.slots = slots;
  }
  p.err = dev->err;
  if (moe_launch_rope(p, dtype, interleaved != 0, f8, dev->num_sms, static_cast<cudaStream_t>(stream)))
    return fail(MOE_ERR_CUDA, "norm and rotation launch: %s", cudaGetErrorString(cudaGetLastError()));
  return MOE_OK;
}

int moe_rope_frequencies(int kind, int rotary_dim, double base, double factor, double original_length, double beta_fast,
                         double beta_slow, double *inv_freq, float *rope_scale) {
  if (kind < MOE_ROPE_PLAIN || kind > MOE_ROPE_YARN) return fail(MOE_ERR_BAD_ARG, "unknown kind of frequencies %d", kind);
  if (rotary_dim < 2 || rotary_dim > 512 || rotary_dim % 2) return fail(MOE_ERR_BAD_ARG, "rotary_dim = %d must be even, in [2, 512]", rotary_dim);
  if (!(base > 1) || !std::isfinite(base) || !(factor >= 1) || !std::isfinite(factor))
    return fail(MOE_ERR_BAD_ARG, "base must be above 1 and factor at least 1");
  if (!inv_freq || !rope_scale) return fail(MOE_ERR_BAD_ARG, "null pointer argument");
  const double pi = 3.14159265358979323846;
  if (kind == MOE_ROPE_NTK) {
    if (rotary_dim == 2) return fail(MOE_ERR_BAD_ARG, "a scaled base needs rotary_dim > 2");
    base *= std::pow(factor, rotary_dim / (rotary_dim - 2.0));
  }
  double first = 0, last = 0;
  if (kind == MOE_ROPE_YARN) {
    if (!(original_length >= 1) || !std::isfinite(original_length) || !(beta_slow > 0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast))
      return fail(MOE_ERR_BAD_ARG, "original_length >= 1 and beta_fast > beta_slow > 0 needed");
    // pair index at which a frequency makes `turns` turns in original_length tokens
    auto pair_of = [&](double turns) { return rotary_dim * std::log(original_length / (turns * 2 * pi)) / (2 * std::log(base)); };
    first = std::max(std::floor(pair_of(beta_fast)), 0.0);
    last = std::min(std::ceil(pair_of(beta_slow)), rotary_dim - 1.0);
    if (last <= first) last = first + 0.001;   // a step
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rotary_dim);
    double keep = 1;   // share of the frequency that is not interpolated
    if (kind == MOE_ROPE_LINEAR) keep = 0;
    if (kind == MOE_ROPE_YARN) keep = 1 - std::min(std::max((i - first) / (last - first), 0.0), 1.0);
    inv_freq[i] = f * (keep + (1 - keep) / factor);
  }
  *rope_scale = kind == MOE_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1) : 1.f;
  return MOE_OK;
}

// Layout of the workspace: partial sums, (maximum, sum) pairs, records of cut segments.
static size_t attn_rows(int n_q, int n_kv, int D) { return 8 * (size_t)moe_attn_tiles(D, n_q / n_kv); }
static size_t attn_o_bytes(size_t rows, int D) { return 2ull * MOE_ATTN_MAX_WORKERS * rows * D * 4; }
static size_t attn_ml_bytes(size_t rows) { return 2ull * MOE_ATTN_MAX_WORKERS * rows * 8; }

size_t moe_attention_decode_workspace_bytes(int n_q, int n_kv, int head_dim) {
  if (n_q < 1 || n_q > 4096 || n_kv < 1 || n_q % n_kv || head_dim < 16 || head_dim > 512 || head_dim % 16) return 0;
  const size_t rows = attn_rows(n_q, n_kv, head_dim);
  return attn_o_bytes(rows, head_dim) + attn_ml_bytes(rows) + MOE_ATTN_MAX_WORKERS * sizeof(int4);
}

int moe_attention_decode(const moe_heads *q, int dtype, const moe_kv_cache *cache, int layer, const int32_t *block_tables,
                         long long table_stride, int max_pages, const int32_t *seq_lens, int B, int n_q, float scale,
                         int window, const moe_heads *out, float *lse, void *workspace, size_t workspace_bytes,
                         void *stream) {
  if (dtype != MOE_DT_BF16 && dtype != MOE_DT_F16) return fail(MOE_ERR_BAD_ARG, "dtype %d is neither bf16 nor fp16", dtype);
  if (!cache || !block_tables || !seq_lens || !workspace) return fail(MOE_ERR_BAD_ARG, "null pointer argument");
  int rc = check_cache(cache, layer, dtype);
  if (!rc) rc = check_heads(q, "q");
  if (!rc) rc = check_heads(out, "out");
  if (rc) return rc;
  if (B < 0 || B > (1 << 30) || n_q < 1 || n_q % cache->n_kv || n_q > 4096)
    return fail(MOE_ERR_BAD_ARG, "bad shape B = %d, n_q = %d over n_kv = %d", B, n_q, cache->n_kv);
  if (max_pages < 1 || table_stride < max_pages || (long long)max_pages * cache->page_size > (1ll << 30))
    return fail(MOE_ERR_BAD_ARG, "max_pages = %d (rows %lld apart) of %d tokens: need 1 <= max_pages <= table_stride and at "
                                 "most 2^30 tokens", max_pages, table_stride, cache->page_size);
  if (window < 0) return fail(MOE_ERR_BAD_ARG, "window = %d < 0", window);
  const float scale_log2 = (float)((double)scale * cache->k_scale * 1.4426950408889634);
  if (!std::isfinite(scale_log2)) return fail(MOE_ERR_BAD_ARG, "scale (times k_scale, log2 e) must be finite");
  const int D = cache->head_dim, rows_b = B > 0 ? B : 1;
  rc = check_apart(out, "out", rows_b, n_q, D);
  if (rc) return rc;
  if (overlap(out, n_q, q, n_q, rows_b, D)) return fail(MOE_ERR_BAD_ARG, "out overlaps q");
  if (!mult_of(block_tables, 4) || !mult_of(seq_lens, 4) || !mult_of(lse, 4))
    return fail(MOE_ERR_BAD_ALIGN, "block_tables, seq_lens and lse must be aligned to their elements");
  if (!mult16(workspace)) return fail(MOE_ERR_BAD_ALIGN, "workspace must be 16-byte aligned");
  const size_t need = moe_attention_decode_workspace_bytes(n_q, cache->n_kv, D);
  if (workspace_bytes < need) return fail(MOE_ERR_BAD_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (B == 0) return MOE_OK;
  Device *dev;
  rc = device(&dev);
  if (rc) return rc;
  const int es = element_bytes(cache->dtype);
  const size_t rows = attn_rows(n_q, cache->n_kv, D);
  AttnParams p{};
  p.q = q->p, p.q_tok = q->token_stride, p.q_head = q->head_stride;
  p.k = static_cast<const char *>(cache->k) + layer * cache->layer_stride * es;
  p.v = static_cast<const char *>(cache->v) + layer * cache->layer_stride * es;
  p.page_b = cache->page_stride * es;
  p.tok_b = cache->token_stride * es;
  p.head_b = cache->head_stride * es;
  p.tables = block_tables;
  p.table_stride = table_stride;
  p.max_tokens = max_pages * cache->page_size;
  p.lens = seq_lens;
  p.B = B;
  p.nq = n_q;
  p.nkv = cache->n_kv;
  p.D = D;
  p.group = n_q / cache->n_kv;
  p.n_groups = (p.group + (int)rows - 1) / (int)rows;
  p.page_size = cache->page_size;
  p.page_shift = (cache->page_size & (cache->page_size - 1)) ? -1 : __builtin_ctz(cache->page_size);
  p.num_pages = cache->num_pages;
  p.window = window;
  p.groups_of_8 = cache->page_size % 8 == 0 && p.tok_b < (1ll << 28);   // row offsets within a group in 32 bits
  p.scale_log2 = scale_log2;
  p.v_scale = cache->v_scale;
  p.out = out->p, p.out_tok = out->token_stride, p.out_head = out->head_stride;
  p.lse = lse;
  char *ws = static_cast<char *>(workspace);
  p.ws_o = reinterpret_cast<float *>(ws);
  p.ws_ml = reinterpret_cast<float2 *>(ws + attn_o_bytes(rows, D));
  p.ws_cut = reinterpret_cast<int4 *>(ws + attn_o_bytes(rows, D) + attn_ml_bytes(rows));
  p.err = dev->err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = cache->dtype == MOE_DT_E4M3 ? moe_launch_attn_e4m3(p, dev->num_sms, dtype == MOE_DT_BF16, s)
       : dtype == MOE_DT_BF16      ? moe_launch_attn_bf16(p, dev->num_sms, s)
                                   : moe_launch_attn_f16(p, dev->num_sms, s);
  if (rc) return fail(MOE_ERR_CUDA, "attention launch: %s", cudaGetErrorString(cudaGetLastError()));
  return MOE_OK;
}

int moe_copy_pages(const moe_kv_cache *cache, const int32_t *src, const int32_t *dst, int n, int32_t *block_tables,
                   long long table_stride, int rows, int cols, void *stream) {
  if (!cache) return fail(MOE_ERR_BAD_ARG, "null pointer argument");
  int rc = check_cache(cache, 0, -1);
  if (rc) return rc;
  if (n < 0) return fail(MOE_ERR_BAD_ARG, "n = %d < 0", n);
  if (n && (!src || !dst)) return fail(MOE_ERR_BAD_ARG, "null pointer argument");
  if (!mult_of(block_tables, 4)) return fail(MOE_ERR_BAD_ALIGN, "block_tables must be aligned to its elements");
  if (block_tables && (rows < 0 || cols < 0 || table_stride < cols))
    return fail(MOE_ERR_BAD_ARG, "block tables of %d x %d, rows %lld apart", rows, cols, table_stride);
  if (n > cache->num_pages) return fail(MOE_ERR_BAD_ARG, "%d copies into %d pages: a page is in dst twice", n, cache->num_pages);
  if (n == 0) return MOE_OK;
  // marks: 1 source, 2 destination; pairs sorted by source for the table look-up
  char *mark = static_cast<char *>(calloc(cache->num_pages, 1));
  int2 *pairs = static_cast<int2 *>(malloc(n * sizeof(int2)));
  auto done = [&](int code) {
    free(mark);
    free(pairs);
    return code;
  };
  if (!mark || !pairs) return done(fail(MOE_ERR_BAD_ARG, "no host memory for a list of %d pages", n));
  bool sorted = true;
  for (int i = 0; i < n; ++i) {
    const int a = src[i], b = dst[i];
    if (a < 0 || a >= cache->num_pages || b < 0 || b >= cache->num_pages)
      return done(fail(MOE_ERR_BAD_ARG, "copy %d: page %d -> %d outside [0, %d)", i, a, b, cache->num_pages));
    if (block_tables && (mark[a] & 1)) return done(fail(MOE_ERR_BAD_ARG, "copy %d: page %d moves twice", i, a));
    if (mark[b] & 2) return done(fail(MOE_ERR_BAD_ARG, "copy %d: page %d is in dst twice", i, b));
    mark[a] |= 1;
    mark[b] |= 2;
    pairs[i] = make_int2(a, b);
    sorted = sorted && (i == 0 || pairs[i - 1].x <= a);
  }
  for (int i = 0; i < n; ++i)
    if (mark[src[i]] & 2) return done(fail(MOE_ERR_BAD_ARG, "page %d is both in src and in dst", src[i]));
  if (block_tables && !sorted) std::sort(pairs, pairs + n, [](const int2 &x, const int2 &y) { return x.x < y.x; });
  Device *dev;
  rc = device(&dev);
  if (rc) return done(rc);
  // the page as runs of contiguous bytes: the tighter of the two dimensions inside
  const long long es = element_bytes(cache->dtype);
  long long run = cache->head_dim * es;
  const bool heads_inner = cache->page_size == 1 || (cache->n_kv > 1 && cache->head_stride < cache->token_stride);
  long long in_b = (heads_inner ? cache->head_stride : cache->token_stride) * es, out_b = (heads_inner ? cache->token_stride : cache->head_stride) * es;
  int in_n = heads_inner ? cache->n_kv : cache->page_size, out_n = heads_inner ? cache->page_size : cache->n_kv;
  CopyParams p{};
  p.pieces = run / 16 * in_n * out_n;
  if (in_n == 1 || in_b == run) run *= in_n, in_n = 1;
  if (in_n == 1 && (out_n == 1 || out_b == run)) run *= out_n, out_n = 1;
  p.k = static_cast<char *>(cache->k);
  p.v = static_cast<char *>(cache->v);
  p.layers = cache->n_layers;
  p.layer_b = cache->layer_stride * es;
  p.page_b = cache->page_stride * es;
  p.outer_b = out_b;
  p.inner_b = in_b;
  p.inner = in_n;
  p.run_pieces = run / 16;
  if (block_tables && rows && cols) {
    p.tables = block_tables;
    p.table_stride = table_stride;
    p.rows = rows;
    p.cols = cols;
  }
  rc = moe_launch_copy_pages(p, pairs, n, static_cast<cudaStream_t>(stream));
  if (rc == -2) return done(fail(MOE_ERR_BAD_ARG, "%d pages in %d layers are too many for one launch", n, cache->n_layers));
  if (rc) return done(fail(MOE_ERR_CUDA, "page copy launch: %s", cudaGetErrorString(cudaGetLastError())));
  return done(MOE_OK);
}

int moe_cache_check(void *stream) {
  Device *dev;
  int rc = device(&dev);
  if (rc) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(s, &capture);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "moe_cache_check: %s", cudaGetErrorString(e));
  if (capture != cudaStreamCaptureStatusNone) return fail(MOE_ERR_BAD_ARG, "moe_cache_check waits for its stream: not while that is captured");
  int slot = -1;
  while (slot < 0) {   // a slot that no other thread's check holds
    uint32_t held = dev->taking.load(std::memory_order_relaxed);
    const int free_slot = ~held ? __builtin_ctz(~held) : -1;
    if (free_slot < 0) std::this_thread::yield();
    else if (dev->taking.compare_exchange_weak(held, held | 1u << free_slot, std::memory_order_acquire)) slot = free_slot;
  }
  uint32_t v = 0;
  k_take_error<<<1, 1, 0, s>>>(slot);
  e = cudaGetLastError();
  if (e == cudaSuccess) moe_prof_count(1);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&v, dev->taken + slot, sizeof v, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  dev->taking.fetch_and(~(1u << slot), std::memory_order_release);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "moe_cache_check: %s", cudaGetErrorString(e));
  switch (v & 0xffffu) {
    case 0: return MOE_OK;
    case MOE_DEV_ERR_BAD_PAGE: return fail(MOE_ERR_BAD_ARG, "a block-table entry inside a sequence was outside [0, num_pages)");
    case MOE_DEV_ERR_BAD_LENGTH: return fail(MOE_ERR_BAD_ARG, "a sequence length was negative or above max_pages * page_size");
    default: return fail(MOE_ERR_BAD_ARG, "a slot was past the cache's last row");
  }
}

}  // extern "C"
