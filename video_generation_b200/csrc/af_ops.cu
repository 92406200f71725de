// af_ops.cu -- the entry points of the attention-layer operators that take no
// model (include/af.h): argument checks, workspace and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>

#include <atomic>

#include "../../include/af.h"
#include "af_cache4.cuh"
#include "af_kernels.h"

namespace af {
void set_error_text(const char* msg);
}

using namespace af;

// What is wrong with a rotary description; null: nothing.
const char* af::rope_fault(const af_rope* r) {
  const int D = r->head_dim;
  if (D != 16 && D != 32 && D != 64 && D != 128 && D != 256) return "head_dim must be 16, 32, 64, 128 or 256";
  int total = 0;
  for (int a = 0; a < 3; ++a) {
    if (r->pairs[a] < 0 || r->pairs[a] > D / 2) return "pairs of an axis must be 0 .. head_dim / 2";
    total += r->pairs[a];
  }
  if (total > D / 2) return "more pairs than head_dim / 2";
  if (!(r->theta >= 1.0) || !isfinite(r->theta) || !(r->eps > 0.f) || !isfinite(r->eps)) return "need finite theta >= 1 and eps > 0";
  if (r->layout != AF_ROPE_PAIRS && r->layout != AF_ROPE_HALVES) return "bad layout";
  return nullptr;
}

namespace {

af_status bad(const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  set_error_text(msg);
  return AF_ERR_ARG;
}

af_status launched(const char* what, cudaError_t e) {
  if (e == cudaSuccess) return AF_OK;
  cudaGetLastError();
  char msg[400];
  snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
  set_error_text(msg);
  return AF_ERR_CUDA;
}

// The current device, after checking that the stream belongs to it (the last
// check of a call: those before it need no device).
af_status op_device(const char* what, cudaStream_t st, int* dev) {
  if (cudaGetDevice(dev) != cudaSuccess) {
    cudaGetLastError();
    set_error_text("no current CUDA device");
    return AF_ERR_CUDA;
  }
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (st && cudaStreamIsCapturing(st, &cap) != cudaSuccess) {
    cudaGetLastError();
    return bad("%s: the stream is not a valid CUDA stream, or its capture has failed", what);
  }
  if (st && cap == cudaStreamCaptureStatusNone) {  // asking a capturing stream for its device ends the capture
    int sdev = -1;
    if (cudaStreamGetDevice(st, &sdev) != cudaSuccess) {
      cudaGetLastError();
      return bad("%s: the stream is not a valid CUDA stream", what);
    }
    if (sdev != *dev) return bad("%s: the stream belongs to device %d but device %d is current", what, sdev, *dev);
  }
  static const int pdl = [] { const char* v = getenv("AF_PDL"); return v ? (atoi(v) != 0) : 1; }();
  g_pdl = pdl;
  return AF_OK;
}

int sms_of(int dev) {
  static int sms[64] = {};
  if (dev < 0 || dev >= 64) return 148;
  if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 148;
  }
  return sms[dev];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// rows that are read: 16-byte aligned (a stride of 0 reads one row again and again)
bool in_stride(int64_t stride, int size) { return stride >= 0 && (stride * size) % 16 == 0; }
// rows of n elements that are written: also apart when there are several
bool out_stride(int64_t stride, int64_t n, int size, int64_t rows) {
  return in_stride(stride, size) && (rows <= 1 || stride >= n);
}
constexpr int kMaxRows = 1 << 30;

bool good_cache(const af_cache_config* c) {
  return c && c->batch >= 0 && c->kv_heads >= 1 && c->capacity >= 1 && c->capacity <= kMaxRows && (c->head_dim == 64 || c->head_dim == 128) &&
         (int64_t)c->batch * c->kv_heads <= (1 << 24);
}
af_status check_cache(const char* what, const af_cache_config* c, const void* cache) {
  if (!good_cache(c))
    return bad("%s: cache config needs batch >= 0, kv_heads >= 1, 1 <= capacity <= 2^30, head_dim 64 or 128, batch * kv_heads <= 2^24", what);
  if (!cache || (reinterpret_cast<uintptr_t>(cache) & 255u)) return bad("%s: the cache is null or not 256-byte aligned", what);
  return AF_OK;
}
Cache4 at(const af_cache_config* c, const void* cache) {
  return cache4_at(cache, c->batch, c->kv_heads, c->head_dim, c->capacity);
}

std::atomic<uint64_t> g_wait_ns{2000000000ull};   // limit of a pipeline wait of the calls here

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Splits and workspace of an attention call.
struct AttnPlan {
  bool tc;
  int nsplit, even;
  size_t opart, ml;   // bytes
};
AttnPlan attn_plan(const af_cache_config* c, int heads, int rows, int sms) {
  AttnPlan p{};
  const int group = heads / c->kv_heads;
  p.tc = attn4_use_tc(c->batch, c->kv_heads, group, rows, c->capacity, c->head_dim, sms);
  p.nsplit = p.tc ? attn4_tc_splits(c->batch, c->kv_heads, group, rows, c->capacity, sms)
                  : attn4_small_splits(c->batch, c->kv_heads, group, rows, c->capacity, sms, &p.even);
  if (p.nsplit > 1) {
    const size_t n = (size_t)p.nsplit * c->batch * heads * rows;
    p.opart = align256(n * c->head_dim * sizeof(float));
    p.ml = align256(n * 2 * sizeof(float));
  }
  return p;
}
bool good_heads(const af_cache_config* c, int heads, int rows) {
  return rows >= 0 && heads >= 1 && heads % c->kv_heads == 0 && (int64_t)rows * (heads / c->kv_heads) <= (1 << 20);
}

}  // namespace

extern "C" {

af_status af_qk_norm_rope(const af_rope* rope, af_dtype dtype, int rows, const void* q, int64_t q_stride, int heads,
                          const void* k, int64_t k_stride, int kv_heads, const float* q_gain, const float* k_gain,
                          const int32_t* pos, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                          void* stream) {
  const char* what = "af_qk_norm_rope";
  if (!rope) return bad("%s: null rope", what);
  if (const char* why = rope_fault(rope)) return bad("%s: %s", what, why);
  const int D = rope->head_dim;
  if (dtype != AF_FP32 && dtype != AF_BF16) return bad("%s: bad dtype", what);
  if (rows < 0 || rows > kMaxRows || heads < 0 || kv_heads < 0 || heads > 65536 || kv_heads > 65536)
    return bad("%s: need 0..2^30 rows and 0..65536 heads", what);
  if (rows == 0 || heads + kv_heads == 0) return AF_OK;
  const int size = dtype == AF_FP32 ? 4 : 2;
  if (!pos) return bad("%s: null pos", what);
  if (heads && (!q || !q_out || !aligned16(q) || !aligned16(q_out) || !in_stride(q_stride, size) ||
                !out_stride(q_out_stride, (int64_t)heads * D, size, rows)))
    return bad("%s: q and q_out must be 16-byte aligned, with 16-byte aligned rows that do not overlap", what);
  if (kv_heads && (!k || !k_out || !aligned16(k) || !aligned16(k_out) ||
                   !in_stride(k_stride, size) ||
                   !out_stride(k_out_stride, (int64_t)kv_heads * D, size, rows)))
    return bad("%s: k and k_out must be 16-byte aligned, with 16-byte aligned rows that do not overlap", what);
  if ((heads && q == q_out && q_stride != q_out_stride && rows > 1) ||
      (kv_heads && k == k_out && k_stride != k_out_stride && rows > 1))
    return bad("%s: an output in its input's place needs its stride", what);
  cudaStream_t st = (cudaStream_t)stream;
  int dev = 0;
  if (af_status s = op_device(what, st, &dev)) return s;
  QkArgs a{};
  a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
  a.q_rs = q_stride; a.k_rs = k_stride; a.qo_rs = q_out_stride; a.ko_rs = k_out_stride;
  a.rows = rows;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.pos = pos;
  a.eps = rope->eps;
  rope_tables(rope->pairs, rope->theta, &a);
  return launched(what, launch_qk_norm_rope(a, dtype == AF_FP32, D, rope->layout == AF_ROPE_HALVES, sms_of(dev), st));
}

size_t af_cache_bytes(const af_cache_config* cfg) {
  if (!good_cache(cfg)) return 0;
  return cache4_bytes(cfg->batch, cfg->kv_heads, cfg->head_dim, cfg->capacity);
}

af_status af_cache_write(const af_cache_config* cfg, void* cache, int rows, const void* k, int64_t k_batch_stride,
                         int64_t k_row_stride, const void* v, int64_t v_batch_stride, int64_t v_row_stride,
                         const int32_t* start, const int32_t* count, void* stream) {
  const char* what = "af_cache_write";
  if (af_status s = check_cache(what, cfg, cache)) return s;
  if (rows < 0 || rows > kMaxRows) return bad("%s: need 0..2^30 rows", what);
  if (rows == 0 || cfg->batch == 0) return AF_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v) || !in_stride(k_row_stride, 2) || !in_stride(k_batch_stride, 2) ||
      !in_stride(v_row_stride, 2) || !in_stride(v_batch_stride, 2))
    return bad("%s: k and v must be 16-byte aligned with 16-byte aligned rows", what);
  cudaStream_t st = (cudaStream_t)stream;
  int dev = 0;
  if (af_status s = op_device(what, st, &dev)) return s;
  Cache4W a{};
  a.c = at(cfg, cache);
  a.k = (const bf16*)k;
  a.v = (const bf16*)v;
  a.k_bs = k_batch_stride; a.k_rs = k_row_stride; a.v_bs = v_batch_stride; a.v_rs = v_row_stride;
  a.rows = rows;
  a.start = start;
  a.count = count;
  return launched(what, launch_cache4_write(a, st));
}

af_status af_cache_read(const af_cache_config* cfg, const void* cache, int rows, const int32_t* start,
                        const int32_t* count, af_dtype dtype, void* k, void* v, int64_t batch_stride,
                        int64_t row_stride, void* stream) {
  const char* what = "af_cache_read";
  if (af_status s = check_cache(what, cfg, cache)) return s;
  if (rows < 0 || rows > kMaxRows || (dtype != AF_FP32 && dtype != AF_BF16))
    return bad("%s: need 0..2^30 rows, dtype AF_FP32 or AF_BF16", what);
  if (rows == 0 || cfg->batch == 0) return AF_OK;
  const int64_t n = (int64_t)cfg->kv_heads * cfg->head_dim;
  const int size = dtype == AF_FP32 ? 4 : 2;
  if (!k || !v || k == v || !aligned16(k) || !aligned16(v) || !out_stride(row_stride, n, size, rows) ||
      !out_stride(batch_stride, n, size, cfg->batch))
    return bad("%s: k and v must be two buffers, 16-byte aligned, with 16-byte aligned rows that do not overlap", what);
  cudaStream_t st = (cudaStream_t)stream;
  int dev = 0;
  if (af_status s = op_device(what, st, &dev)) return s;
  Cache4R a{};
  a.c = at(cfg, cache);
  a.k = k;
  a.v = v;
  a.bs = batch_stride;
  a.rs = row_stride;
  a.rows = rows;
  a.start = start;
  a.count = count;
  return launched(what, launch_cache4_read(a, dtype == AF_FP32, st));
}

size_t af_cache_attention_workspace_bytes(const af_cache_config* cfg, int heads, int rows) {
  if (!good_cache(cfg) || !good_heads(cfg, heads, rows)) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = -1;
  }
  if (cfg->batch == 0 || rows == 0) return 256;
  const AttnPlan p = attn_plan(cfg, heads, rows, sms_of(dev));
  return 256 + p.opart + p.ml;
}

af_status af_cache_attention(const af_cache_config* cfg, const void* cache, int rows, int heads, const void* q,
                             int64_t q_batch_stride, int64_t q_row_stride, const int32_t* length, const int32_t* n_q,
                             int causal, float scale, void* out, int64_t out_batch_stride, int64_t out_row_stride,
                             void* ws, size_t ws_bytes, void* stream) {
  const char* what = "af_cache_attention";
  if (af_status s = check_cache(what, cfg, cache)) return s;
  if (!good_heads(cfg, heads, rows))
    return bad("%s: need heads a multiple of kv_heads, and 0 <= rows * heads / kv_heads <= 2^20", what);
  const float scale_log2 = (float)(scale * 1.4426950408889634);   // scores in units of log2
  if (!(scale > 0.f) || !isfinite(scale_log2)) return bad("%s: scale must be positive and at most 2^127", what);
  if (rows == 0 || cfg->batch == 0) return AF_OK;
  const int64_t n = (int64_t)heads * cfg->head_dim;
  if (!q || !aligned16(q) || !in_stride(q_row_stride, 2) || !in_stride(q_batch_stride, 2))
    return bad("%s: q must be 16-byte aligned with 16-byte aligned rows", what);
  if (!out || out == q || !aligned16(out) || !out_stride(out_row_stride, n, 2, rows) ||
      !out_stride(out_batch_stride, n, 2, cfg->batch))
    return bad("%s: out must be 16-byte aligned, not q, with 16-byte aligned rows that do not overlap", what);
  if (!length) return bad("%s: null length", what);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u)) {
    bad("%s workspace: null or not 256-byte aligned (%p)", what, ws);
    return AF_ERR_WORKSPACE;
  }
  cudaStream_t st = (cudaStream_t)stream;
  int dev = 0;
  if (af_status s = op_device(what, st, &dev)) return s;
  const AttnPlan p = attn_plan(cfg, heads, rows, sms_of(dev));
  const size_t need = 256 + p.opart + p.ml;
  if (ws_bytes < need) {
    bad("%s workspace: need %zu bytes, got %zu", what, need, ws_bytes);
    return AF_ERR_WORKSPACE;
  }
  Attn4Args a{};
  a.c = at(cfg, cache);
  a.q = (const bf16*)q;
  a.o = (bf16*)out;
  a.q_bs = q_batch_stride; a.q_rs = q_row_stride; a.o_bs = out_batch_stride; a.o_rs = out_row_stride;
  a.heads = heads;
  a.rows = rows;
  a.causal = causal != 0;
  a.len = length;
  a.nq = n_q;
  a.scale_log2 = scale_log2;
  a.nsplit = p.nsplit;
  a.even = p.even;
  a.opart = (float*)((char*)ws + 256);
  a.ml = (float*)((char*)ws + 256 + p.opart);
  a.wait_ns = g_wait_ns.load();
  return launched(what, p.tc ? launch_attn4_tc(a, nullptr, st) : launch_attn4_small(a, st));
}

af_status af_operator_wait_limit(double seconds) {
  if (!(seconds > 0.0) || seconds > 60.0) return bad("af_operator_wait_limit: need 0 < seconds <= 60");
  const uint64_t ns = (uint64_t)(seconds * 1e9);
  g_wait_ns = ns < 1 ? 1 : ns;
  return AF_OK;
}

af_status af_operator_error(int* code) {
  int v = 0;
  if (af_status s = launched("af_operator_error", ops_error(&v))) return s;
  if (code) *code = v;
  if (!v) return AF_OK;
  bad("device error code %d", v);
  return AF_ERR_DEVICE;
}

}  // extern "C"
