// serve_api.cu -- the C ABI of the 8-bit integer linear layer and of the
// 4-bit key/value cache (include/q4.h): argument checks and launches.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "q4_internal.h"
#include "serve_internal.h"

using namespace q4;

namespace {
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool in16(int d) { return d == Q4_F16 || d == Q4_BF16; }
inline bool any_float(int d) { return d == Q4_F16 || d == Q4_BF16 || d == Q4_F32; }
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
constexpr int64_t kMaxRows = INT32_MAX;
// Of a product: a row number plus a tile or a grid's stride of rows stays within 32 bits.
constexpr int64_t kMaxLinearRows = Q4_INT8_MAX_ROWS;
constexpr int64_t kMaxKeys = (int64_t)1 << 30;  // of a sequence: positions and windows stay within 32 bits
constexpr int64_t kMaxQueries = (int64_t)1 << 30;  // rows in front of position 0, less a window, do too
constexpr int kDefaultSms = 148;  // sizes asked for without a device are those of a B200
int plan_sms() {
  const DeviceInfo di = device_info();
  return di.ok == Q4_OK ? di.sms : kDefaultSms;
}

int check_linear(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 1 || M > kMaxLinearRows || N > kMaxLinearRows || K > Q4_INT8_MAX_K) return Q4_ERR_SHAPE;
  return Q4_OK;
}

void set_gemv(I8GemvParams &v, int64_t M, const int8_t *W, int64_t ldw, const float *w_scale, int64_t N, int64_t K,
              const void *bias, int32_t bias_dtype, void *Y, int64_t ldy, int32_t y_dtype, int *status) {
  v.W = W, v.ldw = ldw, v.sw = w_scale;
  v.bias = bias, v.bias_dtype = bias_dtype;
  v.Y = Y, v.ldy = ldy, v.y_dtype = y_dtype;
  v.M = (int32_t)M, v.N = (int32_t)N, v.K = (int32_t)K;
  v.status = status;
}

int check_cache(const q4_kv_cache *c, KvView *v) {
  if (!c || !c->k_codes || !c->k_state || !c->v_codes || !c->v_state) return Q4_ERR_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128) || (c->blocksize != 64 && c->blocksize != 128) ||
      c->head_dim % c->blocksize)
    return Q4_ERR_ARG;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return Q4_ERR_ARG;
  if (c->kv_heads < 1 || c->kv_heads > 65535 || c->pages < 1 || c->pages > INT32_MAX) return Q4_ERR_SHAPE;
  if (!aligned16(c->k_codes) || !aligned16(c->k_state) || !aligned16(c->v_codes) || !aligned16(c->v_state))
    return Q4_ERR_ALIGN;
  v->codes[0] = c->k_codes, v->codes[1] = c->v_codes;
  v->state[0] = (uint32_t *)c->k_state, v->state[1] = (uint32_t *)c->v_state;
  v->slots = c->pages * c->page_size;
  v->heads = c->kv_heads;
  v->page_log2 = __builtin_ctz((unsigned)c->page_size);
  return Q4_OK;
}
}  // namespace

extern "C" {

int q4_int8_quantize_rows(const void *X, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ldx, int8_t *codes,
                          int64_t ldc, float *scale, void *stream) {
  if (!X || !codes || !scale || !in16(x_dtype)) return Q4_ERR_ARG;
  if (rows < 1 || cols < 1 || rows > kMaxRows || cols > Q4_INT8_MAX_K || ldx < cols || ldc < cols || ldc % 16)
    return Q4_ERR_SHAPE;
  if (!aligned16(codes)) return Q4_ERR_ALIGN;
  const DeviceInfo di = device_info();
  if (di.ok != Q4_OK) return di.ok;
  I8QuantParams p;
  p.X = (const uint16_t *)X;
  p.rows = rows, p.ldx = ldx, p.ldc = ldc, p.cols = (int32_t)cols;
  p.codes = codes;
  p.scale = scale;
  p.status = di.status;
  return run_int8_quantize(x_dtype, p, (cudaStream_t)stream);
}

int q4_int8_quantize_rows_f32(const float *X, int64_t rows, int64_t cols, int64_t ldx, int8_t *codes, int64_t ldc,
                              float *scale, void *stream) {
  if (!X || !codes || !scale) return Q4_ERR_ARG;
  if (rows < 1 || cols < 1 || rows > kMaxRows || cols > Q4_INT8_MAX_K || ldx < cols || ldc < cols || ldc % 16)
    return Q4_ERR_SHAPE;
  if (!aligned16(codes) || ((uintptr_t)X & 3u)) return Q4_ERR_ALIGN;
  const DeviceInfo di = device_info();
  if (di.ok != Q4_OK) return di.ok;
  I8QuantF32Params p;
  p.X = X;
  p.rows = rows, p.ldx = ldx, p.ldc = ldc, p.cols = (int32_t)cols;
  p.codes = codes;
  p.scale = scale;
  p.status = di.status;
  return run_int8_quantize_f32(p, (cudaStream_t)stream);
}

int q4_int8_gemm_workspace_size(int64_t M, int64_t N, int64_t K, size_t *bytes) {
  if (!bytes) return Q4_ERR_ARG;
  const int rc = check_linear(M, N, K);
  if (rc != Q4_OK) return rc;
  *bytes = 0;
  if (int8_gemv_ok(M, K)) return Q4_OK;
  const I8Plan pl = int8_plan(M, N, K, plan_sms());
  if (!pl.nt) return Q4_ERR_SHAPE;
  *bytes = pl.ws_bytes;
  return Q4_OK;
}

int q4_int8_gemm(const int8_t *A, int64_t lda, const float *a_scale, int64_t M, const int8_t *W, int64_t ldw,
                 const float *w_scale, int64_t N, int64_t K, const void *bias, int32_t bias_dtype, void *Y, int64_t ldy,
                 int32_t y_dtype, void *workspace, size_t workspace_bytes, void *stream) {
  if (!A || !a_scale || !W || !w_scale || !Y || !any_float(y_dtype) || (bias && !any_float(bias_dtype))) return Q4_ERR_ARG;
  int rc = check_linear(M, N, K);
  if (rc != Q4_OK) return rc;
  if (lda < K || ldw < K || ldy < N || lda % 16 || ldw % 16) return Q4_ERR_SHAPE;
  if (!aligned16(A) || !aligned16(W) || !aligned16(workspace)) return Q4_ERR_ALIGN;
  const DeviceInfo di = device_info();
  if (int8_gemv_ok(M, K)) {
    if (di.ok != Q4_OK) return di.ok;
    I8GemvParams v = {};
    v.A = A, v.lda = lda, v.sa = a_scale;
    set_gemv(v, M, W, ldw, w_scale, N, K, bias, bias_dtype, Y, ldy, y_dtype, di.status);
    return run_int8_gemv(0, v, di.sms, (cudaStream_t)stream);
  }
  const I8Plan pl = int8_plan(M, N, K, di.ok == Q4_OK ? di.sms : kDefaultSms);
  if (!pl.nt) return Q4_ERR_SHAPE;
  if (pl.ws_bytes && (!workspace || workspace_bytes < pl.ws_bytes)) return Q4_ERR_WORKSPACE;
  if (di.ok != Q4_OK) return di.ok;
  static thread_local I8GemmParams p;
  memset(&p, 0, sizeof(p));
  p.sa = a_scale, p.sw = w_scale;
  p.bias = bias, p.bias_dtype = bias_dtype;
  p.Y = Y, p.y_dtype = y_dtype, p.ldy = ldy;
  p.M = (int32_t)M, p.N = (int32_t)N;
  p.nk = (int32_t)((K + kI8Bk - 1) / kI8Bk);
  p.tiles_t = pl.tiles_t, p.tiles_n = pl.tiles_n;
  p.whole = pl.whole, p.cut_ctas = pl.cut_ctas;
  p.prefetch = M <= 64 ? 16 : 4;
  p.counts = (unsigned *)workspace;
  p.parts = (int32_t *)((char *)workspace + kI8CountBytes);
  p.stall_copies = g_copy_stall.load(std::memory_order_relaxed);
  p.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  p.status = di.status;
  const I8Operands o = {A, W, lda, ldw, M, N, K};
  return run_int8_gemm(o, pl, p, (cudaStream_t)stream);
}

int q4_int8_linear_scratch_size(int64_t M, int64_t K, size_t *bytes) {
  if (!bytes) return Q4_ERR_ARG;
  const int rc = check_linear(M, 1, K);
  if (rc != Q4_OK) return rc;
  *bytes = int8_gemv_ok(M, K) ? 0 : up256((size_t)M * 4) + (size_t)M * ((size_t)(K + 15) / 16 * 16);
  return Q4_OK;
}

int q4_int8_linear(const void *X, int32_t x_dtype, int64_t ldx, int64_t M, const int8_t *W, int64_t ldw,
                   const float *w_scale, int64_t N, int64_t K, const void *bias, int32_t bias_dtype, void *Y, int64_t ldy,
                   int32_t y_dtype, void *scratch, size_t scratch_bytes, void *workspace, size_t workspace_bytes,
                   void *stream) {
  if (!X || !W || !w_scale || !Y || !in16(x_dtype) || !any_float(y_dtype) || (bias && !any_float(bias_dtype)))
    return Q4_ERR_ARG;
  size_t head = 0, need = 0;
  int rc = q4_int8_gemm_workspace_size(M, N, K, &head);
  if (rc == Q4_OK) rc = q4_int8_linear_scratch_size(M, K, &need);
  if (rc != Q4_OK) return rc;
  if (ldx < K || ldw < K || ldw % 16 || ldy < N) return Q4_ERR_SHAPE;
  if (!aligned16(W) || !aligned16(workspace) || !aligned16(scratch)) return Q4_ERR_ALIGN;
  if ((need && (!scratch || scratch_bytes < need)) || (head && (!workspace || workspace_bytes < head))) return Q4_ERR_WORKSPACE;
  if (int8_gemv_ok(M, K)) {
    const DeviceInfo di = device_info();
    if (di.ok != Q4_OK) return di.ok;
    I8GemvParams v = {};
    v.X = (const uint16_t *)X, v.ldx = ldx;
    set_gemv(v, M, W, ldw, w_scale, N, K, bias, bias_dtype, Y, ldy, y_dtype, di.status);
    return run_int8_gemv(x_dtype, v, di.sms, (cudaStream_t)stream);
  }
  const int64_t ldc = (K + 15) / 16 * 16;
  float *scale = (float *)scratch;
  int8_t *codes = (int8_t *)scratch + up256((size_t)M * 4);
  rc = q4_int8_quantize_rows(X, x_dtype, M, K, ldx, codes, ldc, scale, stream);
  if (rc != Q4_OK) return rc;
  return q4_int8_gemm(codes, ldc, scale, M, W, ldw, w_scale, N, K, bias, bias_dtype, Y, ldy, y_dtype, workspace,
                      workspace_bytes, stream);
}

int q4_kv_append(const q4_kv_cache *cache, const void *K, const void *V, int32_t dtype, int64_t tokens,
                 int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                 const int64_t *slots, void *stream) {
  KvAppendParams p;
  if (!K || !V || !slots || !in16(dtype)) return Q4_ERR_ARG;
  const int rc = check_cache(cache, &p.c);
  if (rc != Q4_OK) return rc;
  if (tokens < 1 || tokens > kMaxRows || k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0)
    return Q4_ERR_SHAPE;
  if (!aligned16(K) || !aligned16(V) || k_token_stride % 8 || k_head_stride % 8 || v_token_stride % 8 || v_head_stride % 8)
    return Q4_ERR_ALIGN;
  const DeviceInfo di = device_info();
  if (di.ok != Q4_OK) return di.ok;
  p.x[0] = (const uint16_t *)K, p.x[1] = (const uint16_t *)V;
  p.ts[0] = k_token_stride, p.ts[1] = v_token_stride;
  p.hs[0] = k_head_stride, p.hs[1] = v_head_stride;
  p.slots = slots;
  p.tokens = tokens;
  p.status = di.status;
  return run_kv_append(dtype, cache->head_dim, cache->blocksize, p, di.sms, (cudaStream_t)stream);
}

int q4_kv_dequantize(const q4_kv_cache *cache, const int64_t *slots, int64_t n, void *K, void *V, int32_t dtype,
                     void *stream) {
  KvDequantParams p;
  if (!K || !V || !slots || !in16(dtype)) return Q4_ERR_ARG;
  const int rc = check_cache(cache, &p.c);
  if (rc != Q4_OK) return rc;
  if (n < 1 || n > kMaxRows) return Q4_ERR_SHAPE;
  if (!aligned16(K) || !aligned16(V)) return Q4_ERR_ALIGN;
  const DeviceInfo di = device_info();
  if (di.ok != Q4_OK) return di.ok;
  p.x[0] = (uint16_t *)K, p.x[1] = (uint16_t *)V;
  p.slots = slots;
  p.n = n;
  p.status = di.status;
  return run_kv_dequantize(dtype, cache->head_dim, cache->blocksize, p, di.sms, (cudaStream_t)stream);
}

int q4_kv_attention_workspace_size(const q4_kv_cache *cache, int64_t batch, int64_t total_q, int32_t q_heads,
                                   size_t *bytes) {
  KvView v;
  if (!bytes) return Q4_ERR_ARG;
  const int rc = check_cache(cache, &v);
  if (rc != Q4_OK) return rc;
  if (batch < 1 || batch > 65535 || total_q < 1 || total_q > kMaxQueries || q_heads < 1 || q_heads % v.heads) return Q4_ERR_SHAPE;
  *bytes = kv_attention_ws(cache->head_dim, plan_sms());
  return Q4_OK;
}

int q4_kv_attention(const q4_kv_cache *cache, const void *Q, int32_t dtype, int64_t total_q, int32_t q_heads,
                    int64_t q_token_stride, int64_t q_head_stride, const int32_t *cu_q, const int32_t *lens,
                    const int32_t *table, int64_t table_stride, int64_t table_pages, int64_t batch, int64_t max_q,
                    float scale, int32_t causal, int64_t window, void *out, float *lse, void *workspace,
                    size_t workspace_bytes, void *stream) {
  KvAttnParams p;
  if (!Q || !lens || !table || !out || !in16(dtype) || (causal != 0 && causal != 1) || !isfinite(scale)) return Q4_ERR_ARG;
  int rc = check_cache(cache, &p.c);
  if (rc != Q4_OK) return rc;
  size_t need = 0;
  rc = q4_kv_attention_workspace_size(cache, batch, total_q, q_heads, &need);
  if (rc != Q4_OK) return rc;
  if ((!cu_q && total_q != batch) || max_q < 1 || window < 0 || table_pages < 1 || table_pages > INT32_MAX || table_stride < table_pages ||
      table_pages * cache->page_size > kMaxKeys || q_token_stride < 0 || q_head_stride < 0)
    return Q4_ERR_SHAPE;
  if (!aligned16(Q) || !aligned16(out) || q_token_stride % 8 || q_head_stride % 8 || !aligned16(workspace)) return Q4_ERR_ALIGN;
  if (need && (!workspace || workspace_bytes < need)) return Q4_ERR_WORKSPACE;
  const DeviceInfo di = device_info();
  if (di.ok != Q4_OK) return di.ok;
  p.Q = (const uint16_t *)Q;
  p.q_ts = q_token_stride, p.q_hs = q_head_stride;
  p.cu_q = cu_q, p.lens = lens, p.table = table;
  p.table_stride = table_stride;
  p.table_pages = (int32_t)table_pages;
  p.batch = (int32_t)batch, p.total_q = (int32_t)total_q, p.q_heads = q_heads;
  p.scale = scale;
  p.causal = causal;
  // a window as long as the table holds every key (and far ones would overflow
  // the kernels' 32-bit positions)
  p.window = window >= table_pages * cache->page_size ? 0 : (int32_t)window;
  p.out = (uint16_t *)out;
  p.lse = lse;
  p.counts = (unsigned *)workspace;
  p.parts = (float *)((char *)workspace + kKvCountBytes);
  p.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  p.sms = di.sms;
  p.stall_copies = g_copy_stall.load(std::memory_order_relaxed);
  p.status = di.status;
  return run_kv_attention(dtype, cache->head_dim, cache->blocksize, p, std::min(max_q, total_q), di.sms,
                          (cudaStream_t)stream);
}

}  // extern "C"
