// serve_internal.h -- launcher entry points of the 8-bit integer and
// key/value-cache kernels (not part of the public C ABI).
#pragma once
#include "int8_gemm.cuh"
#include "int8_gemv.cuh"
#include "int8_quantize.cuh"
#include "kv_attention.cuh"
#include "kv_cache.cuh"
#include "kv_prompt.cuh"

namespace q4 {
struct I8Operands {
  const int8_t *A, *W;
  int64_t lda, ldw, M, N, K;
};
// How a product runs on a device of `sms` SMs (see int8_gemm.cuh).
struct I8Plan {
  int nt = 0;        // tokens per tile (0: too large)
  bool pair = false; // 256-row tiles shared by two CTAs
  int tiles_t = 0, tiles_n = 0, whole = 0, cut_ctas = 0, grid = 0;
  int slots = 0;     // cut tiles
  size_t ws_bytes = 0;
};
I8Plan int8_plan(int64_t M, int64_t N, int64_t K, int sms);
int run_int8_quantize(int dt, const I8QuantParams &p, cudaStream_t st);
int run_int8_quantize_f32(const I8QuantF32Params &p, cudaStream_t st);
// Whether M tokens of K take the one-launch kernel of int8_gemv.cuh.
bool int8_gemv_ok(int64_t M, int64_t K);
int run_int8_gemv(int x_dtype, const I8GemvParams &p, int sms, cudaStream_t st);
int run_int8_gemm(const I8Operands &o, const I8Plan &pl, I8GemmParams &p, cudaStream_t st);
int run_kv_append(int dt, int D, int B, const KvAppendParams &p, int sms, cudaStream_t st);
int run_kv_dequantize(int dt, int D, int B, const KvDequantParams &p, int sms, cudaStream_t st);
int run_kv_attention(int dt, int D, int B, const KvAttnParams &p, int64_t max_q, int sms, cudaStream_t st);
// Workspace of the attention on a device of `sms` SMs.
size_t kv_attention_ws(int D, int sms);
}  // namespace q4
