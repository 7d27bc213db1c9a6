// int8_gemm.cuh -- Y[M, N] = sa[m] sw[n] sum_k A[m, k] W[n, k] + bias[n] with
// 8-bit integer operands and 32-bit integer sums (sm_100a).
#pragma once
#include "q4_common.cuh"

namespace q4 {

struct I8GemmParams {
  const int8_t *A, *W;
  int64_t lda, ldw, ldy;
  const float *sa, *sw;
  const void *bias;
  void *Y;
  int64_t M, N, K;
  int32_t bias_dtype, y_dtype;
  int *status;
};

__device__ __forceinline__ float i8_bias(const void *bias, int dt, int64_t n) {
  if (!bias) return 0.0f;
  if (dt == Q4_F32) return __ldg(reinterpret_cast<const float *>(bias) + n);
  const uint16_t b = __ldg(reinterpret_cast<const uint16_t *>(bias) + n);
  return dt == Q4_BF16 ? Dt<Q4_BF16>::to_f(b) : Dt<Q4_F16>::to_f(b);
}
__device__ __forceinline__ void i8_store(void *Y, int dt, int64_t at, float y) {
  if (dt == Q4_F32) reinterpret_cast<float *>(Y)[at] = y;
  else reinterpret_cast<uint16_t *>(Y)[at] = dt == Q4_BF16 ? Dt<Q4_BF16>::from_f(y) : Dt<Q4_F16>::from_f(y);
}

// 64 x 64 outputs a CTA, 4 x 4 a thread, dot products of four bytes.
static __global__ void __launch_bounds__(256) int8_gemm_kernel(const __grid_constant__ I8GemmParams p) {
  pdl_launch_then_wait();
  __shared__ int sA[64][17], sW[64][17];  // 64 bytes of k a row, as words
  const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int64_t k0 = 0; k0 < p.K; k0 += 64) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
      const int r = i >> 4, w = i & 15;
      const int64_t k = k0 + 4 * w;
      int a = 0, b = 0;
      for (int j = 0; j < 4; ++j) {
        if (k + j < p.K && m0 + r < p.M) a |= (int)(uint8_t)p.A[(m0 + r) * p.lda + k + j] << (8 * j);
        if (k + j < p.K && n0 + r < p.N) b |= (int)(uint8_t)p.W[(n0 + r) * p.ldw + k + j] << (8 * j);
      }
      sA[r][w] = a;
      sW[r][w] = b;
    }
    __syncthreads();
    for (int w = 0; w < 16; ++w)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(sA[ty + 16 * i][w], sW[tx + 16 * j][w], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < p.M && n < p.N) {
        const float y = __fmul_rn((float)acc[i][j], __fmul_rn(__ldg(p.sa + m), __ldg(p.sw + n)));
        i8_store(p.Y, p.y_dtype, m * p.ldy + n, p.bias ? __fadd_rn(y, i8_bias(p.bias, p.bias_dtype, n)) : y);
      }
    }
}

}  // namespace q4
