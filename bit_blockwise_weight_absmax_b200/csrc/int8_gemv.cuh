// int8_gemv.cuh -- the 8-bit integer linear layer for up to four tokens
// (decode), in one launch: each CTA quantizes the tokens itself, each warp
// streams whole weight rows (sm_100a).
//
// Bound by the weights' N K bytes, and by latency where those are few.  A
// lane's first loads of its row (4 KB a warp) are issued before the wait for
// the tokens' maximum, so the quantization (every CTA repeats it: 2 M K bytes
// from L2) hides behind the weights' way from memory.  Sums are dot products
// of four bytes (dp4a) in 32-bit integers, joined over the warp by shuffles:
// no partial tile, no workspace, one launch instead of two.  One token: 4096 x
// 4096 6.4 us (2.6 TB/s), 28672 x 8192 39 us (6.0 TB/s).
// More tokens than four are better on the tensor cores (int8_gemm.cuh): the
// dot products and the tokens' shared-memory reads grow with them.
#pragma once
#include "int8_gemm.cuh"
#include "int8_quantize.cuh"

namespace q4 {

struct I8GemvParams {
  const uint16_t *X;     // 16-bit tokens (FUSED)
  const int8_t *A;       // or their codes
  const float *sa;       // and scales
  const int8_t *W;
  const float *sw;
  const void *bias;
  void *Y;
  int64_t ldx, lda, ldw, ldy;
  int32_t M, N, K;
  int32_t bias_dtype, y_dtype;
  int *status;
};

constexpr int kI8vThreads = 256;
constexpr int kI8vMaxTokens = 4;
constexpr int kI8vMaxBytes = 48 * 1024;  // token codes a CTA holds
constexpr int kI8vDepth = 8;             // 16-byte loads in flight a lane

// CTAs an SM: more tokens need more registers before the loop.
constexpr int i8v_ctas(int mt) { return mt == 1 ? 4 : mt == 2 ? 3 : 2; }

// MT tokens (M of them exist).  DT < 0: the tokens come as codes.
template <int MT, int DT, bool VEC>
__global__ void __launch_bounds__(kI8vThreads, i8v_ctas(MT)) int8_gemv_kernel(const __grid_constant__ I8GemvParams p) {
  pdl_launch_dependents();
  extern __shared__ __align__(16) uint8_t s_codes[];  // [MT][ceil16(K)]
  __shared__ uint32_t s_max[MT][kI8vThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int K = p.K, chunks = (K + 15) / 16;
  pdl_wait();
  // this warp's rows: w, w + all warps, ...; the first loads of the first row
  const int stride = gridDim.x * (kI8vThreads / 32);
  int n = blockIdx.x * (kI8vThreads / 32) + warp;
  uint4 wv[kI8vDepth];
  auto load_row = [&](int row, int first) {
    const uint4 *w = reinterpret_cast<const uint4 *>(p.W + (int64_t)row * p.ldw);
#pragma unroll
    for (int d = 0; d < kI8vDepth; ++d) {
      const int i = first + d * 32 + lane;
      wv[d] = i < chunks ? ldg_stream_v4(w + i) : make_uint4(0, 0, 0, 0);
    }
  };
  if (n < p.N) load_row(n, 0);
  float sa[MT];
  if constexpr (DT >= 0) {
    // the tokens' maxima, then their codes (as int8_quantize_kernel)
    const int pieces = 2 * chunks;  // 8 elements each, zeros past K
    auto load = [&](int m, int i) -> uint4 {
      const uint16_t *x = p.X + m * p.ldx;
      if (VEC && 8 * i + 8 <= K) return __ldcg(reinterpret_cast<const uint4 *>(x) + i);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 8 * i + 2 * j;
        const uint32_t lo = e < K ? __ldcg(x + e) : 0u, hi = e + 1 < K ? __ldcg(x + e + 1) : 0u;
        w[j] = lo | (hi << 16);
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    };
    uint4 keep[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t m2 = 0;
      if (m < p.M) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = tid + k * kI8vThreads;
          keep[m][k] = i < pieces ? load(m, i) : make_uint4(0, 0, 0, 0);
          m2 = __vmaxu2(m2, i8_top8(keep[m][k]));
        }
        for (int i = tid + 2 * kI8vThreads; i < pieces; i += kI8vThreads) m2 = __vmaxu2(m2, i8_top8(load(m, i)));
      }
      const uint32_t t = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
      if (lane == 0) s_max[m][warp] = t;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t t = 0;
#pragma unroll
      for (int j = 0; j < kI8vThreads / 32; ++j) t = max(t, s_max[m][j]);
      const I8Scale sc = i8_scale(Dt<DT>::to_f((uint16_t)t));
      sa[m] = sc.stored;
      if (m >= p.M) continue;
      uint2 *c = reinterpret_cast<uint2 *>(s_codes + m * chunks * 16);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = tid + k * kI8vThreads;
        if (i < pieces) c[i] = i8_codes8<DT>(keep[m][k], sc);
      }
      for (int i = tid + 2 * kI8vThreads; i < pieces; i += kI8vThreads) c[i] = i8_codes8<DT>(load(m, i), sc);
      if (sc.bad && blockIdx.x == 0 && tid == 0) raise_status(p.status, Q4_STATUS_NONFINITE);
    }
  } else {
    for (int m = 0; m < p.M; ++m) {
      const uint4 *a = reinterpret_cast<const uint4 *>(p.A + m * p.lda);
      uint4 *c = reinterpret_cast<uint4 *>(s_codes + m * chunks * 16);
      for (int i = tid; i < chunks; i += kI8vThreads) {
        uint4 v = __ldcg(a + i);
        const int k = K - 16 * i;  // bytes of the piece inside K: the others count as zero
        if (k < 16) {
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int left = k - 4 * j;
            if (left < 4) w[j] = left <= 0 ? 0u : w[j] & (0xFFFFFFFFu >> (8 * (4 - left)));
          }
          v = make_uint4(w[0], w[1], w[2], w[3]);
        }
        c[i] = v;
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) sa[m] = m < p.M ? __ldcg(p.sa + m) : 0.0f;
  }
  __syncthreads();
  const uint4 *codes = reinterpret_cast<const uint4 *>(s_codes);
  for (; n < p.N;) {
    int acc[MT] = {};
    const float sw = __ldcg(p.sw + n);
    const float bias = p.bias ? i8_bias(p.bias, p.bias_dtype, n) : 0.0f;
    const int next = n + stride;
    for (int first = 0; first < chunks; first += 32 * kI8vDepth) {
#pragma unroll
      for (int d = 0; d < kI8vDepth; ++d) {
        const int i = first + d * 32 + lane;
        if (i < chunks) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if (MT > 1 && m >= p.M) continue;
            const uint4 a = codes[m * chunks + i];
            acc[m] = __dp4a((int)wv[d].x, (int)a.x, acc[m]);
            acc[m] = __dp4a((int)wv[d].y, (int)a.y, acc[m]);
            acc[m] = __dp4a((int)wv[d].z, (int)a.z, acc[m]);
            acc[m] = __dp4a((int)wv[d].w, (int)a.w, acc[m]);
          }
        }
      }
      // the other warps of the SM multiply meanwhile
      if (first + 32 * kI8vDepth < chunks) load_row(n, first + 32 * kI8vDepth);
      else if (next < p.N) load_row(next, 0);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int sum = __reduce_add_sync(0xffffffffu, acc[m]);
      if (lane == m && m < p.M) {
        float y = __fmul_rn((float)sum, __fmul_rn(sa[m], sw));
        if (p.bias) y = __fadd_rn(y, bias);
        const int64_t at = (int64_t)m * p.ldy + n;
        if (p.y_dtype == Q4_F32) reinterpret_cast<float *>(p.Y)[at] = y;
        else reinterpret_cast<uint16_t *>(p.Y)[at] = p.y_dtype == Q4_BF16 ? Dt<Q4_BF16>::from_f(y) : Dt<Q4_F16>::from_f(y);
      }
    }
    n = next;
  }
}

}  // namespace q4
