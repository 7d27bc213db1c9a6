// int8_quantize.cuh -- 8-bit codes with one scale per row (sm_100a):
// s = max|x| / 127, q = rint(x / s).
//
// Bound by memory (2 K bytes in, K out per row) and, for a few rows, by
// latency.  One CTA owns a row: each thread keeps up to kI8Keep 8-element
// pieces of it in registers between the maximum and the codes, so a row is
// read from memory once; what a longer row has beyond that is read again
// (from L2).  The quotient is the correctly rounded one (div_markstein, and
// __fdiv_rn for scales outside its range).
#pragma once
#include "q4_common.cuh"

namespace q4 {

struct I8QuantParams {
  const uint16_t *X;
  int64_t rows, ldx, ldc;
  int32_t cols;
  int8_t *codes;
  float *scale;
  int *status;
};

constexpr int kI8Keep = 4;

// Four codes of four floats, low byte first.
__device__ __forceinline__ uint32_t i8_codes4(const float *f, float s, float y, bool fast) {
  uint32_t r = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float q = fast ? div_markstein(f[j], s, y) : __fdiv_rn(f[j], s);
    r |= ((uint32_t)__float2int_rn(q) & 0xFFu) << (8 * j);
  }
  return r;
}

// VEC: rows start at 16-byte boundaries (8-element pieces are one load).
template <int DT, int THREADS, bool VEC>
__global__ void __launch_bounds__(THREADS) int8_quantize_kernel(const __grid_constant__ I8QuantParams p) {
  pdl_launch_then_wait();
  __shared__ uint32_t s_max[THREADS / 32];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const uint16_t *x = p.X + row * p.ldx;
  const int K = p.cols, pieces = (K + 7) / 8;
  auto load = [&](int i) -> uint4 {  // elements 8 i .. 8 i + 7, zeros past the row
    if (VEC && 8 * i + 8 <= K) return __ldg(reinterpret_cast<const uint4 *>(x) + i);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 8 * i + 2 * j;
      const uint32_t lo = e < K ? __ldg(x + e) : 0u, hi = e + 1 < K ? __ldg(x + e + 1) : 0u;
      w[j] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  // max|x| as a bit pattern: both 16-bit formats order their magnitudes as
  // integers, infinities and NaNs last
  auto top8 = [](uint4 v) -> uint32_t {
    const uint32_t a = __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), b = __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
    return __vmaxu2(a, b);
  };
  uint4 keep[kI8Keep];
  uint32_t m2 = 0;
#pragma unroll
  for (int k = 0; k < kI8Keep; ++k) {
    const int i = tid + k * THREADS;
    keep[k] = i < pieces ? load(i) : make_uint4(0, 0, 0, 0);
    m2 = __vmaxu2(m2, top8(keep[k]));
  }
  for (int i = tid + kI8Keep * THREADS; i < pieces; i += THREADS) m2 = __vmaxu2(m2, top8(load(i)));
  uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < THREADS / 32; ++j) m = max(m, s_max[j]);
  const float top = Dt<DT>::to_f((uint16_t)m);
  const bool bad = !(top <= 3.4028235e38f);
  const float s = __fdiv_rn(top, 127.0f);
  const bool fast = markstein_ok(s);
  const float y = fast ? __frcp_rn(s) : 0.0f;
  const bool zero = bad || s == 0.0f;
  int8_t *c = p.codes + row * p.ldc;
  auto store = [&](int i, uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[2 * j] = lo16<DT>(w[j]), f[2 * j + 1] = hi16<DT>(w[j]);
    uint2 o = make_uint2(0, 0);
    if (!zero) o = make_uint2(i8_codes4(f, s, y, fast), i8_codes4(f + 4, s, y, fast));
    if (8 * i + 8 <= K) {
      reinterpret_cast<uint2 *>(c)[i] = o;
    } else {
      for (int j = 0; 8 * i + j < K; ++j) c[8 * i + j] = (int8_t)((j < 4 ? o.x >> (8 * j) : o.y >> (8 * j - 32)) & 0xFFu);
    }
  };
#pragma unroll
  for (int k = 0; k < kI8Keep; ++k) {
    const int i = tid + k * THREADS;
    if (i < pieces) store(i, keep[k]);
  }
  for (int i = tid + kI8Keep * THREADS; i < pieces; i += THREADS) store(i, load(i));
  if (tid == 0) {
    p.scale[row] = bad ? __int_as_float(0x7FFFFFFF) : s;
    if (bad) raise_status(p.status, Q4_STATUS_NONFINITE);
  }
}

}  // namespace q4
