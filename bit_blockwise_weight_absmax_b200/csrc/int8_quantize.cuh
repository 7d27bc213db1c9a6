// int8_quantize.cuh -- 8-bit codes with one scale per row (sm_100a):
// s = max|x| / 127, q = rint(x / s).
//
// Bound by memory (2 K bytes in, K out per row) and, for a few rows, by
// latency.  One CTA owns a row: each thread keeps up to kI8Keep 8-element
// pieces of it in registers between the maximum and the codes, so a row is
// read from memory once; what a longer row has beyond that is read again
// (from L2).  The quotient is the correctly rounded one (div_markstein, and
// __fdiv_rn for scales outside its range).  Rows of binary32 (weights at load
// time) take a plain kernel of two passes.
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
// Threads an SM holds, by registers: 4096 rows of 8192 in 25 us (3.9 TB/s)
// against 30 with a third fewer.
constexpr int kI8QuantThreads = 1536;

// The scale of a row from its largest magnitude.
struct I8Scale {
  float s, y, stored;  // divisor, its reciprocal, the scale as stored (NaN for a bad row)
  bool fast, zero, bad;
};
__device__ __forceinline__ I8Scale i8_scale(float top) {
  I8Scale r;
  r.bad = !(top <= 3.4028235e38f);
  r.s = __fdiv_rn(top, 127.0f);
  r.fast = markstein_ok(r.s);
  r.y = r.fast ? __frcp_rn(r.s) : 0.0f;
  r.zero = r.bad || r.s == 0.0f;
  r.stored = r.bad ? __int_as_float(0x7FFFFFFF) : r.s;
  return r;
}
// max|x| of 8 elements as two bit patterns: both 16-bit formats order their
// magnitudes as integers, infinities and NaNs last.
__device__ __forceinline__ uint32_t i8_top8(uint4 v) {
  const uint32_t a = __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), b = __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
  return __vmaxu2(a, b);
}
// Codes of 8 elements.  |x / s| <= 127 (1 + 2^-23), so adding 1.5 * 2^23
// rounds the quotient to the nearest integer, ties to even, and leaves its
// 8-bit two's complement in the low byte.
template <int DT> __device__ __forceinline__ uint2 i8_codes8(uint4 v, const I8Scale &c) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t b[8];
  if (c.zero) return make_uint2(0, 0);
  if (c.fast) {
    const uint64_t yy = f2_pack(c.y, c.y), ns = f2_pack(-c.s, -c.s), kr = f2_pack(12582912.0f, 12582912.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float r0, r1;
      f2_unpack(f2_add(div_markstein2(f2_pack(lo16<DT>(w[j]), hi16<DT>(w[j])), ns, yy), kr), r0, r1);
      b[2 * j] = __float_as_uint(r0), b[2 * j + 1] = __float_as_uint(r1);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      b[2 * j] = (uint32_t)__float2int_rn(__fdiv_rn(lo16<DT>(w[j]), c.s));
      b[2 * j + 1] = (uint32_t)__float2int_rn(__fdiv_rn(hi16<DT>(w[j]), c.s));
    }
  }
  uint2 o;
  o.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  o.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  return o;
}

// VEC: rows start at 16-byte boundaries (8-element pieces are one load).
template <int DT, int THREADS, bool VEC>
__global__ void __launch_bounds__(THREADS, kI8QuantThreads / THREADS) int8_quantize_kernel(const __grid_constant__ I8QuantParams p) {
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
  uint4 keep[kI8Keep];
  uint32_t m2 = 0;
#pragma unroll
  for (int k = 0; k < kI8Keep; ++k) {
    const int i = tid + k * THREADS;
    keep[k] = i < pieces ? load(i) : make_uint4(0, 0, 0, 0);
    m2 = __vmaxu2(m2, i8_top8(keep[k]));
  }
  for (int i = tid + kI8Keep * THREADS; i < pieces; i += THREADS) m2 = __vmaxu2(m2, i8_top8(load(i)));
  uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < THREADS / 32; ++j) m = max(m, s_max[j]);
  const I8Scale sc = i8_scale(Dt<DT>::to_f((uint16_t)m));
  int8_t *c = p.codes + row * p.ldc;
  auto store = [&](int i, uint4 v) {
    const uint2 o = i8_codes8<DT>(v, sc);
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
    p.scale[row] = sc.stored;
    if (sc.bad) raise_status(p.status, Q4_STATUS_NONFINITE);
  }
}

// Rows of binary32, once at load time: a pass for the maximum, one for the
// codes (from L2 where a row fits).  Magnitudes order as their bit patterns,
// infinities and NaNs last.  A subnormal s is rounded so coarsely that x / s
// may pass 127: clamped.
struct I8QuantF32Params {
  const float *X;
  int64_t rows, ldx, ldc;
  int32_t cols;
  int8_t *codes;
  float *scale;
  int *status;
};
template <int THREADS>
__global__ void __launch_bounds__(THREADS) int8_quantize_f32_kernel(const __grid_constant__ I8QuantF32Params p) {
  pdl_launch_then_wait();
  __shared__ uint32_t s_max[THREADS / 32];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const float *x = p.X + row * p.ldx;
  uint32_t m = 0;
  for (int i = tid; i < p.cols; i += THREADS) m = max(m, __float_as_uint(__ldg(x + i)) & 0x7FFFFFFFu);
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < THREADS / 32; ++j) m = max(m, s_max[j]);
  const I8Scale sc = i8_scale(__uint_as_float(m));
  int8_t *c = p.codes + row * p.ldc;
  for (int i = tid; i < p.cols; i += THREADS)
    c[i] = sc.zero ? (int8_t)0 : (int8_t)max(-127, min(127, __float2int_rn(__fdiv_rn(__ldg(x + i), sc.s))));
  if (tid == 0) {
    p.scale[row] = sc.stored;
    if (sc.bad) raise_status(p.status, Q4_STATUS_NONFINITE);
  }
}

}  // namespace q4
