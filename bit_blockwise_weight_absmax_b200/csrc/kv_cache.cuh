// kv_cache.cuh -- writing keys and values into the paged 4-bit cache, and
// reading them back as 16-bit floats (sm_100a).
//
// Per block of B elements of a token's head vector (the INT4 asymmetric rule
// with binary16 scales): mn = min(0, min x), mx = max(0, max x),
// s = f16((mx - mn) / 15), z = clamp(rint(-mn / s), 0, 15),
// q = clamp(rint(x / s) + z, 0, 15); x^ = s (q - z).
//
// Both kernels are bound by memory: 4 D bytes of K and V and D + 8 D / B bytes
// of cache per token and head.  A thread owns 8 elements = one 16-byte load
// and one word of codes; B / 8 lanes hold a block and find its range by
// shuffles.  Items run over tokens fastest, so that a CTA writes adjacent
// tokens of one head: with slots in order its codes and states are
// contiguous runs of the page.
#pragma once
#include "q4_common.cuh"

namespace q4 {

struct KvView {
  uint8_t *codes[2];   // K, V
  uint32_t *state[2];  // (s, z) binary16 pairs
  int64_t slots;       // pages * page_size
  int32_t heads, page_log2;
};

// Place of (slot, head) in units of one head vector.
__device__ __forceinline__ int64_t kv_vec(const KvView &c, int64_t slot, int head) {
  const int64_t page = slot >> c.page_log2;
  return ((page * c.heads + head) << c.page_log2) + (slot & ((1 << c.page_log2) - 1));
}

struct KvAppendParams {
  KvView c;
  const uint16_t *x[2];
  int64_t ts[2], hs[2];  // token and head strides, elements
  const int64_t *slots;
  int64_t tokens;
  int *status;
};

constexpr int kKvThreads = 256;
constexpr float kKvMaxRange = 61440.0f;  // 15 * 4096: s (q - z) stays within binary16

template <int DT, int D, int B>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
  pdl_launch_then_wait();
  constexpr int TV = D / 8;  // threads per vector
  constexpr int LB = B / 8;  // lanes per block
  constexpr int NB = D / B;
  const int which = blockIdx.y;
  const int64_t item = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) / TV;
  const int w = threadIdx.x % TV;  // elements 8 w .. 8 w + 7
  const int64_t n_items = p.tokens * p.c.heads;
  int64_t slot = -1;
  int head = 0;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (item < n_items) {
    head = (int)(item / p.tokens);
    const int64_t token = item - (int64_t)head * p.tokens;
    slot = __ldg(p.slots + token);
    if (slot >= p.c.slots) {
      if (w == 0) raise_status(p.status, Q4_STATUS_INDEX);
      slot = -1;
    }
    if (slot >= 0) v = ldg_stream_v4(p.x[which] + token * p.ts[which] + head * p.hs[which] + 8 * w);
  }
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) f[2 * j] = lo16<DT>(u[j]), f[2 * j + 1] = hi16<DT>(u[j]);
  float mn = 0.0f, mx = 0.0f, sum = 0.0f;  // sum: NaN or infinite when an element is
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    mn = fminf(mn, f[j]);
    mx = fmaxf(mx, f[j]);
    sum += f[j] * 0.0f;
  }
#pragma unroll
  for (int o = LB / 2; o >= 1; o >>= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  if (slot < 0) return;
  const float range = __fsub_rn(mx, mn);
  const bool bad = !(sum == 0.0f) || !(range <= kKvMaxRange);
  const float s = __half2float(__float2half_rn(__fdiv_rn(range, 15.0f)));
  uint32_t word = 0;
  float z = 0.0f;
  if (!bad && s != 0.0f) {  // a binary16 s is at least 2^-24: inside div_markstein's range
    const float y = __frcp_rn(s);
    z = fminf(fmaxf(rintf(div_markstein(-mn, s, y)), 0.0f), 15.0f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = fminf(fmaxf(rintf(div_markstein(f[j], s, y)) + z, 0.0f), 15.0f);
      word |= (uint32_t)q << (4 * j);
    }
  }
  const int64_t vec = kv_vec(p.c, slot, head);
  const int blk = w / LB, i = w % LB;
  reinterpret_cast<uint32_t *>(p.c.codes[which])[vec * TV + i * NB + blk] = word;
  if (i == 0) {
    const uint32_t sb = bad ? 0x7FFFu : (uint32_t)__half_as_ushort(__float2half_rn(s));
    p.c.state[which][vec * NB + blk] = sb | ((uint32_t)__half_as_ushort(__float2half_rn(z)) << 16);
    if (bad) raise_status(p.status, Q4_STATUS_NONFINITE);
  }
}

struct KvDequantParams {
  KvView c;
  uint16_t *x[2];
  const int64_t *slots;
  int64_t n;
  int *status;
};

template <int DT, int D, int B>
__global__ void __launch_bounds__(kKvThreads) kv_dequantize_kernel(const __grid_constant__ KvDequantParams p) {
  pdl_launch_then_wait();
  constexpr int TV = D / 8, LB = B / 8, NB = D / B;
  const int which = blockIdx.y;
  const int64_t item = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) / TV;
  const int w = threadIdx.x % TV;
  if (item >= p.n * p.c.heads) return;
  const int head = (int)(item / p.n);
  const int64_t row = item - (int64_t)head * p.n;
  const int64_t slot = __ldg(p.slots + row);
  uint4 o = make_uint4(0, 0, 0, 0);
  if (slot >= p.c.slots) {
    if (w == 0) raise_status(p.status, Q4_STATUS_INDEX);
  } else if (slot >= 0) {
    const int64_t vec = kv_vec(p.c, slot, head);
    const int blk = w / LB, i = w % LB;
    const uint32_t word = __ldg(reinterpret_cast<const uint32_t *>(p.c.codes[which]) + vec * TV + i * NB + blk);
    const uint32_t st = __ldg(p.c.state[which] + vec * NB + blk);
    const float s = __half2float(__ushort_as_half((unsigned short)(st & 0xFFFFu)));
    const float z = __half2float(__ushort_as_half((unsigned short)(st >> 16)));
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r[j] = Dt<DT>::pack2(s * ((float)((word >> (8 * j)) & 15u) - z), s * ((float)((word >> (8 * j + 4)) & 15u) - z));
    o = make_uint4(r[0], r[1], r[2], r[3]);
  }
  *reinterpret_cast<uint4 *>(p.x[which] + (row * p.c.heads + head) * D + 8 * w) = o;
}

}  // namespace q4
