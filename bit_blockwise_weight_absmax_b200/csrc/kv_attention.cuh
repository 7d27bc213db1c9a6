// kv_attention.cuh -- softmax(scale Q K^T) V over the paged 4-bit cache (sm_100a).
#pragma once
#include "kv_cache.cuh"

namespace q4 {

struct KvAttnParams {
  KvView c;
  const uint16_t *Q;
  int64_t q_ts, q_hs;
  const int32_t *cu_q;  // NULL: one row a sequence
  const int32_t *lens, *table;
  int64_t table_stride;
  int32_t table_pages, batch, total_q, q_heads;
  float scale;
  int32_t causal, window;  // window 0: none
  uint16_t *out;
  float *lse;
  int *status;
};

struct KvSeq {
  int q0, n, len;  // first query row, rows, keys
};
// Sequence b with its ranges cut to what exists.
__device__ __forceinline__ KvSeq kv_seq(const KvAttnParams &p, int b) {
  KvSeq s;
  int q0 = b, q1 = b + 1;
  if (p.cu_q) q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
  const int len = __ldg(p.lens + b);
  s.q0 = min(max(q0, 0), p.total_q);
  s.n = max(min(q1, p.total_q) - s.q0, 0);
  const int64_t most = (int64_t)p.table_pages << p.c.page_log2;
  s.len = (int)min((int64_t)max(len, 0), most);
  if (s.q0 != q0 || s.q0 + s.n != q1 || s.len != len) raise_status(p.status, Q4_STATUS_INDEX);
  return s;
}
// Page of key block `i` of sequence b, or -1 with the status raised.
__device__ __forceinline__ int kv_page(const KvAttnParams &p, int b, int i, int64_t pages) {
  const int pg = __ldg(p.table + (int64_t)b * p.table_stride + i);
  if (pg >= 0 && pg < pages) return pg;
  raise_status(p.status, Q4_STATUS_INDEX);
  return -1;
}

// One warp for a (row, query head): lanes take keys in turn, each with its own
// running maximum, sum and (in shared memory) none: the values are summed in a
// second pass over the keys with the finished maximum.
template <int DT, int D, int B>
__global__ void __launch_bounds__(128) kv_attention_kernel(const __grid_constant__ KvAttnParams p) {
  pdl_launch_then_wait();
  constexpr int NB = D / B, W = D / 8;
  __shared__ float sq[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * 4 + warp;
  const int row = blockIdx.x;
  int b = 0;
  KvSeq s = {0, 0, 0};
  bool found = false;
  for (b = 0; b < p.batch; ++b) {
    s = kv_seq(p, b);
    if (row >= s.q0 && row < s.q0 + s.n) {
      found = true;
      break;
    }
  }
  if (h >= p.q_heads || !found) return;
  const int hk = h / (p.q_heads / p.c.heads);
  for (int d = lane; d < D; d += 32) sq[warp][d] = Dt<DT>::to_f(p.Q[row * p.q_ts + h * p.q_hs + d]) * p.scale;
  __syncwarp();
  const int pos = s.len - s.n + (row - s.q0);
  const int hi = p.causal ? min(s.len, pos + 1) : s.len;
  const int lo = p.window ? max(0, pos - p.window + 1) : 0;
  const int64_t pages = p.c.slots >> p.c.page_log2;
  auto vec_of = [&](int j) -> int64_t {
    const int pg = kv_page(p, b, j >> p.c.page_log2, pages);
    return pg < 0 ? -1 : ((((int64_t)pg * p.c.heads + hk) << p.c.page_log2) + (j & ((1 << p.c.page_log2) - 1)));
  };
  auto value = [&](int which, int64_t vec, int d) -> float {
    const int blk = d / B, i = (d % B) / 8;
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(p.c.codes[which]) + vec * W + i * NB + blk);
    const uint32_t st = __ldg(p.c.state[which] + vec * NB + blk);
    return __half2float(__ushort_as_half((unsigned short)(st & 0xFFFFu))) *
           ((float)((w >> (4 * (d & 7))) & 15u) - __half2float(__ushort_as_half((unsigned short)(st >> 16))));
  };
  float m = -INFINITY, l = 0.0f;
  float o[D / 32] = {};
  for (int j0 = lo; j0 < hi; j0 += 32) {
    const int j = j0 + lane;
    const int64_t vec = j < hi ? vec_of(j) : -1;
    float x = -INFINITY;
    if (vec >= 0) {
      x = 0.0f;
      for (int d = 0; d < D; ++d) x = fmaf(sq[warp][d], value(0, vec, d), x);
    }
    float mx = x;
    for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    const float mn = fmaxf(m, mx);
    const float ref = mn == -INFINITY ? 0.0f : mn;
    const float f = __expf(m - ref), pr = expf(x - ref);
    float sum = pr;
    for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    l = l * f + sum;
    for (int e = 0; e < D / 32; ++e) o[e] *= f;
    m = mn;
    for (int k = 0; k < 32 && j0 + k < hi; ++k) {
      const int64_t vk = __shfl_sync(0xffffffffu, vec, k);
      const float pk = __shfl_sync(0xffffffffu, pr, k);
      if (vk >= 0)
        for (int e = 0; e < D / 32; ++e) o[e] = fmaf(pk, value(1, vk, lane + 32 * e), o[e]);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  for (int e = 0; e < D / 32; ++e)
    p.out[((int64_t)row * p.q_heads + h) * D + lane + 32 * e] = Dt<DT>::from_f(l == 0.0f ? 0.0f : o[e] * inv);
  if (p.lse && lane == 0) p.lse[(int64_t)row * p.q_heads + h] = l == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m) + logf(l);
}

}  // namespace q4
