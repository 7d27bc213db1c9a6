// k_kv.cu -- launchers of the 4-bit key/value cache kernels.
#include "q4_internal.h"
#include <algorithm>

#include "serve_internal.h"

namespace q4 {
namespace {
// f.template operator()<DT, D, B>() for the cache's format
template <typename F>
int by_format(int dt, int D, int B, F &&f) {
  if (dt == Q4_F16) {
    if (D == 64) return f.template operator()<Q4_F16, 64, 64>();
    return B == 64 ? f.template operator()<Q4_F16, 128, 64>() : f.template operator()<Q4_F16, 128, 128>();
  }
  if (D == 64) return f.template operator()<Q4_BF16, 64, 64>();
  return B == 64 ? f.template operator()<Q4_BF16, 128, 64>() : f.template operator()<Q4_BF16, 128, 128>();
}
int launched() { return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA; }

// Few tokens: one a thread, so that they spread over the SMs; many: kKvItems
// (43 us against 37 for 8191 tokens of 32 heads, the same up to 8192 of 8).
template <int D, int ITEMS> bool kv_grid(int64_t tokens, int heads, dim3 *grid) {
  constexpr int per = kKvThreads / (D / 16) * ITEMS;
  const int64_t groups = (tokens + per - 1) / per;
  *grid = dim3((unsigned)groups, (unsigned)heads, 2);
  return groups <= INT32_MAX;
}
bool kv_many(int64_t tokens, int heads, int D, int sms) {
  return tokens * heads * 2 * (D / 16) >= (int64_t)sms * 2048 * kKvItems;  // the SMs' threads, kKvItems each
}
struct Append {
  const KvAppendParams &p;
  int sms;
  cudaStream_t st;
  template <int DT, int D, int B> int operator()() const {
    dim3 grid;
    if (kv_many(p.tokens, p.c.heads, D, sms)) {
      if (!kv_grid<D, kKvItems>(p.tokens, p.c.heads, &grid)) return Q4_ERR_SHAPE;
      launch_pdl(kv_append_kernel<DT, D, B, kKvItems>, grid, dim3(kKvThreads), 0, st, p);
    } else {
      kv_grid<D, 1>(p.tokens, p.c.heads, &grid);
      launch_pdl(kv_append_kernel<DT, D, B, 1>, grid, dim3(kKvThreads), 0, st, p);
    }
    return launched();
  }
};
struct Dequant {
  const KvDequantParams &p;
  int sms;
  cudaStream_t st;
  template <int DT, int D, int B> int operator()() const {
    dim3 grid;
    if (kv_many(p.n, p.c.heads, D, sms)) {
      if (!kv_grid<D, kKvItems>(p.n, p.c.heads, &grid)) return Q4_ERR_SHAPE;
      launch_pdl(kv_dequantize_kernel<DT, D, B, kKvItems>, grid, dim3(kKvThreads), 0, st, p);
    } else {
      kv_grid<D, 1>(p.n, p.c.heads, &grid);
      launch_pdl(kv_dequantize_kernel<DT, D, B, 1>, grid, dim3(kKvThreads), 0, st, p);
    }
    return launched();
  }
};
// Rows that share a kv head: up to 8 take one column tile of the MMAs, more
// take two at once (the cache is then read half as often).
template <int DT, int D, int B, int NT>
int go_attend(const KvAttnParams &p, int sms, cudaStream_t st) {
  using Sh = KvShape<D, B, NT>;
  constexpr auto kern = kv_attention_kernel<DT, D, B, NT>;
  const int rc = set_smem_attr_once<kern>(Sh::kSmem, true);
  if (rc != Q4_OK) return rc;
  launch_pdl(kern, dim3((unsigned)(Sh::kCtas * sms)), dim3(kKvAttnThreads), Sh::kSmem, st, p);
  return launched();
}
// Many rows: a CTA for each 256 rows of a sequence and kv head; the grid is
// what the rows can make at most (the CTAs past the last tile end at once).
template <int DT, int D, int B>
int go_prompt(const KvAttnParams &p, cudaStream_t st) {
  constexpr auto kern = kv_prompt_kernel<DT, D, B>;
  const int rc = set_smem_attr_once<kern>(KpShape<D>::kSmem, true);
  if (rc != Q4_OK) return rc;
  const int64_t rows = (int64_t)p.total_q * (p.q_heads / p.c.heads);
  const int64_t tiles = (rows / kKpRows + std::min<int64_t>(p.batch, rows)) * p.c.heads + p.sms;  // the last wave's parts
  if (tiles > INT32_MAX) return Q4_ERR_SHAPE;
  launch_pdl(kern, dim3((unsigned)tiles), dim3(kKpThreads), KpShape<D>::kSmem, st, p);
  return launched();
}
// The most rows of a kv head that take the kernel for few rows.  Measured (us,
// 8 kv heads, D = 128), few-rows kernel against the prompt kernel: 32 rows over
// 16384 keys 28 / 63, 32 sequences of 4096 keys 109 / 139; 64 rows 43 / 64 and
// 194 / 143.
constexpr int64_t kFewRows = 48;
struct Attend {
  const KvAttnParams &p;
  int rows, sms;
  cudaStream_t st;
  template <int DT, int D, int B> int operator()() const {
    if (rows > 16) return go_prompt<DT, D, B>(p, st);
    return rows <= 8 ? go_attend<DT, D, B, 1>(p, sms, st) : go_attend<DT, D, B, 2>(p, sms, st);
  }
};
}  // namespace

int run_kv_append(int dt, int D, int B, const KvAppendParams &p, int sms, cudaStream_t st) {
  return by_format(dt, D, B, Append{p, sms, st});
}
int run_kv_dequantize(int dt, int D, int B, const KvDequantParams &p, int sms, cudaStream_t st) {
  return by_format(dt, D, B, Dequant{p, sms, st});
}
int run_kv_attention(int dt, int D, int B, const KvAttnParams &p, int64_t max_q, int sms, cudaStream_t st) {
  const int64_t rows = max_q * (p.q_heads / p.c.heads);
  return by_format(dt, D, B, Attend{p, rows <= 8 ? 8 : rows <= kFewRows ? 16 : 256, sms, st});
}
size_t kv_attention_ws(int D, int sms) {
  // few rows: two segments of 8 or 16 rows a CTA; many: a part of 256 rows an SM
  const size_t few = (size_t)2 * sms * 2 * 16 * (D + 2), many = (size_t)sms * kKpRows * (D + 2);
  return kKvCountBytes + std::max(few, many) * sizeof(float);
}
}  // namespace q4
