// k_kv.cu -- launchers of the 4-bit key/value cache kernels.
#include "q4_internal.h"
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

struct Append {
  const KvAppendParams &p;
  cudaStream_t st;
  template <int DT, int D, int B> int operator()() const {
    const int64_t blocks = (p.tokens * p.c.heads * (D / 8) + kKvThreads - 1) / kKvThreads;
    if (blocks > INT32_MAX) return Q4_ERR_SHAPE;
    launch_pdl(kv_append_kernel<DT, D, B>, dim3((unsigned)blocks, 2), dim3(kKvThreads), 0, st, p);
    return launched();
  }
};
struct Dequant {
  const KvDequantParams &p;
  cudaStream_t st;
  template <int DT, int D, int B> int operator()() const {
    const int64_t blocks = (p.n * p.c.heads * (D / 8) + kKvThreads - 1) / kKvThreads;
    if (blocks > INT32_MAX) return Q4_ERR_SHAPE;
    launch_pdl(kv_dequantize_kernel<DT, D, B>, dim3((unsigned)blocks, 2), dim3(kKvThreads), 0, st, p);
    return launched();
  }
};
struct Attend {
  const KvAttnParams &p;
  cudaStream_t st;
  template <int DT, int D, int B> int operator()() const {
    launch_pdl(kv_attention_kernel<DT, D, B>, dim3((unsigned)p.total_q, (unsigned)((p.q_heads + 3) / 4)), dim3(128), 0, st, p);
    return launched();
  }
};
}  // namespace

int run_kv_append(int dt, int D, int B, const KvAppendParams &p, cudaStream_t st) { return by_format(dt, D, B, Append{p, st}); }
int run_kv_dequantize(int dt, int D, int B, const KvDequantParams &p, cudaStream_t st) {
  return by_format(dt, D, B, Dequant{p, st});
}
int run_kv_attention(int dt, int D, int B, const KvAttnParams &p, cudaStream_t st) { return by_format(dt, D, B, Attend{p, st}); }
}  // namespace q4
