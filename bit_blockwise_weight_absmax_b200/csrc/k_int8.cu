// k_int8.cu -- launchers of the 8-bit integer kernels.
#include "q4_internal.h"
#include "int8_gemm.cuh"
#include "int8_quantize.cuh"

namespace q4 {
namespace {
template <int DT, bool VEC>
int go_quantize(const I8QuantParams &p, cudaStream_t st) {
  // a thread holds up to 32 elements: rows of up to 4096 take 128 threads
  if (p.cols <= 128 * 8 * kI8Keep) {
    launch_pdl(int8_quantize_kernel<DT, 128, VEC>, dim3((unsigned)p.rows), dim3(128), 0, st, p);
  } else {
    launch_pdl(int8_quantize_kernel<DT, 512, VEC>, dim3((unsigned)p.rows), dim3(512), 0, st, p);
  }
  return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}
}  // namespace

int run_int8_quantize(int dt, const I8QuantParams &p, cudaStream_t st) {
  const bool vec = ((uintptr_t)p.X & 15u) == 0 && p.ldx % 8 == 0;
  if (dt == Q4_F16) return vec ? go_quantize<Q4_F16, true>(p, st) : go_quantize<Q4_F16, false>(p, st);
  return vec ? go_quantize<Q4_BF16, true>(p, st) : go_quantize<Q4_BF16, false>(p, st);
}

int run_int8_gemm(const I8GemmParams &p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.N + 63) / 64), (unsigned)((p.M + 63) / 64));
  launch_pdl(int8_gemm_kernel, grid, dim3(256), 0, st, p);
  return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}
}  // namespace q4
