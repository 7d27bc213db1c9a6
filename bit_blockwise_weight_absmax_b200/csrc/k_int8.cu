// k_int8.cu -- planning and launchers of the 8-bit integer kernels.
#include <string.h>

#include <algorithm>

#include "q4_internal.h"
#include "serve_internal.h"

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

template <int NT, bool PAIR>
int go_gemm(const I8Operands &o, const I8Plan &pl, I8GemmParams &p, cudaStream_t st) {
  using Sh = I8Shape<NT, PAIR>;
  constexpr auto kern = int8_gemm_kernel<NT, PAIR>;
  const int rc = set_smem_attr_once<kern>(Sh::kSmem, false);
  if (rc != Q4_OK) return rc;
  if (!make_map(&p.tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.W, o.N, o.K, 1, kI8Bk, kI8Rows, CU_TENSOR_MAP_SWIZZLE_128B, o.ldw) ||
      !make_map(&p.tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.A, o.M, o.K, 1, kI8Bk, Sh::kLoadT, CU_TENSOR_MAP_SWIZZLE_128B, o.lda))
    return Q4_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)pl.grid);
  cfg.blockDim = dim3(kI8Threads);
  cfg.dynamicSmemBytes = Sh::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = PAIR ? 2 : 1;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  cudaLaunchKernelEx(&cfg, kern, p);
  return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}
}  // namespace

int run_int8_quantize(int dt, const I8QuantParams &p, cudaStream_t st) {
  const bool vec = ((uintptr_t)p.X & 15u) == 0 && p.ldx % 8 == 0;
  if (dt == Q4_F16) return vec ? go_quantize<Q4_F16, true>(p, st) : go_quantize<Q4_F16, false>(p, st);
  return vec ? go_quantize<Q4_BF16, true>(p, st) : go_quantize<Q4_BF16, false>(p, st);
}

#ifndef I8_MIN_UNITS
#define I8_MIN_UNITS 4
#endif
I8Plan int8_plan(int64_t M, int64_t N, int64_t K, int sms) {
  I8Plan pl;
  const int nk = (int)((K + kI8Bk - 1) / kI8Bk);
  pl.pair = M > 128;
#ifdef I8_FORCE_NT
  pl.pair = I8_FORCE_NT == 256;
  pl.nt = I8_FORCE_NT;
#else
  pl.nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
#endif
  const int rows = pl.pair ? 2 * kI8Rows : kI8Rows;
  const int g = pl.pair ? sms / 2 : sms;
  const int64_t tt = (M + pl.nt - 1) / pl.nt, tn = (N + rows - 1) / rows, tiles = tt * tn;
  if (tiles > INT32_MAX / 2) {
    pl.nt = 0;  // too many tiles for the kernel's indices
    return pl;
  }
  pl.tiles_t = (int)tt, pl.tiles_n = (int)tn;
  int64_t whole = tiles / g * g;
  const int64_t rest = tiles - whole;
  int64_t cut = rest == 0 ? 0 : std::min<int64_t>(g, std::max<int64_t>(rest, rest * nk / I8_MIN_UNITS));
  if (rest * 8 >= (int64_t)g * 7) whole = tiles, cut = 0;  // the last wave is nearly full
  pl.whole = (int)whole;
  pl.cut_ctas = (int)cut;
  const int per = pl.pair ? 2 : 1;
  pl.grid = (int)(whole ? std::min<int64_t>(g, std::max<int64_t>(whole, cut)) : cut) * per;
  pl.slots = cut > rest ? (int)rest : 0;  // cut == rest: one whole tile each
  if (pl.slots * per * kI8EpiWarps * sizeof(unsigned) > kI8CountBytes) {  // more SMs than the counts have room for
    pl.whole = (int)tiles, pl.cut_ctas = 0, pl.slots = 0;
    pl.grid = (int)std::min<int64_t>(g, tiles) * per;
  }
  pl.ws_bytes = pl.slots ? kI8CountBytes + (size_t)pl.cut_ctas * per * 2 * pl.nt * kI8Rows * 4 : 0;
  return pl;
}

int run_int8_gemm(const I8Operands &o, const I8Plan &pl, I8GemmParams &p, cudaStream_t st) {
  switch (pl.nt) {
    case 16: return go_gemm<16, false>(o, pl, p, st);
    case 32: return go_gemm<32, false>(o, pl, p, st);
    case 64: return go_gemm<64, false>(o, pl, p, st);
    case 128: return go_gemm<128, false>(o, pl, p, st);
    case 256: return go_gemm<256, true>(o, pl, p, st);
  }
  return Q4_ERR_SHAPE;
}
}  // namespace q4
