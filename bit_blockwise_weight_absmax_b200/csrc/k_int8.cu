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
  } else if (p.cols <= 256 * 8 * kI8Keep) {
    launch_pdl(int8_quantize_kernel<DT, 256, VEC>, dim3((unsigned)p.rows), dim3(256), 0, st, p);
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

int run_int8_quantize_f32(const I8QuantF32Params &p, cudaStream_t st) {
  launch_pdl(int8_quantize_f32_kernel<256>, dim3((unsigned)p.rows), dim3(256), 0, st, p);
  return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}

// The plan is the cheapest by this estimate (us, fitted to measured products;
// of 42 of 8 .. 4096 tokens by 576 .. 28672 rows it gives 0.64 to 1.23 of the
// time, two thirds of them within 12 %): a fixed part (set-up, first copies, last epilogue), the
// k-blocks of the busiest CTA or the weights' way from memory, and the round
// trip of sums where tiles are cut.
struct I8Cost {
  int nt;
  float fixed, block, cut;
};
constexpr I8Cost kI8Costs[] = {
    {16, 5.0f, 0.27f, 4.0f}, {32, 5.0f, 0.28f, 4.0f}, {64, 5.0f, 0.29f, 4.0f}, {128, 5.3f, 0.33f, 6.0f}, {256, 8.0f, 0.40f, 14.0f}};
constexpr float kI8BytesPerUs = 6.4e6f;
constexpr int kI8MinRun = 4;  // k-blocks a CTA takes of a cut tile, at least

I8Plan int8_plan(int64_t M, int64_t N, int64_t K, int sms) {
  I8Plan best;
  float best_us = 0.0f;
  const int nk = (int)((K + kI8Bk - 1) / kI8Bk);
  for (const I8Cost &cost : kI8Costs) {
    const bool pair = cost.nt == 256;
    const int rows = pair ? 2 * kI8Rows : kI8Rows, g = pair ? sms / 2 : sms;
    const int64_t tt = (M + cost.nt - 1) / cost.nt, tn = (N + rows - 1) / rows, tiles = tt * tn;
    if (tiles > INT32_MAX / 2) continue;  // too many for the kernel's indices
    const float bytes_us = (float)N * (float)K / kI8BytesPerUs;
    for (int c = 0; c < 2; ++c) {
      int64_t whole = tiles, cut = 0, rest = 0;
      float blocks = (float)((tiles + g - 1) / g * nk);
      if (c) {
        whole = tiles / g * g;
        rest = tiles - whole;
        // an equal number of CTAs for each tile where that keeps most of them
        // busy (then none has two unfinished tiles), else all CTAs
        const int64_t most = nk / kI8MinRun, each = rest ? std::min<int64_t>(g / rest, most) : 0;
        if (!rest || most < 2) continue;
        cut = each >= 2 && (each == most || each * rest * 4 >= 3 * (int64_t)g) ? each * rest
                                                                              : std::min<int64_t>(g, rest * most);
        if (cut <= rest) continue;
        blocks = (float)(whole / g * nk) + (float)(rest * nk) / (float)cut;
      }
      const float us = cost.fixed + std::max(blocks * cost.block, bytes_us) + (c ? cost.cut : 0.0f);
      if (best.nt && us >= best_us) continue;
      best_us = us;
      best.nt = cost.nt;
      best.pair = pair;
      best.tiles_t = (int)tt, best.tiles_n = (int)tn;
      best.whole = (int)whole, best.cut_ctas = (int)cut;
      best.slots = (int)rest;
      const int per = pair ? 2 : 1;
      best.grid = (int)std::min<int64_t>(g, std::max(whole, cut)) * per;
      best.ws_bytes = rest ? kI8CountBytes + (size_t)cut * per * 2 * cost.nt * kI8Rows * 4 : 0;
      if ((size_t)rest * per * kI8EpiWarps * sizeof(unsigned) > kI8CountBytes) best.nt = 0;  // not on a B200's SMs
    }
  }
  return best;
}

namespace {
template <int MT, int DT, bool VEC>
int go_gemv(const I8GemvParams &p, int sms, cudaStream_t st) {
  const int smem = MT * ((p.K + 15) / 16 * 16);
  // without the opt-in the static and the dynamic part together may not pass 48 KB
  constexpr auto kern = int8_gemv_kernel<MT, DT, VEC>;
  const int rc = set_smem_attr_once<kern>(kI8vMaxBytes, false);
  if (rc != Q4_OK) return rc;
  // as many CTAs of 8 warps as the SMs hold, a warp for each row where there are fewer
  const int grid = (int)std::min<int64_t>((p.N + 7) / 8, (int64_t)i8v_ctas(MT) * sms);
  launch_pdl(kern, dim3((unsigned)grid), dim3(kI8vThreads), smem, st, p);
  return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}
template <int DT, bool VEC>
int gemv_tokens(const I8GemvParams &p, int sms, cudaStream_t st) {
  if (p.M == 1) return go_gemv<1, DT, VEC>(p, sms, st);
  if (p.M == 2) return go_gemv<2, DT, VEC>(p, sms, st);
  return go_gemv<4, DT, VEC>(p, sms, st);
}
}  // namespace

bool int8_gemv_ok(int64_t M, int64_t K) {
  return M <= kI8vMaxTokens && (M == 3 ? 4 : M) * ((K + 15) / 16 * 16) <= kI8vMaxBytes;
}
int run_int8_gemv(int x_dtype, const I8GemvParams &p, int sms, cudaStream_t st) {
  if (!p.X) return gemv_tokens<-1, true>(p, sms, st);
  const bool vec = ((uintptr_t)p.X & 15u) == 0 && p.ldx % 8 == 0;
  if (x_dtype == Q4_F16) return vec ? gemv_tokens<Q4_F16, true>(p, sms, st) : gemv_tokens<Q4_F16, false>(p, sms, st);
  return vec ? gemv_tokens<Q4_BF16, true>(p, sms, st) : gemv_tokens<Q4_BF16, false>(p, sms, st);
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
