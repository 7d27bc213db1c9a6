// int8_gemm.cuh -- Y[M, N] = sa[m] sw[n] sum_k A[m, k] W[n, k] + bias[n] with
// 8-bit integer operands and exact 32-bit integer sums, on tcgen05 tensor
// cores (kind::i8, sm_100a).
//
// Bound by the weights' bytes for few tokens (N K of them whatever M) and by
// the tensor pipe and shared memory for many.  One persistent CTA per SM:
//   warp 0      TMA producer: per 128-byte k-block a weight tile [128 rows]
//               and a token tile into a ring of stages (128B swizzle);
//   warp 1      issues 4 MMAs (K = 32) per k-block: the weight tile is on the
//               128-row M side, the tokens are the N side (NT of them), so a
//               decode batch costs a narrow N and not a padded M;
//   warps 2..9  epilogue: a TMEM lane is a weight row, a column a token, so a
//               warp stores runs of 32 outputs of one token.  Two accumulators
//               alternate: an epilogue overlaps the next tile's MMAs.
// PAIR: the two CTAs of a cluster share one 256-row x 256-token tile
// (cta_group::2): each loads its 128 weight rows and half of the tokens, so a
// k-block costs 32 KB of copies per SM and 512 tensor cycles instead of 48 KB
// -- with 48 KB the copies' writes and the MMAs' reads of shared memory need
// more than its 128 bytes per cycle.
//
// Work: tiles are dealt round robin in whole waves; what is left over (all of
// them, for small products) is cut in k into equal runs of k-blocks, one per
// CTA.  The sums of an unfinished tile go to the workspace (a CTA has two at
// most, at the ends of its run) and are counted per epilogue warp in
// k-blocks; the warp that completes a count adds the others' to its own
// (integers: any order gives the same bits), writes Y and zeroes the count.
// (Adding them with atomics instead took 34 us for 128 x 256 tiles: 32-bit
// atomics go at about one element per L2 slice and cycle.)
//
// The weights' first k-blocks are prefetched into L2 before the wait for the
// previous kernel, so they travel while that kernel (the quantization of the
// tokens) still runs; a prefetch changes nothing, so weights that an earlier
// kernel is still writing are read correctly after the wait.
// Measured: 4096 x 28672 x 8192 630 us (3.1 POP/s, tensor pipe busy 0.82 to
// 0.90 of the time); 24 x 11008 x 4096 15.2 us (3.0 TB/s).
// Every wait is bounded: a timeout raises Q4_STATUS_TIMEOUT and ends the
// launch with undefined outputs (the workspace is then zero-filled again by
// the caller).
#pragma once
#include <cuda.h>

#include "gemm.cuh"  // PTX wrappers, bounded waits
#include "q4_common.cuh"

namespace q4 {

constexpr int kI8Bk = 128;                   // bytes of k per stage
constexpr int kI8Rows = 128;                 // weight rows per CTA
constexpr int kI8EpiWarps = 8;
constexpr int kI8Threads = (2 + kI8EpiWarps) * 32;
constexpr int kI8GroupT = 8;                 // token tiles that go together through the weight tiles
constexpr size_t kI8CountBytes = Q4_WORKSPACE_HEAD;  // the counts' part of the workspace, at its start
constexpr int kI8WTile = kI8Rows * kI8Bk;    // 16 KB

template <int NT, bool PAIR> struct I8Shape {
  static constexpr int kLoadT = PAIR ? NT / 2 : NT;  // tokens a CTA copies
  static constexpr int kATile = kLoadT * kI8Bk;
  static constexpr int kStageBytes = kI8WTile + kATile;
  static constexpr int kStages = (222 * 1024 - 2048) / kStageBytes > 12 ? 12 : (222 * 1024 - 2048) / kStageBytes;
  static constexpr int kCols = NT < 32 ? 32 : NT;    // TMEM columns of an accumulator
  static constexpr int kTmem = 2 * kCols < 64 ? 64 : 2 * kCols;
  static constexpr int kSmem = kStages * kStageBytes + 1024 /*align*/;
};

struct alignas(64) I8GemmParams {
  CUtensorMap tmW;  // W [N, K] bytes, box {128, 128}
  CUtensorMap tmA;  // A [M, K] bytes, box {128, kLoadT}
  const float *sa, *sw;
  const void *bias;
  void *Y;
  int64_t ldy;
  int32_t M, N;
  int32_t bias_dtype, y_dtype;
  int32_t nk;              // k-blocks
  int32_t tiles_t, tiles_n;
  int32_t whole;           // tiles dealt whole; the others are cut
  int32_t cut_ctas;        // CTAs (pairs) that share the cut tiles
  int32_t stall_copies;    // test hook: the producer issues no copies
  int32_t prefetch;        // weight boxes prefetched into L2 before the wait
  unsigned *counts;        // cut tiles: [slot][CTA of the pair][epilogue warp] k-blocks done, zero between calls
  int32_t *parts;          // sums of unfinished tiles: [CTA][first or last run][NT / 4][128 rows][4 tokens]
  uint64_t wait_ns;
  int *status;
};

// A run of k-blocks of one tile: [kb0, kb1); slot >= 0: a cut tile.
struct I8Item {
  int tile, kb0, kb1, slot;
};
// The items of CTA (pair) c of g: its share of the cut tiles, then whole ones.
struct I8Walk {
  int64_t u, u1;
  int tile;
  int64_t first;  // the run's first unit
  bool started;   // the current item is not the run's first
};
__device__ __forceinline__ I8Walk i8_walk(const I8GemmParams &p, int c) {
  I8Walk w;
  const int64_t units = (int64_t)(p.tiles_t * p.tiles_n - p.whole) * p.nk;
  w.u = c < p.cut_ctas ? units * c / p.cut_ctas : 0;
  w.u1 = c < p.cut_ctas ? units * (c + 1) / p.cut_ctas : 0;
  w.tile = c;
  w.started = false;
  w.first = w.u;
  return w;
}
// CTA (pair) of the cut tiles' unit u.
__device__ __forceinline__ int i8_owner(const I8GemmParams &p, int64_t units, int64_t u) {
  return (int)(((u + 1) * p.cut_ctas - 1) / units);
}
__device__ __forceinline__ bool i8_next(const I8GemmParams &p, I8Walk &w, int g, I8Item &it) {
  if (w.u < w.u1) {
    const int s = (int)(w.u / p.nk);
    it.slot = s;
    it.tile = p.whole + s;
    it.kb0 = (int)(w.u - (int64_t)s * p.nk);
    it.kb1 = (int)min((int64_t)p.nk, it.kb0 + (w.u1 - w.u));
    w.started = w.u > w.first;
    w.u += it.kb1 - it.kb0;
    return true;
  }
  if (w.tile >= p.whole) return false;
  it.slot = -1;
  it.tile = w.tile;
  it.kb0 = 0;
  it.kb1 = p.nk;
  w.tile += g;
  return true;
}
// Token tiles fastest within groups of kI8GroupT: the CTAs that run at once
// share a few weight tiles and a few token tiles in L2.
__device__ __forceinline__ void i8_tile(const I8GemmParams &p, int tile, int &tt, int &tn) {
  const int per = kI8GroupT * p.tiles_n;
  const int grp = tile / per, r = tile - grp * per;
  const int gt = min(kI8GroupT, p.tiles_t - grp * kI8GroupT);
  tt = grp * kI8GroupT + r % gt;
  tn = r / gt;
}

__device__ __forceinline__ float i8_bias(const void *bias, int dt, int64_t n) {
  if (dt == Q4_F32) return __ldcg(reinterpret_cast<const float *>(bias) + n);
  const uint16_t b = __ldcg(reinterpret_cast<const uint16_t *>(bias) + n);
  return dt == Q4_BF16 ? Dt<Q4_BF16>::to_f(b) : Dt<Q4_F16>::to_f(b);
}

// Outputs of weight row n for tokens t0 .. t0 + 15 from their integer sums:
// sum to binary32, times the product of the scales, plus the bias, each
// rounded once, then to y_dtype.  sa: the tokens' scales, in shared memory.
// A warp's lanes are 32 adjacent n.
__device__ __forceinline__ void i8_store16(const I8GemmParams &p, int n, int t0, float sw, float bias, const float *sa,
                                           const uint32_t (&r)[16]) {
  const int nt = min(16, p.M - t0);
  const int64_t at = (int64_t)t0 * p.ldy + n;
  float y[16];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const float4 s = reinterpret_cast<const float4 *>(sa)[v];
    const float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = 4 * v + e;
      y[j] = __fmul_rn((float)(int32_t)r[j], __fmul_rn(f[e], sw));
      if (p.bias) y[j] = __fadd_rn(y[j], bias);
    }
  }
  if (n >= p.N) return;
  if (p.y_dtype == Q4_F32) {
    float *o = reinterpret_cast<float *>(p.Y) + at;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < nt) o[(int64_t)j * p.ldy] = y[j];
  } else {
    uint16_t *o = reinterpret_cast<uint16_t *>(p.Y) + at;
    const bool bf = p.y_dtype == Q4_BF16;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < nt) o[(int64_t)j * p.ldy] = bf ? Dt<Q4_BF16>::from_f(y[j]) : Dt<Q4_F16>::from_f(y[j]);
  }
}

// Instruction descriptor, kind::i8: D s32 (2 at bit 4), A and B signed (1 at
// bits 7 and 10), K-major, N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t umma_idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
template <bool PAIR>
__device__ __forceinline__ void umma_i8(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
// Arrives on `bar` (in both CTAs of a pair) when all earlier MMAs are done.
template <bool PAIR> __device__ __forceinline__ void i8_commit(uint32_t bar) {
  if constexpr (PAIR) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  } else {
    umma_commit(bar);
  }
}
// The address of `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_l2(const CUtensorMap *map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int NT, bool PAIR>
__global__ void __launch_bounds__(kI8Threads, 1) int8_gemm_kernel(const __grid_constant__ I8GemmParams p) {
  using Sh = I8Shape<NT, PAIR>;
  constexpr int S = Sh::kStages;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t s_bar[2 * S + 4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ __align__(16) float s_sa[kI8EpiWarps][NT < 32 ? 16 : NT / 2];  // the token scales of each epilogue warp's columns
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = PAIR ? (int)(blockIdx.x & 1) : 0;
  const int c = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int g = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  const uint32_t bar0 = smem_u32(s_bar);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto accfull_bar = [&](int b) { return bar0 + 8u * (2 * S + b); };
  auto accempty_bar = [&](int b) { return bar0 + 8u * (2 * S + 2 + b); };
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accfull_bar(b), 1);
      mbar_init(accempty_bar(b), kI8EpiWarps * (PAIR ? 2 : 1));
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_abort = 0;
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(Sh::kTmem));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(Sh::kTmem));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  const int row_of_cta = rank * kI8Rows;  // within the tile's weight rows
  constexpr int kTileN = PAIR ? 2 * kI8Rows : kI8Rows;
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&p.tmW);
    prefetch_tensormap(&p.tmA);
    I8Walk w = i8_walk(p, c);
    I8Item it;
    int left = p.prefetch;
    while (left > 0 && i8_next(p, w, g, it)) {
      int tt, tn;
      i8_tile(p, it.tile, tt, tn);
      for (int kb = it.kb0; kb < it.kb1 && left > 0; ++kb, --left)
        tma_prefetch_l2(&p.tmW, kb * kI8Bk, tn * kTileN + row_of_cta);
    }
  }
  tc_fence_before();
  if constexpr (PAIR) cluster_sync();  // the peer's barriers exist before anything arrives on them
  else __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = s_tmem;
  volatile int *abort = &s_abort;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      I8Walk w = i8_walk(p, c);
      I8Item it;
      uint32_t i = 0;
      bool ok = true;
      while (ok && !*abort && i8_next(p, w, g, it)) {
        int tt, tn;
        i8_tile(p, it.tile, tt, tn);
        const int yw = tn * kTileN + row_of_cta, ya = tt * NT + (PAIR ? rank * Sh::kLoadT : 0);
        for (int kb = it.kb0; kb < it.kb1; ++kb, ++i) {
          const int s = i % S;
          if (!mbar_wait(empty_bar(s), ((i / S) & 1) ^ 1, p.status, abort, p.wait_ns)) {
            ok = false;
            break;
          }
          if (p.stall_copies) continue;
          const uint32_t dw = smem_u32(smem + s * Sh::kStageBytes), da = dw + kI8WTile;
          if constexpr (PAIR) {
            // both CTAs' copies complete on the leader's barrier
            const uint32_t fb = map_rank(full_bar(s), 0);
            if (rank == 0) mbar_arrive_expect_tx(full_bar(s), 2 * Sh::kStageBytes);
            tma_load_2d_pair(dw, &p.tmW, fb, kb * kI8Bk, yw);
            tma_load_2d_pair(da, &p.tmA, fb, kb * kI8Bk, ya);
          } else {
            mbar_arrive_expect_tx(full_bar(s), Sh::kStageBytes);
            tma_load_2d(dw, &p.tmW, full_bar(s), kb * kI8Bk, yw);
            tma_load_2d(da, &p.tmA, full_bar(s), kb * kI8Bk, ya);
          }
        }
      }
      // every copy completes before the CTA (the pair, see the end) may exit; a
      // pair's stages stay unfilled where the other CTA gave up before it copied
      if (rank == 0 && !p.stall_copies)
        for (uint32_t j = i > S ? i - S : 0; j < i; ++j) {
          volatile int no_abort = 0;
          if (!mbar_wait(full_bar(j % S), (j / S) & 1, PAIR ? p.status : nullptr, PAIR ? abort : &no_abort,
                         PAIR ? p.wait_ns : kWaitLimitNs))
            break;
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the pair's leader)
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = umma_idesc_i8(kTileN, NT);
      I8Walk w = i8_walk(p, c);
      I8Item it;
      uint32_t i = 0, count = 0, last_bar = 0, last_par = 0;
      bool ok = true, committed = false;
      for (; ok && !*abort && i8_next(p, w, g, it); ++count) {
        const int b = count & 1;
        const uint32_t ph = (count >> 1) & 1;
        if (!mbar_wait(accempty_bar(b), ph ^ 1, p.status, abort, p.wait_ns)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(b * Sh::kCols);
        for (int kb = it.kb0; kb < it.kb1; ++kb, ++i) {
          const int s = i % S;
          if (!mbar_wait(full_bar(s), (i / S) & 1, p.status, abort, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t dw = smem_u32(smem + s * Sh::kStageBytes), da = dw + kI8WTile;
#pragma unroll
          for (int k = 0; k < kI8Bk / 32; ++k)
            umma_i8<PAIR>(d, umma_desc_sw128(dw + 32 * k), umma_desc_sw128(da + 32 * k), idesc, kb != it.kb0 || k != 0);
          i8_commit<PAIR>(empty_bar(s));
          last_bar = empty_bar(s), last_par = (i / S) & 1, committed = true;
        }
        if (!ok) break;
        i8_commit<PAIR>(accfull_bar(b));
        last_bar = accfull_bar(b), last_par = ph;
      }
      // every MMA issued completes before TMEM is freed, also after a timeout
      if (committed) {
        volatile int no_abort = 0;
        mbar_wait(last_bar, last_par, nullptr, &no_abort);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - 2) >> 2;  // TMEM lane quadrant, which half of the token columns
    constexpr int kChunks = NT / 16, kHalf = (kChunks + 1) / 2;
    const int ch0 = half * kHalf, ch1 = half ? kChunks : kHalf;
    I8Walk w = i8_walk(p, c);
    I8Item it;
    uint32_t count = 0;
    for (; !__any_sync(0xffffffffu, *abort) && i8_next(p, w, g, it); ++count) {
      int tt, tn;
      i8_tile(p, it.tile, tt, tn);
      const int b = count & 1;
      const int nl = q * 32 + lane;
      const int n = tn * kTileN + row_of_cta + nl;
      const float sw = n < p.N ? __ldcg(p.sw + n) : 0.0f;
      const float bias = p.bias && n < p.N ? i8_bias(p.bias, p.bias_dtype, n) : 0.0f;
      const int nt = min(NT, p.M - tt * NT);  // tokens of the tile
      float *sa = s_sa[warp - 2];  // of tokens tt * NT + 16 ch0 ..
      __syncwarp();  // the previous tile's reads are done
      for (int j = lane; j < 16 * (ch1 - ch0); j += 32)
        sa[j] = 16 * ch0 + j < nt ? __ldcg(p.sa + tt * NT + 16 * ch0 + j) : 0.0f;
      __syncwarp();
      if (!mbar_wait_warp(accfull_bar(b), (count >> 1) & 1, p.status, abort, p.wait_ns)) break;
      tc_fence_after();
      const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * Sh::kCols);
      const bool cut = it.slot >= 0 && it.kb1 - it.kb0 < p.nk;
      const bool mine = ch0 < ch1 && 16 * ch0 < nt;  // this warp has columns of the tile
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR) mbar_arrive_cluster(map_rank(accempty_bar(b), 0));
          else mbar_arrive(accempty_bar(b));
        }
      };
      if (!cut) {
#pragma unroll 1
        for (int ch = ch0; ch < ch1 && 16 * ch < nt; ++ch) {
          uint32_t r[16];
          tmem_ld16(ta + 16 * ch, r);
          i8_store16(p, n, tt * NT + 16 * ch, sw, bias, sa + 16 * (ch - ch0), r);
        }
        release();
        continue;
      }
      // [CTA][run][chunk][4 tokens][row]: a warp's 16-byte accesses are adjacent
      constexpr int kPer = PAIR ? 2 : 1;
      auto part = [&](int cta, int run, int ch) {
        return reinterpret_cast<int4 *>(p.parts + ((((int64_t)cta * kPer + rank) * 2 + run) * kChunks + ch) * kI8Rows * 16) + nl;
      };
      bool last = false;
      if (mine) {
        const int run = it.kb0 == 0 && w.started ? 1 : 0;  // the run's second end, or its first
#pragma unroll 1
        for (int ch = ch0; ch < ch1 && 16 * ch < nt; ++ch) {
          uint32_t r[16];
          tmem_ld16(ta + 16 * ch, r);
          int4 *dst = part(c, run, ch);
#pragma unroll
          for (int v = 0; v < 4; ++v) __stcg(dst + v * kI8Rows, make_int4((int)r[4 * v], (int)r[4 * v + 1], (int)r[4 * v + 2], (int)r[4 * v + 3]));
        }
        __threadfence();  // this lane's sums are visible before its warp's count
        __syncwarp();
        unsigned *cnt = p.counts + (it.slot * kPer + rank) * kI8EpiWarps + (warp - 2);
        unsigned old = 0;
        if (lane == 0) old = atomicAdd(cnt, (unsigned)(it.kb1 - it.kb0));
        old = __shfl_sync(0xffffffffu, old, 0);
        last = old + (it.kb1 - it.kb0) == (unsigned)p.nk;
        if (last && lane == 0) *cnt = 0u;
      }
      if (last) {
        __threadfence();
        const int64_t units = (int64_t)(p.tiles_t * p.tiles_n - p.whole) * p.nk, u0 = (int64_t)it.slot * p.nk;
        const int c0 = i8_owner(p, units, u0), others = i8_owner(p, units, u0 + p.nk - 1) - c0;
        // kOC of the others' sums of kCC chunks are on their way at once: one
        // after the other their latencies were most of a small product's time
        constexpr int kCC = kHalf >= 2 ? 2 : 1, kOC = kCC == 2 ? 2 : 4;
#pragma unroll 1
        for (int ch = ch0; ch < ch1 && 16 * ch < nt; ch += kCC) {
          uint32_t r[kCC][16];
#pragma unroll
          for (int e = 0; e < kCC; ++e)
            if (ch + e < ch1) tmem_ld16(ta + 16 * (ch + e), r[e]);
#pragma unroll 1
          for (int o0 = 0; o0 < others; o0 += kOC) {
            int4 t[kOC][kCC][4];
#pragma unroll
            for (int k = 0; k < kOC; ++k) {
              const int o = c0 + o0 + k + (c0 + o0 + k >= c ? 1 : 0);  // the others, past this CTA
              // the tile is the end of a run that began before it, else the run's begin
              const int run = units * o / p.cut_ctas < u0 ? 1 : 0;
#pragma unroll
              for (int e = 0; e < kCC; ++e) {
                const int4 *src = part(o, run, ch + e);
#pragma unroll
                for (int v = 0; v < 4; ++v)
                  t[k][e][v] = o0 + k < others && ch + e < ch1 ? __ldcg(src + v * kI8Rows) : make_int4(0, 0, 0, 0);
              }
            }
#pragma unroll
            for (int k = 0; k < kOC; ++k)
#pragma unroll
              for (int e = 0; e < kCC; ++e)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                  r[e][4 * v] += (uint32_t)t[k][e][v].x, r[e][4 * v + 1] += (uint32_t)t[k][e][v].y;
                  r[e][4 * v + 2] += (uint32_t)t[k][e][v].z, r[e][4 * v + 3] += (uint32_t)t[k][e][v].w;
                }
          }
#pragma unroll
          for (int e = 0; e < kCC; ++e)
            if (ch + e < ch1 && 16 * (ch + e) < nt)
              i8_store16(p, n, tt * NT + 16 * (ch + e), sw, bias, sa + 16 * (ch + e - ch0), r[e]);
        }
      }
      release();
    }
  }

  if (PAIR && *abort && warp == 0 && lane == 0) {
    // after a timeout a pair's CTAs cannot wait for their copies on the stage
    // barriers, which may lack the other's: they give them a millisecond (they
    // take microseconds) before the pair ends
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the peer's copies, commits and arrivals into this CTA have ended
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Sh::kTmem));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Sh::kTmem));
  }
}

}  // namespace q4
