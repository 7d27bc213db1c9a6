// kv_prompt.cuh -- softmax(scale Q K^T) V over the paged 4-bit cache for many
// query rows (prompts, chunks of prompts) on tcgen05 tensor cores (sm_100a).
//
// Bound by the tensor pipe (4 D flops a row and key) and, as close, by the
// exponentials (16 a cycle and SM) and by issue.  One CTA per SM takes 256
// query rows of one sequence and kv head (rows of all the query heads that
// share it: row = token * group + head) against key tiles of 128:
//   warps 0..7    softmax: a thread owns a row.  It reads its 128 scores from
//                 tensor memory and writes the weights back in binary16 over
//                 them.  The reference m of 2^(score - m) stays that of earlier
//                 tiles while the weights fit binary16 (their sum tells); only
//                 then, and for the first tile, the maximum is taken, the
//                 reference set kp_lift() below it and the output rescaled: one
//                 pass over the scores in the common case;
//   warps 8..11   dequantize: a thread owns a key.  Codes come straight from
//                 global memory into registers, a tile ahead; 1024 + code is
//                 one masked OR, minus 1024 + z exact, times s rounded once to
//                 binary16, stored in the 128B-swizzled layouts the MMAs read
//                 (keys K-major, values MN-major).  The order of d inside a
//                 word follows the nibbles; queries are stored alike, outputs
//                 put back at the end;
//   warp 12       issues S = Q K^T (both operands in shared memory) and
//                 O += P V (weights from tensor memory) for the two 128-row
//                 halves in turn: while one half's softmax runs, the other's
//                 products do.
// Work: whole (256 rows, kv head) tiles in as many waves as there are; those of
// the last, partly filled wave are cut along the keys over the idle SMs, their
// partial outputs joined by the CTA that comes last (few rows over many keys
// are all such tiles).
// Measured: 2048 rows of 64 heads over 8192 keys 538 us (894 TFLOP/s, tensor
// pipe busy half the time), 674 with the log sum exp.
// Tensor memory: two score tiles of 128 columns (weights over their first 64)
// and two outputs of D.  Query rows are scaled by a power of two into binary16.
#pragma once
#include <type_traits>

#include "kv_attention.cuh"

namespace q4 {

constexpr int kKpRows = 256;   // query rows of a CTA
constexpr int kKpKeys = 128;   // keys of a tile
constexpr int kKpThreads = 512;
constexpr int kKpMinTiles = 4;         // key tiles a CTA takes of a tile that several share, at least
// The reference is taken kp_lift() below the maximum: the largest weight is
// 2^lift then, and a binary16 weight is off by 2^-25 at most below the normal
// range, so n keys by n 2^(-25 - lift) of the largest: less than 2^-16 up to 2^17
// keys (2^-13 up to 2^20).  64 equal weights of 2^8 sum up to 2^14, inside
// kKpMost.  Not more than the keys need: rows whose scores climb past the
// headroom take the maximum again (2048 rows over 8192 keys, scores of a standard
// deviation of 3: 530 us with this rule's 4, 508 with 0, 738 with 8).
__device__ __forceinline__ float kp_lift(int keys) { return (float)min(8, max(0, 32 - __clz(max(keys - 1, 0)) - 9)); }
constexpr float kKpAhead = 15.0f;    // scores up to this far past the reference keep it
constexpr float kKpMost = 65504.0f;  // of a row's weights in a tile: each is inside binary16 then

template <int D> struct KpShape {
  static constexpr int kHalves = D / 64;                       // 128-byte wide parts of a row
  static constexpr int kTile = kHalves * kKpKeys * 128;        // a key or value tile, also 128 query rows
  static constexpr int kSmem = 2 * kTile + 5 * kTile + 1024;  // queries; keys, values and the keys' remainders
};

// 32 columns of this warp's 32 lanes of tensor memory, without waiting.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The MMAs are issued by a converged warp with one lane's predicate: the
// descriptors then stay in uniform registers.  (Issued inside a one-lane
// branch, 32 of them took 3700 cycles for 2048 of tensor work.)
// D (tensor memory) = A . B (shared memory) [+ D]
// A descriptor's low word carries the address (16-byte units) and moves by
// additions; its high word is the same for all operands here (stride byte
// offset 1024, version 1, 128-byte swizzle).
constexpr uint32_t kUmmaDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate, uint32_t lead) {
  asm volatile(
      "{ .reg .pred p, q; .reg .b64 da, db; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0; mov.b64 da, {%1, %6}; mov.b64 db, {%2, %6}; "
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p; }" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead), "n"(kUmmaDescHi)
      : "memory");
}
// D (tensor memory) = A (tensor memory, 16-bit pairs) . B (shared memory) [+ D]
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate, uint32_t lead) {
  asm volatile(
      "{ .reg .pred p, q; .reg .b64 db; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0; mov.b64 db, {%2, %6}; "
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p; }" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead), "n"(kUmmaDescHi)
      : "memory");
}
__device__ __forceinline__ void umma_commit_lead(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %1, 0; "
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar),
      "r"(lead)
      : "memory");
}
// Low words: K-major operands (leading byte offset unused, 1), and MN-major
// ones: rows of k of 64 elements of n (128 bytes), 8 rows a swizzle atom, the
// next 64 n `lbo` bytes on (leading byte offset).
__device__ __forceinline__ uint32_t desc_lo_k(uint32_t addr) { return (addr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }
constexpr uint32_t kUmmaTransposeB = 1u << 16;

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
template <int DT, int D, int B>
__global__ void __launch_bounds__(kKpThreads, 1) kv_prompt_kernel(const __grid_constant__ KvAttnParams p) {
  using Sh = KpShape<D>;
  constexpr int NB = D / B, W = D / 8;  // words of a vector
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *s_qt = smem;                  // [2 halves of rows][kTile]
  // [2 stages][keys, values][kTile], then what rounding the keys to binary16
  // left over (one stage: two, with one of values, took 694 us instead of 650)
  uint8_t *s_kv = smem + 2 * Sh::kTile;
  auto rest_of = [](int stage) { return (4 - 2 * stage) * Sh::kTile; };  // from a stage's keys to their remainders
  __shared__ uint64_t s_bar[18];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_where[4];  // [3]: this CTA joins the parts
  __shared__ int64_t s_scan[kKpThreads / 32];
  __shared__ uint4 s_bad[4];  // keys of a tile that no row may read
  // values that are the same in a warp are marked so (a shuffle): the MMA
  // warp's addresses and control flow then stay in the uniform datapath
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const uint32_t bar0 = smem_u32(s_bar);
  auto k_full = [&](int s) { return bar0 + 8u * s; };
  auto k_empty = [&](int s) { return bar0 + 8u * (2 + s); };
  auto v_full = [&](int s) { return bar0 + 8u * (4 + s); };
  auto v_empty = [&](int s) { return bar0 + 8u * (6 + s); };
  auto s_full = [&](int h) { return bar0 + 8u * (8 + h); };
  // the weights of keys 64 u .. of a tile (a barrier each: a warp may be done
  // with both before another is with the first); the first phase of u = 0 is
  // the queries'
  auto p_full = [&](int h, int u) { return bar0 + 8u * (10 + 2 * h + u); };
  auto pv_done = [&](int h, int u) { return bar0 + 8u * (14 + 2 * h + u); };
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(k_full(s), 4);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), 4);
      mbar_init(v_empty(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s, 0), 4);
      mbar_init(p_full(s, 1), 4);
      mbar_init(pv_done(s, 0), 1);
      mbar_init(pv_done(s, 1), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_abort = 0;
    s_where[0] = -1, s_where[1] = s_where[2] = 0;  // no tile
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  // this CTA's tile: a prefix sum over the sequences' (row tile, kv head)
  // tiles, heads fastest, a sequence's last rows (the longest) first
  const int group = p.q_heads / p.c.heads;
  const int per = (p.batch + kKpThreads - 1) / kKpThreads;
  auto tiles_of = [&](int b) -> int64_t {
    const KvSeq s = kv_seq(p, b);
    return ((int64_t)s.n * group + kKpRows - 1) / kKpRows * p.c.heads;
  };
  int64_t mine = 0;
  for (int b = tid * per; b < min(p.batch, (tid + 1) * per); ++b) mine += tiles_of(b);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  for (int w = 0; w < warp; ++w) incl += s_scan[w];
  int64_t all = 0;
  for (int w = 0; w < kKpThreads / 32; ++w) all += s_scan[w];
  // the last wave's tiles: `share` CTAs each, where the grid has room for them
  // (row ranges that overlap make more tiles than it was sized for: those past
  // it stay undone and are reported)
  const int64_t whole = all / p.sms * p.sms;
  const int rest = (int)(all - whole);
  int share = rest ? p.sms / rest : 1;
  if (whole + (int64_t)rest * share > gridDim.x) share = 1;
  if (all > gridDim.x && tid == 0) raise_status(p.status, Q4_STATUS_INDEX);
  int64_t x = blockIdx.x;
  const int part = x < whole ? 0 : (int)((x - whole) % share);
  const int slot = (int)max((int64_t)0, x - whole) / share;  // which of the last wave's tiles
  if (x >= whole) x = whole + (x - whole) / share;
  if (x >= incl - mine && x < incl) {
    int64_t at = incl - mine;
    int b = tid * per;
    while (x >= at + tiles_of(b)) at += tiles_of(b++);
    const int rt = (int)(tiles_of(b) / p.c.heads);
    s_where[0] = b;
    s_where[1] = (rt - 1 - (int)((x - at) / p.c.heads)) * kKpRows;
    s_where[2] = (int)((x - at) % p.c.heads);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)s_tmem);
  const int b = s_where[0], r0 = s_where[1], hk = s_where[2];
  volatile int *abort = &s_abort;
  KvSeq sq = {0, 0, 0};
  int rows = 0, tiles = 0, tile0 = 0, lo_first = 0, hi_last = 0;  // keys some row attends to
  int lo_all = 0, hi_all = 0;                                    // keys all rows do
  if (b >= 0) {
    sq = kv_seq(p, b);
    rows = min(kKpRows, sq.n * group - r0);
    const int p0 = sq.len - sq.n, i0 = r0 / group, i1 = (r0 + rows - 1) / group;
    lo_first = p.window ? max(0, p0 + i0 - p.window + 1) : 0;
    hi_last = p.causal ? min(sq.len, p0 + i1 + 1) : sq.len;
    lo_all = p.window ? max(0, p0 + i1 - p.window + 1) : 0;
    hi_all = p.causal ? min(sq.len, p0 + i0 + 1) : sq.len;
    tile0 = lo_first / kKpKeys;
    tiles = max(0, (hi_last + kKpKeys - 1) / kKpKeys - tile0);
  }
  // s (q - z) has up to 15 bits, binary16 holds 11.  The output is rounded to
  // 16 bits itself and hardly shows it (relative error 2.1e-4 with exact keys,
  // 2.3e-4 with rounded ones, binary16), but the log sum exp does: 2e-6 over
  // 2000 keys, 2e-4 over one.  Where it is asked for, the remainders are
  // multiplied too: 1e-7.  Values and weights are rounded to binary16 in any
  // case, since the product takes no wider operands at its rate: binary16
  // outputs are off by 2.5e-4 to 2.9e-4, 2.1e-4 with all in binary32.
  const bool exact = p.lse != nullptr;
  // this CTA's part of the keys
  const int parts = (int)blockIdx.x < whole ? 1 : max(1, min(share, tiles / kKpMinTiles));
  if (part >= parts) {
    rows = 0;  // not needed: it ends like a CTA past the last tile
    tiles = 0;
  } else {
    const int from = (int)((int64_t)tiles * part / parts);
    tiles = (int)((int64_t)tiles * (part + 1) / parts) - from;
    tile0 += from;
  }
  tiles = uniform(tiles);
  const uint32_t s_addr = tmem, o_addr = tmem + 256;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int half = warp >> 2;
    const int rl = tid & 127;                 // row within the half: its lane of tensor memory
    const int r = half * 128 + rl, row = r0 + r;
    const bool real = r < rows;
    const int i = row / group, h = hk * group + row % group;
    const int p0 = sq.len - sq.n;
    const int hi = p.causal ? min(sq.len, p0 + i + 1) : sq.len, lo = p.window ? max(0, p0 + i - p.window + 1) : 0;
    float hf = 0.0f;
    // the query row: scaled into binary16, words in the cache's order, nibble
    // order within a word
    {
      const uint16_t *q = p.Q + (int64_t)(sq.q0 + i) * p.q_ts + (int64_t)h * p.q_hs;
      float top = 0.0f;
      uint4 raw[W];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        raw[w] = make_uint4(0, 0, 0, 0);
        if (real) raw[w] = __ldcg(reinterpret_cast<const uint4 *>(q + (w % NB) * B + 8 * (w / NB)));
        const uint32_t u[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(lo16<DT>(u[e])), fabsf(hi16<DT>(u[e]))));
      }
      const int ex = top > 0.0f ? max((int)(__float_as_uint(top) >> 23) - 127, -110) : 0;
      // 2^(14 - ex), with the scale's sign: scores then grow with the products
      const float up = copysignf(__uint_as_float((uint32_t)(127 + 14 - ex) << 23), p.scale);
      hf = fmaxf(ldexpf(fabsf(p.scale) * 1.4426950408889634f, ex - 14), 1e-37f);
      uint8_t *dst = s_qt + half * Sh::kTile + rl * 128;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const uint32_t u[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[2 * e] = lo16<DT>(u[e]) * up, f[2 * e + 1] = hi16<DT>(u[e]) * up;
        uint4 o;
        o.x = Dt<Q4_F16>::pack2(f[0], f[4]);
        o.y = Dt<Q4_F16>::pack2(f[1], f[5]);
        o.z = Dt<Q4_F16>::pack2(f[2], f[6]);
        o.w = Dt<Q4_F16>::pack2(f[3], f[7]);
        *reinterpret_cast<uint4 *>(dst + (w >> 3) * (kKpKeys * 128) + (((w & 7) ^ (rl & 7)) << 4)) = o;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(half, 0));
    }
    const uint32_t st = s_addr + (uint32_t)(half * 128) + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ot = o_addr + (uint32_t)(half * D) + ((uint32_t)((warp & 3) * 32) << 16);
    float m = -INFINITY, l = 0.0f;
    const uint64_t hf2 = f2_pack(hf, hf);
    const float lift = kp_lift(tiles * kKpKeys);
    bool ok = true, fresh = true;  // fresh: a row of the warp has no reference yet
    for (int j = 0; j < tiles && ok; ++j) {
      // the whole warp goes on or none of it: what follows are its collectives
      if (!__all_sync(0xffffffffu, mbar_wait(s_full(half), j & 1, p.status, abort, p.wait_ns))) {
        ok = false;
        break;
      }
      __syncwarp();
      tc_fence_after();
      const int key0 = (tile0 + j) * kKpKeys;
      // 64 keys at a time: the first product starts while the second half's
      // weights are made
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t s[2][32];
        tmem_ld32(st + 64 * u, s[0]);
        tmem_ld32(st + 64 * u + 32, s[1]);
        const uint4 bad4 = s_bad[j & 3];
        const uint32_t bad[2] = {u ? bad4.z : bad4.x, u ? bad4.w : bad4.y};
        const bool masked = key0 < lo_all || key0 + kKpKeys > hi_all || (bad[0] | bad[1]) != 0;
        auto mask = [&] {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int from = lo - key0 - 64 * u - 32 * c, to = hi - key0 - 64 * u - 32 * c;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (k < from || k >= to || ((bad[c] >> k) & 1u)) s[c][k] = 0xFF800000u;  // -inf
          }
        };
        tmem_wait_ld();
        if (masked) mask();
        uint32_t w[32];  // the weights, pairs of keys
        float sum;
        auto weigh = [&] {
          const float mm = m == -INFINITY ? 0.0f : -m;
          const uint64_t mm2 = f2_pack(mm, mm);
          uint64_t l2[2] = {0, 0};  // two packed sums
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            float x, y;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[k >> 4][2 * (k & 15)]), __uint_as_float(s[k >> 4][2 * (k & 15) + 1])), hf2, mm2), x, y);
            x = ex2(x), y = ex2(y);
            l2[k & 1] = f2_add(l2[k & 1], f2_pack(x, y));
            w[k] = Dt<Q4_F16>::pack2(x, y);
          }
          float x, y;
          f2_unpack(f2_add(l2[0], l2[1]), x, y);
          sum = x + y;
        };
        // the reference of the keys before serves as long as no weight leaves
        // binary16, which the row's sum of weights tells; else (and for the
        // first keys) it moves to the maximum
        bool move = m == -INFINITY;
        if (!fresh) {
          weigh();
          move = !(sum <= kKpMost);
        }
        if (__any_sync(0xffffffffu, move)) {
          if (!fresh) {  // the scores again: their registers held the exponents
            tmem_ld32(st + 64 * u, s[0]);
            tmem_ld32(st + 64 * u + 32, s[1]);
            tmem_wait_ld();
            if (masked) mask();
          }
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < 64; ++k) top = fmaxf(top, __uint_as_float(s[k >> 5][k & 31]));
          top *= hf;
          if (fresh) move = !(top <= m + kKpAhead);
          top = fmaxf(m, top - lift);
          const float f = !move || m == -INFINITY ? 1.0f : ex2(m - top);
          if (move) m = top, l *= f;
          if ((j | u) && __any_sync(0xffffffffu, f != 1.0f)) {
            // the output so far takes the new reference, once its last product is in
            ok = __all_sync(0xffffffffu, mbar_wait(pv_done(half, 1 - u), (j - 1 + u) & 1, p.status, abort, p.wait_ns));
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(ot + 16 * c, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(ot + 16 * c, o);
            }
          }
          weigh();
          fresh = __any_sync(0xffffffffu, m == -INFINITY);
        }
        l += sum;
        tmem_st16(st + 32 * u, w);
        tmem_st16(st + 32 * u + 16, w + 16);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(half, u));
      }
    }
    // ---- the row's output ----
    if (ok && tiles > 0) ok = mbar_wait_warp(pv_done(half, 1), (tiles - 1) & 1, p.status, abort, p.wait_ns);
    tc_fence_after();
    const int64_t at = (int64_t)(sq.q0 + i) * p.q_heads + h;
    auto finish = [&](int c, const float (&o)[32], float inv) {  // columns 32 c .. of the row
#pragma unroll
      for (int v = 0; v < 4; ++v) {  // word 4 c + v of the row
        const int w = 4 * c + v;
        uint4 out;
        out.x = Dt<DT>::pack2(o[8 * v] * inv, o[8 * v + 2] * inv);
        out.y = Dt<DT>::pack2(o[8 * v + 4] * inv, o[8 * v + 6] * inv);
        out.z = Dt<DT>::pack2(o[8 * v + 1] * inv, o[8 * v + 3] * inv);
        out.w = Dt<DT>::pack2(o[8 * v + 5] * inv, o[8 * v + 7] * inv);
        *reinterpret_cast<uint4 *>(p.out + at * D + (w % NB) * B + 8 * (w / NB)) = out;
      }
    };
    auto finish_lse = [&] {
      // (a row whose scores are all NaN has no reference, and the sum NaN)
      if (p.lse) p.lse[at] = l == 0.0f ? -INFINITY : ((m == -INFINITY ? 0.0f : m) + log2f(l)) * 0.69314718055994531f;
    };
    auto output = [&](int c, float (&o)[32]) {  // columns 32 c .. from tensor memory
      uint32_t t[32];
      if (tiles > 0) {
        tmem_ld32(ot + 32 * c, t);
        tmem_wait_ld();
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = tiles > 0 ? __uint_as_float(t[e]) : 0.0f;
    };
    if (ok && rows > 0 && parts == 1) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        output(c, o);
        if (l == 0.0f)
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.0f;
        if (real) finish(c, o, inv);
      }
      if (real) finish_lse();
    } else if (rows > 0 && parts > 1) {  // after a timeout too: all warps meet
      // one of several parts: [part][D / 4][256 rows] float4, then (m, l)
      constexpr int kPart = kKpRows * (D + 2);
      float *base = p.parts + (int64_t)(slot * share) * kPart;
      float4 *mine4 = reinterpret_cast<float4 *>(base + part * kPart) + r;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        output(c, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) __stcg(mine4 + (8 * c + e) * kKpRows, make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
      }
      __stcg(reinterpret_cast<float2 *>(base + part * kPart + kKpRows * D) + r, make_float2(m, l));
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (tid == 0) {
        __threadfence();  // the part (ordered by the barrier) before its count
        const unsigned old = atomicAdd(p.counts + slot, 1u);
        s_where[3] = old == (unsigned)(parts - 1);
        if (s_where[3]) p.counts[slot] = 0u;
        __threadfence();
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (s_where[3]) {
        m = -INFINITY;
        for (int k = 0; k < parts; ++k)
          m = fmaxf(m, __ldcg(reinterpret_cast<const float2 *>(base + k * kPart + kKpRows * D) + r).x);
        l = 0.0f;
        for (int k = 0; k < parts; ++k) {
          const float2 ml = __ldcg(reinterpret_cast<const float2 *>(base + k * kPart + kKpRows * D) + r);
          l = fmaf(ml.y, ml.x == -INFINITY ? 0.0f : ex2(ml.x - m), l);
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.0f;
#pragma unroll 1
          for (int k = 0; k < parts; ++k) {
            const float mk = __ldcg(reinterpret_cast<const float2 *>(base + k * kPart + kKpRows * D) + r).x;
            const float f = mk == -INFINITY ? 0.0f : ex2(mk - m);
            const float4 *src = reinterpret_cast<const float4 *>(base + k * kPart) + r;
            float4 t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = ldcg_v4(reinterpret_cast<const float *>(src + (8 * c + e) * kKpRows));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              o[4 * e] = fmaf(t[e].x, f, o[4 * e]), o[4 * e + 1] = fmaf(t[e].y, f, o[4 * e + 1]);
              o[4 * e + 2] = fmaf(t[e].z, f, o[4 * e + 2]), o[4 * e + 3] = fmaf(t[e].w, f, o[4 * e + 3]);
            }
          }
          if (real) finish(c, o, inv);
        }
        if (real) finish_lse();
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ dequantize
    const int kk = tid - 256;  // key of a tile
    const int pages = (int)(p.c.slots >> p.c.page_log2), page_mask = (1 << p.c.page_log2) - 1;
    const int32_t *table = b >= 0 ? p.table + (int64_t)b * p.table_stride : nullptr;
    constexpr int kNone = INT_MIN;
    auto page_of = [&](int j) -> int {  // table entry of this thread's key of tile j
      const int key = (tile0 + j) * kKpKeys + kk;
      if (j >= tiles || key >= hi_last || key < lo_first) return kNone;
      return __ldg(table + (key >> p.c.page_log2));
    };
    constexpr int V4 = D / 32;
    uint4 raw[2][V4];      // codes of the key and of the value
    uint32_t state[2][NB];
    bool bad_page = false, there = false;
    auto load = [&](int j, int pg) {
      const int key = (tile0 + j) * kKpKeys + kk;
      there = pg >= 0 && pg < pages;
      bad_page = !there && pg != kNone;
      if (bad_page) raise_status(p.status, Q4_STATUS_INDEX);
      // a key that may not be read takes page 0's codes (they are finite) and
      // a zero state
      const int64_t vec = ((int64_t)((there ? pg : 0) * p.c.heads + hk) << p.c.page_log2) + (key & page_mask);
      const uint4 *c0 = reinterpret_cast<const uint4 *>(p.c.codes[0] + vec * (D / 2));
      const uint4 *c1 = reinterpret_cast<const uint4 *>(p.c.codes[1] + vec * (D / 2));
#pragma unroll
      for (int v = 0; v < V4; ++v) raw[0][v] = __ldg(c0 + v), raw[1][v] = __ldg(c1 + v);
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int n = 0; n < NB; ++n) state[w][n] = there ? __ldg(p.c.state[w] + vec * NB + n) : 0u;
    };
    auto store = [&](auto remainder, int which, int stage, bool poison) {
      // the row's base with the swizzle's XOR in it: chunk c lies at base ^ 16 c
      const uint32_t dst = smem_u32(s_kv + (stage * 2 + which) * Sh::kTile + kk * 128) + ((kk & 7) << 4);
      const uint32_t to_rest = rest_of(stage);
      __half2 s[NB], z64[NB], z1024[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const __half2 sz = *reinterpret_cast<const __half2 *>(&state[which][n]);
        s[n] = __low2half2(sz);
        if (poison) s[n] = __half2half2(__ushort_as_half(which == 0 ? 0x7FFF : 0));
        z64[n] = kv_z64(sz);
        z1024[n] = kv_z1024(sz);
      }
#pragma unroll
      for (int v = 0; v < V4; ++v) {
        const uint32_t w4[4] = {raw[which][v].x, raw[which][v].y, raw[which][v].z, raw[which][v].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int w = 4 * v + e, n = w % NB;
          const uint32_t at = (dst ^ ((w & 7) << 4)) + (w >> 3) * (kKpKeys * 128);
          const KvDiff d = kv_diff(w4[e], z64[n], z1024[n]);
          st_shared_v4(at, kv_scaled(d, s[n]));
          if constexpr (decltype(remainder)::value) st_shared_v4(at + to_rest, kv_rest(d, s[n]));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    auto tiles_in = [&](auto exact_tag) {
      if (tiles > 0) load(0, page_of(0));
      int pg_next = page_of(1);
      for (int j = 0; j < tiles && !p.stall_copies; ++j) {
        const int st = j & 1;
        // a value that is not finite must not meet the zero weights of rows that
        // do not attend to it: it becomes zero, and its key NaN, so that the rows
        // that do attend give NaN
        bool poison = false;
#pragma unroll
        for (int n = 0; n < NB; ++n) poison |= (state[1][n] & 0x7C00u) == 0x7C00u;
        const uint32_t bad = __ballot_sync(0xffffffffu, bad_page);
        if (lane == 0) reinterpret_cast<uint32_t *>(&s_bad[j & 3])[warp - 8] = bad;
        if (!mbar_wait_warp(k_empty(st), ((j >> 1) & 1) ^ 1, p.status, abort, p.wait_ns)) break;
        // the tile before has been multiplied, its remainders too
        if (exact_tag && j > 0 && !mbar_wait_warp(k_empty(st ^ 1), ((j - 1) >> 1) & 1, p.status, abort, p.wait_ns)) break;
        store(exact_tag, 0, st, poison);
        if (lane == 0) mbar_arrive(k_full(st));
        if (!mbar_wait_warp(v_empty(st), ((j >> 1) & 1) ^ 1, p.status, abort, p.wait_ns)) break;
        store(std::false_type{}, 1, st, poison);
        if (lane == 0) mbar_arrive(v_full(st));
        if (j + 1 < tiles) load(j + 1, pg_next);
        pg_next = page_of(j + 2);
      }
    };
    if (exact) tiles_in(std::true_type{});
    else tiles_in(std::false_type{});
  } else {
    if (warp == 12) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t id_s = umma_idesc_f16(0, 128, kKpKeys);
      constexpr uint32_t id_o = umma_idesc_f16(0, 128, D) | kUmmaTransposeB;
      const uint32_t q0 = smem_u32(s_qt), kv0 = smem_u32(s_kv);
      const uint32_t lead = lane == 0;
      const uint32_t dq = desc_lo_k(q0), dk = desc_lo_k(kv0), dv = desc_lo_mn(kv0 + Sh::kTile, kKpKeys * 128);
      auto scores = [&](auto exact_tag, int half, int st) {
        const uint32_t a0 = dq + half * (Sh::kTile >> 4), b0 = dk + st * (2 * Sh::kTile >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * (kKpKeys * 128) + (k & 3) * 32) >> 4;
          umma_f16_ss(s_addr + half * 128, a0 + off, b0 + off, id_s, k != 0, lead);
        }
        if constexpr (decltype(exact_tag)::value) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * (kKpKeys * 128) + (k & 3) * 32) >> 4;
            umma_f16_ss(s_addr + half * 128, a0 + off, b0 + (rest_of(st) >> 4) + off, id_s, true, lead);
          }
        }
      };
      auto output = [&](int half, int st, int u, bool first) {  // of keys 64 u .. 64 u + 63
        const uint32_t b0 = dv + st * (2 * Sh::kTile >> 4);
#pragma unroll
        for (int k = u * (kKpKeys / 32); k < (u + 1) * (kKpKeys / 32); ++k)
          umma_f16_ts(o_addr + half * D, s_addr + half * 128 + 8 * k, b0 + (2048 * k >> 4), id_o, !first || k != 0, lead);
      };
      auto wait = [&](uint32_t bar, uint32_t par) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, par, p.status, abort, p.wait_ns));
        tc_fence_after();
        return ok;
      };
      bool ok = true;
      uint32_t last_bar = 0, last_par = 0;
      bool committed = false;
      auto commit = [&](uint32_t bar, uint32_t par) {
        umma_commit_lead(bar, lead);
        last_bar = bar, last_par = par, committed = true;
      };
      // (two versions of the loop: one with a test inside took 6 % longer)
      auto products = [&](auto exact_tag) {
        if (tiles > 0) {
          ok = wait(p_full(0, 0), 0) && wait(p_full(1, 0), 0) && wait(k_full(0), 0);  // queries, first keys
          if (ok) {
            scores(exact_tag, 0, 0);
            commit(s_full(0), 0);
            scores(exact_tag, 1, 0);
            commit(s_full(1), 0);
            commit(k_empty(0), 0);
          }
        }
        for (int j = 0; j < tiles && ok; ++j) {
          const int st = j & 1, nx = (j + 1) & 1;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = wait(p_full(half, 0), (j + 1) & 1) && (half || wait(v_full(st), (j >> 1) & 1));
            if (!ok) break;
            output(half, st, 0, j == 0);
            commit(pv_done(half, 0), j & 1);
            ok = wait(p_full(half, 1), j & 1);
            if (!ok) break;
            output(half, st, 1, false);
            commit(pv_done(half, 1), j & 1);
            if (half) commit(v_empty(st), (j >> 1) & 1);
            if (j + 1 < tiles) {
              ok = half || wait(k_full(nx), ((j + 1) >> 1) & 1);
              if (!ok) break;
              scores(exact_tag, half, nx);
              commit(s_full(half), (j + 1) & 1);
              if (half) commit(k_empty(nx), ((j + 1) >> 1) & 1);
            }
          }
        }
      };
      if (exact) products(std::true_type{});
      else products(std::false_type{});
      // every MMA issued completes before TMEM is freed, also after a timeout
      if (committed) {
        volatile int no_abort = 0;
        mbar_wait(last_bar, last_par, nullptr, &no_abort);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

}  // namespace q4
