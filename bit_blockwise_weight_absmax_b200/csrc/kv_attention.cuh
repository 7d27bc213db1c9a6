// kv_attention.cuh -- softmax(scale Q K^T) V over the paged 4-bit cache: the
// kernel for single and few query rows (sm_100a).
//
// What it cannot do without are the cache's bytes (D + 8 D / B per key and
// head); instructions come close behind (637 a warp and 32 keys, in 0.45 of the
// issue slots), so the codes go into the tensor cores as they are.
//  - A 4-bit code masked out of a packed word is a binary16 number already:
//    w & 0x000f000f holds two codes as multiples of 2^-24 (binary16
//    subnormals, which the MMAs take exactly), w & 0x00f000f0 two more times
//    16.  Eight codes cost 5 integer instructions and no conversion.  The
//    factors 2^24 and 16 go into the query and the output.
//  - s (q - z) = s q - s z: per block, score = s_k (acc - z_k sum(Q)), and the
//    values' scale goes into the weights: w = p s_v, O = sum w code - sum w z_v.
//  - mma.sync m16n8k16, keys on the 16-row side, query rows (8 or 16 of the
//    rows that share a kv head) on the 8-column side.  The contraction over d
//    may run in any order, so a lane takes the words of a row as they lie.
//  - Online softmax in base 2 with a running reference m, kKvLift below the
//    maximum of score + log2(s_v), so that the weights w = 2^(score - m) s_v use
//    binary16's range well whatever the values' sizes: the largest is 2^10 when
//    m is taken, and weights have all of binary16's bits down to 2^-24 of it and
//    are dropped below 2^-35 (with the largest at 1, 131072 keys at 2^-25 counted
//    in the sum and not in the output).  m moves only when a weight passes the
//    range (a packed maximum finds it), which is rare after the first
//    unit: no reduction over lanes and no rescaling in the common case.  The
//    zero-points' sum is one more MMA with the weights.  Query rows are scaled
//    by a power of two into binary16 (exact for both 16-bit types down to 2^-38
//    of the row's largest).
// Work: the (sequence, row tile, kv head) segments, each in units of 32 keys,
// are one list that is cut into equal runs, one per CTA, whatever the lengths;
// a CTA's 8 warps take its units in turn, each with its own ring of bulk
// copies.  Warps join through shared memory; a segment's CTAs join through the
// workspace, the last to arrive in the order of the keys.  (tcgen05 has no
// tile below 128 rows on the key side that would pay for 8 query rows, and
// needs dequantized operands in shared memory; here registers feed the MMAs.)
// Measured: 100 keys 8.7 us; 16 sequences of up to 8192 keys, 64 heads over 8,
// 43 us (2.4 TB/s); 131071 keys 55 us (2.8 TB/s); about 6 us before the first
// unit and 5 for a join are fixed, units stream at 4.7 TB/s between them.
#pragma once
#include <limits.h>

#include "gemm.cuh"  // PTX wrappers, bounded waits
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
  unsigned *counts;  // [CTA] arrivals at the segment that the CTA is the first of, zero between calls
  float *parts;      // [CTA][first or last segment][kPart] results of cut segments
  uint64_t wait_ns;
  int32_t sms;
  int32_t stall_copies;  // test hook: no keys and values are brought in
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

constexpr int kKvUnit = 32;    // keys per unit
constexpr int kKvWarps = 8;
// Of a segment in units of the list, beside its units: its begin and join (us
// at 16 / 24 / 32 / 40: 16 sequences 46.0 / 45.6 / 45.1 / 46.1, 24 of five
// drafted tokens 24.4 / 21.5 / 20.6 / 18.6, 64 of 4096 keys 71 / 68 / 69 / 71).
constexpr int kKvSegmentCost = 32;
// Segments of up to this many units a warp are not cut, where there are CTAs
// enough (us, whole / cut: one sequence of 500 keys 10.7 / 13.3, of 777 13.5 /
// 13.4, four of up to 100 9.6 / 13.4; a join costs what four more units do).
constexpr int kKvWholeTurns = 3;
constexpr float kKvLift = 10.0f;  // the largest weight when the reference is taken: 2^10, six binades below binary16's end
constexpr float kKvMasked = -3.4028235e38f;  // in the place of a score that does not count
constexpr int kKvAttnThreads = kKvWarps * 32;
constexpr size_t kKvCountBytes = Q4_WORKSPACE_HEAD;

template <int D, int B, int NT> struct KvShape {
  static constexpr int NB = D / B, R = 8 * NT;
  static constexpr int kCodes = kKvUnit * D / 2, kState = kKvUnit * NB * 4;  // bytes of K or V in a unit
  static constexpr int kStage = 2 * (kCodes + kState);
  static constexpr int kCtas = NT == 1 ? 2 : 1;  // per SM: two column tiles need more than 128 registers
  static constexpr int kStages = NT == 1 ? 2 : 4;
  static constexpr int kQRow = D * 2 + 16;   // bytes of a query row in shared memory
  static constexpr int kORow = D + 4;        // floats of an output row
  static constexpr int kFactors = 4 * kORow > 320 ? 4 * kORow : 320;  // most CTAs of a segment
  static constexpr int kRing = kKvWarps * kStages * kStage;
  static constexpr int kSmem = kRing + R * kQRow + R * kFactors * 4 + 2 * kKvWarps * R * 4;
  static constexpr int kPart = R * (D + 2);  // floats of a partial result: O, then M and l
  static constexpr int kRowsPerWarp = (R + kKvWarps - 1) / kKvWarps;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// Transposes an 8 x 8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float2 half_pair(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
// Issued where it stands: a batch of them is on its way at once.
__device__ __forceinline__ float4 ldcg_v4(const float *p) {
  float4 r;
  asm volatile("ld.global.cg.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ void kv_bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
      "r"(bytes), "r"(bar)
      : "memory");
}

// After a wait that ran out: waits for the `n` stages from use `no` on, whose
// copies are on their way, so that they have landed before the CTA ends.
static __device__ __noinline__ void kv_drain(uint32_t bar, uint32_t no, int n, int stages) {
  volatile int no_abort = 0;
  for (int s = 0; s < n; ++s) mbar_wait(bar + 8 * ((no + s) % stages), ((no + s) / stages) & 1, nullptr, &no_abort);
}

// a / b for a >= 0, b > 0: in 32 bits where they are enough.
__device__ __forceinline__ int64_t kv_div(int64_t a, int b) {
  return (uint64_t)a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

__device__ __forceinline__ int64_t kv_div64(int64_t a, int64_t b) {
  return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The units of sequence b: u0 .. u0 + units - 1 (at least one where it has
// rows, so that empty rows are written) for each of rt row tiles.
struct KvSpan {
  KvSeq s;
  int u0, units, rt;
  int cost;  // units in the list: those, and kKvSegmentCost for a segment's begin and join
};
template <int R> __device__ __forceinline__ KvSpan kv_span(const KvAttnParams &p, int b, int group) {
  KvSpan v;
  v.s = kv_seq(p, b);
  v.rt = (int)(((int64_t)v.s.n * group + R - 1) / R);
  const int lo = p.window ? max(0, v.s.len - v.s.n - p.window + 1) : 0;
  v.u0 = lo / kKvUnit;
  v.units = v.s.n > 0 ? max(1, (v.s.len + kKvUnit - 1) / kKvUnit - v.u0) : 0;
  v.cost = v.s.n > 0 ? v.units + kKvSegmentCost : 0;
  return v;
}

// What a warp keeps of its query rows over a segment: columns 8 n + 2 t + e.
template <int D, int B, int NT> struct KvRun {
  static constexpr int NB = D / B;
  float o[NT][D / 16][4];           // output^T: rows d, columns query rows
  float zs[NT][NB][4];              // sum w z per block (all rows alike)
  float m[NT][2], l[NT][2];         // reference (-inf before the first key), sum of 2^(score - m)
  float hf[NT][2], qs[NT][NB][2];   // score factor, the query's block sums
  bool pending;                     // a row has no reference yet
};

// One unit: 32 keys whose codes and states lie in shared memory.  inside: all
// of them count for every row; else hi, lo (in shared memory) bound a row's
// keys, and hi_any, lo_any and parts say which keys can be read at all.
template <int D, int B, int NT, bool inside>
__device__ __forceinline__ void kv_unit(KvRun<D, B, NT> &run, const uint8_t *kc, const uint8_t *s_q, const int *s_hi,
                                        const int *s_lo, int key0, int lane, bool first, int hi_any, int lo_any,
                                        uint32_t parts, int part_log2) {
  using Sh = KvShape<D, B, NT>;
  constexpr int NB = Sh::NB, W4 = D / 32, MT = D / 16;
  const int g = lane >> 2, t = lane & 3;
  const uint8_t *ks = kc + Sh::kCodes, *vc = ks + Sh::kState, *vs = vc + Sh::kCodes;
  // a key can be read: inside the lengths, and its page was there
  auto real_key = [&](int kk) {
    return key0 + kk < hi_any && key0 + kk >= lo_any && ((parts >> (kk >> part_log2)) & 1u);
  };
  float sv[2][2][NB];   // values' scales, [16-key tile][row g, g + 8][block]
  float xs[2][NT][4];   // scores before the factor hf
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    float acc[NT][NB][4];
    uint32_t wa[W4], wb[W4];
    // Inside a sequence the codes themselves: the zero-point's part, taken off
    // afterwards, is some times the score, and the roundings of the sums average
    // out over many keys.  Over few they do not, so units at the ends multiply
    // code - 8, near the differences code - z (one to three keys: log sum exp
    // off by 4e-7 of its size instead of 1.4e-6).
    auto operand = [&](uint32_t w, bool high) -> uint32_t {
      const uint32_t v = w & (high ? 0x00F000F0u : 0x000F000Fu);
      if (inside) return v;
      const uint32_t u = v | 0x64006400u;  // 1024 + v
      const __half2 c = __hadd2(*reinterpret_cast<const __half2 *>(&u), __half2half2(__ushort_as_half(high ? 0xE480 : 0xE408)));
      return *reinterpret_cast<const uint32_t *>(&c);
    };
    const uint8_t *ra = kc + (16 * mt + g) * (D / 2) + t * (W4 * 4);
    if constexpr (W4 == 4) {
      const uint4 a = *reinterpret_cast<const uint4 *>(ra), bb = *reinterpret_cast<const uint4 *>(ra + 8 * (D / 2));
      wa[0] = a.x, wa[1] = a.y, wa[2] = a.z, wa[3] = a.w;
      wb[0] = bb.x, wb[1] = bb.y, wb[2] = bb.z, wb[3] = bb.w;
    } else {
      const uint2 a = *reinterpret_cast<const uint2 *>(ra), bb = *reinterpret_cast<const uint2 *>(ra + 8 * (D / 2));
      wa[0] = a.x, wa[1] = a.y;
      wb[0] = bb.x, wb[1] = bb.y;
    }
#pragma unroll
    for (int w = 0; w < W4; ++w) {
      const int j = w % NB;
      const uint32_t a8 = wa[w] >> 8, b8 = wb[w] >> 8;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 q = *reinterpret_cast<const uint4 *>(s_q + (8 * n + g) * Sh::kQRow + (W4 * t + w) * 16);
        if (w < NB) mma_f16_first(acc[n][j], operand(wa[w], false), operand(wb[w], false), operand(wa[w], true), operand(wb[w], true), q.x, q.y);
        else mma_f16(acc[n][j], operand(wa[w], false), operand(wb[w], false), operand(wa[w], true), operand(wb[w], true), q.x, q.y);
        mma_f16(acc[n][j], operand(a8, false), operand(b8, false), operand(a8, true), operand(b8, true), q.z, q.w);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kk = 16 * mt + g + 8 * h;
      float sk[NB], kz[NB];
      uint32_t ka[NB], va[NB];
      if constexpr (NB == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(ks + kk * 8), w = *reinterpret_cast<const uint2 *>(vs + kk * 8);
        ka[0] = u.x, ka[1] = u.y, va[0] = w.x, va[1] = w.y;
      } else {
        ka[0] = *reinterpret_cast<const uint32_t *>(ks + kk * 4), va[0] = *reinterpret_cast<const uint32_t *>(vs + kk * 4);
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const float2 k2 = half_pair(ka[j]);
        sk[j] = k2.x, kz[j] = inside ? k2.y : k2.y - 8.0f;
        sv[mt][h][j] = half_pair(va[j]).x;
      }
      // NaN where a block of the value could not be held: its key's score is
      // NaN then, and so is the whole row, log sum exp included
      float spoil = sv[mt][h][0] * 0.0f;
      if constexpr (NB == 2) spoil = fmaf(sv[mt][h][1], 0.0f, spoil);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // the zero-point first: it cancels most of the sum of codes
          auto block = [&](int j) {
            const float a = acc[n][j][2 * h + e];
            return fmaf(-kz[j], run.qs[n][j][e], inside ? a : a * 5.9604644775390625e-08f);  // 2^-24, as the codes
          };
          float s = fmaf(sk[0], block(0), spoil);
          if constexpr (NB == 2) s = fmaf(sk[1], block(1), s);
          xs[mt][n][2 * h + e] = s;
        }
    }
    if (!inside) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int kk = 16 * mt + g + 8 * h;
        const bool ok = real_key(kk);
#pragma unroll
        for (int j = 0; j < NB; ++j)
          if (!ok) sv[mt][h][j] = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * n + 2 * t + e;
            if (!ok || key0 + kk >= s_hi[r] || key0 + kk < s_lo[r]) xs[mt][n][2 * h + e] = kKvMasked;
          }
      }
    }
  }
  // the reference moves to kKvLift below the maximum so far of score + log2(s_v)
  auto move = [&] {
    run.pending = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float to = run.m[n][e];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float top = sv[mt][h][0];
            if constexpr (NB == 2) top = fmaxf(top, sv[mt][h][1]);
            const float s = xs[mt][n][2 * h + e];
            if (s != kKvMasked) to = fmaxf(to, fmaf(s, run.hf[n][e], fmaxf(lg2(top), -24.0f) - kKvLift));
          }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
        const float f = run.m[n][e] == -INFINITY ? 0.0f : ex2(run.m[n][e] - to);
        run.m[n][e] = to;
        run.l[n][e] *= f;
#pragma unroll
        for (int j = 0; j < NB; ++j) run.zs[n][j][e] *= f;
#pragma unroll
        for (int m = 0; m < MT; ++m) run.o[n][m][e] *= f, run.o[n][m][2 + e] *= f;
        run.pending |= __any_sync(0xffffffffu, to == -INFINITY) != 0;
      }
  };
  uint32_t ww[2][NT][NB][2];  // weights, pairs of query rows
  float lsum[NT][2];
  auto weigh = [&]() -> uint32_t {  // the largest weight's bits, in either half
    uint32_t top = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float mm[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) mm[e] = run.m[n][e] == -INFINITY ? 0.0f : -run.m[n][e], lsum[n][e] = 0.0f;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float pr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) pr[e] = ex2(fmaf(xs[mt][n][2 * h + e], run.hf[n][e], mm[e]));
          float w[NB][2];
#pragma unroll
          for (int j = 0; j < NB; ++j) w[j][0] = pr[0] * sv[mt][h][j], w[j][1] = pr[1] * sv[mt][h][j];
          if (!inside) {  // a masked weight is zero whatever the key's state holds
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (xs[mt][n][2 * h + e] == kKvMasked) {
                pr[e] = 0.0f;
#pragma unroll
                for (int j = 0; j < NB; ++j) w[j][e] = 0.0f;
              }
          }
          lsum[n][0] += pr[0], lsum[n][1] += pr[1];
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            // rounded to binary16, the MMA's type beside the codes: half a step,
            // 2^-11, as the output's own in binary16 (which is off by 2.1e-4 and
            // 2.3e-4 in the norm, 2.1e-4 and 2.2e-4 with binary32 weights)
            ww[mt][n][j][h] = Dt<Q4_F16>::pack2(w[j][0], w[j][1]);
            top = __vmaxu2(top, ww[mt][n][j][h]);
          }
        }
    }
    return top;
  };
  if (first || !inside || run.pending) move();
  const uint32_t top = weigh();
  if (__any_sync(0xffffffffu, (top & 0xFFFFu) >= 0x7C00u || (top >> 16) >= 0x7C00u)) {  // past binary16
    move();
    weigh();
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) run.l[n][0] += lsum[n][0], run.l[n][1] += lsum[n][1];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    uint32_t bw[NT][NB][2];  // the weights as B operand: key pairs of one query row
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < NB; ++j) bw[n][j][0] = movmatrix(ww[mt][n][j][0]), bw[n][j][1] = movmatrix(ww[mt][n][j][1]);
    // zero-points of keys 2t, 2t + 1 and 2t + 8, 2t + 9, the same in all rows
    uint32_t z[NB][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kk = 16 * mt + 2 * t + 8 * h;
      uint32_t a[NB], c[NB];
      if constexpr (NB == 2) {
        const uint4 u = *reinterpret_cast<const uint4 *>(vs + kk * 8);
        a[0] = u.x, a[1] = u.y, c[0] = u.z, c[1] = u.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(vs + kk * 4);
        a[0] = u.x, c[0] = u.y;
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) z[j][h] = __byte_perm(a[j], c[j], 0x7632u);
    }
    if (!inside) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int kk = 16 * mt + 2 * t + 8 * h;
        const uint32_t keep = (real_key(kk) ? 0xFFFFu : 0u) | (real_key(kk + 1) ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int j = 0; j < NB; ++j) z[j][h] &= keep;
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < NB; ++j) mma_f16(run.zs[n][j], z[j][0], z[j][0], z[j][1], z[j][1], bw[n][j][0], bw[n][j][1]);
    // values: the same keys, this lane's words of each
    constexpr int WS = D / 64;
    uint32_t vw[4][WS];
    const uint8_t *rv = vc + (16 * mt + 2 * t) * (D / 2) + g * (WS * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t *r = rv + ((i & 1) + 8 * (i >> 1)) * (D / 2);
      if constexpr (WS == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(r);
        vw[i][0] = u.x, vw[i][1] = u.y;
      } else {
        vw[i][0] = *reinterpret_cast<const uint32_t *>(r);
      }
    }
#pragma unroll
    for (int ws = 0; ws < WS; ++ws) {
      const int j = ws % NB;
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // elements 0..3, 4..7 of the words
        const uint32_t sel = half ? 0x7632u : 0x5410u;
        const uint32_t a = __byte_perm(vw[0][ws], vw[1][ws], sel), c = __byte_perm(vw[2][ws], vw[3][ws], sel);
        const uint32_t a8 = a >> 8, c8 = c >> 8;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(run.o[n][4 * ws + 2 * half], a & 0x000F000Fu, a & 0x00F000F0u, c & 0x000F000Fu, c & 0x00F000F0u,
                  bw[n][j][0], bw[n][j][1]);
          mma_f16(run.o[n][4 * ws + 2 * half + 1], a8 & 0x000F000Fu, a8 & 0x00F000F0u, c8 & 0x000F000Fu, c8 & 0x00F000F0u,
                  bw[n][j][0], bw[n][j][1]);
        }
      }
    }
  }
}

// A run of units of one segment: a row tile of a sequence and a kv head.
template <int R> struct KvSegment {
  KvSpan v;
  int64_t base;            // the sequence's first unit in the list
  int b, seg, first, count;
  int r0, hk, rows;
  int key0, key_end;                   // keys of the run (key_end: also where no row attends further)
  int hi_all, hi_any, lo_all, lo_any;  // keys that all and that some rows of the tile attend to
  __device__ __forceinline__ void ranges(const KvAttnParams &p, int group) {
    r0 = seg / p.c.heads * R, hk = seg % p.c.heads;
    rows = min(R, v.s.n * group - r0);
    const int i0 = r0 / group, i1 = (r0 + rows - 1) / group;
    hi_all = hi(p, i0), hi_any = hi(p, i1), lo_all = lo(p, i1), lo_any = lo(p, i0);
  }
  __device__ __forceinline__ int hi(const KvAttnParams &p, int i) const {
    return p.causal ? min(v.s.len, v.s.len - v.s.n + i + 1) : v.s.len;
  }
  __device__ __forceinline__ int lo(const KvAttnParams &p, int i) const {
    return p.window ? max(0, v.s.len - v.s.n + i - p.window + 1) : 0;
  }
};

template <int DT, int D, int B, int NT>
__global__ void __launch_bounds__(kKvAttnThreads, KvShape<D, B, NT>::kCtas) kv_attention_kernel(const __grid_constant__ KvAttnParams p) {
  using Sh = KvShape<D, B, NT>;
  constexpr int NB = Sh::NB, R = Sh::R;
  constexpr int MT = D / 16;  // 16-row tiles of the output's d
  pdl_launch_dependents();
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *s_q = smem + Sh::kRing;
  float *s_o = reinterpret_cast<float *>(s_q + R * Sh::kQRow);  // [4][R][kORow], then [R][kFactors]
  float *s_m = s_o + R * Sh::kFactors, *s_l = s_m + kKvWarps * R;
  __shared__ uint64_t s_bar[kKvWarps * Sh::kStages];
  __shared__ float s_hf[R], s_qs[NB][R];
  __shared__ int s_hi[R], s_lo[R];
  __shared__ int64_t s_scan[kKvWarps], s_first[2];
  __shared__ int2 s_segs[kKvWarps];
  __shared__ int s_abort;
  __shared__ unsigned s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int group = p.q_heads / p.c.heads;
  const uint8_t *ring = smem + warp * Sh::kStages * Sh::kStage;
  const uint32_t ring_u = smem_u32(ring);
  const uint32_t bar = smem_u32(s_bar) + warp * Sh::kStages * 8;
  if (lane < Sh::kStages) mbar_init(bar + 8 * lane, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (tid == 0) s_abort = 0;
  pdl_wait();

  // this CTA's run of the list of units: a prefix sum over the sequences (the
  // spans of a batch of up to 256 stay in shared memory)
  __shared__ KvSpan s_span[kKvAttnThreads];
  const int per = (p.batch + kKvAttnThreads - 1) / kKvAttnThreads;
  int64_t mine = 0;
  int my_segs = 0, longest = 0;
  for (int b = tid * per; b < min(p.batch, (tid + 1) * per); ++b) {
    const KvSpan v = kv_span<R>(p, b, group);
    if (per == 1) s_span[b] = v;
    mine += (int64_t)v.rt * p.c.heads * v.cost;
    my_segs = min(my_segs + min(v.rt, 1 << 16) * p.c.heads, 1 << 20);
    longest = max(longest, v.units);
  }
  int64_t incl = mine;
  int incl_segs = my_segs;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    const int v = __shfl_up_sync(0xffffffffu, incl_segs, o);
    if (lane >= o) incl += u, incl_segs = min(incl_segs + v, 1 << 20);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) s_scan[warp] = incl, s_segs[warp] = make_int2(incl_segs, longest);
  __syncthreads();
  int64_t before = 0, total = 0;
  int before_segs = 0, segs = 0;
  for (int w = 0; w < kKvWarps; ++w) {
    if (w < warp) before += s_scan[w], before_segs += s_segs[w].x;
    total += s_scan[w];
    segs += s_segs[w].x, longest = max(longest, s_segs[w].y);
  }
  incl += before;
  if (total == 0) return;
  // all CTAs, or where that leaves less than a unit for each warp, fewer; a
  // multiple of the segments where there are few and that keeps nearly all
  // CTAs: equal ones are then cut alike, and none lies in two pieces of a CTA
  const int grid = min((int)gridDim.x, Sh::kFactors);
  int ctas = (int)min((int64_t)grid, (total + kKvWarps - 1) / kKvWarps);
  // short segments, a CTA for each: as if they all had the longest's cost
  const int uniform = segs <= grid && longest <= kKvWholeTurns * kKvWarps ? longest : 0;
  if (uniform) {
    mine = (int64_t)my_segs * uniform, incl = (int64_t)(before_segs + incl_segs) * uniform, total = (int64_t)segs * uniform;
    ctas = segs;
  } else if (segs <= grid) {
    const int each = (int)min((int64_t)(grid / segs), kv_div(total + kKvWarps * segs - 1, kKvWarps * segs));
    if (each * segs * 16 >= grid * 15 || ctas < grid) ctas = each * segs;
  }
  const int c = blockIdx.x;
  if (c >= ctas) return;
  auto begin_of = [&](int cta) { return kv_div(total * cta, ctas); };
  int64_t x = begin_of(c);
  const int64_t x1 = begin_of(c + 1);
  if (x >= incl - mine && x < incl) s_first[0] = tid * per, s_first[1] = incl - mine;
  __syncthreads();
  const int pages = (int)(p.c.slots >> p.c.page_log2);
  const int page_mask = (1 << p.c.page_log2) - 1;
  const int part_log2 = min(p.c.page_log2, 5);  // keys of a part: a page's, at most a unit's
  constexpr float kLog2e = 1.4426950408889634f;

  KvSegment<R> sg;
  sg.b = (int)s_first[0];
  sg.base = s_first[1];
  auto span_of = [&](int b) {
    KvSpan v = per == 1 ? s_span[b] : kv_span<R>(p, b, group);
    if (uniform) v.cost = uniform;
    return v;
  };
  sg.v = span_of(sg.b);
  // sg: the segment that unit x of the list belongs to, as far as this CTA
  // takes it, and x past it; false where the run has no more
  auto locate = [&]() -> bool {
    while (x < x1) {
      while (x >= sg.base + (int64_t)sg.v.rt * p.c.heads * sg.v.cost) {
        sg.base += (int64_t)sg.v.rt * p.c.heads * sg.v.cost;
        sg.v = span_of(++sg.b);
      }
      sg.seg = (int)kv_div(x - sg.base, sg.v.cost);
      sg.first = (int)((x - sg.base) - (int64_t)sg.seg * sg.v.cost);
      sg.count = (int)min((int64_t)(sg.v.units - sg.first), x1 - x);
      x = min(x1, sg.base + (int64_t)(sg.seg + 1) * sg.v.cost);
      if (sg.count > 0) break;  // else the run began in the segment's own cost
      if (x >= x1) return false;
    }
    sg.ranges(p, group);
    sg.key0 = (sg.v.u0 + sg.first) * kKvUnit;
    sg.key_end = min(sg.hi_any, sg.key0 + sg.count * kKvUnit);
    return true;
  };
  // copies of a unit: lane 4 part + kind copies (codes or states of K or V) a
  // page's part; what does not change is kept per lane
  const int part = lane >> 2, which = lane & 1;
  const bool copier = part < (32 >> part_log2);
  const uint32_t vec_bytes = (lane & 2) ? NB * 4 : D / 2;
  const uint32_t copy_bytes = vec_bytes << part_log2;
  const uint32_t copy_dst = ring_u + which * (Sh::kCodes + Sh::kState) + ((lane & 2) ? Sh::kCodes : 0) + part * copy_bytes;
  const uint8_t *const copy_src = (lane & 2) ? reinterpret_cast<const uint8_t *>(p.c.state[which]) : p.c.codes[which];
  const int key_off = part << part_log2;
  const int32_t *table = nullptr;  // the segment's row of the table
  constexpr int kNoPage = INT_MIN;
  // the table's entry for this lane's part of the unit at `key` (looked at
  // only when the copy is issued, a unit later)
  auto page_of = [&](int key) -> int {
    key += key_off;
    // parts outside what any row attends to may have no page: left out
    if (!copier || key >= sg.key_end || key + (1 << part_log2) <= sg.lo_any) return kNoPage;
    return __ldg(table + (key >> p.c.page_log2));
  };
  uint32_t there = 0;  // bit stage * 2 + part: the part was copied
  bool gave_up = false;  // a wait of this warp ran out: no more copies
  auto issue = [&](int key, int pg, uint32_t no) {
    if (p.stall_copies || gave_up) return;
    const int st = no % Sh::kStages;
    const bool good = pg >= 0 && pg < pages;
    if (!good && pg != kNoPage) raise_status(p.status, Q4_STATUS_INDEX);
    const uint32_t ok = __ballot_sync(0xffffffffu, good);
    const uint32_t parts = (ok & 1u) | ((ok >> 3) & 2u);
    there = (there & ~(3u << (2 * st))) | (parts << (2 * st));
    if (lane == 0) mbar_arrive_expect_tx(bar + 8 * st, (__popc(parts) * 2 * (D / 2 + NB * 4)) << part_log2);
    __syncwarp();
    if (good) {
      const uint64_t vec = ((uint64_t)(uint32_t)(pg * p.c.heads + sg.hk) << p.c.page_log2) + (uint32_t)((key + key_off) & page_mask);
      kv_bulk_load(copy_dst + st * Sh::kStage, copy_src + vec * vec_bytes, copy_bytes, bar + 8 * st);
    }
  };
  uint32_t seq_no = 0;  // stages this warp has used
  int pg_next = kNoPage;
  uint4 q_raw[Sh::kRowsPerWarp];
  // the first units' copies and the query rows of a segment are on their way
  // before the previous one's results are joined
  const int wj = lane % NB, wi = lane / NB;  // the word of a query row this lane prepares
  auto begin = [&] {
    table = p.table + (int64_t)sg.b * p.table_stride;
    int pg[Sh::kStages];
#pragma unroll
    for (int s = 0; s < Sh::kStages; ++s) pg[s] = page_of(sg.key0 + (warp + s * kKvWarps) * kKvUnit);
    pg_next = page_of(sg.key0 + (warp + Sh::kStages * kKvWarps) * kKvUnit);
#pragma unroll
    for (int i = 0; i < Sh::kRowsPerWarp; ++i) {
      const int r = warp + i * kKvWarps, row = sg.r0 + r;
      q_raw[i] = make_uint4(0, 0, 0, 0);
      if (r < sg.rows && lane < D / 8)
        q_raw[i] = __ldcg(reinterpret_cast<const uint4 *>(p.Q + (int64_t)(sg.v.s.q0 + row / group) * p.q_ts +
                                                          (int64_t)(sg.hk * group + row % group) * p.q_hs + wj * B + 8 * wi));
    }
#pragma unroll
    for (int s = 0; s < Sh::kStages; ++s)
      if (warp + s * kKvWarps < sg.count) issue(sg.key0 + (warp + s * kKvWarps) * kKvUnit, pg[s], seq_no + s);
  };
  if (!locate()) return;
  begin();

  while (true) {
    // the query rows, scaled into binary16, in the order of the words, and
    // their sums
#pragma unroll
    for (int i = 0; i < Sh::kRowsPerWarp; ++i) {
      const int r = warp + i * kKvWarps;
      const uint32_t w[4] = {q_raw[i].x, q_raw[i].y, q_raw[i].z, q_raw[i].w};
      float f[8], top = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) f[2 * e] = lo16<DT>(w[e]), f[2 * e + 1] = hi16<DT>(w[e]);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int ex = top > 0.0f ? max((int)(__float_as_uint(top) >> 23) - 127, -110) : 0;
      const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);  // 2^(14 - ex)
      float sum = 0.0f;
      __half hq[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // nibbles 1, 3, 5, 7 of a word are read 16 times their code
        hq[e] = __float2half_rn(f[e] * up);
        sum += __half2float(hq[e]);
        if (e & 1) hq[e] = __float2half_rn(f[e] * up * 0.0625f);
      }
      if (lane < D / 8) {
        auto pk = [&](int a, int b2) { return (uint32_t)__half_as_ushort(hq[a]) | ((uint32_t)__half_as_ushort(hq[b2]) << 16); };
        *reinterpret_cast<uint4 *>(s_q + r * Sh::kQRow + lane * 16) = make_uint4(pk(0, 4), pk(1, 5), pk(2, 6), pk(3, 7));
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        float s = lane < D / 8 && wj == j ? sum : 0.0f;
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) s_qs[j][r] = s * 5.9604644775390625e-08f;  // 2^-24, as the codes
      }
      if (lane == 0) {
        const int i = (sg.r0 + r) / group;
        s_hf[r] = ldexpf(p.scale * kLog2e, 24 - 14 + ex);
        s_hi[r] = sg.hi(p, i), s_lo[r] = sg.lo(p, i);
      }
    }
    __syncthreads();

    KvRun<D, B, NT> acc;
    acc.pending = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
        acc.hf[n][e] = s_hf[r];
#pragma unroll
        for (int j = 0; j < NB; ++j) acc.qs[n][j][e] = s_qs[j][r], acc.zs[n][j][e] = acc.zs[n][j][2 + e] = 0.0f;
        acc.m[n][e] = -INFINITY, acc.l[n][e] = 0.0f;
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc.o[n][m][e] = 0.0f;
    }

    int key = sg.key0 + warp * kKvUnit;
    for (int k = warp; k < sg.count && !gave_up; k += kKvWarps, ++seq_no, key += kKvWarps * kKvUnit) {
      const int st = seq_no % Sh::kStages;
      // the whole warp goes on or none of it: what follows are its collectives
      if (!__all_sync(0xffffffffu, mbar_wait(bar + 8 * st, (seq_no / Sh::kStages) & 1, p.status, &s_abort, p.wait_ns))) {
        gave_up = true;
        if (!p.stall_copies) kv_drain(bar, seq_no, min(Sh::kStages, (sg.count - k + kKvWarps - 1) / kKvWarps), Sh::kStages);
        break;
      }
      const uint32_t parts = (there >> (2 * st)) & 3u;
      const uint8_t *kc = ring + st * Sh::kStage;
      const bool inside = key >= sg.lo_all && key + kKvUnit <= sg.hi_all && parts == (part_log2 == 5 ? 1u : 3u);
      if (inside) kv_unit<D, B, NT, true>(acc, kc, s_q, s_hi, s_lo, key, lane, k == warp, sg.hi_any, sg.lo_any, parts, part_log2);
      else kv_unit<D, B, NT, false>(acc, kc, s_q, s_hi, s_lo, key, lane, k == warp, sg.hi_any, sg.lo_any, parts, part_log2);
      __syncwarp();  // the stage has been read
      if (k + Sh::kStages * kKvWarps < sg.count) issue(key + Sh::kStages * kKvWarps * kKvUnit, pg_next, seq_no + Sh::kStages);
      pg_next = page_of(key + (Sh::kStages + 1) * kKvWarps * kKvUnit);
    }

    // the next segment's copies start while this one's results are joined
    const KvSegment<R> done = sg;
    const bool more = x < x1 && locate();
    if (more) begin();

    // ---- the warps join ----
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) acc.l[n][e] += __shfl_xor_sync(0xffffffffu, acc.l[n][e], o);
        if (g == 0) {
          s_m[warp * R + 8 * n + 2 * t + e] = acc.m[n][e];
          s_l[warp * R + 8 * n + 2 * t + e] = acc.l[n][e];
        }
      }
    __syncthreads();
    auto join_max = [&](int r) {
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kKvWarps; ++w) m = fmaxf(m, s_m[w * R + r]);
      return m;
    };
    {
      auto put = [&](bool add) {
        float *o = s_o + (warp & 3) * R * Sh::kORow;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * n + 2 * t + e;
            const float m = join_max(r);
            const float f = acc.m[n][e] == -INFINITY ? 0.0f : ex2(acc.m[n][e] - m);
#pragma unroll
            for (int ws = 0; ws < D / 64; ++ws) {
              const int j = ws % NB;
              // word (D / 64) g + ws of the row: element 8 i of block j
              const int word = (D / 64) * g + ws, d0 = (word % NB) * B + 8 * (word / NB);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                float2 val;
                val.x = f * fmaf(acc.o[n][4 * ws + q][e], 16777216.0f, -acc.zs[n][j][e]);
                val.y = f * fmaf(acc.o[n][4 * ws + q][2 + e], 1048576.0f, -acc.zs[n][j][e]);
                float2 *dst = reinterpret_cast<float2 *>(o + r * Sh::kORow + d0 + 2 * q);
                if (add) {
                  const float2 old = *dst;
                  val.x += old.x, val.y += old.y;
                }
                *dst = val;
              }
            }
          }
      };
      if (warp >= 4) put(false);
      __syncthreads();
      if (warp < 4) put(true);
      __syncthreads();
    }
    const int units = done.v.units, rows = done.rows;
    const bool whole = done.count == units;
    const int64_t seg0 = done.base + (int64_t)done.seg * done.v.cost;  // the segment's units in the list
    // a run's slot: its first segment, or the one it ends in
    auto part_of = [&](int cta, bool began_before) { return p.parts + ((int64_t)cta * 2 + (began_before ? 1 : 0)) * Sh::kPart; };
    // row r of the tile, elements d .. d + 3, from the sums o, the maximum and l
    auto finish = [&](int r, int d, float4 o, float m, float l) {
      if (r >= rows) return;
      const int i = (done.r0 + r) / group, h = done.hk * group + (done.r0 + r) % group;
      const int64_t at = (int64_t)(done.v.s.q0 + i) * p.q_heads + h;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      uint2 out;
      out.x = Dt<DT>::pack2(o.x * inv, o.y * inv);
      out.y = Dt<DT>::pack2(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2 *>(p.out + at * D + d) = out;
      if (d == 0 && p.lse) p.lse[at] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
    };
    for (int i = tid; i < R * D / 4; i += kKvAttnThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float4 o = *reinterpret_cast<const float4 *>(s_o + r * Sh::kORow + d);
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        const float4 a = *reinterpret_cast<const float4 *>(s_o + (w * R + r) * Sh::kORow + d);
        o.x += a.x, o.y += a.y, o.z += a.z, o.w += a.w;
      }
      const float m = join_max(r);
      float l = 0.0f;
#pragma unroll
      for (int w = 0; w < kKvWarps; ++w) {
        const float mw = s_m[w * R + r];
        l += s_l[w * R + r] * (mw == -INFINITY ? 0.0f : ex2(mw - m));  // 0 * NaN keeps a NaN
      }
      if (whole) {
        finish(r, d, o, m, l);
      } else {
        float *part = part_of(c, begin_of(c) < seg0);
        __stcg(reinterpret_cast<float4 *>(part + r * D + d), o);
        if (d == 0) __stcg(reinterpret_cast<float2 *>(part + R * D) + r, make_float2(m, l));
      }
    }
    if (!whole) {
      // the CTAs of the segment join: counted on the first one's word
      const int c0 = (int)kv_div64((seg0 + 1) * ctas - 1, total), c1 = (int)kv_div64((seg0 + units) * ctas - 1, total);
      __syncthreads();
      if (tid == 0) {
        __threadfence();  // the CTA's results (ordered by the barrier) before its count
        const unsigned old = atomicAdd(p.counts + c0, 1u);
        s_last = old == (unsigned)(c1 - c0);
        if (s_last) p.counts[c0] = 0u;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        const int n = c1 - c0 + 1;
        const bool early = begin_of(c0) < seg0;  // only the first can have begun before the segment
        // a warp for each row: the maximum and sum over the partial results;
        // their factors go to shared memory (s_o is free)
        constexpr int kFactors = Sh::kFactors;
        float *s_f = s_o;
        for (int r = warp; r < R; r += kKvWarps) {
          const float *src = part_of(c0, false) + R * D + 2 * r;
          constexpr int kHold = (Sh::kFactors + 31) / 32;
          float2 ml[kHold];
          float m = -INFINITY, l = 0.0f;
#pragma unroll
          for (int i = 0; i < kHold; ++i) {
            const int a = lane + 32 * i;
            ml[i] = make_float2(-INFINITY, 0.0f);
            if (a < n) ml[i] = __ldcg(reinterpret_cast<const float2 *>(src + (int64_t)(2 * a + (a == 0 && early ? 1 : 0)) * Sh::kPart));
            m = fmaxf(m, ml[i].x);
          }
#pragma unroll
          for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
          for (int i = 0; i < kHold; ++i) {
            const int a = lane + 32 * i;
            const float f = ml[i].x == -INFINITY ? 0.0f : ex2(ml[i].x - m);
            if (a < n) s_f[r * kFactors + a] = f;
            l = fmaf(ml[i].y, f, l);
          }
#pragma unroll
          for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
          if (lane == 0) s_m[r] = m, s_l[r] = l;
        }
        __syncthreads();
        for (int i = tid; i < R * D / 4; i += kKvAttnThreads) {
          const int r = i / (D / 4), d = i % (D / 4) * 4;
          if (r >= rows) continue;
          float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          constexpr int kAhead = 16;  // partial results on their way at once
          const float *src = part_of(c0, false) + r * D + d;
          for (int a0 = 0; a0 < n; a0 += kAhead) {
            float4 po[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
              const int k = min(a0 + a, n - 1);
              po[a] = ldcg_v4(src + (int64_t)(2 * k + (k == 0 && early ? 1 : 0)) * Sh::kPart);
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
              const float f = a0 + a < n ? s_f[r * kFactors + a0 + a] : 0.0f;
              if (a0 + a < n) {
                o.x = fmaf(po[a].x, f, o.x), o.y = fmaf(po[a].y, f, o.y);
                o.z = fmaf(po[a].z, f, o.z), o.w = fmaf(po[a].w, f, o.w);
              }
            }
          }
          finish(r, d, o, s_m[r], s_l[r]);
        }
      }
    }
    if (!more) break;
    __syncthreads();  // shared memory is free for the next segment
  }
}

}  // namespace q4
