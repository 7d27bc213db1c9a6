// kv_cache.cuh -- writing keys and values into the paged 4-bit cache, and
// reading them back as 16-bit floats (sm_100a).
//
// Per block of B elements of a token's head vector (the INT4 asymmetric rule
// with binary16 scales): mn = min(0, min x), mx = max(0, max x),
// s = f16((mx - mn) / 15), z = clamp(rint(-mn / s), 0, 15),
// q = clamp(rint(x / s) + z, 0, 15); x^ = s (q - z).
//
// Both kernels are bound by memory: 4 D bytes of K and V and D + 8 D / B bytes
// of cache per token and head; append, close behind, by issue.  A thread owns
// two pieces of 8 elements of a block (a 16-byte load and a word of codes
// each; with one piece the block's own work, its range, scale and place, was
// done twice as often: 52 us for 37); B / 16 lanes hold a block and find its
// range by shuffles.  A CTA takes adjacent tokens of one head: with slots in
// order its codes and states are contiguous runs of the page.  Calls of many
// tokens give a thread kKvItems of them, whose loads are on their way together.
// 8191 tokens of 32 heads, D = 128: append 37 us (4.6 TB/s; one token a thread
// 43), dequantize 32 us (5.3 TB/s; 34).
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
constexpr int kKvItems = 4;
constexpr float kKvMaxRange = 61440.0f;  // 15 * 4096: s (q - z) stays within binary16

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A thread's place in a vector: pieces of 8 elements at e and e + B / 2 of
// one block, whose words of codes stand at `word` and `word` + step.
template <int D, int B> struct KvPiece {
  static constexpr int TV = D / 16, LB = B / 16;  // threads of a vector, of a block
  int blk, i;
  __device__ __forceinline__ explicit KvPiece(int w) : blk(w / LB), i(w % LB) {}
  __device__ __forceinline__ int at(int h) const { return blk * B + 8 * i + h * (B / 2); }
  __device__ __forceinline__ int word(int h) const { return (i + h * LB) * (D / B) + blk; }
};

// grid: (token groups, heads, K or V)
template <int DT, int D, int B, int ITEMS>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
  pdl_launch_then_wait();
  using Piece = KvPiece<D, B>;
  constexpr int TV = Piece::TV, LB = Piece::LB, NB = D / B, TPB = kKvThreads / TV;
  const int which = blockIdx.z, head = blockIdx.y;
  const Piece me(threadIdx.x % TV);
  const int64_t token0 = (int64_t)blockIdx.x * (TPB * ITEMS) + threadIdx.x / TV;
  const uint16_t *x = p.x[which] + head * p.hs[which];
  int64_t slot[ITEMS];
  uint4 v[ITEMS][2];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int64_t token = token0 + k * TPB;
    slot[k] = token < p.tokens ? __ldg(p.slots + token) : -1;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      v[k][h] = token < p.tokens ? ldg_stream_v4(x + token * p.ts[which] + me.at(h)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    float f[2][8];
    float mn = 0.0f, mx = 0.0f;  // NaN where an element is
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t u[4] = {v[k][h].x, v[k][h].y, v[k][h].z, v[k][h].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) f[h][2 * j] = lo16<DT>(u[j]), f[h][2 * j + 1] = hi16<DT>(u[j]);
#pragma unroll
      for (int j = 0; j < 8; ++j) mn = min_nan(mn, f[h][j]), mx = max_nan(mx, f[h][j]);
    }
#pragma unroll
    for (int o = LB / 2; o >= 1; o >>= 1) {
      mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if (slot[k] < 0) continue;
    if (slot[k] >= p.c.slots) {
      if (threadIdx.x % TV == 0) raise_status(p.status, Q4_STATUS_INDEX);
      continue;
    }
    const float range = __fsub_rn(mx, mn);
    const bool bad = !(range <= kKvMaxRange);
    const float s = __half2float(__float2half_rn(__fdiv_rn(range, 15.0f)));
    uint32_t word[2] = {0, 0};
    float z = 0.0f;
    if (!bad && s != 0.0f) {  // a binary16 s is at least 2^-24: inside div_markstein's range
      const float y = __frcp_rn(s);
      z = fminf(fmaxf(rintf(div_markstein(-mn, s, y)), 0.0f), 15.0f);
      // rint(x / s) + z stands in the low 16 bits of a sum with 1.5 * 2^23 (|x / s|
      // is a few times 15 at most), clamped there to 0 .. 15, two at a time
      const uint64_t yy = f2_pack(y, y), ns = f2_pack(-s, -s), zz = f2_pack(z, z);
      const uint64_t kr = f2_pack(12582912.0f, 12582912.0f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float r0, r1;
          f2_unpack(f2_add(f2_add(div_markstein2(f2_pack(f[h][2 * j], f[h][2 * j + 1]), ns, yy), kr), zz), r0, r1);
          q[j] = __vimin_s16x2_relu(__byte_perm(__float_as_uint(r0), __float_as_uint(r1), 0x5410), 0x000F000Fu);
        }
        const uint32_t a = __byte_perm(q[0], q[1], 0x6240), b = __byte_perm(q[2], q[3], 0x6240);  // even codes, odd codes
        word[h] = __byte_perm(a, b, 0x5410) + 16u * __byte_perm(a, b, 0x7632);
      }
    }
    const int64_t vec = kv_vec(p.c, slot[k], head);
    uint32_t *codes = reinterpret_cast<uint32_t *>(p.c.codes[which]) + vec * (D / 8);
    codes[me.word(0)] = word[0], codes[me.word(1)] = word[1];
    if (me.i == 0) {
      const uint32_t sb = bad ? 0x7FFFu : (uint32_t)__half_as_ushort(__float2half_rn(s));
      p.c.state[which][vec * NB + me.blk] = sb | ((uint32_t)__half_as_ushort(__float2half_rn(z)) << 16);
      if (bad) raise_status(p.status, Q4_STATUS_NONFINITE);
    }
  }
}

// Eight codes of a word as binary16 code - z, pairs in the order of the nibbles
// 04 15 26 37: 1024 + code is one masked OR, the difference exact.
// z64 = -(64 + z), z1024 = -(1024 + z), both pairs.
struct KvDiff {
  __half2 d[4];
};
__device__ __forceinline__ KvDiff kv_diff(uint32_t w, __half2 z64, __half2 z1024) {
  const __half2 sixteenth = __half2half2(__ushort_as_half(0x2C00));  // 1 / 16
  auto h2 = [](uint32_t v) { return *reinterpret_cast<__half2 *>(&v); };
  const uint32_t w8 = w >> 8;
  KvDiff r;
  r.d[0] = __hadd2(h2((w & 0x000F000Fu) | 0x64006400u), z1024);
  r.d[1] = __hfma2(h2((w & 0x00F000F0u) | 0x64006400u), sixteenth, z64);
  r.d[2] = __hadd2(h2((w8 & 0x000F000Fu) | 0x64006400u), z1024);
  r.d[3] = __hfma2(h2((w8 & 0x00F000F0u) | 0x64006400u), sixteenth, z64);
  return r;
}
// Their products with s, rounded once.
__device__ __forceinline__ uint4 kv_scaled(const KvDiff &v, __half2 s) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 r = __hmul2(v.d[i], s);
    o[i] = *reinterpret_cast<const uint32_t *>(&r);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// What that rounding left over: s d minus the rounded product, exact.
__device__ __forceinline__ uint4 kv_rest(const KvDiff &v, __half2 s) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 r = __hfma2(v.d[i], s, __hneg2(__hmul2(v.d[i], s)));
    o[i] = *reinterpret_cast<const uint32_t *>(&r);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// -(64 + z) and -(1024 + z) of a state's word, in pairs.
__device__ __forceinline__ __half2 kv_z64(__half2 state) {
  return __hsub2(__half2half2(__ushort_as_half(0xD400)), __high2half2(state));
}
__device__ __forceinline__ __half2 kv_z1024(__half2 state) {
  return __hsub2(__half2half2(__ushort_as_half(0xE400)), __high2half2(state));
}

struct KvDequantParams {
  KvView c;
  uint16_t *x[2];
  const int64_t *slots;
  int64_t n;
  int *status;
};

template <int DT, int D, int B, int ITEMS>
__global__ void __launch_bounds__(kKvThreads) kv_dequantize_kernel(const __grid_constant__ KvDequantParams p) {
  pdl_launch_then_wait();
  using Piece = KvPiece<D, B>;
  constexpr int TV = Piece::TV, NB = D / B, TPB = kKvThreads / TV;
  const int which = blockIdx.z, head = blockIdx.y;
  const Piece me(threadIdx.x % TV);
  const int64_t row0 = (int64_t)blockIdx.x * (TPB * ITEMS) + threadIdx.x / TV;
  int64_t slot[ITEMS];
  uint32_t word[ITEMS][2], st[ITEMS];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) slot[k] = row0 + k * TPB < p.n ? __ldg(p.slots + row0 + k * TPB) : -1;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    word[k][0] = word[k][1] = st[k] = 0;  // zeros
    if (slot[k] >= p.c.slots) {
      if (threadIdx.x % TV == 0) raise_status(p.status, Q4_STATUS_INDEX);
    } else if (slot[k] >= 0) {
      const int64_t vec = kv_vec(p.c, slot[k], head);
      const uint32_t *codes = reinterpret_cast<const uint32_t *>(p.c.codes[which]) + vec * (D / 8);
      word[k][0] = __ldg(codes + me.word(0)), word[k][1] = __ldg(codes + me.word(1));
      st[k] = __ldg(p.c.state[which] + vec * NB + me.blk);
    }
  }
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int64_t row = row0 + k * TPB;
    if (row >= p.n) break;
    const __half2 sz = *reinterpret_cast<const __half2 *>(&st[k]);
    // binary16: the products themselves; bf16: the exact differences, times s
    // in binary32
    const __half2 s = DT == Q4_F16 ? __low2half2(sz) : __half2half2(__ushort_as_half(0x3C00));
    const __half2 z64 = kv_z64(sz), z1024 = kv_z1024(sz);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 r = kv_scaled(kv_diff(word[k][h], z64, z1024), s);  // pairs 04 15 26 37
      uint4 o;
      if constexpr (DT == Q4_F16) {
        o.x = __byte_perm(r.x, r.y, 0x5410), o.y = __byte_perm(r.z, r.w, 0x5410);
        o.z = __byte_perm(r.x, r.y, 0x7632), o.w = __byte_perm(r.z, r.w, 0x7632);
      } else {
        const float sf = __low2float(sz);
        auto f2 = [](uint32_t v) { return __half22float2(*reinterpret_cast<__half2 *>(&v)); };
        const float2 a = f2(r.x), b = f2(r.y), c = f2(r.z), d = f2(r.w);
        o.x = Dt<DT>::pack2(sf * a.x, sf * b.x), o.y = Dt<DT>::pack2(sf * c.x, sf * d.x);
        o.z = Dt<DT>::pack2(sf * a.y, sf * b.y), o.w = Dt<DT>::pack2(sf * c.y, sf * d.y);
      }
      *reinterpret_cast<uint4 *>(p.x[which] + (row * p.c.heads + head) * D + me.at(h)) = o;
    }
  }
}

}  // namespace q4
