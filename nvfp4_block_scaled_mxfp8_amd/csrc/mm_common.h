// Shared by the kernels on 16-bit operands (grouped products, low-rank adapters, expert dispatch).
#pragma once
#include "device_common.h"
#include "kernels.h"

namespace gmlp {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));

// The two 16-bit operand types: conversions round to nearest even.  mma32_pair is c0 += a0 b, c1 += a1 b
// where I < live (uniform), accumulators in place and the branch inside the asm: written
// as a branch around the builtins, the two paths leave the accumulators in different registers and
// the compiler copies and spills all of them.  The wait states it would put between a product and
// a read of its result are then the caller's: mma32_settle before the first such read.
template <int TYPE>
struct Elem;
template <>
struct Elem<MM_BF16> {
  static __device__ __forceinline__ float up(uint16_t v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ uint16_t down(float f) { return (uint16_t)f32_to_bf16_bits(f); }
  static __device__ __forceinline__ uint32_t down2(float lo, float hi) { return pack_bf16x2(lo, hi); }
  static __device__ __forceinline__ v16f mma32(v4i a, v4i b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  }
  template <int I>
  static __device__ __forceinline__ void mma32_pair(int live, v4i a0, v4i a1, v4i b, v16f& c0, v16f& c1) {
    asm volatile("s_cmp_le_i32 %5, %6\n\ts_cbranch_scc1 L_mma_%=\n\t"
                 "v_mfma_f32_32x32x16_bf16 %0, %2, %4, %0\n\tv_mfma_f32_32x32x16_bf16 %1, %3, %4, %1\n\t"
                 "L_mma_%=:" : "+v"(c0), "+v"(c1) : "v"(a0), "v"(a1), "v"(b), "s"(live), "n"(I) : "scc");
  }
  static __device__ __forceinline__ v4f mma16(v4i a, v4i b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  }
};
template <>
struct Elem<MM_FP16> {
  static __device__ __forceinline__ float up(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ uint16_t down(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
  static __device__ __forceinline__ uint32_t down2(float lo, float hi) {
    return (uint32_t)down(lo) | ((uint32_t)down(hi) << 16);
  }
  static __device__ __forceinline__ v16f mma32(v4i a, v4i b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
  template <int I>
  static __device__ __forceinline__ void mma32_pair(int live, v4i a0, v4i a1, v4i b, v16f& c0, v16f& c1) {
    asm volatile("s_cmp_le_i32 %5, %6\n\ts_cbranch_scc1 L_mma_%=\n\t"
                 "v_mfma_f32_32x32x16_f16 %0, %2, %4, %0\n\tv_mfma_f32_32x32x16_f16 %1, %3, %4, %1\n\t"
                 "L_mma_%=:" : "+v"(c0), "+v"(c1) : "v"(a0), "v"(a1), "v"(b), "s"(live), "n"(I) : "scc");
  }
  static __device__ __forceinline__ v4f mma16(v4i a, v4i b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
};

// The accumulators pass through the asm, so that no use of them can be moved above its 32 wait states (a
// 32x32x16 product takes 16 passes).
__device__ __forceinline__ void mma32_settle(v16f (&c)[4][2]) {
  asm volatile("s_nop 15\n\ts_nop 15 ; settled %0 %1 %2 %3 %4 %5 %6 %7"
               : "+v"(c[0][0]), "+v"(c[0][1]), "+v"(c[1][0]), "+v"(c[1][1]), "+v"(c[2][0]), "+v"(c[2][1]), "+v"(c[3][0]),
                 "+v"(c[3][1]) :: "memory");
}

// ----------------------------------------------------------------------------- loads from any even address
// Eight elements of a row from p, the first `valid` of which exist, zeros behind them, in two steps so
// that many loads can be in flight: load8_raw issues one 16-byte load (the hardware takes any
// alignment; a ragged end is read as the row's last eight elements) and shift8 moves a ragged end
// down.  Rows of fewer than eight elements are read by element (load8_short, no shift).
__device__ __forceinline__ v4i load8_raw(const uint16_t* p, int valid) {
  v4i v{0, 0, 0, 0};
  if (valid > 0) __builtin_memcpy(&v, p - max(8 - valid, 0), 16);
  return v;
}
__device__ __forceinline__ v4i shift8(v4i v, int valid) {
  uint64_t lo = (uint32_t)v.x | ((uint64_t)(uint32_t)v.y << 32), hi = (uint32_t)v.z | ((uint64_t)(uint32_t)v.w << 32);
  const int s = 16 * min(max(8 - valid, 0), 8);
  if (s >= 64) {
    lo = s >= 128 ? 0 : hi >> (s - 64);
    hi = 0;
  } else if (s > 0) {
    lo = (lo >> s) | (hi << (64 - s));
    hi >>= s;
  }
  return v4i{(int)(uint32_t)lo, (int)(uint32_t)(lo >> 32), (int)(uint32_t)hi, (int)(uint32_t)(hi >> 32)};
}
__device__ __forceinline__ v4i load8_short(const uint16_t* p, int valid) {
  uint32_t w[4] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < valid) w[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
  return v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
}

// ----------------------------------------------------------------------------- split sizes
// Every wave walks m_splits by itself, 64 groups at a time (no table, no launch before the
// product, no barrier).  Row counts are clamped like the split scan's: a negative count is 0 and
// the running sum stops at M (M <= 2^30, so the unsigned sums below do not wrap).
struct Span {
  uint32_t start, end;     // rows of this lane's group
};
__device__ __forceinline__ uint32_t wave_incl_add(uint32_t v, int lane, uint32_t cap) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t u = (uint32_t)__shfl_up((int)v, o, 64);
    if (lane >= o) v = min(v + u, cap);
  }
  return v;
}
// Spans of groups [base, base + 64), the rows before them in `done` (updated).
__device__ __forceinline__ Span wave_spans(const int32_t* m_splits, int G, uint32_t M, int base, int lane, uint32_t& done) {
  const int g = base + lane;
  const int raw = g < G ? m_splits[g] : 0;
  const uint32_t m = min((uint32_t)max(raw, 0), M);
  const uint32_t incl = wave_incl_add(m, lane, M);
  const uint32_t prev = (uint32_t)__shfl_up((int)incl, 1, 64);
  Span s;
  s.start = min(done + (lane ? prev : 0u), M);
  s.end = min(done + incl, M);
  done = (uint32_t)__builtin_amdgcn_readlane((int)s.end, 63);
  return s;
}
// The flag word of a call (one wave): bit 0 negative count, bit 1 sum past M, bit 2 sum short of M.
__device__ __forceinline__ uint32_t wave_split_flags(const int32_t* m_splits, int G, int64_t M, int lane) {
  long long sum = 0;
  bool neg = false;
  for (int g = lane; g < G; g += 64) {
    const int v = m_splits[g];
    neg |= v < 0;
    sum += max(v, 0);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
  return (__any(neg) ? 1u : 0u) | (sum > M ? 2u : 0u) | (sum < M ? 4u : 0u);
}

// Output tiles of the row-wise layouts: every group's rows in tiles of `tm`, `ntn` column tiles
// each, and (rest) the rows behind the last group as one more group G.
struct RowTile {
  int g;              // group; G: the rows behind the last one; -1: past the last tile
  uint32_t row0, m;   // the group's first row and its rows
  uint32_t t;         // tile within the group, [0, ceil(m / tm) ntn)
};
__device__ __forceinline__ uint32_t row_tiles_total(const int32_t* m_splits, int G, uint32_t M, uint32_t tm, uint32_t ntn,
                                                    bool rest, int lane) {
  uint32_t done = 0, tiles = 0;
  for (int base = 0; base < G; base += 64) {
    const Span s = wave_spans(m_splits, G, M, base, lane, done);
    uint32_t v = (s.end - s.start + tm - 1) / tm;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += (uint32_t)__shfl_xor((int)v, o, 64);
    tiles += v;
  }
  if (rest) tiles += (M - done + tm - 1) / tm;
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)(tiles * ntn));
}
__device__ __forceinline__ RowTile find_row_tile(const int32_t* m_splits, int G, uint32_t M, uint32_t tm, uint32_t ntn,
                                                 bool rest, uint32_t tile, int lane) {
  RowTile r;
  uint32_t done = 0, before = 0;
  for (int base = 0; base < G; base += 64) {
    const Span s = wave_spans(m_splits, G, M, base, lane, done);
    const uint32_t mine = (s.end - s.start + tm - 1) / tm * ntn;
    const uint32_t incl = wave_incl_add(mine, lane, 0x7FFFFFFFu);
    const uint64_t hit = __ballot(tile < before + incl);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      r.g = base + l;
      r.row0 = (uint32_t)__builtin_amdgcn_readlane((int)s.start, l);
      r.m = (uint32_t)__builtin_amdgcn_readlane((int)s.end, l) - r.row0;
      r.t = tile - before - ((uint32_t)__builtin_amdgcn_readlane((int)incl, l) - (uint32_t)__builtin_amdgcn_readlane((int)mine, l));
      return r;
    }
    before += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
  }
  r.g = G;
  r.row0 = done;
  r.m = M - done;
  r.t = tile - before;
  if (!rest || r.t >= (r.m + tm - 1) / tm * ntn) r.g = -1;
  return r;
}
// Rows of group g.
__device__ __forceinline__ RowTile find_group_rows(const int32_t* m_splits, int G, uint32_t M, int g, int lane) {
  uint32_t done = 0;
  Span s{0, 0};
  for (int base = 0; base <= g; base += 64) s = wave_spans(m_splits, G, M, base, lane, done);
  RowTile r;
  r.g = g;
  r.row0 = (uint32_t)__builtin_amdgcn_readlane((int)s.start, g & 63);
  r.m = (uint32_t)__builtin_amdgcn_readlane((int)s.end, g & 63) - r.row0;
  r.t = 0;
  return r;
}

}  // namespace gmlp
