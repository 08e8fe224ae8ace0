// Grouped products of few rows with weights of 4 bits: y[r] = x[r] w[g]^T.  Bound by the read of the weights
// (half a byte an element and the scales), so a weight is read once, decoded in registers and multiplied on the
// matrix cores.
//
// K is taken in chunks of 128.  Of a chunk a lane loads 16 bytes of a column's codes, 32 elements of one
// row of w: the operand of a product 16 x 16 x 32 holds 8 consecutive elements of a column per lane, the 16
// columns in the lanes of a row of 16, so each of the four words is one product's operand.  Which elements of K
// a product takes together is free as long as x's operand has the same:
//   without scales outside (NVFP4) or with one scale for the chunk: product i has elements 32 q + 8 i + (0..7)
//     of the chunk in lanes 16 q..16 q + 15, as they were loaded;
//   groups of 32 and 64: a product may hold one group only, so the four words of the lanes l, l + 16,
//     l + 32, l + 48 are transposed (four exchanges), and product i has the elements 32 i + 8 q + (0..7).
// Exactness: NVFP4 weights E2M1 x E4M3 have at most 6 significant bits, and integers q - zero at most 5, exact in
// both types; an integer group's sum is taken in fp32 before its scale multiplies it.
#include "block_ops.h"
#include "block_sizes.h"
#include "mm_common.h"
#include "wave_ops.h"

#include <type_traits>

namespace gmlp {

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint16_t v2us __attribute__((ext_vector_type(2)));
typedef int16_t v2ss __attribute__((ext_vector_type(2)));

constexpr int kW4Chunk = sizes::kW4Chunk;

// The four words of lanes l, l + 16, l + 32, l + 48 transposed.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  v2u a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  v2u b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const v2u c = __builtin_amdgcn_permlane16_swap(a.x, b.x, false, false);
  const v2u d = __builtin_amdgcn_permlane16_swap(a.y, b.y, false, false);
  w[0] = c.x;
  w[1] = c.y;
  w[2] = d.x;
  w[3] = d.y;
}

// What a group's codes and sums are multiplied by (s16: the scale's bits in the rows' type R).
//   fp16 operands: zero2 = the pair of -(1024 + zero), sc the scale.
//   bf16 operands: the scale's power of two goes into the integers (exact: they have 5 bits) and the rest, in [1, 2),
//   multiplies their sum, so that sums of the largest and the smallest rows are as large as the result's parts are; the
//   power stays within 2^-126 and 2^123, where 15 times it is a number.
struct IntGroup {
  float sc, pow, zero;
  uint32_t zero2;
};
template <int R, int U>
__device__ __forceinline__ IntGroup int_group(uint32_t s16, uint32_t z) {
  IntGroup o{Elem<R>::up((uint16_t)s16), 1.0f, 0.0f, 0u};
  if constexpr (U == MM_FP16) {
    o.zero2 = 0xE400E400u + z * 0x00010001u;
  } else {
    const uint32_t e = min(max((s16 >> 7) & 255u, 1u), 250u);
    o.pow = __uint_as_float(e << 23);
    o.sc *= __uint_as_float((254u - e) << 23);
    o.zero = -o.pow * (float)z;
  }
  return o;
}
// Eight codes -> eight integers q - zero (bf16: times the group's power of two), exact in 16 bits.  fp16 takes the pairs
// k, k + 4 that a mask leaves in one word: 1024 + q is a number whose last bits are q, and 1024 + 16 q the same four
// bits higher, so a mask, an or and one addition (or one product with 1/16 and addition) of pairs do; x's operand
// is then in that order too (pairs_apart).
template <int U>
__device__ __forceinline__ v4i decode_int(uint32_t w, const IntGroup& g) {
  if constexpr (U == MM_FP16) {
    const v2h low = __builtin_bit_cast(v2h, g.zero2);
    const v2h high = low + v2h{(_Float16)960, (_Float16)960};             // -(64 + zero)
    const v2h sixteenth{(_Float16)0.0625f, (_Float16)0.0625f};
    v4i o;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint32_t v = w >> (4 * i);
      const v2h a = __builtin_bit_cast(v2h, (v & 0x000F000Fu) | 0x64006400u), b = __builtin_bit_cast(v2h, (v & 0x00F000F0u) | 0x64006400u);
      o[i] = __builtin_bit_cast(int, a + low);
      o[i + 1] = __builtin_bit_cast(int, __builtin_elementwise_fma(b, sixteenth, high));
    }
    return o;
  }
  const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  auto pair = [&](int at) {
    return (int)Elem<U>::down2(fmaf((float)((even >> at) & 255u), g.pow, g.zero), fmaf((float)((odd >> at) & 255u), g.pow, g.zero));
  };
  return v4i{pair(0), pair(8), pair(16), pair(24)};
}
// Eight values (0 1)(2 3)(4 5)(6 7) -> (0 4)(1 5)(2 6)(3 7).
__device__ __forceinline__ v4i pairs_apart(v4i v) {
  const uint32_t a = (uint32_t)v.x, b = (uint32_t)v.y, c = (uint32_t)v.z, d = (uint32_t)v.w;
  return v4i{(int)__builtin_amdgcn_perm(c, a, 0x05040100u), (int)__builtin_amdgcn_perm(c, a, 0x07060302u),
             (int)__builtin_amdgcn_perm(d, b, 0x05040100u), (int)__builtin_amdgcn_perm(d, b, 0x07060302u)};
}
// Eight E2M1 codes times an E4M3 block scale, exact in 16 bits.
template <int TYPE>
__device__ __forceinline__ v4i decode_fp4(uint32_t w, float sc) {
  if constexpr (TYPE == MM_BF16)
    return v4i{(int)e2m1x2_scaled_bf16<0>(w, sc), (int)e2m1x2_scaled_bf16<1>(w, sc), (int)e2m1x2_scaled_bf16<2>(w, sc),
               (int)e2m1x2_scaled_bf16<3>(w, sc)};
  const v2h s{(_Float16)sc, (_Float16)sc};
  return v4i{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s),
             __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s),
             __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s),
             __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s)};
}

// ----------------------------------------------------------------------------- few tiles
// A workgroup has 16 rows of one group and 16 NT columns; its waves take a part of K each, a batch of chunks' loads in
// flight at once, and join their sums in LDS.  Of one group with up to 16 rows, a single token's layer, all loads
// are on their way before the split size that says how many rows there are.
// What bounds it is the number of requests, 64 bytes of a row each: one token, 7168 x 4096, groups of 64 (us): no loads 3.1,
// codes 5.2, scales and zeros chunk by chunk 8.8, x 10.5, products 11.4.  So a batch's scales come in one load (10.5 in
// all), and where tiles have many rows, whose part of x is four requests a row and chunk, four column tiles share it
// (32 rows: 29.8 -> 18.9).
template <int KIND, int GROUP, int NT>
struct W4Batch {
  static constexpr bool INT = KIND == W4_INT;
  static constexpr int B = 2;                                  // chunks (four leave one workgroup on a CU: 12.3 us for 10.5)
  static constexpr int NS = INT ? B * kW4Chunk / GROUP : B;    // 16-bit words of scales
  v4i w[B][NT];
  uint32_t s[NT][NS / 2];    // integers: the column's scales in order; NVFP4: the lane's two blocks of each chunk
  uint32_t z[NT][(NS + 3) / 4];
  v4i a[B][4];
};
template <int TYPE, int KIND, int GROUP, int NT>
__global__ __launch_bounds__(512) void w4_split_kernel(W4Args p, uint32_t ntn, int64_t blocks) {
  using E = Elem<TYPE>;
  constexpr bool INT = KIND == W4_INT, TRANS = INT && GROUP < 128, APART = INT && TYPE == MM_FP16;
  constexpr int PER = INT ? kW4Chunk / GROUP : 2;              // scales a lane has in a chunk
  using Batch = W4Batch<KIND, GROUP, NT>;
  constexpr int B = Batch::B, NS = Batch::NS, SLOTS = 4 * NT;
  extern __shared__ float s_sum[];                             // [waves][SLOTS][64]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t block = (int64_t)blockIdx.x + (int64_t)blockIdx.y * p.row_blocks;
  if (block >= blocks) return;
  const int col = lane & 15, q = lane >> 4, N = p.N, K = p.K;
  const int chunks = (K + kW4Chunk - 1) / kW4Chunk;
  const int first = chunks * wave / waves, last = chunks * (wave + 1) / waves;      // waves <= chunks: at least one
  const uint16_t* x;
  const uint8_t* codes[NT];
  int64_t meta[NT];                                            // the column's first scale
  // rows and columns behind the last read the last one's values: a product's row or column reaches its own results only
  auto operands = [&](int g, int64_t row0, int last_row, int n0) {
    x = static_cast<const uint16_t*>(p.x) + (row0 + min(col, last_row)) * p.ldx;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t n = (int64_t)g * N + min(n0 + 16 * j + col, N - 1);
      codes[j] = p.codes + n * (K / 2);
      meta[j] = n * (K / GROUP);
    }
  };
  Batch l;
  auto load = [&](int from) {
    const bool whole = (from + B) * kW4Chunk <= K;
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        l.w[b][j] = *reinterpret_cast<const v4i*>(codes[j] + min((from + b) * (kW4Chunk / 2) + 16 * q, K / 2 - 16));
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (!INT) {
        const uint8_t* s = static_cast<const uint8_t*>(p.scales) + meta[j];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          uint16_t v;
          __builtin_memcpy(&v, s + min((from + b) * 8 + 2 * q, K / 16 - 2), 2);
          l.s[j][b / 2] = b % 2 ? l.s[j][b / 2] | (uint32_t)v << 16 : v;
        }
      } else {
        const int at = from * PER;
        const uint16_t* s = static_cast<const uint16_t*>(p.scales) + meta[j] + at;
        if (whole) {
          __builtin_memcpy(l.s[j], s, 2 * NS);
          if (p.zeros) __builtin_memcpy(l.z[j], p.zeros + meta[j] + at, NS);
        } else {                                               // up to K's end, the last one's again behind it
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const int e = min(i, K / GROUP - 1 - at);
            const uint32_t v = s[e], z = p.zeros ? p.zeros[meta[j] + at + e] : 0;
            l.s[j][i / 2] = i % 2 ? l.s[j][i / 2] | v << 16 : v;
            l.z[j][i / 4] = i % 4 ? l.z[j][i / 4] | z << (8 * (i % 4)) : z;
          }
        }
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __builtin_memcpy(&l.a[b][i], x + min((from + b) * kW4Chunk + (TRANS ? 32 * i + 8 * q : 32 * q + 8 * i), K - 8), 16);
  };
  const bool early = p.G == 1 && p.M <= 16 && block < ntn;
  RowTile tile;
  int n0, rows;
  if (early) {
    n0 = (int)block * (16 * NT);
    operands(0, 0, (int)p.M - 1, n0);
    load(first);
    tile = RowTile{0, 0, (uint32_t)min((int64_t)max(p.m_splits[0], 0), p.M), 0};
    rows = (int)tile.m;
  } else {
    tile = find_row_tile(p.m_splits, p.G, (uint32_t)p.M, 16, ntn, p.zero_rest, (uint32_t)block, lane);
    if (tile.g < 0) return;
    // a column tile's row tiles follow each other: they read the same weights
    const uint32_t nrt = (tile.m + 15) / 16, r0 = tile.t % nrt * 16;
    n0 = (int)(tile.t / nrt) * (16 * NT);
    rows = (int)min(tile.m - r0, 16u);
    tile.row0 += r0;
  }
  uint16_t* y = static_cast<uint16_t*>(p.y) + (int64_t)tile.row0 * p.ldy;
  if (tile.g == p.G || rows == 0) {                            // rows behind the groups; all of them where the one group has none
    const int n = n0 + (int)threadIdx.x % (16 * NT);
    if (n < N && p.zero_rest)
      for (int m = threadIdx.x / (16 * NT); m < (early ? (int)p.M : rows); m += blockDim.x / (16 * NT)) y[(int64_t)m * p.ldy + n] = 0;
    return;
  }
  if (!early) {
    operands(tile.g, tile.row0, rows - 1, n0);
    load(first);
  }
  // NVFP4, bf16 rows: the largest power of two up to 1 / S goes into the block scales, so that products are
  // no larger than those of the weights themselves (above 2^-60: below it they would leave the exact values)
  const float global = INT ? 1.0f : nvfp4_global_scale(p.amax[tile.g]);
  const int down = INT || TYPE != MM_BF16 ? 0 : min(max(ilogbf(global), -126), 59) + 1;
  const float downf = ldexpf(1.0f, -down);
  v4f acc[NT] = {};
  for (int from = first; from < last; from += B) {
    if (from > first) load(from);
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int k0 = (from + b) * kW4Chunk;
      if (from + b >= last) break;
      const bool whole = k0 + kW4Chunk <= K, have = k0 + 32 * q < K;
      if (!TRANS && !whole)                                    // lanes behind K's end: zeros
#pragma unroll
        for (int i = 0; i < 4; ++i) l.a[b][i] = have ? l.a[b][i] : v4i{0, 0, 0, 0};
      if (APART)
#pragma unroll
        for (int i = 0; i < 4; ++i) l.a[b][i] = pairs_apart(l.a[b][i]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const v4i v = l.w[b][j];
        uint32_t w[4] = {(uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w};
        if (TRANS) transpose4(w);
        float sc[PER];
        IntGroup grp[PER];
#pragma unroll
        for (int s = 0; s < PER; ++s) {
          const int at = b * PER + s;
          if (INT) {
            grp[s] = int_group<TYPE, TYPE>((l.s[j][at / 2] >> (16 * (at & 1))) & 0xFFFFu, p.zeros ? (l.z[j][at / 4] >> (8 * (at & 3))) & 255u : 8u);
          } else {
            sc[s] = downf * __builtin_amdgcn_cvt_f32_fp8((int)(l.s[j][b / 2] >> (16 * (b & 1) + 8 * s)), 0);
            if (!whole && !have) sc[s] = 0.0f;
          }
        }
        v4f part = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (TRANS && !whole && k0 + 32 * i >= K) break;
          const int s = INT ? i * 32 / GROUP : i / 2;
          if (!INT) {
            acc[j] = E::mma16(l.a[b][i], decode_fp4<TYPE>(w[i], sc[s]), acc[j]);
          } else {
            part = E::mma16(l.a[b][i], decode_int<TYPE>(w[i], grp[s]), part);
            if ((i + 1) * 32 % GROUP == 0) {
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[j][r] = fmaf(grp[s].sc, part[r], acc[j][r]);
              part = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            }
          }
        }
      }
    }
  }
  // the waves' sums, joined in order
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) s_sum[(wave * SLOTS + 4 * j + r) * 64 + lane] = acc[j][r];
  __syncthreads();
  const float rest = ldexpf(global, -down);
  for (int s = wave; s < SLOTS; s += waves) {
    float v = s_sum[s * 64 + lane];
    for (int o = 1; o < waves; ++o) v += s_sum[(o * SLOTS + s) * 64 + lane];
    if (!INT) v = __fdiv_rn(v, rest);
    const int m = 4 * q + s % 4, n = n0 + s / 4 * 16 + col;
    if (m < rows && n < N) y[(int64_t)m * p.ldy + n] = E::down(v);
  }
}

// ----------------------------------------------------------------------------- many tiles
// Where the tiles alone fill the device: a workgroup has 16 MT rows of one group and 16 columns a wave, and walks K in
// spans of SPAN chunks: a wave's loads of the next span (512 elements of each of its columns) are all in
// flight while it multiplies this one, and x's part of a span lies in LDS for all waves.  What is left of K
// behind the last whole span goes chunk by chunk.
// bf16 rows of a single tile become fp16 on their way into LDS, times a power of two by row and span that brings the
// span's largest to [2^14, 2^15): the same value as long as the smallest is no less than 2^-31 of it.  So both types decode
// by the packed operations that fp16 has and bf16 lacks: 9 instead of 23 operations a product of integers, 8 instead of 20
// with NVFP4.  At 6 TB/s a SIMD has 44 ns for a product's 512 weights: 22 to 26 operations at 2.0 to 2.4 GHz.
// A row's span that spreads further, or whose power of two leaves fp32 together with NVFP4's global scale, is left out, and
// done behind the others with bf16 operands, chunk by chunk: of normally distributed elements one in 10^9 is that small;
// where every row has one in every span the launch below takes 553 us.
// Loads alone, 16 rows of 64 bytes each, reach 6.0 TB/s where eight are in flight per wave, 3.5 to 4 with one or two.
// 64 bf16 rows that reach 50 of 128 experts of 4096 x 7168, NVFP4 (us, whole launches in a graph): one chunk ahead 234;
// spans in workgroups of eight waves, bf16 decode 246, fp16 195; of four waves 175; loads through the caches, not past
// them, 164 to 167 (5.0 TB/s of the 50 experts' weights).
template <int KIND, int GROUP, int SPAN>
struct W4Span {
  static constexpr bool INT = KIND == W4_INT;
  static constexpr int NS = INT ? SPAN * kW4Chunk / GROUP : SPAN;          // 16-bit words of scales a lane has
  v4i w[SPAN];
  uint32_t s[NS / 2];        // integers: the column's, in order; NVFP4: of each four chunks, the one q's eight bytes
  uint32_t z[INT ? NS / 4 : 1];
};
// Scale bytes of four chunks, chunk q in lane row q -> the pairs of blocks 2 q, 2 q + 1 of every chunk.
__device__ __forceinline__ void scales_by_lane(uint32_t& d0, uint32_t& d1) {
  const v2u a = __builtin_amdgcn_permlane32_swap(d0, d1, false, false);
  const v2u b = __builtin_amdgcn_permlane16_swap(a.x, a.y, false, false);
  const uint32_t lo = __builtin_amdgcn_perm(b.y, b.x, 0x05040100u), hi = __builtin_amdgcn_perm(b.y, b.x, 0x07060302u);
  const v2u c = __builtin_amdgcn_permlane16_swap(lo, hi, false, false);
  d0 = c.x;
  d1 = c.y;
}

template <int TYPE, int KIND, int GROUP, int MT, int SPAN, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void w4_wide_kernel(W4Args p, uint32_t ntn, int64_t blocks) {
  using E = Elem<TYPE>;
  using F = Elem<MM_FP16>;
  constexpr bool SCALED = TYPE == MM_BF16 && MT == 1;          // rows become fp16 times a power of two
  constexpr int T = SCALED ? MM_FP16 : TYPE;
  constexpr bool INT = KIND == W4_INT, TRANS = INT && GROUP < 128, APART = INT && T == MM_FP16;
  constexpr int SK = SPAN * kW4Chunk, XLD = SK + 8, PIECES = SK / 8, ROWS = 16 * MT;
  constexpr int NTH = 64 * WAVES, STAGE = ROWS * PIECES / NTH;                   // 16-byte pieces of x a thread stages at most
  using Span = W4Span<KIND, GROUP, SPAN>;
  static_assert(PIECES % 64 == 0, "a wave stages pieces of one row");
  extern __shared__ __align__(16) uint16_t s_x[];              // [2][ROWS][XLD]: rows 16 bytes apart in the banks
  __shared__ __align__(16) float s_factor[2][PIECES / 64][ROWS];            // what brings a row's sums over a span back; 0: left out
  __shared__ int s_left[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t block = (int64_t)blockIdx.x + (int64_t)blockIdx.y * p.row_blocks;
  if (block >= blocks) return;
  const RowTile tile = find_row_tile(p.m_splits, p.G, (uint32_t)p.M, ROWS, ntn, p.zero_rest, (uint32_t)block, lane);
  if (tile.g < 0) return;
  const uint32_t nrt = (tile.m + ROWS - 1) / ROWS;
  const uint32_t r0 = tile.t % nrt * ROWS;
  const int n0 = (int)(tile.t / nrt) * (16 * WAVES) + 16 * wave;
  const int rows = (int)min(tile.m - r0, (uint32_t)ROWS);
  const int col = lane & 15, q = lane >> 4, N = p.N, K = p.K;
  uint16_t* y = static_cast<uint16_t*>(p.y) + (int64_t)(tile.row0 + r0) * p.ldy + n0 + col;
  if (tile.g == p.G) {
    if (n0 + col < N)
      for (int m = q; m < rows; m += 4) y[(int64_t)m * p.ldy] = 0;
    return;
  }
  const uint16_t* x0 = static_cast<const uint16_t*>(p.x) + (int64_t)(tile.row0 + r0) * p.ldx;
  const int64_t n = (int64_t)tile.g * N + min(n0 + col, N - 1);
  const uint8_t* codes = p.codes + n * (K / 2);
  const int64_t meta = n * (K / GROUP);
  const float global = INT ? 1.0f : nvfp4_global_scale(p.amax[tile.g]);
  const int down = INT || TYPE != MM_BF16 ? 0 : min(max(ilogbf(global), -126), 59) + 1;
  const float downf = ldexpf(1.0f, -down);
  const int spans = K / SK, chunks = (K + kW4Chunk - 1) / kW4Chunk;

  auto load = [&](int s, Span& l) {
#pragma unroll
    for (int c = 0; c < SPAN; ++c) l.w[c] = *reinterpret_cast<const v4i*>(codes + s * (SK / 2) + c * 64 + 16 * q);
    if (INT) {
      __builtin_memcpy(l.s, static_cast<const uint16_t*>(p.scales) + meta + s * Span::NS, 2 * Span::NS);
      if (p.zeros) __builtin_memcpy(l.z, p.zeros + meta + s * Span::NS, Span::NS);
    } else {
#pragma unroll
      for (int h = 0; h < SPAN / 4; ++h) __builtin_memcpy(&l.s[2 * h], static_cast<const uint8_t*>(p.scales) + meta + (s * SPAN + 4 * h + q) * 8, 8);
    }
  };
  bool left = false;                                           // of the wave's rows: spans left out
  auto load_x = [&](int s, int tid, v4i (&xr)[STAGE]) {
#pragma unroll
    for (int i = 0; i < STAGE; ++i) {
      const int at = tid + NTH * i;
      if (at / PIECES < rows) __builtin_memcpy(&xr[i], x0 + (int64_t)(at / PIECES) * p.ldx + s * SK + at % PIECES * 8, 16);
    }
  };
  auto store_x = [&](int s, int tid, const v4i (&xr)[STAGE]) {
#pragma unroll
    for (int i = 0; i < STAGE; ++i) {
      const int at = tid + NTH * i, row = at / PIECES;
      if (row >= rows) continue;
      v4i v = xr[i];
      if constexpr (SCALED) {
        v2ss most2{128, 128};                                  // the largest finite magnitude's bits + 128: infinities and NaN are negative
        v2us least2{65535, 65535};                             // the smallest's that is not 0, less 1
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const v2us u = __builtin_bit_cast(v2us, v[j] & 0x7FFF7FFF);
          most2 = __builtin_elementwise_max(most2, __builtin_bit_cast(v2ss, u + v2us{128, 128}));
          least2 = __builtin_elementwise_min(least2, u - v2us{1, 1});
          f[2 * j] = E::up((uint16_t)v[j]);
          f[2 * j + 1] = E::up((uint16_t)((uint32_t)v[j] >> 16));
        }
        const int most = (int)lanes_reduce<64>((uint32_t)max((int)most2.x, (int)most2.y), [](uint32_t a, uint32_t b) { return a > b ? a : b; }) - 128;
        const uint32_t least = min((uint32_t)least2.x, (uint32_t)least2.y);
        // fp16's step below 2^-14 is 2^-24: all 8 bits from 2^-17 on, 31 binades below the largest
        const int e = most ? min(141 - (most >> 7), 126) : 0;
        // and the power of two that brings the sums back is a number
        const bool fits = !__any(least < (uint32_t)max(((most >> 7) - 31) * 128 - 1, 0)) && (INT || (down + e <= 126 && down + e >= -127));
        left |= !fits;
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (int)F::down2(f[2 * j] * up, f[2 * j + 1] * up);
        if (lane == 0) s_factor[s & 1][at % PIECES / 64][row] = !fits ? 0.0f : INT ? ldexpf(1.0f, -e) : ldexpf(downf, -e);
      }
      *reinterpret_cast<v4i*>(s_x + ((s & 1) * ROWS + row) * XLD + at % PIECES * 8) = APART ? pairs_apart(v) : v;
    }
  };
  v4f acc[MT] = {}, sum[MT];
  // one chunk into `to`: a(m, i) gives x's operand, w the codes, grp the chunk's groups (NVFP4: sc the scales of the
  // lane's two blocks); products of k >= K are left out (live of the four)
  auto multiply = [&](auto type, v4f (&to)[MT], auto a, v4i codes4, const float* sc, const IntGroup* grp, int live) {
    constexpr int U = decltype(type)::value;
    uint32_t w[4] = {(uint32_t)codes4.x, (uint32_t)codes4.y, (uint32_t)codes4.z, (uint32_t)codes4.w};
    if (TRANS) transpose4(w);
    v4f part[MT] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= live) break;
      const int s = INT ? i * 32 / GROUP : i / 2;
      const v4i b = INT ? decode_int<U>(w[i], grp[s]) : decode_fp4<U>(w[i], sc[s]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (!INT) {
          to[m] = Elem<U>::mma16(a(m, i), b, to[m]);
        } else {
          part[m] = Elem<U>::mma16(a(m, i), b, part[m]);
          if ((i + 1) * 32 % GROUP == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) to[m][r] = fmaf(grp[s].sc, part[m][r], to[m][r]);
            part[m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
          }
        }
      }
    }
  };
  constexpr int PER = INT ? kW4Chunk / GROUP : 2;
  auto zero_of = [&](uint32_t z8) { return p.zeros ? z8 & 255u : 8u; };
  int row_at[MT];                                              // rows behind the last read the last one's
#pragma unroll
  for (int m = 0; m < MT; ++m) row_at[m] = min(16 * m + col, rows - 1) * XLD;
  auto span = [&](int s, Span& l) {
    const uint16_t* xs = s_x + (s & 1) * ROWS * XLD;
    if (!INT)
#pragma unroll
      for (int h = 0; h < SPAN / 4; ++h) scales_by_lane(l.s[2 * h], l.s[2 * h + 1]);
#pragma unroll
    for (int c = 0; c < SPAN; ++c) {
      if (SCALED && c % 4 == 0)
#pragma unroll
        for (int m = 0; m < MT; ++m) sum[m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      float sc[PER];
      IntGroup grp[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int at = c * PER + i;
        if (INT) grp[i] = int_group<TYPE, T>((l.s[at / 2] >> (16 * (at & 1))) & 0xFFFFu, zero_of(l.z[INT ? at / 4 : 0] >> (8 * (at & 3))));
        else sc[i] = (SCALED ? 1.0f : downf) * __builtin_amdgcn_cvt_f32_fp8((int)((l.s[c / 2] >> (16 * (c & 1))) >> (8 * i)), 0);
      }
      multiply(std::integral_constant<int, T>{}, SCALED ? sum : acc, [&](int m, int i) { return *reinterpret_cast<const v4i*>(xs + row_at[m] + c * kW4Chunk + (TRANS ? 32 * i + 8 * q : 32 * q + 8 * i)); },
               l.w[c], sc, grp, 4);
      if (SCALED && c % 4 == 3)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const v4f f = *reinterpret_cast<const v4f*>(&s_factor[s & 1][c / 4][16 * m + 4 * q]);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][r] = f[r] != 0.0f ? fmaf(f[r], sum[m][r], acc[m][r]) : acc[m][r];
        }
      __builtin_amdgcn_sched_barrier(0);                       // a chunk's values only are live at once
    }
  };
  Span l0, l1;
  v4i xr[STAGE];
  load_x(0, tid, xr);
  load(0, l0);
  store_x(0, tid, xr);
  __syncthreads();
  for (int s = 0; s < spans; s += 2) {
    const bool more = s + 1 < spans;
    if (more) {
      load_x(s + 1, tid, xr);
      load(s + 1, l1);
    }
    span(s, l0);
    if (!more) break;
    store_x(s + 1, tid, xr);
    __syncthreads();
    const bool yet = s + 2 < spans;
    if (yet) {
      load_x(s + 2, tid, xr);
      load(s + 2, l0);
    }
    span(s + 1, l1);
    if (!yet) break;
    store_x(s + 2, tid, xr);
    __syncthreads();
  }
  int behind = spans * SPAN;                                   // chunks that were done
  if constexpr (SCALED) {
    if (lane == 0) s_left[wave] = left;
    __syncthreads();
    for (int i = 0; i < WAVES; ++i) behind = s_left[i] ? 0 : behind;
  }
  bool mine[4] = {true, true, true, true};                     // the lane's rows that take part
  for (int c = behind; c < chunks; ++c) {                      // the rest of K, and before it the spans that were left out
    if constexpr (SCALED) {
      static_assert(PIECES == 64, "a span has one factor");
      if (c <= spans * SPAN && c % SPAN == 0) {
        v4f f{0.0f, 0.0f, 0.0f, 0.0f};
        if (c < spans * SPAN) {
          v4i again[STAGE] = {};
          int t = tid;
          asm("" : "+v"(t));                                   // addresses of its own: none kept from above in registers
          load_x(c / SPAN, t, again);
          store_x(c / SPAN, t, again);
          __syncthreads();
          f = *reinterpret_cast<const v4f*>(&s_factor[c / SPAN & 1][0][4 * q]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) mine[r] = f[r] == 0.0f && 4 * q + r < rows;
        if (!__any(mine[0] || mine[1] || mine[2] || mine[3])) {          // the same in every wave
          c += SPAN - 1;
          continue;
        }
      }
    }
    const int k0 = c * kW4Chunk, live = min((K - k0) / 32, 4);
    const v4i w = *reinterpret_cast<const v4i*>(codes + min(k0 / 2 + 16 * q, K / 2 - 16));
    v4i a[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + (TRANS ? 32 * i + 8 * q : 32 * q + 8 * i);
        v4i v;
        __builtin_memcpy(&v, x0 + (int64_t)min(16 * m + col, rows - 1) * p.ldx + min(k, K - 8), 16);
        if (!TRANS) v = k < K ? v : v4i{0, 0, 0, 0};
        a[m][i] = APART && TYPE == MM_FP16 ? pairs_apart(v) : v;
      }
    float sc[PER];
    IntGroup grp[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (INT) {
        const int64_t at = meta + min((k0 + i * GROUP) / GROUP, K / GROUP - 1);
        grp[i] = int_group<TYPE, TYPE>(static_cast<const uint16_t*>(p.scales)[at], zero_of(p.zeros ? p.zeros[at] : 0));
      } else {
        const int k = k0 + 32 * q + 16 * i;
        sc[i] = k < K ? downf * __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(p.scales)[meta + k / 16], 0) : 0.0f;
      }
    }
    v4f to[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) to[m] = acc[m];
    multiply(std::integral_constant<int, TYPE>{}, to, [&](int m, int i) { return a[m][i]; }, w, sc, grp, TRANS ? live : 4);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[m][r] = mine[r] ? to[m][r] : acc[m][r];
  }
  const float rest = ldexpf(global, -down);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float v = INT ? acc[m][r] : __fdiv_rn(acc[m][r], rest);
      if (16 * m + 4 * q + r < rows && n0 + col < N) y[(int64_t)(16 * m + 4 * q + r) * p.ldy] = E::down(v);
    }
}

// ----------------------------------------------------------------------------- launches
template <int TYPE, int KIND, int GROUP, int NT>
static hipError_t run_split(W4Args p, hipStream_t s) {
  const int64_t ntn = (p.N + 16 * NT - 1) / (16 * NT), blocks = sizes::row_tiles_bound(p.M, p.G, 16) * ntn;
  const int waves = sizes::w4_waves(p.K);
  const FoldedGrid g = fold_grid(blocks, 64 * waves);
  p.row_blocks = g.x;
  hipLaunchKernelGGL((w4_split_kernel<TYPE, KIND, GROUP, NT>), dim3(g.x, g.y), dim3(64 * waves), (size_t)waves * NT * 4 * 64 * sizeof(float), s, p,
                     (uint32_t)ntn, blocks);
  return hipGetLastError();
}
template <int TYPE, int KIND, int GROUP, int MT, int SPAN, int WAVES>
static hipError_t run_wide(W4Args p, hipStream_t s) {
  const int64_t ntn = (p.N + 16 * WAVES - 1) / (16 * WAVES), blocks = sizes::row_tiles_bound(p.M, p.G, 16 * MT) * ntn;
  const FoldedGrid g = fold_grid(blocks, 64 * WAVES);
  p.row_blocks = g.x;
  hipLaunchKernelGGL((w4_wide_kernel<TYPE, KIND, GROUP, MT, SPAN, WAVES>), dim3(g.x, g.y), dim3(64 * WAVES), 2 * 16 * MT * (SPAN * kW4Chunk + 8) * sizeof(uint16_t),
                     s, p, (uint32_t)ntn, blocks);
  return hipGetLastError();
}
template <int TYPE, int KIND, int GROUP>
static hipError_t run_w4(const W4Args& p, hipStream_t s) {
  constexpr int SPAN = 4;
  // Spans where there are 2048 tiles of 16 x 16, a wave each eight a CU; near where the two cross for the larger tiles too (us,
  // split K / spans): 64 rows over 128 experts of 4096 x 7168, NVFP4 305 / 161; 4, 8 and 16 rows over 16 experts of 2048 x 2048,
  // NVFP4 (512, 1024 and 2048 tiles) 7.2 / 9.3, 12.8 / 9.6, 16.8 / 11.9; dense 7168 x 4096, groups of 128, 48, 64 and 96 rows (1792,
  // 2240 and 3136) 28.5 / 35.0, 28.8 / 36.7, 41.7 / 37.2, 64 rows NVFP4 34.0 / 34.1, groups of 64 34.2 / 31.5, of 32 37.6 / 43.4
  const int64_t waves = sizes::row_tiles_bound(p.M, p.G, 16) * ((p.N + 15) / 16);
  if (waves < 2048 || p.K < SPAN * kW4Chunk)
    return p.M / p.G > 4 && waves >= 512 ? run_split<TYPE, KIND, GROUP, 4>(p, s) : run_split<TYPE, KIND, GROUP, 1>(p, s);
  if (p.M / p.G <= 16) return run_wide<TYPE, KIND, GROUP, 1, SPAN, 4>(p, s);
  // 512 rows in 8 groups of 4096 x 4096, their sizes drawn, by tiles of 64 / 32 rows: groups of 128 80 / 88 us; groups of 64 (whose
  // larger tiles spill) 146 / 94, of 32 343 / 132
  return run_wide<TYPE, KIND, GROUP, KIND == W4_INT && GROUP < 128 ? 2 : 4, SPAN, 8>(p, s);
}
template <int TYPE>
static hipError_t run_w4(const W4Args& p, hipStream_t s) {
  if (p.kind == W4_NVFP4) return run_w4<TYPE, W4_NVFP4, 16>(p, s);
  if (p.group == 32) return run_w4<TYPE, W4_INT, 32>(p, s);
  if (p.group == 64) return run_w4<TYPE, W4_INT, 64>(p, s);
  return run_w4<TYPE, W4_INT, 128>(p, s);
}
hipError_t launch_w4(const W4Args& p, hipStream_t s) {
  return p.type == MM_BF16 ? run_w4<MM_BF16>(p, s) : run_w4<MM_FP16>(p, s);
}

}  // namespace gmlp
