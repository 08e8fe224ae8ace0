// Low-rank adapters of many requests: v = W_l x (shrink), y = base + W_l v (expand), the adapters'
// gradients sum_m v_m x_m^T (outer), each over rows taken in the order of their adapter.
//
// All three are bound by the read (and write) of the [M, C] tensors: 2 R flops per element read.
// Rows of one adapter are consecutive positions; a workgroup takes a tile of positions of one
// adapter and gathers their rows through `order`, so requests need not be sorted or equal in
// length.  The rank-sized factor v is summed in fp32 and enters the 16-bit matrix products as
// hi + lo, two values of the operands' type (at least 16 of its bits), split once where v is made:
// one V_MFMA_F32_16X16X32 takes 16 ranks, hi in its lower and lo in its upper sixteen contraction
// steps.  fp16 scales each position's v by a power of two first, so that neither half leaves the range.
#include "mm_common.h"
#include "op_sizes.h"

#include <algorithm>

namespace gmlp {

// ----------------------------------------------------------------------------- loads
// Eight consecutive elements of a row from p, of which `valid` exist: load8 then fix8 (which moves the
// ragged end of an unaligned row down).  brief: rows of fewer than eight elements.
template <bool VEC>
__device__ __forceinline__ v4i load8(const uint16_t* p, int valid, bool brief) {
  if constexpr (VEC) return valid > 0 ? *reinterpret_cast<const v4i*>(p) : v4i{0, 0, 0, 0};
  else return brief ? load8_short(p, valid) : load8_raw(p, valid);
}
template <bool VEC>
__device__ __forceinline__ v4i fix8(v4i v, int valid, bool brief) {
  if constexpr (VEC) return v;
  else return brief ? v : shift8(v, valid);
}

// v as a factor of the 16-bit products: hi = T(v), lo = T(v - hi); hi is the largest finite value where a finite
// v rounds to infinity (bf16 above 2^128 (1 - 2^-9); lo then holds the rest).
template <int TYPE>
__device__ __forceinline__ void split(float v, uint16_t& hi, uint16_t& lo) {
  using E = Elem<TYPE>;
  hi = E::down(v);
  if (__builtin_isfinite(v) && !__builtin_isfinite(E::up(hi))) --hi;
  const float h = E::up(hi);
  lo = E::down(__builtin_isfinite(h) ? v - h : 0.0f);
}
// W's (or X's) elements for the product with lo: infinities and NaN as zeros.  hi times them is already what v
// times them is; lo, zero or of the other sign, would make a NaN of an infinity.
template <int TYPE>
__device__ __forceinline__ v4i finite_only(v4i w) {
  constexpr uint32_t E = TYPE == MM_BF16 ? 0x7F80u : 0x7C00u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v = (uint32_t)w[i];
    if ((v & E) == E) v &= 0xFFFF0000u;
    if ((v >> 16 & E) == E) v &= 0xFFFFu;
    w[i] = (int)v;
  }
  return w;
}
// The largest magnitude of elements, by their bits.
template <int TYPE>
struct Top {
  typedef uint16_t v2u __attribute__((ext_vector_type(2)));
  v2u m = {0, 0};
  __device__ __forceinline__ void add(v4i v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(v2u, v[i] & 0x7FFF7FFF));
  }
  __device__ __forceinline__ bool not_finite() const {
    constexpr uint16_t E = TYPE == MM_BF16 ? 0x7F80 : 0x7C00;
    return m.x >= E || m.y >= E;
  }
};
__device__ __forceinline__ int any_nan(v4f c) { return (int)__builtin_isunordered(c[0], c[1]) | (int)__builtin_isunordered(c[2], c[3]); }
// A power of two that brings a largest magnitude m to [2^14, 2^15) (fp16 operands: hi then never
// overflows and lo resolves 2^-39 of m), 1 where m is zero or not finite.  Exponents are kept where
// the factor and its inverse are normal numbers.
__device__ __forceinline__ float fp16_scale(float m) {
  const uint32_t ex = __float_as_uint(m) >> 23;
  if (ex == 0 || ex >= 255) return 1.0f;
  return __uint_as_float(min(253u, max(1u, 268u - min(ex, 267u))) << 23);
}
__device__ __forceinline__ float inverse_pow2(float s) { return __uint_as_float((254u - (__float_as_uint(s) >> 23)) << 23); }

// ----------------------------------------------------------------------------- shrink
// RB x 16 positions by RT x 16 ranks per workgroup, the contraction in blocks of 32 SPB dealt to its
// NW waves, fragments straight from memory.  The waves are joined through LDS, in order.  A workgroup
// for the whole contraction keeps v out of memory until it is whole; the waves of a workgroup give
// the loads in flight that few positions cannot.  16384 rows of 4096, rank 16: 31 us, 4.3 TB/s of X;
// 6001 rows of 7168, rank 64: 45 us (W, read once per tile, is twice X there).
template <int TYPE, bool VEC, int RB, int RT, int NW>
__global__ __launch_bounds__(64 * NW) void lora_shrink_kernel(LoraShrink p) {
  using E = Elem<TYPE>;
  // A lane has 256 registers with 8 waves and holds two blocks; 128 with 16, whose other waves cover the
  // loads of one.  Blocks of 64 at least where they fit: a row's 128-byte line is then read by one wave.
  // (Unaligned rows take more registers for their addresses: three of these shapes spill 14 to 38 then.)
  constexpr bool TWO = NW <= 8;
  constexpr int F = RB + RT, SPB = TWO ? (F <= 3 ? 4 : F <= 6 ? 2 : 1) : (F <= 2 ? 8 : F <= 3 ? 4 : 2);
  constexpr int LD = RT * 16 + 4;
  __shared__ __align__(16) float red[NW * RB * 16 * LD];
  __shared__ float s_mul[RB * 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const RowTile rt = find_row_tile(p.rows.count, p.rows.L, (uint32_t)p.rows.M, RB * 16, 1, false,
                                   blockIdx.x + blockIdx.y * p.row_blocks, lane);
  if (rt.g < 0) return;
  const int64_t pos0 = (int64_t)rt.row0 + rt.t * (RB * 16);
  const int valid = min((int)(rt.m - rt.t * (RB * 16)), RB * 16);
  const int q = lane & 15, j = lane >> 4;
  const uint16_t* xr[RB];
  const uint16_t* wr[RT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
    xr[b] = static_cast<const uint16_t*>(p.x) + p.rows.order[pos0 + min(16 * b + q, valid - 1)] * p.ldx + 8 * j;
#pragma unroll
  for (int t = 0; t < RT; ++t)
    wr[t] = static_cast<const uint16_t*>(p.w) + rt.g * p.w_stride + min(16 * t + q, p.R - 1) * p.ldw + 8 * j;
  v4f acc[RB][RT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[b][t] = v4f{0, 0, 0, 0};
  constexpr int64_t step = 32 * SPB;
  const bool brief = p.C < 8;
  const int64_t nblk = (p.C + step - 1) / step;
  v4i xf[TWO ? 2 : 1][SPB][RB], wf[TWO ? 2 : 1][SPB][RT];
  auto fetch = [&](int64_t blk, int s) {
    const int64_t c0 = blk * step;
#pragma unroll
    for (int k = 0; k < SPB; ++k) {
      const int64_t c = c0 + 32 * k;
      const int left = (int)min(p.C - c - 8 * j, (int64_t)8);
#pragma unroll
      for (int b = 0; b < RB; ++b) xf[s][k][b] = load8<VEC>(xr[b] + c, left, brief);
#pragma unroll
      for (int t = 0; t < RT; ++t) wf[s][k][t] = load8<VEC>(wr[t] + c, left, brief);
    }
  };
  auto mul = [&](int64_t blk, int s) {
    if constexpr (!VEC) {
#pragma unroll
      for (int k = 0; k < SPB; ++k) {
        const int left = (int)min(p.C - blk * step - 32 * k - 8 * j, (int64_t)8);
#pragma unroll
        for (int b = 0; b < RB; ++b) xf[s][k][b] = fix8<VEC>(xf[s][k][b], left, brief);
#pragma unroll
        for (int t = 0; t < RT; ++t) wf[s][k][t] = fix8<VEC>(wf[s][k][t], left, brief);
      }
    }
#pragma unroll
    for (int k = 0; k < SPB; ++k)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[b][t] = E::mma16(wf[s][k][t], xf[s][k][b], acc[b][t]);
  };
  int64_t blk = wave;
  if constexpr (!TWO) {
    for (; blk < nblk; blk += NW) {
      fetch(blk, 0);
      mul(blk, 0);
    }
  } else if (blk < nblk) {
    fetch(blk, 0);
    while (true) {
      if (blk + NW < nblk) fetch(blk + NW, 1);
      mul(blk, 0);
      blk += NW;
      if (blk >= nblk) break;
      if (blk + NW < nblk) fetch(blk + NW, 0);
      mul(blk, 1);
      blk += NW;
      if (blk >= nblk) break;
    }
  }
  // lane: position 16 b + q, ranks 16 t + 4 j + i
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < RT; ++t)
      *reinterpret_cast<v4f*>(red + ((wave * RB + b) * 16 + q) * LD + 16 * t + 4 * j) = acc[b][t];
  __syncthreads();
  const float sc = p.scales ? p.scales[rt.g] : 1.0f;
  const int rp = (p.R + 15) & ~15;
  constexpr int N = RB * 16 * RT * 16, PER = (N + 64 * NW - 1) / (64 * NW);
  float v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid + i * 64 * NW, row = e / (RT * 16), r = e % (RT * 16);
    v[i] = 0.0f;
    if (e < N && row < valid && r < p.R) {
      for (int w = 0; w < NW; ++w) v[i] += red[(w * RB * 16 + row) * LD + r];
      v[i] *= sc;
    }
  }
  if (TYPE == MM_FP16) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + i * 64 * NW;
      if (e < N) red[e / (RT * 16) * LD + e % (RT * 16)] = v[i];
    }
    __syncthreads();
    for (int row = wave; row < RB * 16; row += NW) {
      float top = 0.0f;
#pragma unroll
      for (int r = 0; r < RT * 16; r += 64)
        if (r + lane < RT * 16) {                        // zero behind rank R
          const float f = fabsf(red[row * LD + r + lane]);
          top = fmaxf(top, __builtin_isfinite(f) ? f : 0.0f);
        }
      const float s = fp16_scale(wave_max(top));
      if (lane == 0) {
        s_mul[row] = s;
        if (row < valid) p.out.inv[pos0 + row] = inverse_pow2(s);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid + i * 64 * NW, row = e / (RT * 16), r = e % (RT * 16);
    if (e >= N || row >= valid || r >= rp) continue;
    uint16_t hi, lo;
    split<TYPE>(TYPE == MM_FP16 ? v[i] * s_mul[row] : v[i], hi, lo);
    uint16_t* d = p.out.hi + (pos0 + row) * 2 * rp + r;
    d[0] = hi;
    d[rp] = lo;
    if (p.out.v && r < p.R) p.out.v[(pos0 + row) * p.R + r] = v[i];
  }
}

using sizes::tiles_bound;

template <int TYPE, bool VEC, int RB, int RT, int NW>
static hipError_t run_shrink(LoraShrink p, hipStream_t s) {
  const FoldedGrid grid = fold_grid(tiles_bound(p.rows.M, p.rows.L, 16 * RB), 64 * NW);
  p.row_blocks = grid.x;
  hipLaunchKernelGGL((lora_shrink_kernel<TYPE, VEC, RB, RT, NW>), dim3(grid.x, grid.y), dim3(64 * NW), 0, s, p);
  return hipGetLastError();
}
// 32 positions a tile where those fill the device, 16 waves while one tile a CU is all there is, else 8;
// 16 positions below.  (Above 64 ranks a wave's registers allow 8.)  Measured (bf16, us, whole forward, rows
// of 4096 to 4096 / of 7168 to 2048, by 16 positions, by 32 with 16 waves, with 8):
//   tiles of 32      rank 16                                   rank 64
//       71      29.2 33.1 33.3 / 30.1 36.2 36.0       47.7 51.5 51.9 / 55.4 61.9 62.0
//      135      35.8 39.3 40.2 / 35.7 41.1 41.1       58.8 62.4 62.9 / 61.5 67.4 67.5
//      195      53.6 49.8 49.9 / 51.6 44.4 44.3       86.0 71.0 71.8 / 93.8 68.9 69.1
//      519       122  119  119 /  119  108  108        185  155  157 /  211  157  158
// so the sides meet at about 150 tiles, and 16 waves or 8 make 1% at most (fp16, 6001 rows of 7168, rank 64:
// 100.6 and 102.0).  Rank 128: 65.0 69.6 at 71 tiles, 86.8 90.9 at 135, 145 116 at 195.
template <int TYPE, bool VEC, int RT>
static hipError_t shrink_rank(const LoraShrink& p, hipStream_t s) {
  constexpr int NW = RT > 4 ? 8 : 16;
  const int64_t tiles = tiles_bound(p.rows.M, p.rows.L, 32);
  if (tiles >= 512) return run_shrink<TYPE, VEC, 2, RT, 8>(p, s);
  if (tiles >= 128) return run_shrink<TYPE, VEC, 2, RT, NW>(p, s);
  return run_shrink<TYPE, VEC, 1, RT, NW>(p, s);
}
template <int TYPE, bool VEC>
static hipError_t shrink_rows(const LoraShrink& p, hipStream_t s) {
  if (p.R <= 16) return shrink_rank<TYPE, VEC, 1>(p, s);
  if (p.R <= 32) return shrink_rank<TYPE, VEC, 2>(p, s);
  if (p.R <= 64) return shrink_rank<TYPE, VEC, 4>(p, s);
  return shrink_rank<TYPE, VEC, 8>(p, s);
}
static bool vec16(const void* p, int64_t ld, int64_t cols) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ((ld | cols) & 7) == 0;
}
hipError_t launch_lora_shrink(const LoraShrink& p, hipStream_t s) {
  const bool v = vec16(p.x, p.ldx, p.C) && vec16(p.w, p.ldw, p.w_stride);
  if (p.type == MM_BF16) return v ? shrink_rows<MM_BF16, true>(p, s) : shrink_rows<MM_BF16, false>(p, s);
  return v ? shrink_rows<MM_FP16, true>(p, s) : shrink_rows<MM_FP16, false>(p, s);
}

// ----------------------------------------------------------------------------- expand
// A tile of 16 RB positions by 256 columns, 64 per wave.  A wave keeps W_l's fragments of its columns
// in registers and takes the positions 16 at a time, all rows of base on their way from the start.
// The product is taken transposed with the columns dealt so that a lane ends with 16 consecutive
// ones of one row: 32 bytes of base and y.  16384 rows of 4096, rank 16: 37 us with base (268 MB, part
// of it in the last-level cache); 6001 rows of 4096, rank 64: 40 us, bound by the chain of loads of
// the few waves that W's fragments leave room for.
template <int TYPE, bool VEC, bool VECW, int RB, int RT>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraExpand p) {
  using E = Elem<TYPE>;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const RowTile rt = find_row_tile(p.rows.count, p.rows.L + 1, (uint32_t)p.rows.M, 16 * RB, 1, false, blockIdx.x, lane);
  if (rt.g < 0) return;
  const bool rest = rt.g == p.rows.L;                    // rows without an adapter
  if (rest && p.base == p.y) return;
  const int64_t pos0 = (int64_t)rt.row0 + (int64_t)rt.t * (16 * RB);
  const int valid = min((int)(rt.m - rt.t * (16 * RB)), 16 * RB);
  const int q = lane & 15, j = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.y * 256 + wave * 64;
  if (n0 >= p.C) return;
  const int64_t c = n0 + 16 * j;
  const int cols = (int)min(p.C - c, (int64_t)16);       // of this lane
  int32_t row[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) row[b] = p.rows.order[pos0 + min(16 * b + q, valid - 1)];
  v4i wf[4][RT];
  if (!rest) {
    const uint16_t* w = static_cast<const uint16_t*>(p.w) + rt.g * p.w_stride;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int64_t n = min(n0 + 16 * (q >> 2) + 4 * f + (q & 3), p.C - 1);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int r = 16 * t + 8 * (j & 1);
        wf[f][t] = load8<VECW>(w + n * p.ldw + r, min(p.R - r, 8), p.R < 8);
      }
    }
  }
  v4i old[RB][2];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    old[b][0] = old[b][1] = v4i{0, 0, 0, 0};
    if (p.base && 16 * b + q < valid) {
      const uint16_t* src = static_cast<const uint16_t*>(p.base) + row[b] * p.ldbase + c;
      old[b][0] = load8<VEC>(src, cols, p.C < 8);
      old[b][1] = load8<VEC>(src + 8, cols - 8, p.C < 8);
    }
  }
  if (!VECW && !rest) {
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int t = 0; t < RT; ++t) wf[f][t] = fix8<VECW>(wf[f][t], min(p.R - 16 * t - 8 * (j & 1), 8), p.R < 8);
  }
  const float sc = !rest && p.scales ? p.scales[rt.g] : 1.0f;
  const int rp = (p.R + 15) & ~15;
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    if (16 * b >= valid) break;
    old[b][0] = fix8<VEC>(old[b][0], cols, p.C < 8);
    old[b][1] = fix8<VEC>(old[b][1], cols - 8, p.C < 8);
    v4f acc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = v4f{0, 0, 0, 0};
    float mul = sc;
    if (!rest) {
      const int64_t at = pos0 + min(16 * b + q, valid - 1);
      const uint16_t* src = p.v.hi + at * 2 * rp + (j >= 2 ? rp : 0) + 8 * (j & 1);
      v4i u[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) u[t] = 16 * t < rp ? *reinterpret_cast<const v4i*>(src + 16 * t) : v4i{0, 0, 0, 0};
      if (p.v.inv) mul *= p.v.inv[at];
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[f] = E::mma16(wf[f][t], u[t], acc[f]);
      if (__any(any_nan(acc[0]) | any_nan(acc[1]) | any_nan(acc[2]) | any_nan(acc[3]))) {      // again, lo times finite W
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          acc[f] = v4f{0, 0, 0, 0};
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            if (j >= 2) wf[f][t] = finite_only<TYPE>(wf[f][t]);
            acc[f] = E::mma16(wf[f][t], u[t], acc[f]);
          }
        }
      }
    }
    // mul is its row's: the accumulator's column is the lane's own position q
    if (16 * b + q >= valid) continue;
    uint16_t* dst = static_cast<uint16_t*>(p.y) + row[b] * p.ldy + c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint16_t o = (uint16_t)((uint32_t)old[b][h][i / 2] >> (16 * (i & 1)));
        y[i] = rest ? 0.0f : mul * acc[2 * h + i / 4][i & 3];
        y[i] = p.base ? E::up(o) + y[i] : y[i];
      }
      v4i out;
      if (rest) out = old[b][h];                         // bit for bit
      else
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = (int)E::down2(y[2 * i], y[2 * i + 1]);
      if constexpr (VEC) {
        if (cols > 8 * h) *reinterpret_cast<v4i*>(dst + 8 * h) = out;
      } else if (cols >= 8 * h + 8) {
        __builtin_memcpy(dst + 8 * h, &out, 16);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * h + i < cols) dst[8 * h + i] = (uint16_t)((uint32_t)out[i / 2] >> (16 * (i & 1)));
      }
    }
  }
}

template <int TYPE, bool VEC, bool VECW, int RB>
static hipError_t run_expand_rows(const LoraExpand& p, hipStream_t s) {
  const dim3 grid((uint32_t)tiles_bound(p.rows.M, p.rows.L + 1, 16 * RB), (uint32_t)((p.C + 255) / 256));
  if (p.R <= 16) hipLaunchKernelGGL((lora_expand_kernel<TYPE, VEC, VECW, RB, 1>), grid, dim3(256), 0, s, p);
  else if (p.R <= 32) hipLaunchKernelGGL((lora_expand_kernel<TYPE, VEC, VECW, RB, 2>), grid, dim3(256), 0, s, p);
  else if (p.R <= 64) hipLaunchKernelGGL((lora_expand_kernel<TYPE, VEC, VECW, RB, 4>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((lora_expand_kernel<TYPE, VEC, VECW, RB, 8>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}
template <int TYPE, bool VEC, bool VECW>
static hipError_t run_expand(const LoraExpand& p, hipStream_t s) {
  // W is read once per tile: 128 positions where those give three workgroups a CU, 16 where those give
  // fewer than eight, else 64.  Measured (bf16, us, whole forward, by 16, 64 and 128 positions):
  //   workgroups of 16 (of 128)   rank 16              rank 64              rank 128
  //     1136 (240), 4096 wide    22.6 24.4 26.7       41.0 40.0 40.6       66.5 61.5 59.2
  //     2160 (368)               29.3 29.2 32.2       55.0 47.7 48.9       88.8 65.0 77.4
  //     4208 (624)               41.7 39.2 41.1       79.3 62.4 54.2        134 90.9 85.1
  //     8304 (1136)              54.9 51.5 56.1        123 84.2 74.4        218  125  122
  //    16496 (2160)               118  120  119        246  170  157        443  255  250
  // and 16384 rows of 4096, rank 16, with gradients 289 by 64 and 280 by 128.
  const int64_t cols = (p.C + 255) / 256;
  if (tiles_bound(p.rows.M, p.rows.L + 1, 16) * cols < 2048) return run_expand_rows<TYPE, VEC, VECW, 1>(p, s);
  if (tiles_bound(p.rows.M, p.rows.L + 1, 128) * cols < 768) return run_expand_rows<TYPE, VEC, VECW, 4>(p, s);
  return run_expand_rows<TYPE, VEC, VECW, 8>(p, s);
}
template <int TYPE>
static hipError_t expand_vec(const LoraExpand& p, hipStream_t s) {
  const bool v = (!p.base || vec16(p.base, p.ldbase, p.C)) && vec16(p.y, p.ldy, p.C);
  const bool w = vec16(p.w, p.ldw, p.w_stride) && (p.R & 7) == 0;     // rows of whole 16-byte chunks
  if (v) return w ? run_expand<TYPE, true, true>(p, s) : run_expand<TYPE, true, false>(p, s);
  return w ? run_expand<TYPE, false, true>(p, s) : run_expand<TYPE, false, false>(p, s);
}
hipError_t launch_lora_expand(const LoraExpand& p, hipStream_t s) {
  return p.type == MM_BF16 ? expand_vec<MM_BF16>(p, s) : expand_vec<MM_FP16>(p, s);
}

// ----------------------------------------------------------------------------- outer
// part[chunk][r][c] = sum over the chunk's positions of v[p, r] X[row p, c]: a chunk of positions of
// one adapter by 256 columns, 64 positions a stage.  Both factors are contracted over positions, so
// both are read from LDS by ds_read_b64_tr_b16 (as the ring kernel's transposed units).  The chunks
// of an adapter are joined in order by lora_outer_sum_kernel.  16384 rows of 4096, rank 16: 43 us and 5.
constexpr int OP = sizes::kOuterRows, OC = sizes::kOuterCols;

template <int TYPE, bool VEC, int RT>
__global__ __launch_bounds__(256) void lora_outer_kernel(LoraOuter p, int chunk_rows) {
  using E = Elem<TYPE>;
  constexpr int VW = RT * 16;                                     // ranks in LDS
  __shared__ __align__(1024) uint16_t sx[OP * OC];
  __shared__ __align__(1024) uint16_t sv[2][OP * VW];             // hi, lo
  __shared__ float s_top[4];
  __shared__ int s_odd[2];                                        // a stage's X holds what is not finite
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid < 2) s_odd[tid] = 0;
  const RowTile rt = find_row_tile(p.rows.count, p.rows.L, (uint32_t)p.rows.M, chunk_rows, 1, false, blockIdx.x, lane);
  if (rt.g < 0) return;
  const int64_t pos0 = (int64_t)rt.row0 + (int64_t)rt.t * chunk_rows;
  const int valid = min((int)(rt.m - rt.t * chunk_rows), chunk_rows);
  const int64_t c0 = (int64_t)blockIdx.y * OC;
  const int rp = (p.R + 15) & ~15;
  float scale = 1.0f;
  if (TYPE == MM_FP16) {                                          // one power of two for the chunk
    float top = 0.0f;
    for (int i = tid; i < valid * p.R; i += 256) {
      const float f = fabsf(p.v.v[pos0 * p.R + i]);
      if (__builtin_isfinite(f)) top = fmaxf(top, f);
    }
    top = wave_max(top);
    if (lane == 0) s_top[wave] = top;
    __syncthreads();
    scale = fp16_scale(fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3])));
  }
  v4f acc[RT][4];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[t][f] = v4f{0, 0, 0, 0};

  // a thread stages 8 columns of rows tid / 32 + 8 i
  const int xr = tid >> 5, xc = (tid & 31) * 8;
  const int xcols = (int)min(p.C - c0 - xc, (int64_t)8);
  // Two stages of rows in flight, their indices one stage further ahead.
  v4i xs[2][OP / 8];
  int32_t idx[OP / 8];
  auto rows_of = [&](int b) {
#pragma unroll
    for (int i = 0; i < OP / 8; ++i) idx[i] = p.rows.order[pos0 + min(b + xr + 8 * i, valid - 1)];
  };
  auto fetch = [&](int b, v4i* x) {
#pragma unroll
    for (int i = 0; i < OP / 8; ++i)
      x[i] = b + xr + 8 * i < valid ? load8<VEC>(static_cast<const uint16_t*>(p.x) + (int64_t)idx[i] * p.ldx + c0 + xc, xcols, p.C < 8)
                                    : v4i{0, 0, 0, 0};
  };
  rows_of(0);
  fetch(0, xs[0]);
  rows_of(OP);
  fetch(OP, xs[1]);
  rows_of(2 * OP);
  const int i16 = lane & 15, r4 = i16 >> 2, j = lane >> 4;
  const uint32_t sx0 = (uint32_t)(uintptr_t)sx, sv0 = (uint32_t)(uintptr_t)sv;
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  auto tr = [](uint32_t a, uint32_t step) {
    const v2i lo = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)a));
    const v2i hi = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)(a + step)));
    return v4i{lo.x, lo.y, hi.x, hi.y};
  };
  auto stage = [&](int b, v4i* x) {
    const int odd = b / OP & 1;
    __syncthreads();
    if (tid == 0) s_odd[odd ^ 1] = 0;                             // the next stage's
    Top<TYPE> top;
#pragma unroll
    for (int i = 0; i < OP / 8; ++i) {
      const int r = xr + 8 * i;
      const v4i v = fix8<VEC>(x[i], xcols, p.C < 8);
      top.add(v);
      *reinterpret_cast<v4i*>(sx + r * OC + (((xc >> 3) ^ ((r & 3) << 2)) << 3)) = v;
    }
    if (top.not_finite()) s_odd[odd] = 1;
    if (TYPE == MM_FP16) {
      for (int i = tid; i < OP * VW; i += 256) {
        const int m = i / VW, r = i % VW;
        split<TYPE>((b + m < valid && r < p.R) ? scale * p.v.v[(pos0 + b + m) * p.R + r] : 0.0f, sv[0][i], sv[1][i]);
      }
    } else {
      for (int i = tid; i < OP * RT * 4; i += 256) {              // 8 ranks of hi or lo
        const int m = i / (RT * 4), h = i / (RT * 2) & 1, r = i % (RT * 2) * 8;
        *reinterpret_cast<v4i*>(sv[h] + m * VW + r) =
            b + m < valid && r < rp ? *reinterpret_cast<const v4i*>(p.v.hi + (pos0 + b + m) * 2 * rp + h * rp + r) : v4i{0, 0, 0, 0};
      }
    }
    if (b + 2 * OP < valid) {
      fetch(b + 2 * OP, x);
      rows_of(b + 3 * OP);
    }
    __syncthreads();
    const bool clean = __builtin_amdgcn_readfirstlane(s_odd[odd]) != 0;
#pragma unroll
    for (int ks = 0; ks < OP / 32; ++ks) {
      const int row = 32 * ks + 8 * j + r4;
      v4i xf[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int chunk = ((wave * 64 + 16 * f) / 8 + ((i16 & 3) >> 1)) ^ (r4 << 2);
        xf[f] = tr(sx0 + row * (OC * 2) + chunk * 16 + (i16 & 1) * 8, 4 * OC * 2);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && clean) {
#pragma unroll
          for (int f = 0; f < 4; ++f) xf[f] = finite_only<TYPE>(xf[f]);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const v4i vf = tr(sv0 + h * (OP * VW * 2) + row * (VW * 2) + t * 32 + (i16 & 3) * 8, 4 * VW * 2);
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[t][f] = E::mma16(vf, xf[f], acc[t][f]);
        }
      }
    }
  };
  for (int b = 0; b < valid; b += 2 * OP) {
    stage(b, xs[0]);
    if (b + OP < valid) stage(b + OP, xs[1]);
  }
  // lane: ranks 16 t + 4 j + i, column 16 f + lane % 16
  const float inv = inverse_pow2(scale);
  float* out = p.part + (int64_t)blockIdx.x * p.R * p.C;
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * t + 4 * j + i;
        const int64_t c = c0 + wave * 64 + 16 * f + i16;
        if (r < p.R && c < p.C) out[r * p.C + c] = inv * acc[t][f][i];
      }
}

// Chunks of the adapters before l, and of l.
struct ChunkSpan {
  uint32_t first, n;
};
__device__ __forceinline__ ChunkSpan find_chunks(const int32_t* count, int L, uint32_t M, uint32_t h, int l, int lane) {
  uint32_t done = 0, before = 0;
  ChunkSpan s{0, 0};
  for (int base = 0; base <= l; base += 64) {
    const Span sp = wave_spans(count, L, M, base, lane, done);
    const uint32_t mine = (sp.end - sp.start + h - 1) / h;
    const uint32_t incl = wave_incl_add(mine, lane, 0x7FFFFFFFu);
    const int at = min(l - base, 63);
    s.n = (uint32_t)__builtin_amdgcn_readlane((int)mine, at);
    s.first = before + (uint32_t)__builtin_amdgcn_readlane((int)incl, at) - s.n;
    before += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
  }
  return s;
}

// Four ranks of 256 columns of one adapter, four chunks' loads in flight.
template <int TYPE, bool TRANSPOSED>
__global__ __launch_bounds__(256) void lora_outer_sum_kernel(LoraOuter p, int chunk_rows) {
  using E = Elem<TYPE>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int l = blockIdx.z, r0 = blockIdx.y * 4;
  const int64_t c = (int64_t)blockIdx.x * 256 + tid;
  const ChunkSpan s = find_chunks(p.rows.count, p.rows.L, (uint32_t)p.rows.M, chunk_rows, l, lane);
  if (c >= p.C) return;
  const int live = min(p.R - r0, 4);
  float acc[4] = {};
  for (uint32_t k = 0; k < s.n; k += 4) {
    float v[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[u][i] = k + u < s.n && i < live ? p.part[((int64_t)(s.first + k + u) * p.R + r0 + i) * p.C + c] : 0.0f;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += v[u][i];
  }
  const float sc = p.scales ? p.scales[l] : 1.0f;
  uint16_t* out = static_cast<uint16_t*>(p.out);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= live) break;
    const uint16_t v = s.n ? E::down(sc * acc[i]) : (uint16_t)0;
    if (TRANSPOSED) out[((int64_t)l * p.C + c) * p.R + r0 + i] = v;
    else out[((int64_t)l * p.R + r0 + i) * p.C + c] = v;
  }
}

int64_t lora_outer_part_floats(int64_t M, int64_t C, int R, int L) { return sizes::outer_part_floats(M, C, R, L); }
template <int TYPE, bool VEC>
static hipError_t run_outer(const LoraOuter& p, hipStream_t s) {
  const int rows = sizes::outer_rows(p.rows.M, p.C);
  const dim3 grid((uint32_t)tiles_bound(p.rows.M, p.rows.L, rows), (uint32_t)((p.C + OC - 1) / OC));
  if (p.R <= 16) hipLaunchKernelGGL((lora_outer_kernel<TYPE, VEC, 1>), grid, dim3(256), 0, s, p, rows);
  else if (p.R <= 32) hipLaunchKernelGGL((lora_outer_kernel<TYPE, VEC, 2>), grid, dim3(256), 0, s, p, rows);
  else if (p.R <= 64) hipLaunchKernelGGL((lora_outer_kernel<TYPE, VEC, 4>), grid, dim3(256), 0, s, p, rows);
  else hipLaunchKernelGGL((lora_outer_kernel<TYPE, VEC, 8>), grid, dim3(256), 0, s, p, rows);
  if (hipError_t e = hipGetLastError()) return e;
  const dim3 sum((uint32_t)((p.C + 255) / 256), (uint32_t)((p.R + 3) / 4), (uint32_t)p.rows.L);
  if (p.transposed) hipLaunchKernelGGL((lora_outer_sum_kernel<TYPE, true>), sum, dim3(256), 0, s, p, rows);
  else hipLaunchKernelGGL((lora_outer_sum_kernel<TYPE, false>), sum, dim3(256), 0, s, p, rows);
  return hipGetLastError();
}
hipError_t launch_lora_outer(const LoraOuter& p, hipStream_t s) {
  const bool v = vec16(p.x, p.ldx, p.C);
  if (p.type == MM_BF16) return v ? run_outer<MM_BF16, true>(p, s) : run_outer<MM_BF16, false>(p, s);
  return v ? run_outer<MM_FP16, true>(p, s) : run_outer<MM_FP16, false>(p, s);
}

// ----------------------------------------------------------------------------- transposed weights
// dst[l][c][r] = src[l][r][c] through 64 x 64 tiles, two stacks in one launch; adapters without rows are
// left out.
struct TransposeArgs {
  LoraTranspose t[2];
  int64_t tiles[2], cols[2];      // tiles of one adapter, and along C
  const int32_t* count;
};
__global__ __launch_bounds__(256) void lora_transpose_kernel(TransposeArgs a) {
  __shared__ uint16_t s[64][66];
  const int l = blockIdx.y;
  if (a.count[l] <= 0) return;
  const int w = blockIdx.x < a.tiles[0] ? 0 : 1;
  const int64_t i = blockIdx.x - (w ? a.tiles[0] : 0);
  const LoraTranspose t = a.t[w];
  const int64_t r0 = i / a.cols[w] * 64, c0 = i % a.cols[w] * 64;
  const uint16_t* src = static_cast<const uint16_t*>(t.src) + l * t.src_stride;
  uint16_t* dst = static_cast<uint16_t*>(t.dst) + l * t.dst_stride;
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  uint16_t v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t r = r0 + y + 4 * i;
    v[i] = r < t.R && c0 + x < t.C ? src[r * t.lds + c0 + x] : (uint16_t)0;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) s[y + 4 * i][x] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t c = c0 + y + 4 * i;
    if (c < t.C && r0 + x < t.ldd) dst[c * t.ldd + r0 + x] = s[x][y + 4 * i];
  }
}
hipError_t launch_lora_transpose(const LoraTranspose* t, int n, const int32_t* count, int L, hipStream_t s) {
  TransposeArgs a{};
  for (int i = 0; i < n; ++i) {
    a.t[i] = t[i];
    a.cols[i] = (t[i].C + 63) / 64;
    a.tiles[i] = a.cols[i] * ((t[i].R + 63) / 64);
  }
  a.count = count;
  hipLaunchKernelGGL(lora_transpose_kernel, dim3((uint32_t)(a.tiles[0] + a.tiles[1]), (uint32_t)L), dim3(256), 0, s, a);
  return hipGetLastError();
}

__global__ void zero16_kernel(uint16_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) p[i] = 0;
}
hipError_t launch_zero16(void* p, int64_t n, hipStream_t s) {
  const int64_t blocks = std::min<int64_t>((n + 255) / 256, 4096);
  hipLaunchKernelGGL(zero16_kernel, dim3((uint32_t)blocks), dim3(256), 0, s, static_cast<uint16_t*>(p), n);
  return hipGetLastError();
}

}  // namespace gmlp
