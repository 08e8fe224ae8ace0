// Grouped products on bf16 / fp16 operands, rows grouped by expert with ragged sizes:
//   FPROP  y[r, :] = x[r, :] w[g]^T      DGRAD  dx[r, :] = dy[r, :] w[g]      WGRAD  dw[g] = dy_g^T x_g
// accumulated in fp32 on the matrix cores and rounded once.  The split sizes are read on the
// device by every workgroup (mm_common.h).
#include "mm_common.h"

#include <algorithm>

namespace gmlp {

// ----------------------------------------------------------------------------- any alignment
// 64 x 64 tile, 4 waves of 32 x 32, 32-deep stages through registers into LDS, every element
// checked.  Takes every stride, size and alignment; what the 16-byte loads of the other kernels
// cannot read runs here.
constexpr int ST = 64, SK = 32, SLD = SK + 8;

template <int TYPE, int LAYOUT, int OUT>
__global__ __launch_bounds__(256) void gmm_any_kernel(MmArgs p) {
  using E = Elem<TYPE>;
  __shared__ uint16_t sa[ST * SLD], sb[ST * SLD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (blockIdx.x == 0 && wave == 0) {
    const uint32_t f = wave_split_flags(p.m_splits, p.G, p.M, lane);
    if (lane == 0) *p.flags = f;
  }
  const uint16_t* A = static_cast<const uint16_t*>(p.a);
  const uint16_t* B = static_cast<const uint16_t*>(p.b);
  int64_t crow0, kn;                 // first C row of the tile, contraction length
  int arows, bcols, col0;            // valid rows and columns of the tile, first column
  if (LAYOUT == MM_WGRAD) {
    const uint32_t ntm = (p.n + ST - 1) / ST, ntn = (p.k + ST - 1) / ST;
    const int g = (int)(blockIdx.x / (ntm * ntn));
    const uint32_t t = blockIdx.x % (ntm * ntn);
    const RowTile rt = find_group_rows(p.m_splits, p.G, (uint32_t)p.M, g, lane);
    const int tm = t % ntm * ST;
    col0 = t / ntm * ST;
    arows = min(ST, p.n - tm);
    bcols = min(ST, p.k - col0);
    kn = rt.m;
    A += (int64_t)rt.row0 * p.lda + tm;
    B += (int64_t)rt.row0 * p.ldb + col0;
    crow0 = tm;
    p.c = static_cast<uint8_t*>(p.c) + (int64_t)g * p.c_stride * (OUT == MM_OUT_SAME ? 2 : 4);
    if (OUT == MM_OUT_ACC32 && kn == 0) return;
  } else {
    const uint32_t ntn = (p.n + ST - 1) / ST;
    const RowTile rt = find_row_tile(p.m_splits, p.G, (uint32_t)p.M, ST, ntn, p.zero_rest, blockIdx.x, lane);
    if (rt.g < 0) return;
    const uint32_t tm = rt.t / ntn * ST;
    col0 = rt.t % ntn * ST;
    arows = min((uint32_t)ST, rt.m - tm);
    bcols = min(ST, p.n - col0);
    kn = rt.g < p.G ? p.k : 0;
    crow0 = (int64_t)rt.row0 + tm;
    A += crow0 * p.lda;
    if (rt.g < p.G) B += (int64_t)rt.g * p.b_stride + (LAYOUT == MM_FPROP ? (int64_t)col0 * p.ldb : (int64_t)col0);
  }
  constexpr bool AT = LAYOUT == MM_WGRAD, BT = LAYOUT != MM_FPROP;     // contraction along the rows in memory
  auto load = [&](const uint16_t* src, int64_t ld, bool tr, int valid, int64_t k0, uint16_t* dst) {
    if (!tr) {
      const int r = tid >> 2, c = (tid & 3) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        dst[r * SLD + c + i] = (r < valid && k0 + c + i < kn) ? src[r * ld + k0 + c + i] : (uint16_t)0;
    } else {
      const int r = tid >> 3, c = (tid & 7) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        dst[(c + i) * SLD + r] = (c + i < valid && k0 + r < kn) ? src[(k0 + r) * ld + c + i] : (uint16_t)0;
    }
  };
  v16f acc = {};
  const int wm = wave >> 1, wn = wave & 1;
  for (int64_t k0 = 0; k0 < kn; k0 += SK) {
    load(A, p.lda, AT, arows, k0, sa);
    load(B, p.ldb, BT, bcols, k0, sb);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < SK; s += 16) {
      const int o = (lane & 31) * SLD + s + 8 * (lane >> 5);
      const v4i fa = *reinterpret_cast<const v4i*>(sa + wm * 32 * SLD + o);
      const v4i fb = *reinterpret_cast<const v4i*>(sb + wn * 32 * SLD + o);
      acc = E::mma32(fa, fb, acc);
    }
    __syncthreads();
  }
  // lane l, element i: row 8 (i / 4) + 4 (l / 32) + i % 4, column l % 32
  const int c = wn * 32 + (lane & 31);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = wm * 32 + 8 * (i / 4) + 4 * (lane >> 5) + (i & 3);
    if (r >= arows || c >= bcols) continue;
    const int64_t o = (crow0 + r) * p.ldc + col0 + c;
    if (OUT == MM_OUT_SAME) static_cast<uint16_t*>(p.c)[o] = E::down(acc[i]);
    else if (OUT == MM_OUT_FP32) static_cast<float*>(p.c)[o] = acc[i];
    else static_cast<float*>(p.c)[o] += acc[i];
  }
}

// The most row tiles of height h that any splits of M rows give: at most min(G + 1, M) runs of rows
// (the groups and the rows behind them), each with less than one tile of padding.
static int64_t row_tiles_bound(const MmArgs& p, int h) {
  return (p.M + (h - 1) * std::min<int64_t>((int64_t)p.G + 1, p.M)) / h;
}

template <int TYPE, int LAYOUT, int OUT>
static hipError_t run_any(const MmArgs& p, hipStream_t s) {
  int64_t grid;
  if (LAYOUT == MM_WGRAD) grid = (int64_t)p.G * ((p.n + ST - 1) / ST) * ((p.k + ST - 1) / ST);
  else grid = row_tiles_bound(p, ST) * ((p.n + ST - 1) / ST);
  grid = std::max<int64_t>(grid, 1);
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gmm_any_kernel<TYPE, LAYOUT, OUT>), dim3((uint32_t)grid), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <int TYPE>
static hipError_t run_type(const MmArgs& p, hipStream_t s) {
  if (p.layout == MM_FPROP) return run_any<TYPE, MM_FPROP, MM_OUT_SAME>(p, s);
  if (p.layout == MM_DGRAD) return run_any<TYPE, MM_DGRAD, MM_OUT_SAME>(p, s);
  if (p.out == MM_OUT_SAME) return run_any<TYPE, MM_WGRAD, MM_OUT_SAME>(p, s);
  if (p.out == MM_OUT_FP32) return run_any<TYPE, MM_WGRAD, MM_OUT_FP32>(p, s);
  return run_any<TYPE, MM_WGRAD, MM_OUT_ACC32>(p, s);
}

hipError_t launch_grouped_matmul(const MmArgs& p, hipStream_t s) {
  return p.type == MM_BF16 ? run_type<MM_BF16>(p, s) : run_type<MM_FP16>(p, s);
}

}  // namespace gmlp
