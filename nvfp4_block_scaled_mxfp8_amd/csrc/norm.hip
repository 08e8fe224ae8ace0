// The residual sum behind a block with the norms on both sides of it, and its gradients:
//   n = b rb wb, rb = (mean b^2 + eps)^-1/2;  y = x + s g n;  h = y ry w, ry = (mean y^2 + eps)^-1/2
// Bound by memory: forward 8 bytes an element (x, branch, y, h), backward 12 (x, branch, dy, dh, dx, dbranch).
//
// A row belongs to one workgroup (rows of up to 2048 in the forward: to one wave), 8 C values a thread in registers, so
// that each tensor is read once.  Squares are summed in 64 bits: a square of a 16-bit value is exact in them, and
// neither the largest nor the smallest rows leave their range (the conversions hide behind the loads).
#include "block_ops.h"
#include "block_sizes.h"
#include "mm_common.h"
#include "wave_ops.h"

namespace gmlp {

// ----------------------------------------------------------------------------- eight values
// The hardware takes any alignment; the last values of a row that is not whole eights go one by one.
template <int TYPE>
__device__ __forceinline__ void load8(const void* base, int64_t at, int valid, float* f) {
  using E = Elem<TYPE>;
  const uint16_t* p = static_cast<const uint16_t*>(base) + at;
  uint16_t e[8] = {};
  if (valid >= 8) {
    __builtin_memcpy(e, p, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) e[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = E::up(e[i]);
}
template <int TYPE>
__device__ __forceinline__ void store8(void* base, int64_t at, int valid, const float* f) {
  using E = Elem<TYPE>;
  uint16_t* p = static_cast<uint16_t*>(base) + at;
  if (valid >= 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = E::down2(f[2 * i], f[2 * i + 1]);
    __builtin_memcpy(p, w, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = E::down(f[i]);
  }
}
// Parameters: of the rows' type or fp32.
template <int TYPE>
__device__ __forceinline__ void load8p(const void* base, int fp32, int64_t at, int valid, float* f) {
  if (!fp32) return load8<TYPE>(base, at, valid, f);
  const float* p = static_cast<const float*>(base) + at;
  if (valid >= 8) {
    __builtin_memcpy(f, p, 32);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < valid ? p[i] : 0.0f;
  }
}
template <int TYPE>
__device__ __forceinline__ void store1p(void* base, int fp32, int64_t at, float v) {
  if (fp32) static_cast<float*>(base)[at] = v;
  else static_cast<uint16_t*>(base)[at] = Elem<TYPE>::down(v);
}
template <int TYPE>
__device__ __forceinline__ float load1p(const void* base, int fp32, int64_t at) {
  return fp32 ? static_cast<const float*>(base)[at] : Elem<TYPE>::up(static_cast<const uint16_t*>(base)[at]);
}

// Sum over the row's threads: a wave, or the workgroup's waves in order through LDS.
template <bool WAVE, class T>
__device__ __forceinline__ T row_sum(T v, T* lds, int waves) {
  v = lanes_sum<64>(v);
  if constexpr (WAVE) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  T s = lds[0];
  for (int w = 1; w < waves; ++w) s += lds[w];
  return s;
}
__device__ __forceinline__ float inv_root(double sum, int H, float eps) { return (float)(1.0 / sqrt(sum / H + (double)eps)); }

// ----------------------------------------------------------------------------- forward
template <int TYPE, int C, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_kernel(NormArgs p) {
  __shared__ double s_red[2][16];
  const int waves = blockDim.x >> 6;
  const int64_t block = (int64_t)blockIdx.x + (int64_t)blockIdx.y * p.row_blocks;
  const int64_t t = WAVE ? block * waves + (threadIdx.x >> 6) : block;
  const int tid = WAVE ? threadIdx.x & 63 : threadIdx.x, nt = WAVE ? 64 : blockDim.x;
  if (t >= p.T) return;                                        // WAVE: whole waves; else whole workgroups
  const int H = p.H;
  float y[C][8], b[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = (c * nt + tid) * 8;
    load8<TYPE>(p.x, t * p.ldx + at, H - at, y[c]);
  }
  if (p.branch) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * nt + tid) * 8;
      load8<TYPE>(p.branch, t * p.ldbranch + at, H - at, b[c]);
    }
    float rb = 1.0f;
    if (p.branch_weight) {
      double ss = 0.0;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma((double)b[c][i], (double)b[c][i], ss);
      rb = inv_root(row_sum<WAVE>(ss, s_red[0], waves), H, p.eps);
      if (p.stats && tid == 0) p.stats[t] = rb;
    }
    const float st = p.gate_kind == GATE_TOKEN ? p.scale * load1p<TYPE>(p.gate, p.gate_fp32, t * p.ld_gate) : p.scale;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * nt + tid) * 8;
      float f[8];
      if (p.branch_weight) {
        load8p<TYPE>(p.branch_weight, p.branch_weight_fp32, at, H - at, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[c][i] = b[c][i] * rb * f[i];
      }
      if (p.gate_kind == GATE_CHANNEL || p.gate_kind == GATE_FULL) {
        load8p<TYPE>(p.gate, p.gate_fp32, (p.gate_kind == GATE_FULL ? t * p.ld_gate : 0) + at, H - at, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[c][i] *= f[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[c][i] = fmaf(st, b[c][i], y[c][i]);
      store8<TYPE>(p.y, t * p.ldy + at, H - at, y[c]);
    }
  }
  if (!p.weight) return;
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma((double)y[c][i], (double)y[c][i], ss);
  const float ry = inv_root(row_sum<WAVE>(ss, s_red[1], waves), H, p.eps);
  if (p.stats && tid == 0) p.stats[p.T + t] = ry;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = (c * nt + tid) * 8;
    float f[8];
    load8p<TYPE>(p.weight, p.weight_fp32, at, H - at, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = y[c][i] * ry * f[i];
    store8<TYPE>(p.h, t * p.ldh + at, H - at, f);
  }
}

// ----------------------------------------------------------------------------- backward
// With u = dh w and yh = y ry:    d = dx = dy + ry (u - yh mean(u yh))
// With q = s g d and bh = b rb:   dbranch = rb (q wb - bh mean(q wb bh)), or q without a branch norm
//   dgate = s d n (summed over the columns: by token; over the rows: by channel), dweight = sum of dh yh,
//   dbranch_weight = sum of q bh
// mean(q wb bh) = s mean(g n d) opens into sums of g n dy, g n u and g n yh, so a row has one reduction.
// Workgroups take rows in turn and keep their column sums in registers; a second launch adds the workgroups'
// sums in order.
struct RowSums {
  float uy, ndy, nu, ny;
};
template <int TYPE, int C>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormArgs p) {
  __shared__ RowSums s_red[2][16];
  const int tid = threadIdx.x, nt = blockDim.x, waves = nt >> 6, H = p.H;
  float w[C][8], wb[C][8], g[C][8];
  float aw[C][8] = {}, ab[C][8] = {}, ag[C][8] = {};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = (c * nt + tid) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[c][i] = wb[c][i] = g[c][i] = 1.0f;
    if (p.weight) load8p<TYPE>(p.weight, p.weight_fp32, at, H - at, w[c]);
    if (p.branch_weight) load8p<TYPE>(p.branch_weight, p.branch_weight_fp32, at, H - at, wb[c]);
    if (p.gate_kind == GATE_CHANNEL) load8p<TYPE>(p.gate, p.gate_fp32, at, H - at, g[c]);
  }
  int turn = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
    float x[C][8], b[C][8] = {}, dy[C][8] = {}, dh[C][8] = {};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * nt + tid) * 8;
      load8<TYPE>(p.x, t * p.ldx + at, H - at, x[c]);
      if (p.branch) load8<TYPE>(p.branch, t * p.ldbranch + at, H - at, b[c]);
      if (p.dy) load8<TYPE>(p.dy, t * p.lddy + at, H - at, dy[c]);
      if (p.weight) load8<TYPE>(p.dh, t * p.lddh + at, H - at, dh[c]);
      if (p.gate_kind == GATE_FULL) load8p<TYPE>(p.gate, p.gate_fp32, t * p.ld_gate + at, H - at, g[c]);
    }
    const float rb = p.branch_weight ? p.stats[t] : 1.0f;
    const float ry = p.weight ? p.stats[p.T + t] : 0.0f;
    const float gt = p.gate_kind == GATE_TOKEN ? load1p<TYPE>(p.gate, p.gate_fp32, t * p.ld_gate) : 1.0f;
    // x becomes yh, b becomes bh
    RowSums s{};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        b[c][i] *= rb;
        const float n = b[c][i] * wb[c][i], gn = g[c][i] * n;
        x[c][i] = fmaf(p.scale * gt, gn, x[c][i]) * ry;
        const float u = dh[c][i] * w[c][i];
        s.uy = fmaf(u, x[c][i], s.uy);
        s.ndy = fmaf(gn, dy[c][i], s.ndy);
        s.nu = fmaf(gn, u, s.nu);
        s.ny = fmaf(gn, x[c][i], s.ny);
      }
    s.uy = lanes_sum<64>(s.uy);
    s.ndy = lanes_sum<64>(s.ndy);
    s.nu = lanes_sum<64>(s.nu);
    s.ny = lanes_sum<64>(s.ny);
    if ((tid & 63) == 0) s_red[turn][tid >> 6] = s;
    __syncthreads();                     // the other turn's slots are free: every thread has read them
    s = s_red[turn][0];
    for (int i = 1; i < waves; ++i) {
      const RowSums o = s_red[turn][i];
      s.uy += o.uy;
      s.ndy += o.ndy;
      s.nu += o.nu;
      s.ny += o.ny;
    }
    const float c1 = s.uy / (float)H;
    const float gnd = s.ndy + ry * (s.nu - c1 * s.ny);         // sum of g n d
    const float c2 = p.branch_weight ? p.scale * gt * gnd / (float)H : 0.0f;
    if (p.dgate && p.gate_kind == GATE_TOKEN && tid == 0) store1p<TYPE>(p.dgate, p.gate_fp32, t, p.scale * gnd);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * nt + tid) * 8;
      float d[8], o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = dy[c][i] + ry * (dh[c][i] * w[c][i] - x[c][i] * c1);
        aw[c][i] = fmaf(dh[c][i], x[c][i], aw[c][i]);
      }
      if (p.dx) store8<TYPE>(p.dx, t * p.lddx + at, H - at, d);
      if (!p.branch) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] *= p.scale * gt;
        o[i] = d[i] * b[c][i] * wb[c][i];
        ag[c][i] += o[i];
        d[i] *= g[c][i];
        ab[c][i] = fmaf(d[i], b[c][i], ab[c][i]);
      }
      if (p.dgate && p.gate_kind == GATE_FULL) {
        if (p.gate_fp32) {
          float* q = static_cast<float*>(p.dgate) + t * H + at;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (at + i < H) q[i] = o[i];
        } else {
          store8<TYPE>(p.dgate, t * H + at, H - at, o);
        }
      }
      if (p.dbranch) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = p.branch_weight ? rb * (d[i] * wb[c][i] - b[c][i] * c2) : d[i];
        store8<TYPE>(p.dbranch, t * p.lddbranch + at, H - at, o);
      }
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * H;
  const int64_t stride = (int64_t)gridDim.x * H;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = (c * nt + tid) * 8 + i;
      if (at >= H) continue;
      if (p.dweight) part[at] = aw[c][i];
      if (p.dbranch_weight) part[stride + at] = ab[c][i];
      if (p.dgate && p.gate_kind == GATE_CHANNEL) part[2 * stride + at] = ag[c][i];
    }
}

// Column sums over the workgroups' parts: 64 columns a workgroup, its waves a sixteenth of the parts each.
template <int TYPE>
__global__ __launch_bounds__(1024) void norm_columns_kernel(NormArgs p, int parts) {
  __shared__ float s_sum[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, which = blockIdx.y;
  const int at = blockIdx.x * 64 + lane;
  void* out = which == 0 ? p.dweight : which == 1 ? p.dbranch_weight : p.gate_kind == GATE_CHANNEL ? p.dgate : nullptr;
  const int fp32 = which == 0 ? p.weight_fp32 : which == 1 ? p.branch_weight_fp32 : p.gate_fp32;
  if (!out) return;
  const float* part = p.part + (int64_t)which * parts * p.H;
  float s = 0.0f;
  if (at < p.H)
    for (int i = wave; i < parts; i += 16) s += part[(int64_t)i * p.H + at];
  s_sum[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || at >= p.H) return;
  for (int i = 1; i < 16; ++i) s += s_sum[i][lane];
  store1p<TYPE>(out, fp32, at, s);
}

// ----------------------------------------------------------------------------- launches
template <int TYPE, int C, bool WAVE>
static hipError_t run_norm(NormArgs p, hipStream_t s) {
  const int threads = WAVE ? 256 : sizes::norm_threads(p.H, C);
  const FoldedGrid g = fold_grid(WAVE ? (p.T + 3) / 4 : p.T, threads);
  p.row_blocks = g.x;
  hipLaunchKernelGGL((norm_kernel<TYPE, C, WAVE>), dim3(g.x, g.y), dim3(threads), 0, s, p);
  return hipGetLastError();
}
template <int TYPE>
static hipError_t run_norm(const NormArgs& p, hipStream_t s) {
  const int chunks = (p.H + 7) / 8;
  if (chunks <= 64) return run_norm<TYPE, 1, true>(p, s);
  if (chunks <= 128) return run_norm<TYPE, 2, true>(p, s);
  if (chunks <= 256) return run_norm<TYPE, 4, true>(p, s);
  if (chunks <= 2048) return run_norm<TYPE, 2, false>(p, s);
  return run_norm<TYPE, 4, false>(p, s);
}
hipError_t launch_norm(const NormArgs& p, hipStream_t s) {
  return p.type == MM_BF16 ? run_norm<MM_BF16>(p, s) : run_norm<MM_FP16>(p, s);
}

template <int TYPE, int C>
static hipError_t run_backward(const NormArgs& p, hipStream_t s) {
  const int blocks = sizes::norm_bwd_blocks(p.T);
  hipLaunchKernelGGL((norm_backward_kernel<TYPE, C>), dim3(blocks), dim3(sizes::norm_threads(p.H, C)), 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (!p.dweight && !p.dbranch_weight && !(p.dgate && p.gate_kind == GATE_CHANNEL)) return e;
  hipLaunchKernelGGL((norm_columns_kernel<TYPE>), dim3((p.H + 63) / 64, 3), dim3(1024), 0, s, p, blocks);
  return hipGetLastError();
}
template <int TYPE>
static hipError_t run_backward(const NormArgs& p, hipStream_t s) {
  const int chunks = (p.H + 7) / 8;
  if (chunks <= 256) return run_backward<TYPE, 1>(p, s);
  if (chunks <= 2048) return run_backward<TYPE, 2>(p, s);
  return run_backward<TYPE, 4>(p, s);
}
hipError_t launch_norm_backward(const NormArgs& p, hipStream_t s) {
  return p.type == MM_BF16 ? run_backward<MM_BF16>(p, s) : run_backward<MM_FP16>(p, s);
}

}  // namespace gmlp
