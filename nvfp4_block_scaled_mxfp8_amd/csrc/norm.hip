// The residual sum behind a block with the norms on both sides of it, and its gradients:
//   n = b rb wb, rb = (mean b^2 + eps)^-1/2;  y = x + s g n;  h = y ry w, ry = (mean y^2 + eps)^-1/2
// Bound by memory: forward 8 bytes an element (x, branch, y, h), backward 12 (x, branch, dy, dh, dx, dbranch).
//
// 8192 rows of 7168 (bf16, fp32 parameters): forward 100 to 104 us (4.6 TB/s), backward 165 to 180 and 6 us of column sums (4.0 TB/s;
// a copy reaches 4.9).
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
// Loads without branches, so that many are in flight (the hardware takes any alignment): the eight at a row's ragged
// end, and those of threads behind it, are the row's last eight, moved down where they are used; rows of fewer
// than eight (SHORT) go one by one.  partial (uniform): there are such threads.
template <bool SHORT>
__device__ __forceinline__ v4i raw8(const void* base, int64_t row, int at, int H) {
  const uint16_t* p = static_cast<const uint16_t*>(base) + row;
  if constexpr (SHORT) return load8_short(p + at, H - at);
  v4i v;
  __builtin_memcpy(&v, p + min(at, H - 8), 16);
  return v;
}
template <int TYPE, bool SHORT>
__device__ __forceinline__ void up8(v4i v, int valid, bool partial, float* f) {
  if (!SHORT && partial) v = shift8(v, valid);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = Elem<TYPE>::up((uint16_t)((uint32_t)v[i / 2] >> (16 * (i & 1))));
}
// Parameters: of the rows' type or fp32.
template <int TYPE, bool SHORT>
__device__ __forceinline__ void load8p(const void* base, int fp32, int64_t row, int at, int H, bool partial, float* f) {
  if (!fp32) return up8<TYPE, SHORT>(raw8<SHORT>(base, row, at, H), H - at, partial, f);
  const float* p = static_cast<const float*>(base) + row;
  if (!SHORT && !partial) {
    __builtin_memcpy(f, p + at, 32);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = p[min(at + i, H - 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = at + i < H ? f[i] : 0.0f;
  }
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
// The factor 1 / sqrt(mean + eps).  Without eps, that of a row below 2^-127 (but not of zeros, whose is infinite) has no
// place in fp32: then the row is multiplied by kTinyRow, exactly, and the factor is for that; stats hold it with a minus.
constexpr float kTinyRow = 0x1p64f;
struct RowFactor {
  float f, row;
  __device__ __forceinline__ float stat() const { return row == 1.0f ? f : -f; }
};
__device__ __forceinline__ RowFactor inv_root(double sum, int H, float eps) {
  const double f = 1.0 / sqrt(sum / H + (double)eps);
  if (eps == 0.0f && f > 0x1p127 && f < (double)INFINITY) return {(float)(f * 0x1p-64), kTinyRow};
  return {(float)f, 1.0f};
}
// Of a workgroup's row; TINY: it may be such a row.
template <bool TINY>
__device__ __forceinline__ RowFactor row_factor(float stat) {
  if (!TINY) return {stat, 1.0f};
  return {fabsf(stat), stat < 0.0f ? kTinyRow : 1.0f};
}

// ----------------------------------------------------------------------------- forward
template <int TYPE, int C, bool WAVE, bool SHORT>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_kernel(NormArgs p) {
  __shared__ double s_red[2][16];
  const int waves = blockDim.x >> 6;
  const int64_t block = (int64_t)blockIdx.x + (int64_t)blockIdx.y * p.row_blocks;
  const int64_t t = WAVE ? block * waves + (threadIdx.x >> 6) : block;
  const int tid = WAVE ? threadIdx.x & 63 : threadIdx.x, nt = WAVE ? 64 : blockDim.x;
  if (t >= p.T) return;                                        // WAVE: whole waves; else whole workgroups
  const int H = p.H;
  const bool partial = H != nt * C * 8;
  v4i xr[C], br[C];
#pragma unroll
  for (int c = 0; c < C; ++c) xr[c] = raw8<SHORT>(p.x, t * p.ldx, (c * nt + tid) * 8, H);
  if (p.branch)
#pragma unroll
    for (int c = 0; c < C; ++c) br[c] = raw8<SHORT>(p.branch, t * p.ldbranch, (c * nt + tid) * 8, H);
  float y[C][8];
  if (p.branch) {
    float b[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) up8<TYPE, SHORT>(br[c], H - (c * nt + tid) * 8, partial, b[c]);
    float rb = 1.0f;
    if (p.branch_weight) {
      double ss = 0.0;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma((double)b[c][i], (double)b[c][i], ss);
      const RowFactor r = inv_root(row_sum<WAVE>(ss, s_red[0], waves), H, p.eps);
      rb = r.f;
      if (p.stats && tid == 0) p.stats[t] = r.stat();
      if (r.row != 1.0f)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) b[c][i] *= r.row;
    }
    const float st = p.gate_kind == GATE_TOKEN ? p.scale * load1p<TYPE>(p.gate, p.gate_fp32, t * p.ld_gate) : p.scale;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * nt + tid) * 8;
      float f[8];
      if (p.branch_weight) {
        load8p<TYPE, SHORT>(p.branch_weight, p.branch_weight_fp32, 0, at, H, partial, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[c][i] = b[c][i] * rb * f[i];
      }
      if (p.gate_kind == GATE_CHANNEL || p.gate_kind == GATE_FULL) {
        load8p<TYPE, SHORT>(p.gate, p.gate_fp32, p.gate_kind == GATE_FULL ? t * p.ld_gate : 0, at, H, partial, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[c][i] *= f[i];
      }
      up8<TYPE, SHORT>(xr[c], H - at, partial, y[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[c][i] = fmaf(st, b[c][i], y[c][i]);
      store8<TYPE>(p.y, t * p.ldy + at, H - at, y[c]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) up8<TYPE, SHORT>(xr[c], H - (c * nt + tid) * 8, partial, y[c]);
  }
  if (!p.weight) return;
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma((double)y[c][i], (double)y[c][i], ss);
  const RowFactor r = inv_root(row_sum<WAVE>(ss, s_red[1], waves), H, p.eps);
  const float ry = r.f;
  if (p.stats && tid == 0) p.stats[p.T + t] = r.stat();
  if (r.row != 1.0f)
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[c][i] *= r.row;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = (c * nt + tid) * 8;
    float f[8];
    load8p<TYPE, SHORT>(p.weight, p.weight_fp32, 0, at, H, partial, f);
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
// Workgroups take rows in turn, the next row's loads in flight (rows of up to 8192), the parameters in LDS, and keep
// their column sums in registers; a second launch adds the workgroups' sums in order.  What made the difference on 8192
// rows of 7168: loads by branches on the row's end 425 us; without branches but with selects for absent inputs and 1024
// threads' 128 registers (spills wait for the row ahead) 464; 512 threads 308; no selects 220; values of four
// columns live at once 171 (with 1024 threads 213).
// Rows above 8192 have 32 values a thread: no row ahead, parameters by element, and registers spilled; 4096 x 12288 1100 us,
// 4096 x 16384 1350, 2048 x 32768 2290.
struct RowSums {
  float uy, ndy, nu, ny;
};
enum { BWD_GATE_NONE, BWD_GATE_CHANNEL, BWD_GATE_FULL, BWD_GATE_FULL32 };      // none: or by token
template <int C>
struct RawRow {
  v4i x[C], b[C], dy[C], dh[C], g[C];      // g: a gate of every element, 16 bits
};
// Four of the eight.
template <int TYPE>
__device__ __forceinline__ void up4(v4i v, int half, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = Elem<TYPE>::up((uint16_t)((uint32_t)v[2 * half + i / 2] >> (16 * (i & 1))));
}
__device__ __forceinline__ void store_raw(void* base, int64_t at, int valid, v4i v) {
  uint16_t* p = static_cast<uint16_t*>(base) + at;
  if (valid >= 8) {
    __builtin_memcpy(p, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = (uint16_t)((uint32_t)v[i / 2] >> (16 * (i & 1)));
  }
}
template <int TYPE, int C, int MAXT, int GATE, bool SHORT, bool TINY>
__global__ __launch_bounds__(MAXT) void norm_backward_kernel(NormArgs p) {
  constexpr bool AHEAD = C <= 2;         // the next row in registers, the parameters in LDS
  extern __shared__ __align__(16) float s_param[];     // [3][P]: weight, branch_weight, gate by channel
  __shared__ RowSums s_red[2][16];
  const int tid = threadIdx.x, nt = blockDim.x, waves = nt >> 6, H = p.H, P = nt * C * 8;
  float aw[C][8] = {}, ab[C][8] = {}, ag[C][8] = {};
  const bool post = p.branch_weight != nullptr, partial = H != P;
  // four parameters: w is 0 without a weight, wb 1 without a branch norm
  auto param = [&](int which, const void* base, int fp32, int at, float* f) {
    if (AHEAD) {
      const v4f v = *reinterpret_cast<const v4f*>(s_param + which * P + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = !base ? (which == 0 ? 0.0f : 1.0f) : at + i < H ? load1p<TYPE>(base, fp32, at + i) : 0.0f;
    }
  };
  if (AHEAD) {                           // each thread reads back its own values only
    auto keep = [&](int which, const void* base, int fp32) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int at = (c * nt + tid) * 8;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = which == 0 ? 0.0f : 1.0f;
        if (base) load8p<TYPE, SHORT>(base, fp32, 0, at, H, partial, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s_param[which * P + at + i] = f[i];
      }
    };
    keep(0, p.weight, p.weight_fp32);
    keep(1, p.branch_weight, p.branch_weight_fp32);
    if (GATE == BWD_GATE_CHANNEL) keep(2, p.gate, p.gate_fp32);
  }
  auto load = [&](int64_t t, RawRow<C>& r) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * nt + tid) * 8;
      r.x[c] = raw8<SHORT>(p.x, t * p.ldx, at, H);
      r.b[c] = p.branch ? raw8<SHORT>(p.branch, t * p.ldbranch, at, H) : v4i{0, 0, 0, 0};
      r.dy[c] = p.dy ? raw8<SHORT>(p.dy, t * p.lddy, at, H) : v4i{0, 0, 0, 0};
      r.dh[c] = p.weight ? raw8<SHORT>(p.dh, t * p.lddh, at, H) : v4i{0, 0, 0, 0};
      if (GATE == BWD_GATE_FULL) r.g[c] = raw8<SHORT>(p.gate, t * p.ld_gate, at, H);
    }
  };
  // bh, n, g n, yh, u = dh w of four columns from `at`, and the gate and wb
  auto columns = [&](int64_t t, const RawRow<C>& r, int c, int half, RowFactor rb, RowFactor ry, float gt, float* bh, float* n, float* g, float* wb,
                     float* yh, float* u, float* dh) {
    const int at = (c * nt + tid) * 8 + 4 * half;
    float x[4], w[4];
    up4<TYPE>(r.b[c], half, bh);
    up4<TYPE>(r.x[c], half, x);
    up4<TYPE>(r.dh[c], half, dh);
    param(0, p.weight, p.weight_fp32, at, w);
    param(1, p.branch_weight, p.branch_weight_fp32, at, wb);
    if (GATE == BWD_GATE_CHANNEL) param(2, p.gate, p.gate_fp32, at, g);
    if (GATE == BWD_GATE_FULL) up4<TYPE>(r.g[c], half, g);
    if (GATE == BWD_GATE_FULL32)
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = static_cast<const float*>(p.gate)[t * p.ld_gate + min(at + i, H - 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (GATE == BWD_GATE_NONE) g[i] = 1.0f;
      bh[i] = bh[i] * rb.row * rb.f;
      n[i] = bh[i] * wb[i];
      yh[i] = fmaf(gt, GATE == BWD_GATE_NONE ? n[i] : g[i] * n[i], x[i]) * ry.row * ry.f;
      u[i] = dh[i] * w[i];
    }
    if (!p.weight)                       // what is not finite in y stays out of the gradients that do not have it
#pragma unroll
      for (int i = 0; i < 4; ++i) yh[i] = 0.0f;
  };
  const float inv_h = 1.0f / (float)H;
  int turn = 0;
  RawRow<C> next;
  if (AHEAD && blockIdx.x < p.T) load(blockIdx.x, next);
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
    RawRow<C> r;
    if (AHEAD) {
      r = next;
      if (t + gridDim.x < p.T) load(t + gridDim.x, next);
    } else {
      load(t, r);
    }
    if (!SHORT && partial)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int valid = H - (c * nt + tid) * 8;
        r.x[c] = shift8(r.x[c], valid);
        r.b[c] = shift8(r.b[c], valid);
        r.dy[c] = shift8(r.dy[c], valid);
        r.dh[c] = shift8(r.dh[c], valid);
        if (GATE == BWD_GATE_FULL) r.g[c] = shift8(r.g[c], valid);
      }
    const RowFactor rb = row_factor<TINY>(post ? p.stats[t] : 1.0f);
    const RowFactor ry = row_factor<TINY>(p.weight ? p.stats[p.T + t] : 0.0f);
    const float gt = p.scale * (p.gate_kind == GATE_TOKEN ? load1p<TYPE>(p.gate, p.gate_fp32, t * p.ld_gate) : 1.0f);
    RowSums s{};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float bh[4], n[4], g[4], wb[4], yh[4], u[4], dh[4], dy[4];
        columns(t, r, c, half, rb, ry, gt, bh, n, g, wb, yh, u, dh);
        up4<TYPE>(r.dy[c], half, dy);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float gn = GATE == BWD_GATE_NONE ? n[i] : g[i] * n[i];
          s.ndy = fmaf(gn, dy[i], s.ndy);
          if (!p.weight) continue;
          s.uy = fmaf(u[i], yh[i], s.uy);
          s.nu = fmaf(gn, u[i], s.nu);
          s.ny = fmaf(gn, yh[i], s.ny);
        }
        __builtin_amdgcn_sched_barrier(0);      // a half's values only are live at once: no spills beside the row ahead
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
    const float c1 = s.uy * inv_h;
    const float gnd = p.weight ? s.ndy + ry.f * ((s.nu - c1 * s.ny) * ry.row) : s.ndy;      // sum of g n d
    const float c2 = post ? gt * gnd * inv_h : 0.0f;
    if (p.dgate && p.gate_kind == GATE_TOKEN && tid == 0) store1p<TYPE>(p.dgate, p.gate_fp32, t, p.scale * gnd);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * nt + tid) * 8;
      v4i dx, db, dg;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float bh[4], n[4], g[4], wb[4], yh[4], u[4], dh[4], d[4];
        columns(t, r, c, half, rb, ry, gt, bh, n, g, wb, yh, u, dh);
        up4<TYPE>(r.dy[c], half, d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          aw[c][4 * half + i] = fmaf(dh[i], yh[i], aw[c][4 * half + i]);
          d[i] = fmaf(ry.f, fmaf(-yh[i], c1, u[i]) * ry.row, d[i]);
        }
        dx[2 * half] = (int)Elem<TYPE>::down2(d[0], d[1]);
        dx[2 * half + 1] = (int)Elem<TYPE>::down2(d[2], d[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float q = gt * d[i];
          n[i] *= q;                                           // the gate's gradient
          if (GATE == BWD_GATE_CHANNEL) ag[c][4 * half + i] += n[i];
          d[i] = GATE == BWD_GATE_NONE ? q : q * g[i];
          ab[c][4 * half + i] = fmaf(d[i], bh[i], ab[c][4 * half + i]);
        }
        if (post)
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = rb.f * (fmaf(-bh[i], c2, d[i] * wb[i]) * rb.row);
        db[2 * half] = (int)Elem<TYPE>::down2(d[0], d[1]);
        db[2 * half + 1] = (int)Elem<TYPE>::down2(d[2], d[3]);
        if (GATE == BWD_GATE_FULL) {
          dg[2 * half] = (int)Elem<TYPE>::down2(n[0], n[1]);
          dg[2 * half + 1] = (int)Elem<TYPE>::down2(n[2], n[3]);
        }
        if (GATE == BWD_GATE_FULL32 && p.dgate) {
          float* out = static_cast<float*>(p.dgate) + t * H + at + 4 * half;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (at + 4 * half + i < H) out[i] = n[i];
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (p.dx) store_raw(p.dx, t * p.lddx + at, H - at, dx);
      if (p.dbranch) store_raw(p.dbranch, t * p.lddbranch + at, H - at, db);
      if (GATE == BWD_GATE_FULL && p.dgate) store_raw(p.dgate, t * H + at, H - at, dg);
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
      if (GATE == BWD_GATE_CHANNEL && p.dgate) part[2 * stride + at] = ag[c][i];
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
    for (int i0 = wave; i0 < parts; i0 += 16 * 8) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = i0 + 16 * j < parts ? part[(int64_t)(i0 + 16 * j) * p.H + at] : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
  s_sum[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || at >= p.H) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += s_sum[i][lane];
  store1p<TYPE>(out, fp32, at, s);
}

// ----------------------------------------------------------------------------- launches
template <int TYPE, int C, bool WAVE, bool SHORT = false>
static hipError_t run_norm(NormArgs p, hipStream_t s) {
  const int threads = WAVE ? 256 : sizes::norm_threads(p.H, C);
  const FoldedGrid g = fold_grid(WAVE ? (p.T + 3) / 4 : p.T, threads);
  p.row_blocks = g.x;
  hipLaunchKernelGGL((norm_kernel<TYPE, C, WAVE, SHORT>), dim3(g.x, g.y), dim3(threads), 0, s, p);
  return hipGetLastError();
}
template <int TYPE>
static hipError_t run_norm(const NormArgs& p, hipStream_t s) {
  // A wave a row up to 2048, then 16 values a thread: 8192 x 7168 98 us against 150 with 8, 2049 x 2048 (fp16) 11.6 us by waves
  // against 12.2 by workgroups of 8 a thread.
  const int chunks = (p.H + 7) / 8;
  if (p.H < 8) return run_norm<TYPE, 1, true, true>(p, s);
  if (chunks <= 64) return run_norm<TYPE, 1, true>(p, s);
  if (chunks <= 128) return run_norm<TYPE, 2, true>(p, s);
  if (chunks <= 256) return run_norm<TYPE, 4, true>(p, s);
  if (chunks <= 2048) return run_norm<TYPE, 2, false>(p, s);
  return run_norm<TYPE, 4, false>(p, s);
}
hipError_t launch_norm(const NormArgs& p, hipStream_t s) {
  return p.type == MM_BF16 ? run_norm<MM_BF16>(p, s) : run_norm<MM_FP16>(p, s);
}

template <int TYPE, int C, int MAXT, int GATE, bool SHORT>
static hipError_t run_backward(const NormArgs& p, hipStream_t s) {
  const int blocks = sizes::norm_bwd_blocks(p.T, p.H), threads = sizes::norm_threads(p.H, C);
  const size_t lds = C <= 2 ? 3 * 8 * C * sizeof(float) * threads : 0;
  // four more products a value for rows that only eps 0 can have: 8192 x 7168, a gate by channel 170 -> 181 us, by token 160 -> 192
  if (p.eps == 0.0f)
    hipLaunchKernelGGL((norm_backward_kernel<TYPE, C, MAXT, GATE, SHORT, true>), dim3(blocks), dim3(threads), lds, s, p);
  else
    hipLaunchKernelGGL((norm_backward_kernel<TYPE, C, MAXT, GATE, SHORT, false>), dim3(blocks), dim3(threads), lds, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (!p.dweight && !p.dbranch_weight && !(p.dgate && p.gate_kind == GATE_CHANNEL)) return e;
  hipLaunchKernelGGL((norm_columns_kernel<TYPE>), dim3((p.H + 63) / 64, 3), dim3(1024), 0, s, p, blocks);
  return hipGetLastError();
}
template <int TYPE, int C, int MAXT, bool SHORT = false>
static hipError_t run_backward(const NormArgs& p, hipStream_t s) {
  if (p.gate_kind == GATE_CHANNEL) return run_backward<TYPE, C, MAXT, BWD_GATE_CHANNEL, SHORT>(p, s);
  if (p.gate_kind != GATE_FULL) return run_backward<TYPE, C, MAXT, BWD_GATE_NONE, SHORT>(p, s);
  return p.gate_fp32 ? run_backward<TYPE, C, MAXT, BWD_GATE_FULL32, SHORT>(p, s) : run_backward<TYPE, C, MAXT, BWD_GATE_FULL, SHORT>(p, s);
}
template <int TYPE>
static hipError_t run_backward(const NormArgs& p, hipStream_t s) {
  const int chunks = (p.H + 7) / 8;
  if (p.H < 8) return run_backward<TYPE, 1, 512, true>(p, s);
  if (chunks <= 512) return run_backward<TYPE, 1, 512>(p, s);
  if (chunks <= 1024) return run_backward<TYPE, 2, 512>(p, s);
  if (chunks <= 2048) return run_backward<TYPE, 4, 512>(p, s);
  return run_backward<TYPE, 4, 1024>(p, s);
}
hipError_t launch_norm_backward(const NormArgs& p, hipStream_t s) {
  return p.type == MM_BF16 ? run_backward<MM_BF16>(p, s) : run_backward<MM_FP16>(p, s);
}

}  // namespace gmlp
