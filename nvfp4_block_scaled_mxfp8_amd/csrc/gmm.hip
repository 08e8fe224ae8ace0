// Grouped products on bf16 / fp16 operands, rows grouped by expert with ragged sizes:
//   FPROP  y[r, :] = x[r, :] w[g]^T      DGRAD  dx[r, :] = dy[r, :] w[g]      WGRAD  dw[g] = dy_g^T x_g
// accumulated in fp32 on the matrix cores and rounded once.  The split sizes are read on the
// device (mm_common.h).
#include "mm_common.h"
#include "op_sizes.h"

#include <algorithm>
#include <type_traits>

namespace gmlp {


// ----------------------------------------------------------------------------- ring kernel
// 128 x 128 tiles, 2 x 2 waves of 64 x 64, contraction in stages of 64.  A stage is two units, A's
// and B's 64-deep slabs of the tile (128 x 128 bytes each), and the units of all stages run through a
// ring of five LDS slots filled by buffer-to-LDS DMA: while stage s is read, both units of stage
// s + 1 and A of s + 2 are on their way.  One barrier a stage: at it every wave has the stage's last
// fragments in registers and its share of the next stage's units has landed, so the two slots read
// last are refilled and the next stage's first fragments read while the last sixteen-deep step's
// MFMAs run.  80 KB: two workgroups per CU, whose ends and beginnings overlap.
//
// A unit whose operand is contiguous along the contraction (x, dy and FPROP's w) holds rows of 128
// bytes, 16-byte chunks XOR-swizzled by row so that 16 consecutive rows meet all 16 bank groups;
// fragments are ds_read_b128.  A unit whose operand has the contraction along its rows in memory
// (DGRAD's w, both of WGRAD's) holds 64 rows of T elements as they are in memory; its fragments
// are transposed on the way out by ds_read_b64_tr_b16 (16 lanes read four rows of 16 elements and
// get one column of four each), chunks XORed by (row % 4) so that the four rows fall into four
// different 64-byte windows of the banks.  Conflicts: 1% of the LDS cycles (counter).
//
// Rows, columns and contraction past the operand's end read as zero by the buffer range check;
// a contraction tail inside a row (k % 64) is cut per lane in the last stage.
//
// Where rows are not multiples of 16 bytes the DMA cannot read them: the units then come through
// registers into two pairs of slots, 16 bytes per lane from any address; the ragged chunk at a row's
// end is the row's last eight elements, shifted down (by element in rows of fewer than eight).
//
// Few tiles with a long contraction (PART): the contraction is cut over blockIdx.y, each part's
// fp32 tile goes to scratch, and gmm_sum_kernel adds the parts in order.
//
// Measured: 64 rows over 128 experts of 4096 x 7168 470 to 520 us from run to run, 5.7 to 6.3 TB/s of
// weights (bound by their read); 6144 rows, Zipf over 60 of 64 experts of 2816 x 2048 (752 MB), 174 to 190 us,
// 4.0 to 4.3 TB/s (the large groups' MFMAs beside the small ones' reads); 32768 x 4096 x 1536, forward, 503 us, 820 TFLOP/s (bound by what
// 128-wide tiles fetch from L2; the stream's 256-wide ones take 430).  Unaligned rows: 16384 rows,
// 8 x 4095 x 2047, 730 us (4096 x 2048: 270), bound by the trip through registers.
constexpr int MM_OUT_PART = 3;

typedef __attribute__((address_space(3))) v4s lds_v4s;

__device__ __forceinline__ int sgpr(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t sgpr64(uint64_t v) {
  return (uint64_t)(uint32_t)sgpr((int)(uint32_t)v) | ((uint64_t)(uint32_t)sgpr((int)(uint32_t)(v >> 32)) << 32);
}
// 16 bytes per lane from a buffer into LDS at m0 + 16 lane.  Inline asm, as the compiler would wait
// for every outstanding DMA before each LDS read; the kernel counts them itself.  The compiler may
// have written the scalar operands by a vector instruction just before (a lane read), which a
// vector-memory instruction must not read for five wait states: the move and the s_nop are those.
// m0 is reserved, so the compiler keeps nothing in it; no code of its own here may use it (none does).
__device__ __forceinline__ void dma16(v4i rsrc, uint32_t voff, uint32_t soff, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(soff), "s"(m0) : "memory");
}
// The same, non-temporal where the tile's group has at most T rows (one row tile).  The comparison is
// part of the asm: a truth value would come out of a vector register.
template <int T>
__device__ __forceinline__ void dma16_once(v4i rsrc, uint32_t voff, uint32_t soff, uint32_t m0, uint32_t rows) {
  asm volatile("s_mov_b32 m0, %3\n\ts_cmp_gt_u32 %4, %5\n\ts_nop 2\n\ts_cbranch_scc1 L_all_%=\n\t"
               "buffer_load_dwordx4 %0, %1, %2 offen nt lds\n\ts_branch L_end_%=\n"
               "L_all_%=:\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds\nL_end_%=:"
               :: "v"(voff), "s"(rsrc), "s"(soff), "s"(m0), "s"(rows), "n"(T) : "memory", "scc");
}
template <int VM>
__device__ __forceinline__ void wait_stage() {      // all LDS reads back, at most VM DMAs in flight
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"(VM) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

constexpr uint32_t kNoLane = 0x80000000u;            // past every range: the lane reads zeros

// One operand's stream of units.  ONCE: non-temporal loads where the tile's group has no other row tile.
template <bool TR, int T, int NT, bool ONCE = false>
struct Feed {
  static constexpr int kDma = T * 128 / (NT * 16);   // DMAs per unit and wave
  uint64_t base;                // address of the current stage's unit
  int64_t rest;                 // !TR: bytes of all but the last valid row;  TR: bytes behind the current stage's first row
  int32_t left;                 // contraction elements from the current stage on (clamped)
  uint32_t voff, vtail;         // lane offset; in the last stage
  uint32_t step;                // bytes between a wave's DMAs of one unit
  uint32_t row_bytes;           // 2 ld
  uint32_t cols_bytes;          // TR: bytes from the tile's first column to the end of a row
  v4i rsrc;                     // the unit being issued
  uint32_t v;
  uint32_t group_rows;

  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld, int valid, int64_t kn, int tid) {
    base = sgpr64((uint64_t)(uintptr_t)p);
    row_bytes = (uint32_t)(2 * ld);
    left = sgpr((int)min(kn, (int64_t)0x40000000));
    if (!TR) {
      const int r = tid >> 3, c = (tid & 7) ^ ((r >> 1) & 7);
      voff = r * row_bytes + c * 16;
      vtail = 8 * c < ((left + 63) % 64 + 1) ? voff : kNoLane;
      step = (NT / 8) * row_bytes;
      rest = (int64_t)(valid - 1) * row_bytes;
    } else {
      constexpr int CPR = T / 8;
      const int r = tid / CPR, c = (tid % CPR) ^ ((r & 3) << 2);
      voff = 8 * c < valid ? r * row_bytes + c * 16 : kNoLane;
      vtail = voff;
      step = (NT / CPR) * row_bytes;
      cols_bytes = 2 * min(valid, T);
    }
  }
  // The unit's descriptor, then on to the next stage.
  __device__ __forceinline__ void next() {
    int32_t n;
    if (!TR) n = left > 0 ? (int32_t)rest + 2 * left : 0;
    else n = left > 0 ? (int32_t)min((uint64_t)(uint32_t)(left - 1) * row_bytes + cols_bytes, (uint64_t)0x7FFFFFFF) : 0;
    rsrc = v4i{(int)(uint32_t)base, (int)((uint32_t)(base >> 32) & 0xFFFFu), n, 0x00020000};
    v = left <= 64 ? vtail : voff;
    base += TR ? 64ull * row_bytes : 128ull;
    left -= 64;
  }
  // DMA number i of the unit (after next()).
  __device__ __forceinline__ void issue(int i, uint32_t slot, int wave) {
    const uint32_t so = (uint32_t)sgpr(i * step), m0 = (uint32_t)sgpr(slot + i * NT * 16 + wave * 1024);
    if constexpr (ONCE) dma16_once<T>(rsrc, v, so, m0, group_rows);
    else dma16(rsrc, v, so, m0);
  }
  __device__ __forceinline__ void issue_all(uint32_t slot, int wave) {
    next();
#pragma unroll
    for (int i = 0; i < kDma; ++i) issue(i, slot, wave);
  }
};

// Fragments of one 16-deep step: N tiles of 32 rows (columns) of the unit from row `first`.
template <bool TR, int T, int N>
struct Frags {
  uint32_t off[4];              // lane offsets: !TR by step, TR by tile
  uint32_t at[4];               // the same in the current unit
  __device__ __forceinline__ void init(int first, int lane) {
    if (!TR) {
      const int r = lane & 31, j = lane >> 5;
#pragma unroll
      for (int s = 0; s < 4; ++s) off[s] = (first + r) * 128 + (((2 * s + j) ^ ((r >> 1) & 7)) << 4);
    } else {
      const int i = lane & 15, r = i >> 2, j = lane >> 5;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int chunk = ((first / 8 + 4 * t + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1)) ^ (r << 2));
        off[t] = (8 * j + r) * (T * 2) + chunk * 16 + (i & 1) * 8;
      }
    }
  }
  // The bases stay opaque, so that the steps and tiles are instruction offsets.
  __device__ __forceinline__ void enter(uint32_t unit) {
#pragma unroll
    for (int i = 0; i < (TR ? N : 4); ++i) {
      at[i] = unit + off[i];
      asm volatile("" : "+v"(at[i]));
    }
  }
  __device__ __forceinline__ v4i read(int s, int t) const {
    if (!TR) return *(const __attribute__((address_space(3))) v4i*)(uintptr_t)(at[s] + t * 32 * 128);
    const uint32_t a = at[t] + s * 16 * (T * 2);
    const v2i lo = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)a));
    const v2i hi = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)(a + 4 * (T * 2))));
    return v4i{lo.x, lo.y, hi.x, hi.y};
  }
};

#define MM_FENCE() __builtin_amdgcn_sched_barrier(0)

// The same units as a Feed's, through registers.
template <bool TR, int T, int NT>
struct Staged {
  static constexpr int N = T * 128 / (NT * 16);
  const uint16_t* ptr;          // this thread's chunk of the next unit
  int64_t ld;
  int left, valid, row, chunk;
  int have;                     // elements of the chunk that exist, in the unit loaded last
  bool brief;                   // rows of fewer than eight elements
  v4i v[N];
  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld_, int valid_, int64_t kn, bool brief_, int tid) {
    ld = ld_;
    valid = valid_;
    brief = brief_;
    left = (int)min(kn, (int64_t)0x40000000);
    if (!TR) {
      row = tid >> 3;
      chunk = (tid & 7) ^ ((row >> 1) & 7);
    } else {
      row = tid / (T / 8);
      chunk = (tid % (T / 8)) ^ ((row & 3) << 2);
    }
    ptr = p + row * ld + chunk * 8;
  }
  __device__ __forceinline__ void load() {
    constexpr int ROWS = TR ? NT / (T / 8) : NT / 8;
    have = (TR ? valid : left) - 8 * chunk;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int n = row + i * ROWS < (TR ? left : valid) ? have : 0;
      v[i] = brief ? load8_short(ptr + i * ROWS * ld, n) : load8_raw(ptr + i * ROWS * ld, n);
    }
    ptr += TR ? 64 * ld : 64;
    left -= 64;
  }
  __device__ __forceinline__ void store(uint32_t slot, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      *(__attribute__((address_space(3))) v4i*)(uintptr_t)(slot + (i * NT + tid) * 16) = brief ? v[i] : shift8(v[i], have);
  }
};

template <int TYPE, int LAYOUT, int OUT, bool VEC, bool ONCE>
__global__ __launch_bounds__(256, 2) void gmm_ring_kernel(MmArgs p) {
  using E = Elem<TYPE>;
  constexpr int T = 128, NWN = 2, NT = 256, SLOT = T * 128;
  constexpr bool AT = LAYOUT == MM_WGRAD, BT = LAYOUT != MM_FPROP;
  constexpr int WM = 64, WN = 64, NA = WM / 32, NB = WN / 32;
  __shared__ __align__(1024) uint8_t lds[(VEC ? 5 : 4) * SLOT];
  const int tid = threadIdx.x, lane = tid & 63, wave = sgpr(tid >> 6);
  const uint32_t block = blockIdx.x + blockIdx.z * p.row_blocks;
  if (block == 0 && blockIdx.y == 0 && wave == 0) {
    const uint32_t f = wave_split_flags(p.m_splits, p.G, p.M, lane);
    if (lane == 0) *p.flags = f;
  }
  const uint16_t* A = static_cast<const uint16_t*>(p.a);
  const uint16_t* B = static_cast<const uint16_t*>(p.b);
  constexpr int EB = OUT == MM_OUT_SAME ? 2 : 4;
  uint8_t* C = static_cast<uint8_t*>(p.c);
  int64_t crow0, kn, ldc = p.ldc;
  int arows, bcols, col0, ncols;
  uint32_t group_rows = 0;
  constexpr uint32_t GR = 4;             // four row tiles to a column sweep
  if (LAYOUT == MM_WGRAD) {
    const uint32_t ntm = (p.n + T - 1) / T, ntn = (p.k + T - 1) / T, tpg = ntm * ntn;
    uint32_t g, t;
    if (tpg >= 64) {                     // XCD x takes the x-th eighth of every group's tiles
      const uint32_t per = (tpg + 7) / 8, x = block & 7, l = block >> 3;
      g = l / per;
      t = x * per + l % per;
      if (t >= tpg || (int)g >= p.G) return;
    } else {
      g = block / tpg;
      t = block % tpg;
      if ((int)g >= p.G) return;
    }
    const RowTile rt = find_group_rows(p.m_splits, p.G, (uint32_t)p.M, (int)g, lane);
    const uint32_t grp = t / (GR * ntn), rem = t % (GR * ntn), rh = min(GR, ntm - grp * GR);
    const int tm = (int)((grp * GR + rem % rh) * T);
    col0 = (int)(rem / rh * T);
    arows = p.n - tm;
    ncols = p.k;
    kn = rt.m;
    if (OUT == MM_OUT_ACC32 && kn == 0) return;
    A += (int64_t)rt.row0 * p.lda + tm;
    B += (int64_t)rt.row0 * p.ldb + col0;
    crow0 = tm;
    C += (int64_t)g * (OUT == MM_OUT_PART ? (int64_t)p.n * p.k : p.c_stride) * EB;
  } else {
    const uint32_t ntn = (p.n + T - 1) / T;
    const uint32_t total = row_tiles_total(p.m_splits, p.G, (uint32_t)p.M, T, ntn, p.zero_rest, lane);
    const uint32_t per = (total + 7) / 8, l = block >> 3;          // XCD x takes the x-th eighth of the tiles
    if (l >= per) return;
    const RowTile rt = find_row_tile(p.m_splits, p.G, (uint32_t)p.M, T, ntn, p.zero_rest, (block & 7) * per + l, lane);
    if (rt.g < 0) return;
    const uint32_t ntm = (rt.m + T - 1) / T;
    const uint32_t grp = rt.t / (GR * ntn), rem = rt.t % (GR * ntn), rh = min(GR, ntm - grp * GR);
    const uint32_t tm = (grp * GR + rem % rh) * T;
    col0 = (int)(rem / rh * T);
    arows = (int)(rt.m - tm);
    ncols = p.n;
    kn = rt.g < p.G ? p.k : 0;
    group_rows = (uint32_t)sgpr((int)rt.m);
    crow0 = (int64_t)rt.row0 + tm;
    A += crow0 * p.lda;
    if (rt.g < p.G) B += (int64_t)rt.g * p.b_stride + (LAYOUT == MM_FPROP ? (int64_t)col0 * p.ldb : (int64_t)col0);
  }
  if (OUT == MM_OUT_PART) {              // this part's stages
    const int64_t nst = (kn + 63) / 64, z = blockIdx.y;
    const int64_t k0 = 64 * (nst * z / p.parts), k1 = min(kn, 64 * (nst * (z + 1) / p.parts));
    A += AT ? k0 * p.lda : k0;
    B += BT ? k0 * p.ldb : k0;
    kn = max(k1 - k0, (int64_t)0);
    ldc = ncols;
    C = reinterpret_cast<uint8_t*>(p.part + z * p.part_stride) + (LAYOUT == MM_WGRAD ? C - static_cast<uint8_t*>(p.c) : 0);
  }
  arows = sgpr(min(arows, T));
  bcols = sgpr(min(ncols - col0, T));

  const int wm = wave / NWN, wn = wave % NWN;
  v16f acc[NA][NB];
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = v16f{};

  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  const int nst = sgpr((int)((kn + 63) / 64));
  if (nst > 0) {
    Frags<AT, T, NA> ra;
    Frags<BT, T, NB> rb;
    ra.init(wm * WM, lane);
    rb.init(wn * WN, lane);
    v4i a[2][NA], b[2][NB];
    constexpr int NR = NA + NB, NM = NA * NB;
    // fragment reads in the order the MFMAs want them: b0 a0 b1 a1
    auto read_one = [&](int step, int n, v4i* xa, v4i* xb) {
      if (!(n & 1)) xb[n / 2] = rb.read(step, n / 2);
      else xa[n / 2] = ra.read(step, n / 2);
    };
    static_assert(NA == 2 && NB == 2, "reads alternate between the operands");
    if constexpr (VEC) {
      Feed<AT, T, NT> fa;
      Feed<BT, T, NT, ONCE> fb;
      fa.init(A, p.lda, arows, kn, tid);
      fb.init(B, p.ldb, bcols, kn, tid);
      fb.group_rows = group_rows;
      constexpr int P = Feed<AT, T, NT>::kDma;
      fa.issue_all(lds0 + 0 * SLOT, wave);
      fb.issue_all(lds0 + 1 * SLOT, wave);
      fa.issue_all(lds0 + 2 * SLOT, wave);
      fb.issue_all(lds0 + 3 * SLOT, wave);
      fa.issue_all(lds0 + 4 * SLOT, wave);
      uint32_t ua = lds0, ub = lds0 + SLOT;       // the stage's units
      const uint32_t end = lds0 + 5 * SLOT;
      wait_stage<3 * P>();
      ra.enter(ua);
      rb.enter(ub);
#pragma unroll
      for (int n = 0; n < NR; ++n) read_one(0, n, a[0], b[0]);
      for (int s = 0; s < nst; ++s) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const int cur = ks & 1, nxt = cur ^ 1;
          uint32_t da = 0, db = 0;
          if (ks == 3) {
            wait_stage<P>();
            da = ub;                                // A of stage s + 3 goes into B's slot,
            db = ua;                                // B of s + 2 into A's
            ua += 2 * SLOT;
            ub += 2 * SLOT;
            if (ua >= end) ua -= 5 * SLOT;
            if (ub >= end) ub -= 5 * SLOT;
            ra.enter(ua);
            rb.enter(ub);
            fb.next();
            fa.next();
          }
          MM_FENCE();
          // the transposed product: a lane then holds consecutive columns of one row.  One read of the
          // next step behind each MFMA, and at the stage's end its DMAs.
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            const int i = m / NB, j = m % NB;
            acc[i][j] = E::mma32(b[cur][j], a[cur][i], acc[i][j]);
            MM_FENCE();
            if (m < NR) read_one(ks < 3 ? ks + 1 : 0, m, a[nxt], b[nxt]);
            if (ks == 3) {
              constexpr int D = (2 * P + NM - 1) / NM;
#pragma unroll
              for (int d = m * D; d < (m + 1) * D && d < 2 * P; ++d) {
                if (d < P) fb.issue(d, db, wave);
                else fa.issue(d - P, da, wave);
              }
            }
            MM_FENCE();
          }
        }
      }
      wait_stage<0>();
    } else {
      Staged<AT, T, NT> fa;
      Staged<BT, T, NT> fb;
      fa.init(A, p.lda, arows, kn, (AT ? p.n : p.k) < 8, tid);
      fb.init(B, p.ldb, bcols, kn, (BT ? ncols : p.k) < 8, tid);
      fa.load();
      fb.load();
      for (int s = 0; s < nst; ++s) {
        const uint32_t u = lds0 + (s & 1) * 2 * SLOT;
        fa.store(u, tid);
        fb.store(u + SLOT, tid);
        __syncthreads();                          // the other pair's readers are past the barrier before
        if (s + 1 < nst) {
          fa.load();
          fb.load();
        }
        ra.enter(u);
        rb.enter(u + SLOT);
#pragma unroll
        for (int n = 0; n < NR; ++n) read_one(0, n, a[0], b[0]);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            const int i = m / NB, j = m % NB;
            if (ks < 3) read_one(ks + 1, m, a[(ks & 1) ^ 1], b[(ks & 1) ^ 1]);
            acc[i][j] = E::mma32(b[ks & 1][j], a[ks & 1][i], acc[i][j]);
          }
        }
      }
      __syncthreads();
    }
  }

  // acc[i][j][e]: row 32 i + lane % 32, column 32 j + 8 (e / 4) + 4 (lane / 32) + e % 4 of the wave's
  // tile.  Each wave stages its own rows of 128 bytes and stores whole ones.
  const uint32_t reg = lds0 + wave * (WM * 128);
  const int m = lane & 31, h = lane >> 5, msw = (m >> 1) & 7;
  const int sr = lane >> 3, sc = lane & 7;
  typedef __attribute__((address_space(3))) v4i lds_v4i;
  typedef __attribute__((address_space(3))) v2i lds_v2i;
  constexpr int PASSES = OUT == MM_OUT_SAME ? 1 : NB;
  constexpr int CE = 16 / EB;                       // elements of a 16-byte chunk
#pragma unroll
  for (int ps = 0; ps < PASSES; ++ps) {
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const uint32_t row = reg + (32 * i + m) * 128;
      if constexpr (OUT == MM_OUT_SAME) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const v2i v{(int)E::down2(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                         (int)E::down2(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3])};
            *(lds_v2i*)(uintptr_t)(row + (((4 * j + q) ^ msw) << 4) + h * 8) = v;
          }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v4f v{acc[i][ps][4 * q], acc[i][ps][4 * q + 1], acc[i][ps][4 * q + 2], acc[i][ps][4 * q + 3]};
          *(lds_v4i*)(uintptr_t)(row + (((2 * q + h) ^ msw) << 4)) = __builtin_bit_cast(v4i, v);
        }
      }
    }
#pragma unroll
    for (int r0 = 0; r0 < WM; r0 += 8) {
      const int r = r0 + sr, tr = wm * WM + r;
      const v4i v = *(lds_v4i*)(uintptr_t)(reg + r * 128 + ((sc ^ ((r >> 1) & 7)) << 4));
      const int c = wn * WN + (OUT == MM_OUT_SAME ? 0 : ps * 32) + sc * CE;
      if (tr >= arows || c >= bcols) continue;
      uint8_t* dst = C + ((crow0 + tr) * ldc + col0 + c) * EB;
      if (VEC || c + CE <= bcols) {
        v4i out = v;
        if (OUT == MM_OUT_ACC32) {
          v4f old;
          __builtin_memcpy(&old, dst, 16);
          out = __builtin_bit_cast(v4i, old + __builtin_bit_cast(v4f, v));
        }
        if constexpr (VEC) *reinterpret_cast<v4i*>(dst) = out;
        else __builtin_memcpy(dst, &out, 16);
      } else {
#pragma unroll
        for (int e = 0; e < CE; ++e) {
          if (c + e >= bcols) break;
          if constexpr (OUT == MM_OUT_SAME) {
            reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)((uint32_t)v[e / 2] >> (16 * (e & 1)));
          } else {
            float* f = reinterpret_cast<float*>(dst) + e;
            const float x = __builtin_bit_cast(v4f, v)[e];
            *f = OUT == MM_OUT_ACC32 ? *f + x : x;
          }
        }
      }
    }
  }
}

// c = the parts' sum in order, one element per thread.  FPROP, DGRAD: rows behind the last group are
// zeroed or left; adding to c, a zero sum (an empty group's) leaves it as it is.
template <int TYPE, int LAYOUT, int OUT>
__global__ __launch_bounds__(256) void gmm_sum_kernel(MmArgs p) {
  const int64_t cols = LAYOUT == MM_WGRAD ? p.k : p.n;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  long long used = 0;                    // rows of all groups
  if (LAYOUT != MM_WGRAD) {
    for (int g = threadIdx.x & 63; g < p.G; g += 64) used += max(p.m_splits[g], 0);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) used += __shfl_xor(used, o, 64);
  }
  if (i >= p.part_stride) return;
  const int64_t row = i / cols, col = i - row * cols;
  int64_t o = row * p.ldc + col;
  bool live = true;
  if (LAYOUT == MM_WGRAD) {
    const int64_t g = row / p.n;
    o = g * p.c_stride + (row - g * p.n) * p.ldc + col;
  } else {
    live = row < used;
    if (!live && !p.zero_rest) return;
  }
  float f = 0.0f;
  if (live)
    for (int z = 0; z < p.parts; ++z) f += p.part[z * p.part_stride + i];
  if (OUT == MM_OUT_SAME) static_cast<uint16_t*>(p.c)[o] = Elem<TYPE>::down(f);
  else if (OUT == MM_OUT_FP32) static_cast<float*>(p.c)[o] = f;
  else if (f != 0.0f) static_cast<float*>(p.c)[o] += f;
}

// ----------------------------------------------------------------------------- stream kernel
// The ring kernel made persistent: one workgroup per CU walks a list of 256 x 256 tiles and the
// units of all its tiles form one sequence through the ring, so that a tile's first units are on
// their way while the one before it ends, and its stores drain under the next one's products.
//
// At a tile's last stage the slot that held B is not refilled: it takes the tile's results (4 KB per
// wave, 32 rows of 128 bytes at a time), which are read back as whole rows, and is refilled then; 16-bit
// results are stored behind those DMAs, so that the next tile's first stage need not wait for them.  Every
// wave issues the same count of DMAs and stores for every tile (the buffer range check drops what lies
// outside), which is what the vmcnt bounds count on.  fp32 results (WGRAD) are stored piece by piece before
// the refill, and added to c each of a tile's 32 pieces waits for its old values, and so for the stores and
// DMAs before them: 8 x 4096 x 1536 of 32768 rows 381 us in 16 bits, 388 in fp32, 444 added; 128 x 4096 x
// 7168 of 65536 rows 4.50, 5.43 and 9.3 ms.
//
// Measured: 32768 x 4096 x 7168 in one group 1.28 PFLOP/s forward, 1.26 dgrad, 1.14 wgrad; 8 experts
// of 4096 x 1536 three products 1.14 to 1.16 ms (1.07 PFLOP/s); 128 uneven experts of 4096 x 7168 12.3 ms
// (0.94 PFLOP/s, a third of it the 7.5 GB of weight gradients and the ragged tiles).  Counters on the
// one-group case: the matrix cores busy 66% of the cycles at 1.84 GHz (1.61 PFLOP/s on zeros, where
// the clock stays up), LDS 26%, bank conflicts 1%, L2 hits 80%.
//
// A tile has three stages at least (empty ones read and multiply nothing): the units issued while
// one tile is computed then belong to it or to its successor.  A wave multiplies only the 32-row
// blocks of its half that hold a row, and the last stage only the 16-deep steps that hold an
// element, so that a group's last tile costs what it holds.
//
// The groups come from a table that gmm_table_kernel writes first, largest first (with static shares the
// small tiles then even out the workgroups' ends), rows cut into ceil(m / 256) tiles of equal height,
// a multiple of 32: eight words {group, its first row tile in the table's order, its row tiles, first
// row, rows, tile height} per row tile; WGRAD reads one such entry per group.
//
// A workgroup's share: rounds of one tile per workgroup; within a round an XCD takes consecutive
// tiles, so that those resident together share A rows and B columns in its L2, and from round to
// round a workgroup moves on by one within its XCD, as tiles of one group's full and last row
// blocks alternate.
using sizes::kTableWords;
constexpr int kTableSort = 1024;       // groups that one workgroup sorts; more keep their order

// n / d for any n < 2^32: the product with floor((2^32 - 1) / d) is at most two below.
struct UDiv {
  uint32_t d, m;
  UDiv() = default;
  explicit UDiv(uint32_t v) : d(v), m(0xFFFFFFFFu / v) {}
  __device__ __forceinline__ uint32_t div(uint32_t n, uint32_t& r) const {
    uint32_t q = (uint32_t)(((uint64_t)n * m) >> 32);
    r = n - q * d;
    if (r >= d) { ++q; r -= d; }
    if (r >= d) { ++q; r -= d; }
    return q;
  }
};
struct StreamArgs {
  MmArgs p;
  uint32_t* table;
  UDiv ntn, sweep, per;  // column tiles; tiles of a four-row sweep; WGRAD: an XCD's tiles of a group
  uint32_t ntm, tpg;     // WGRAD: row tiles and tiles of a group
};

__global__ __launch_bounds__(1024) void gmm_table_kernel(StreamArgs args, bool by_rows) {
  const MmArgs& p = args.p;
  __shared__ uint32_t s_rows[kTableSort], s_row0[kTableSort];
  __shared__ uint16_t s_group[kTableSort];
  uint32_t* table = args.table;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = p.G + (by_rows && p.zero_rest ? 1 : 0);      // the rows behind the last group are group G
  const bool sort = n <= kTableSort;
  if (wave == 15) {
    const uint32_t f = wave_split_flags(p.m_splits, p.G, p.M, lane);
    if (lane == 0) *p.flags = f;
  }
  auto spans = [&](int base, uint32_t& done) {
    Span s = wave_spans(p.m_splits, p.G, (uint32_t)p.M, base, lane, done);
    if (base + lane == p.G && n > p.G) s.end = (uint32_t)p.M;
    if (base + lane >= n) s.end = s.start;
    return s;
  };
  if (sort) {
    uint32_t done = 0;
    for (int base = 0; base < n; base += 64) {
      const Span s = spans(base, done);
      if (wave == 0 && base + lane < n) {
        s_row0[base + lane] = s.start;
        s_rows[base + lane] = s.end - s.start;
      }
    }
    __syncthreads();
    if (tid < n) {
      const uint32_t mine = s_rows[tid];
      int rank = 0;
      for (int i = 0; i < n; ++i) rank += s_rows[i] > mine || (s_rows[i] == mine && i < tid);
      s_group[rank] = (uint16_t)tid;
    }
    __syncthreads();
  }
  uint32_t done = 0, tiles = 0;
  for (int base = 0; base < n; base += 64) {
    const int at = base + lane;
    uint32_t g = at, row0 = 0, m = 0;
    if (sort) {
      if (at < n) {
        g = s_group[at];
        row0 = s_row0[g];
        m = s_rows[g];
      }
    } else {
      const Span s = spans(base, done);
      row0 = s.start;
      m = s.end - s.start;
    }
    const uint32_t nt = by_rows ? (m + 255) / 256 : 1;
    const uint32_t count = at < n ? nt : 0;
    const uint32_t incl = wave_incl_add(count, lane, 0x7FFFFFFFu);
    const uint32_t first = tiles + incl - count;
    const uint32_t h = by_rows && nt ? ((m + nt - 1) / nt + 31) / 32 * 32 : 0;
    for (uint32_t t = wave; t < count; t += 16) {
      uint32_t* e = table + 8 + (uint64_t)(first + t) * kTableWords;
      e[0] = g;
      e[1] = first;
      e[2] = nt;
      e[3] = row0;
      e[4] = m;
      e[5] = h;
    }
    tiles += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
  }
  if (tid == 0) table[0] = tiles;
}

// One output tile (uniform values).
struct StreamTile {
  const uint16_t* a;
  const uint16_t* b;
  uint8_t* c;              // its first element
  int arows, bcols;        // valid rows and columns, at most T; 0 rows: no tile
  int kn, nst;
};

template <int LAYOUT, int OUT, int T>
struct TileWalk {
  uint32_t round, rounds, x, w, nw, total;
  __device__ __forceinline__ void init(const StreamArgs& s) {
    nw = gridDim.x >> 3;
    x = blockIdx.x & 7;
    w = blockIdx.x >> 3;
    round = 0;
    total = LAYOUT == MM_WGRAD ? (s.tpg >= 64 ? s.per.d : s.tpg) * (uint32_t)s.p.G : s.table[0] * s.ntn.d;
    // WGRAD with many tiles a group: every XCD has the same count of tiles of its own
    const uint32_t each = LAYOUT == MM_WGRAD && s.tpg >= 64 ? nw : nw * 8;
    rounds = (total + each - 1) / each;
  }
  // The next tile of this workgroup.
  __device__ __forceinline__ StreamTile next(const StreamArgs& s) {
    constexpr uint32_t GR = 4;           // four row tiles to a column sweep
    const MmArgs& p = s.p;
    StreamTile t{};
    while (round < rounds) {
      const bool own = LAYOUT == MM_WGRAD && s.tpg >= 64;
      const uint32_t l = (own ? round : round * 8 + x) * nw + w;
      ++round;
      w = w + 1 == nw ? 0 : w + 1;
      if (l >= total) continue;
      uint32_t i, rem;
      const uint32_t* e;
      if (LAYOUT == MM_WGRAD) {
        uint32_t q = s.per.div(l, i);
        if (own) i += x * s.per.d;
        if (i >= s.tpg) continue;
        e = s.table + 8 + q * kTableWords;
      } else {
        e = s.table + 8 + (uint64_t)s.ntn.div(l, i) * kTableWords;
        i = l - e[1] * s.ntn.d;
      }
      const uint32_t g = e[0], row0 = e[3], m = e[4];
      const uint32_t ntm = LAYOUT == MM_WGRAD ? s.ntm : e[2];
      if (OUT == MM_OUT_ACC32 && m == 0) continue;
      const uint32_t grp = s.sweep.div(i, rem), rh = min(GR, ntm - grp * GR);
      const uint32_t col = rh == 4 ? rem >> 2 : rh == 3 ? (uint32_t)(((uint64_t)rem * 0xAAAAAAABu) >> 33) : rh == 2 ? rem >> 1 : rem;
      const uint32_t tm = grp * GR + rem - col * rh;
      const int col0 = (int)(col * T);
      if (LAYOUT == MM_WGRAD) {
        const int r = (int)(tm * T);
        t.a = static_cast<const uint16_t*>(p.a) + (int64_t)row0 * p.lda + r;
        t.b = static_cast<const uint16_t*>(p.b) + (int64_t)row0 * p.ldb + col0;
        t.c = static_cast<uint8_t*>(p.c) + ((int64_t)g * p.c_stride + (int64_t)r * p.ldc + col0) * (OUT == MM_OUT_SAME ? 2 : 4);
        t.arows = min(p.n - r, T);
        t.bcols = min(p.k - col0, T);
        t.kn = (int)m;
      } else {
        const uint32_t h = e[5];
        const int64_t row = (int64_t)row0 + tm * h;
        t.a = static_cast<const uint16_t*>(p.a) + row * p.lda;
        t.b = static_cast<const uint16_t*>(p.b);
        if ((int)g < p.G) t.b += (int64_t)g * p.b_stride + (LAYOUT == MM_FPROP ? (int64_t)col0 * p.ldb : (int64_t)col0);
        t.c = static_cast<uint8_t*>(p.c) + (row * p.ldc + col0) * 2;
        t.arows = (int)min(m - tm * h, h);
        t.bcols = min(p.n - col0, T);
        t.kn = (int)g < p.G ? p.k : 0;
      }
      t.nst = max(3, (t.kn + 63) / 64);
      return t;
    }
    t.nst = 1 << 30;                     // behind the last tile: empty units
    return t;
  }
};

// A Feed that moves on to the next tile by itself.
template <bool TR, int T, int NT>
struct StreamFeed : Feed<TR, T, NT> {
  int todo;
  __device__ __forceinline__ void set(const uint16_t* ptr, int64_t ld, int valid, const StreamTile& t, int tid) {
    this->init(ptr, ld, valid, t.kn, tid);
    todo = t.nst;
  }
  __device__ __forceinline__ void advance(const uint16_t* ptr, int64_t ld, int valid, const StreamTile& nt, int tid) {
    if (todo == 0) set(ptr, ld, valid, nt, tid);
    --todo;
    this->next();
  }
};

template <int TYPE, int LAYOUT, int OUT>
__global__ __launch_bounds__(512, 2) void gmm_stream_kernel(StreamArgs args) {
  const MmArgs& p = args.p;
  using E = Elem<TYPE>;
  constexpr int T = 256, NWN = 4, NT = 512, SLOT = T * 128;
  constexpr bool AT = LAYOUT == MM_WGRAD, BT = LAYOUT != MM_FPROP;
  constexpr int WM = 128, NA = 4, NB = 2, NR = NA + NB;
  constexpr int NST = 16;                          // a wave's stores per tile (16-bit results)
  typedef __attribute__((address_space(3))) v4i lds_v4i;
  typedef __attribute__((address_space(3))) v2i lds_v2i;
  __shared__ __align__(1024) uint8_t lds[5 * SLOT];
  const int tid = threadIdx.x, lane = tid & 63, wave = sgpr(tid >> 6);
  const int wm = wave / NWN, wn = wave % NWN;

  TileWalk<LAYOUT, OUT, T> walk;
  walk.init(args);
  StreamTile cur = walk.next(args);
  if (cur.arows == 0) return;
  StreamTile nt = walk.next(args);

  StreamFeed<AT, T, NT> fa;
  StreamFeed<BT, T, NT> fb;
  fa.set(cur.a, p.lda, cur.arows, cur, tid);
  fb.set(cur.b, p.ldb, cur.bcols, cur, tid);
  auto next_a = [&]() { fa.advance(nt.a, p.lda, nt.arows, nt, tid); };
  auto next_b = [&]() { fb.advance(nt.b, p.ldb, nt.bcols, nt, tid); };
  constexpr int P = Feed<AT, T, NT>::kDma;
  auto issue_a = [&](uint32_t slot) {
    next_a();
#pragma unroll
    for (int i = 0; i < P; ++i) fa.issue(i, slot, wave);
  };
  auto issue_b = [&](uint32_t slot) {
    next_b();
#pragma unroll
    for (int i = 0; i < P; ++i) fb.issue(i, slot, wave);
  };
  Frags<AT, T, NA> ra;
  Frags<BT, T, NB> rb;
  ra.init(wm * WM, lane);
  rb.init(wn * 64, lane);

  const uint32_t lds0 = (uint32_t)(uintptr_t)lds, end = lds0 + 5 * SLOT;
  issue_a(lds0);
  issue_b(lds0 + SLOT);
  issue_a(lds0 + 2 * SLOT);
  issue_b(lds0 + 3 * SLOT);
  issue_a(lds0 + 4 * SLOT);
  uint32_t ua = lds0, ub = lds0 + SLOT;            // the stage's units
  uint32_t sa = 0, sb = 0;                         // the units read before them
  v4i a[2][NA], b[2][NB];
  auto read_one = [&](int step, int n, v4i* xa, v4i* xb) {
    if (n < 2 * NB && !(n & 1)) xb[n / 2] = rb.read(step, n / 2);
    else if (n < 2 * NB) xa[n / 2] = ra.read(step, n / 2);
    else xa[n - NB] = ra.read(step, n - NB);
  };
  v16f acc[NA][NB];
  auto turn = [&]() {                              // on to the next stage's units
    sa = ua;
    sb = ub;
    ua += 2 * SLOT;
    ub += 2 * SLOT;
    if (ua >= end) ua -= 5 * SLOT;
    if (ub >= end) ub -= 5 * SLOT;
    ra.enter(ua);
    rb.enter(ub);
  };
  int nal = 0;                                     // 32-row blocks of this wave's half that hold a row
  // One 16-deep step: behind each pair of MFMAs the reads of the step after it and, in a stage's last
  // step, DMAs into the units just left.  A tile's last step reads nothing and leaves B's slot free.
  // Row blocks without a row
  // and steps without an element are not multiplied.
  auto step = [&](auto more_, int ks, int left) {
    constexpr bool MORE = decltype(more_)::value;
    const int cu = ks & 1, nx = cu ^ 1;
    const int live = sgpr(16 * ks < left ? nal : 0);
    MM_FENCE();
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      if (i == 0) E::template mma32_pair<0>(live, b[cu][0], b[cu][1], a[cu][0], acc[0][0], acc[0][1]);
      if (i == 1) E::template mma32_pair<1>(live, b[cu][0], b[cu][1], a[cu][1], acc[1][0], acc[1][1]);
      if (i == 2) E::template mma32_pair<2>(live, b[cu][0], b[cu][1], a[cu][2], acc[2][0], acc[2][1]);
      if (i == 3) E::template mma32_pair<3>(live, b[cu][0], b[cu][1], a[cu][3], acc[3][0], acc[3][1]);
      MM_FENCE();
      if (MORE) {
#pragma unroll
        for (int r = 2 * i; r < 2 * i + 2 && r < NR; ++r) read_one((ks + 1) & 3, r, a[nx], b[nx]);
      }
      if (ks == 3) {
#pragma unroll
        for (int d = 2 * i; d < 2 * i + 2; ++d) {
          if (d < P) fb.issue(d, sa, wave);
          else if (MORE) fa.issue(d - P, sb, wave);
        }
      }
      MM_FENCE();
    }
  };
  static_assert(P == NA && NB == 2, "two DMAs behind each pair of MFMAs of a stage's last step");
  using No = std::integral_constant<bool, false>;
  using Yes = std::integral_constant<bool, true>;
  bool stores = false;                             // the tile before left stores behind its DMAs
  auto stage = [&](auto more_, int s) {
    constexpr bool MORE = decltype(more_)::value;
    const int left = cur.kn - 64 * s;
    step(Yes{}, 0, left);
    step(Yes{}, 1, left);
    step(Yes{}, 2, left);
    if (OUT == MM_OUT_SAME && s == 0 && stores) wait_stage<P + NST>();
    else wait_stage<P>();
    turn();
    next_b();
    if (MORE) next_a();
    step(more_, 3, left);
  };

  wait_stage<3 * P>();
  ra.enter(ua);
  rb.enter(ub);
  while (true) {
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = v16f{};
    nal = sgpr(min(max((cur.arows - wm * WM + 31) / 32, 0), 4));
    // first fragments of the tile (its first two units have landed)
#pragma unroll
    for (int n = 0; n < NR; ++n) read_one(0, n, a[0], b[0]);
    for (int s = 0; s + 1 < cur.nst; ++s) stage(Yes{}, s);
    stage(No{}, cur.nst - 1);
    mma32_settle(acc);
    MM_FENCE();
    // acc[i][j][e]: row 32 i + lane % 32, column 32 j + 8 (e / 4) + 4 (lane / 32) + e % 4 of the wave's
    // 128 x 64; staged by 32 rows of 128 bytes in the wave's 4 KB of the slot B left
    const uint32_t reg = sb + wave * 4096;
    const int m = lane & 31, h = lane >> 5, msw = (m >> 1) & 7;
    const int sr = lane >> 3, sc = lane & 7;
    constexpr int EB = OUT == MM_OUT_SAME ? 2 : 4;
    const uint32_t ldb = (uint32_t)(p.ldc * EB);
    const uint64_t cb = sgpr64((uint64_t)(uintptr_t)cur.c);
    const v4i rc{(int)(uint32_t)cb, (int)((uint32_t)(cb >> 32) & 0xFFFFu),
                 sgpr((int)((uint32_t)(cur.arows - 1) * ldb + (uint32_t)(cur.bcols * EB))), 0x00020000};
    auto staged = [&](int r) {                     // 16 bytes of row 8 r + sr
      return *(lds_v4i*)(uintptr_t)(reg + (8 * r + sr) * 128 + ((sc ^ (((8 * r + sr) >> 1) & 7)) << 4));
    };
    auto store = [&](v4i v, uint32_t vo, uint32_t so) {
      asm volatile("s_nop 4\n\tbuffer_store_dwordx4 %0, %1, %2, %3 offen nt\n\ts_nop 1" :: "v"(v), "v"(vo), "s"(rc), "s"((uint32_t)sgpr((int)so)) : "memory");
    };
    if constexpr (OUT == MM_OUT_SAME) {
      v4i out[NA][4];
#pragma unroll
      for (int i = 0; i < NA; ++i) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const v16f& c = acc[i][j];
            const v2i v{(int)E::down2(c[4 * q], c[4 * q + 1]), (int)E::down2(c[4 * q + 2], c[4 * q + 3])};
            *(lds_v2i*)(uintptr_t)(reg + m * 128 + (((4 * j + q) ^ msw) << 4) + h * 8) = v;
          }
#pragma unroll
        for (int r = 0; r < 4; ++r) out[i][r] = staged(r);
      }
      wait_stage<63>();                            // every wave's rows are out of the slot
      issue_a(sb);
      const int c = wn * 64 + sc * 8;
      const uint32_t vo = c < cur.bcols ? (uint32_t)(wm * WM + sr) * ldb + (uint32_t)(c * EB) : kNoLane;
#pragma unroll
      for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) store(out[i][r], vo, (32 * i + 8 * r) * ldb);
    } else {
#pragma unroll
      for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const v16f& c = acc[i][j];
            const v4f v{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
            *(lds_v4i*)(uintptr_t)(reg + m * 128 + (((2 * q + h) ^ msw) << 4)) = __builtin_bit_cast(v4i, v);
          }
          const int c = wn * 64 + j * 32 + sc * 4;
          const uint32_t vo = c < cur.bcols ? (uint32_t)(wm * WM + sr) * ldb + (uint32_t)(c * EB) : kNoLane;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            v4f f = __builtin_bit_cast(v4f, staged(r));
            if (OUT == MM_OUT_ACC32) {
              const int row = wm * WM + 32 * i + 8 * r + sr;
              if (row < cur.arows && c < cur.bcols) f = *reinterpret_cast<const v4f*>(cur.c + (int64_t)row * ldb + c * EB) + f;
            }
            store(__builtin_bit_cast(v4i, f), vo, (32 * i + 8 * r) * ldb);
          }
        }
      wait_stage<63>();
      issue_a(sb);
    }
    stores = OUT == MM_OUT_SAME;
    if (nt.arows == 0) break;
    cur = nt;
    nt = walk.next(args);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no DMA may land after the LDS is given away
}

static int cu_count() {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess || hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 8)
    return 256;
  return n;
}

int grouped_matmul_parts(int layout, int G, int64_t M, int64_t n, int64_t k) { return sizes::parts(layout == MM_WGRAD, G, M, n, k); }
int64_t grouped_matmul_part_floats(int layout, int G, int64_t M, int64_t n, int64_t k) {
  return sizes::part_floats(layout == MM_WGRAD, G, M, n, k);
}
size_t grouped_matmul_table_bytes(int G, int64_t M) { return sizes::table_bytes(G, M); }

// Non-temporal loads of the weights of groups with one row tile, where the weights pass twice the
// last-level cache, so that none is still there from the call before.  Measured (us, forward, plain /
// non-temporal): 128 x 4096 x 7168 with 64 rows 556 / 512, with 128 rows 848 / 768; 64 x 2816 x 2048
// (738 MB) at 16 rows a group 133 / 120, at 32 149 / 145, at 64 154 / 162 (dgrad 145 / 140), at 128
// (most groups two tiles) 204 / 205, Zipf with 96 a group 187 / 176; 8 x 4096 x 4096 (268 MB) at 4
// rows 53 / 59.
static bool weights_once(const MmArgs& p) { return 2.0 * std::min<int64_t>(p.G, p.M) * p.n * p.k > 512e6; }

template <int TYPE, int LAYOUT, int OUT, bool VEC>
static hipError_t run_ring(MmArgs p, hipStream_t s) {
  const FoldedGrid f = fold_grid(sizes::ring_blocks(LAYOUT == MM_WGRAD, p.G, p.M, p.n, p.k), 256);
  p.row_blocks = f.x;
  const bool once = VEC && LAYOUT != MM_WGRAD && weights_once(p);
  auto* k = once ? gmm_ring_kernel<TYPE, LAYOUT, OUT, VEC, VEC && LAYOUT != MM_WGRAD> : gmm_ring_kernel<TYPE, LAYOUT, OUT, VEC, false>;
  hipLaunchKernelGGL(k, dim3(f.x, OUT == MM_OUT_PART ? p.parts : 1, f.y), dim3(256), 0, s, p);
  return hipGetLastError();
}
template <int TYPE, int LAYOUT, int OUT, bool VEC>
static hipError_t run_tiles(const MmArgs& p, hipStream_t s) {
  if (p.parts <= 1) return run_ring<TYPE, LAYOUT, OUT, VEC>(p, s);
  MmArgs q = p;
  q.part_stride = sizes::part_stride(LAYOUT == MM_WGRAD, p.G, p.M, p.n, p.k);
  q.zero_rest = 0;
  if (hipError_t e = run_ring<TYPE, LAYOUT, MM_OUT_PART, VEC>(q, s)) return e;
  q.zero_rest = p.zero_rest;
  hipLaunchKernelGGL((gmm_sum_kernel<TYPE, LAYOUT, OUT>), dim3((uint32_t)((q.part_stride + 255) / 256)), dim3(256), 0, s, q);
  return hipGetLastError();
}

template <int TYPE, int LAYOUT, int OUT>
static hipError_t run_stream(const MmArgs& p, hipStream_t s) {
  constexpr bool W = LAYOUT == MM_WGRAD;
  StreamArgs a;
  a.p = p;
  a.table = static_cast<uint32_t*>(p.table);
  a.ntn = UDiv((uint32_t)(((W ? p.k : p.n) + 255) / 256));
  a.sweep = UDiv(4 * a.ntn.d);
  a.ntm = W ? (uint32_t)((p.n + 255) / 256) : 0;
  a.tpg = a.ntm * a.ntn.d;
  a.per = UDiv(W ? (a.tpg >= 64 ? (a.tpg + 7) / 8 : a.tpg) : 1);
  hipLaunchKernelGGL(gmm_table_kernel, dim3(1), dim3(1024), 0, s, a, !W);
  if (hipError_t e = hipGetLastError()) return e;
  auto* k = gmm_stream_kernel<TYPE, LAYOUT, OUT>;
  hipLaunchKernelGGL(k, dim3((uint32_t)(cu_count() / 8 * 8)), dim3(512), 0, s, a);
  return hipGetLastError();
}
// The 256 x 256 tiles where they fill the device and hold rows enough.  Measured (bf16, us, 128-tile
// ring / stream): 8 x 512 rows, 4096 x 2048: forward 71.7 / 64.7, at 256 rows a group 38.6 / 64.6;
// 64 x 256 rows, 1024 x 2048: 104 / 78; 64 x 128 rows, 2816 x 2048: 206 / 200 and dgrad 157 / 159;
// 32 x 64 rows, 4096 x 2048: 133 / 138.  WGRAD by its tiles alone: 8 x 128 rows, 4096 x 2048 (1024
// tiles) 49.1 / 44.1, one group 2048 rows 4096 x 4096 (256 tiles) 71.0 / 67.0, 16384 rows 1024 x
// 1024 (16 tiles) 134 / 335.
static bool use_stream(const MmArgs& p) {
  const int64_t tn = (p.n + 255) / 256, tk = (p.k + 255) / 256;
  if (p.layout == MM_WGRAD) return p.G * tn * tk >= 256;
  return p.M >= (int64_t)160 * p.G && sizes::row_tiles_even(p.M, p.G, 256) * tn >= 256;
}
// 16-byte loads and stores throughout.
static bool vec_ok(const MmArgs& p) {
  const uintptr_t addr = reinterpret_cast<uintptr_t>(p.a) | reinterpret_cast<uintptr_t>(p.b) | reinterpret_cast<uintptr_t>(p.c);
  return (addr & 15) == 0 && ((p.n | p.k | p.lda | p.ldb | p.ldc | p.b_stride | p.c_stride) & 7) == 0;
}

template <int TYPE, int LAYOUT, int OUT>
static hipError_t run_sized(const MmArgs& p, hipStream_t s) {
  if (!vec_ok(p)) return run_tiles<TYPE, LAYOUT, OUT, false>(p, s);
  if (use_stream(p)) return run_stream<TYPE, LAYOUT, OUT>(p, s);
  return run_tiles<TYPE, LAYOUT, OUT, true>(p, s);
}

template <int TYPE>
static hipError_t run_type(const MmArgs& p, hipStream_t s) {
  if (p.layout == MM_FPROP) return run_sized<TYPE, MM_FPROP, MM_OUT_SAME>(p, s);
  if (p.layout == MM_DGRAD) return run_sized<TYPE, MM_DGRAD, MM_OUT_SAME>(p, s);
  if (p.out == MM_OUT_SAME) return run_sized<TYPE, MM_WGRAD, MM_OUT_SAME>(p, s);
  if (p.out == MM_OUT_FP32) return run_sized<TYPE, MM_WGRAD, MM_OUT_FP32>(p, s);
  return run_sized<TYPE, MM_WGRAD, MM_OUT_ACC32>(p, s);
}

hipError_t launch_grouped_matmul(const MmArgs& p, hipStream_t s) {
  return p.type == MM_BF16 ? run_type<MM_BF16>(p, s) : run_type<MM_FP16>(p, s);
}

}  // namespace gmlp
