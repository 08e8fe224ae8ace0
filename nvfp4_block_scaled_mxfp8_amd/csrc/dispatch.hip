// The order of rows by group (a stable counting sort), and the moves between token order and expert
// order: dispatch, combine and their gradients.  All of it is bound by memory (or, in a decode
// step, by the launch): every tensor is read and written once, 16 bytes per lane.  8192 tokens, top-8
// of 128 experts, rows of 7168: order 10 us, moves 190 to 230 us each (4.6 to 5.6 TB/s; a plain copy
// reaches 5.2).
#include "mm_common.h"
#include "op_sizes.h"

#include <algorithm>

namespace gmlp {

// ----------------------------------------------------------------------------- group order
// A block takes a contiguous chunk of the slots, each of its 16 waves a contiguous part of that, 64
// slots at a time.  Within a wave the lanes with the same id find each other by one ballot per bit
// of the id; a wave's running position per group sits in LDS.  So positions depend on nothing but
// the ids: the sort is stable and every run gives the same order.
//   counting pass (many slots): the chunk's slots per group -> ws[block][G]
//   placing pass: a group's first position (the slots of lower groups, and of this group in earlier
//   blocks and waves), then one walk that places every slot.  Without a counting pass (no ws) every
//   block counts all slots by itself.
constexpr int OT = sizes::kOrderThreads, OW = OT / 64;

__device__ __forceinline__ uint64_t same_id_lanes(int id, int bits, bool in) {
  uint64_t m = __ballot(in);
  for (int b = 0; b < bits; ++b) {
    const uint64_t v = __ballot((id >> b) & 1);
    m &= ((id >> b) & 1) ? v : ~v;
  }
  return m;
}

template <bool PLACE>
__global__ __launch_bounds__(OT) void order_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t chunk, int G,
                                                   int bits, int nblocks, bool rest,
                                                   int32_t* __restrict__ ws,
                                                   int32_t* __restrict__ count, int32_t* __restrict__ rows,
                                                   int32_t* __restrict__ order) {
  __shared__ int32_t at[OW][kOrderMaxGroups];      // a wave's slots per group, then its next position
  __shared__ int32_t part[OW];
  __shared__ int32_t s_total;
  __shared__ int32_t s_before[kOrderMaxGroups], s_all[kOrderMaxGroups];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t lo = (int64_t)blockIdx.x * chunk, hi = min(lo + chunk, n);
  const int64_t wchunk = chunk / OW;               // chunk is a multiple of OT
  const int64_t wlo = lo + wave * wchunk, whi = min(wlo + wchunk, hi);
  int32_t before = 0, all = 0;                     // of group tid: slots in earlier blocks, in all
  if (PLACE && nblocks > 1 && !ws) {
    int32_t* rep = &at[0][0];                      // sixteen counters per group, one per lane % 16
    auto count_ids = [&](int64_t from, int64_t to) {
      for (int64_t i = from + tid; i < to; i += 4 * OT) {
        int id[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          id[u] = i + u * OT < to ? ids[i + u * OT] : -1;
          if (rest && i + u * OT < to && (uint32_t)id[u] >= (uint32_t)G) id[u] = G - 1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if ((uint32_t)id[u] < (uint32_t)G) atomicAdd(&rep[id[u] * OW + (lane & (OW - 1))], 1);
      }
      __syncthreads();
      int32_t sum = 0;
      if (tid < G)
        for (int w = 0; w < OW; ++w) sum += rep[tid * OW + w];
      __syncthreads();
      return sum;
    };
    for (int i = tid; i < G * OW; i += OT) rep[i] = 0;
    __syncthreads();
    before = count_ids(0, lo);
    all = count_ids(lo, n);                        // the counters run on
  }
  for (int g = lane; g < G; g += 64) at[wave][g] = 0;
  // LDS within a wave is in order; other waves read at[][] only after the barrier
  for (int64_t i = wlo; i < whi; i += 64) {
    int id = i + lane < whi ? ids[i + lane] : -1;
    if (rest && i + lane < whi && (uint32_t)id >= (uint32_t)G) id = G - 1;
    if ((uint32_t)id < (uint32_t)G) atomicAdd(&at[wave][id], 1);
  }
  __syncthreads();
  // the block's slots of group tid (G <= OT), as a running sum over its waves
  int32_t mine = 0;
  if (tid < G) {
    for (int w = 0; w < OW; ++w) {
      const int32_t v = at[w][tid];
      at[w][tid] = mine;
      mine += v;
    }
    if (!PLACE) {
      ws[(int64_t)blockIdx.x * G + tid] = mine;
    } else {
      s_before[tid] = s_all[tid] = 0;
    }
  }
  if (!PLACE) return;
  if (nblocks > 1 && ws) {                         // all threads add up the blocks' counts
    __syncthreads();
    const int g = tid & ((1 << bits) - 1), per = OT >> bits;
    if (g < G) {
      int32_t b0 = 0, a0 = 0;
#pragma unroll 4
      for (int b = tid >> bits; b < nblocks; b += per) {
        const int32_t v = ws[(int64_t)b * G + g];
        b0 += b < (int)blockIdx.x ? v : 0;
        a0 += v;
      }
      atomicAdd(&s_before[g], b0);
      atomicAdd(&s_all[g], a0);
    }
    __syncthreads();
  }
  if (tid < G && (nblocks == 1 || ws)) {
    before = nblocks > 1 ? s_before[tid] : 0;
    all = nblocks > 1 ? s_all[tid] : mine;
  }
  // first position of each group: exclusive scan of `all` over the block
  int32_t incl = all;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t u = __shfl_up(incl, o, 64);
    if (lane >= o) incl += u;
  }
  if (lane == 63) part[wave] = incl;
  __syncthreads();
  int32_t base = 0;
  for (int w = 0; w < wave; ++w) base += part[w];
  if (tid == OT - 1) s_total = base + incl;
  if (tid < G) {
    const int32_t first = base + incl - all + before;
    for (int w = 0; w < OW; ++w) at[w][tid] += first;
    if (blockIdx.x == 0) count[tid] = all;
  }
  __syncthreads();
  for (int64_t i = wlo; i < whi; i += 64) {
    const int64_t slot = i + lane;
    int id = slot < whi ? ids[slot] : -1;
    if (rest && slot < whi && (uint32_t)id >= (uint32_t)G) id = G - 1;
    const bool in = (uint32_t)id < (uint32_t)G;
    const uint64_t peers = same_id_lanes(id, bits, in);
    const int rank = __popcll(peers & ((1ull << lane) - 1));
    const int32_t pos = in ? at[wave][id] + rank : -1;
    if (in && rank == 0) at[wave][id] = pos + __popcll(peers);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");      // the next 64 slots read what the leaders wrote
    if (slot < whi) {
      if (rows) rows[slot] = pos;
      if (order && in) order[pos] = (int32_t)slot;
    }
  }
  if (order)
    for (int64_t i = s_total + (int64_t)blockIdx.x * OT + tid; i < n; i += (int64_t)gridDim.x * OT) order[i] = -1;
}

int order_blocks(int64_t n) { return sizes::order_blocks(n); }

hipError_t launch_group_order(const int32_t* ids, int64_t n, int G, bool rest, int32_t* count, int32_t* rows,
                              int32_t* order, int32_t* ws, hipStream_t s) {
  const int nb = sizes::order_grid(n);
  const int64_t chunk = sizes::order_chunk(n);
  int bits = 0;
  while ((1 << bits) < G) ++bits;
  if (order_blocks(n) == 1) ws = nullptr;
  if (ws)
    hipLaunchKernelGGL(order_kernel<false>, dim3(nb), dim3(OT), 0, s, ids, n, chunk, G, bits, nb, rest, ws, count, rows, order);
  hipLaunchKernelGGL(order_kernel<true>, dim3(nb), dim3(OT), 0, s, ids, n, chunk, G, bits, nb, rest, ws, count, rows, order);
  return hipGetLastError();
}

// ----------------------------------------------------------------------------- moves
// A thread owns V consecutive elements of one token's row and its k rows on the other side: 16 bytes,
// one element where a row holds less.  Rows that are not whole 16-byte chunks: the last chunk is the
// row's last eight elements (the hardware takes any alignment), so it overlaps the one before, with
// the same values.
constexpr int MT = 256;

template <int V>
struct Chunk {
  uint16_t e[V];
};
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));
template <int V>
__device__ __forceinline__ int chunk_start(int c, int H) { return V == 8 ? min(c * 8, H - 8) : c; }
// NT: non-temporal, for rows in expert order that do not fit the last-level cache: they are read or
// written once, and dirty lines left in the cache slow the kernels behind.  Measured on 65536 rows of
// 7168 (940 MB; us, plain / loads alone / loads and stores): combine 285 / 233 / 210, its gradient
// for probs 259 / 237 / 177, dispatch 200 / 214 / 226, all moves of a training step 1180 / 1118 / 1041.
// 12294 rows of 2048 (50 MB): combine 12.5 / 14.7 with loads.
template <int V, bool NT = false>
__device__ __forceinline__ Chunk<V> load_chunk(const uint16_t* p) {
  if constexpr (V == 8) {
    const v4i_any* q = reinterpret_cast<const v4i_any*>(p);
    return __builtin_bit_cast(Chunk<8>, NT ? __builtin_nontemporal_load(q) : *q);
  }
  Chunk<V> c;
  c.e[0] = *p;
  return c;
}
template <int V, bool NT = false>
__device__ __forceinline__ void store_chunk(uint16_t* p, const Chunk<V>& c) {
  if constexpr (V == 8) {
    v4i_any* q = reinterpret_cast<v4i_any*>(p);
    if (NT) __builtin_nontemporal_store(__builtin_bit_cast(v4i_any, c), q);
    else *q = __builtin_bit_cast(v4i_any, c);
  } else {
    *p = c.e[0];
  }
}

// Token and column chunk of a thread: whole tokens per block where a row has fewer chunks than
// threads, else blocks per token.
struct Place {
  int64_t t;
  int c;
};
__device__ __forceinline__ Place place_of(int chunks, int64_t T, int64_t block, int tid) {
  Place p;
  if (chunks >= MT) {
    const int per = (chunks + MT - 1) / MT;
    p.t = block / per;
    p.c = (int)(block % per) * MT + tid;
    if (p.c >= chunks || p.t >= T) p.t = -1;
  } else {
    const int per = MT / chunks;
    p.t = block * per + tid / chunks;
    p.c = tid % chunks;
    if (tid / chunks >= per || p.t >= T) p.t = -1;
  }
  return p;
}
static int64_t place_blocks(int chunks, int64_t T) {
  return chunks >= MT ? T * ((chunks + MT - 1) / MT) : (T + MT / chunks - 1) / (MT / chunks);
}
__device__ __forceinline__ int64_t block_number(const MoveArgs& p) { return blockIdx.x + (int64_t)blockIdx.y * p.row_blocks; }

constexpr int kRestBlocks = 64;      // blocks that clear the rows behind the last used one

template <int TYPE, int V, bool SCALE, bool NT>
__global__ __launch_bounds__(MT) void dispatch_kernel(MoveArgs p, int chunks, int64_t blocks) {
  using E = Elem<TYPE>;
  uint16_t* dst = static_cast<uint16_t*>(p.dst);
  const int64_t M = p.T * p.k, block = block_number(p);
  if (block >= blocks) {
    if (!p.zero_rest || block >= blocks + kRestBlocks) return;
    long long used = 0;
    for (int e = threadIdx.x & 63; e < p.E; e += 64) used += max(p.count[e], 0);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) used += __shfl_xor(used, o, 64);
    const Chunk<V> zero = {};
    for (int64_t r = used + (block - blocks); r < M; r += kRestBlocks)
      for (int c = threadIdx.x; c < chunks; c += MT) store_chunk<V>(dst + r * p.ld_dst + chunk_start<V>(c, p.H), zero);
    return;
  }
  const Place w = place_of(chunks, p.T, block, threadIdx.x);
  if (w.t < 0) return;
  const int at = chunk_start<V>(w.c, p.H);
  const Chunk<V> x = load_chunk<V>(static_cast<const uint16_t*>(p.src) + w.t * p.ld_src + at);
  for (int j = 0; j < p.k; ++j) {
    const int32_t r = p.rows[w.t * p.k + j];
    if ((uint64_t)(int64_t)r >= (uint64_t)M) continue;
    Chunk<V> y = x;
    if (SCALE) {
      const float f = p.probs[w.t * p.k + j];
#pragma unroll
      for (int i = 0; i < V; ++i) y.e[i] = E::down(f * E::up(x.e[i]));
    }
    store_chunk<V, NT>(dst + r * p.ld_dst + at, y);
  }
}

template <int TYPE, int V, bool SCALE, bool NT>
__global__ __launch_bounds__(MT) void combine_kernel(MoveArgs p, int chunks) {
  using E = Elem<TYPE>;
  const uint16_t* src = static_cast<const uint16_t*>(p.src);
  const int64_t M = p.T * p.k;
  const Place w = place_of(chunks, p.T, block_number(p), threadIdx.x);
  if (w.t < 0) return;
  const int at = chunk_start<V>(w.c, p.H);
  float acc[V] = {};
  for (int j0 = 0; j0 < p.k; j0 += 8) {      // eight rows' loads in flight
    Chunk<V> x[8];
    float f[8];
    bool live[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = j0 + j < p.k;
      const int32_t r = in ? p.rows[w.t * p.k + j0 + j] : -1;
      live[j] = (uint64_t)(int64_t)r < (uint64_t)M;
      f[j] = SCALE && in ? p.probs[w.t * p.k + j0 + j] : 1.0f;
      if (live[j]) x[j] = load_chunk<V, NT>(src + r * p.ld_src + at);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (live[j])
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(f[j], E::up(x[j].e[i]), acc[i]);
  }
  Chunk<V> y;
#pragma unroll
  for (int i = 0; i < V; ++i) y.e[i] = E::down(acc[i]);
  store_chunk<V>(static_cast<uint16_t*>(p.dst) + w.t * p.ld_dst + at, y);
}

// One block per token: the products of its gradient with its k rows, in fp32, summed by thread, by
// wave and over the waves in order.
template <int TYPE, int V, bool NT>
__global__ __launch_bounds__(MT) void combine_dprobs_kernel(MoveArgs p, int chunks) {
  using E = Elem<TYPE>;
  __shared__ float red[MT / 64][8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t = block_number(p), M = p.T * p.k;
  if (t >= p.T) return;
  const uint16_t* dy = static_cast<const uint16_t*>(p.src) + t * p.ld_src;
  const uint16_t* v = static_cast<const uint16_t*>(p.src2);
  for (int j0 = 0; j0 < p.k; j0 += 8) {
    float acc[8] = {};
    int32_t r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r[j] = j0 + j < p.k ? p.rows[t * p.k + j0 + j] : -1;
      if ((uint64_t)(int64_t)r[j] >= (uint64_t)M) r[j] = -1;
    }
    for (int c = tid; c < chunks; c += MT) {
      const int at = chunk_start<V>(c, p.H);
      const Chunk<V> d = load_chunk<V>(dy + at);
      Chunk<V> x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (r[j] >= 0) x[j] = load_chunk<V, NT>(v + r[j] * p.ld_src2 + at);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (r[j] >= 0)
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (at + i >= c * V) acc[j] = fmaf(E::up(d.e[i]), E::up(x[j].e[i]), acc[j]);   // not the chunk before's
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) acc[j] += __shfl_xor(acc[j], o, 64);
      if (lane == 0) red[wave][j] = acc[j];
    }
    __syncthreads();
    if (tid < 8 && j0 + tid < p.k) {
      float s = 0.0f;
      for (int w = 0; w < MT / 64; ++w) s += red[w][tid];
      p.dprobs[t * p.k + j0 + tid] = s;
    }
    __syncthreads();
  }
}

static dim3 grid_of(int64_t blocks, MoveArgs& p) {
  const FoldedGrid g = fold_grid(blocks, MT);
  p.row_blocks = g.x;
  return dim3(g.x, g.y);
}

// Half the 256 MB last-level cache.
static bool past_cache(const MoveArgs& p) { return (double)p.T * p.k * p.H * 2 > 128e6; }

template <int TYPE, int V, bool NT>
static hipError_t run_dispatch_nt(MoveArgs p, hipStream_t s) {
  const int chunks = (p.H + V - 1) / V;
  const int64_t blocks = place_blocks(chunks, p.T);
  const dim3 grid = grid_of(blocks + (p.zero_rest ? kRestBlocks : 0), p);
  if (p.probs) hipLaunchKernelGGL((dispatch_kernel<TYPE, V, true, NT>), grid, dim3(MT), 0, s, p, chunks, blocks);
  else hipLaunchKernelGGL((dispatch_kernel<TYPE, V, false, NT>), grid, dim3(MT), 0, s, p, chunks, blocks);
  return hipGetLastError();
}
template <int TYPE, int V>
static hipError_t run_dispatch(const MoveArgs& p, hipStream_t s) {
  return V == 8 && past_cache(p) ? run_dispatch_nt<TYPE, V, V == 8>(p, s) : run_dispatch_nt<TYPE, V, false>(p, s);
}
template <int TYPE, int V, bool NT>
static hipError_t run_combine_nt(MoveArgs p, hipStream_t s) {
  const int chunks = (p.H + V - 1) / V;
  const dim3 grid = grid_of(place_blocks(chunks, p.T), p);
  if (p.probs) hipLaunchKernelGGL((combine_kernel<TYPE, V, true, NT>), grid, dim3(MT), 0, s, p, chunks);
  else hipLaunchKernelGGL((combine_kernel<TYPE, V, false, NT>), grid, dim3(MT), 0, s, p, chunks);
  return hipGetLastError();
}
template <int TYPE, int V>
static hipError_t run_combine(const MoveArgs& p, hipStream_t s) {
  return V == 8 && past_cache(p) ? run_combine_nt<TYPE, V, V == 8>(p, s) : run_combine_nt<TYPE, V, false>(p, s);
}
template <int TYPE, int V>
static hipError_t run_dprobs(MoveArgs p, hipStream_t s) {
  const int chunks = (p.H + V - 1) / V;
  const dim3 grid = grid_of(p.T, p);
  if (V == 8 && past_cache(p))
    hipLaunchKernelGGL((combine_dprobs_kernel<TYPE, V, V == 8>), grid, dim3(MT), 0, s, p, chunks);
  else
    hipLaunchKernelGGL((combine_dprobs_kernel<TYPE, V, false>), grid, dim3(MT), 0, s, p, chunks);
  return hipGetLastError();
}

hipError_t launch_dispatch(const MoveArgs& p, hipStream_t s) {
  if (p.type == MM_BF16) return p.H >= 8 ? run_dispatch<MM_BF16, 8>(p, s) : run_dispatch<MM_BF16, 1>(p, s);
  return p.H >= 8 ? run_dispatch<MM_FP16, 8>(p, s) : run_dispatch<MM_FP16, 1>(p, s);
}
hipError_t launch_combine(const MoveArgs& p, hipStream_t s) {
  if (p.type == MM_BF16) return p.H >= 8 ? run_combine<MM_BF16, 8>(p, s) : run_combine<MM_BF16, 1>(p, s);
  return p.H >= 8 ? run_combine<MM_FP16, 8>(p, s) : run_combine<MM_FP16, 1>(p, s);
}
hipError_t launch_combine_dprobs(const MoveArgs& p, hipStream_t s) {
  if (p.type == MM_BF16) return p.H >= 8 ? run_dprobs<MM_BF16, 8>(p, s) : run_dprobs<MM_BF16, 1>(p, s);
  return p.H >= 8 ? run_dprobs<MM_FP16, 8>(p, s) : run_dprobs<MM_FP16, 1>(p, s);
}

}  // namespace gmlp
