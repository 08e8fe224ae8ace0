// C ABI of the operators on bf16 / fp16 tensors: validation, workspace carving and launches.
#include "gmlp.h"
#include "kernels.h"
#include "planner.h"

#include <algorithm>

using namespace gmlp;

namespace {

constexpr int64_t kMaxRows = 1LL << 30;
constexpr int64_t kMaxLd = 1LL << 20;      // a tile's rows then span less than 2^31 bytes
// Every workgroup of a grouped product walks the split sizes, 64 groups at a time, so that the time grows with the
// groups' square where each has a tile: 0.6 ms for 4096 groups of one row, 9 ms for 16384, 147 ms for 65536; 2^20
// would take 40 s and 2^24 hours.
constexpr int32_t kMaxGroups = 1 << 16;

gmlp_status fine() { return set_error(GMLP_OK, "%s", ""); }
gmlp_status launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return fine();
  return set_error(GMLP_HIP_ERROR, "system: launching %s failed: %s", what, hipGetErrorString(e));
}
bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

gmlp_status check_dtype(int32_t t) {
  if (t != GMLP_BF16 && t != GMLP_FP16) return set_error(GMLP_UNSUPPORTED, "dtype: bf16 or fp16 is required, got %d", t);
  return GMLP_OK;
}

// Workspace of a grouped product: the flag word, the tile table, the parts of a cut contraction.
constexpr size_t kMmFlagBytes = 256;
size_t mm_table_bytes(int32_t G, int64_t M) { return (grouped_matmul_table_bytes(G, M) + 255) & ~size_t(255); }

gmlp_status check_mm_sizes(int32_t layout, int32_t G, int64_t M, int64_t n, int64_t k) {
  if (layout != GMLP_GEMM_FPROP && layout != GMLP_GEMM_WGRAD && layout != GMLP_GEMM_DGRAD)
    return set_error(GMLP_INVALID_ARG, "layout: unknown layout %d", layout);
  if (G < 1) return set_error(GMLP_INVALID_ARG, "dims: number of groups must be >= 1, got %d", G);
  if (G > kMaxGroups) return set_error(GMLP_UNSUPPORTED, "dims: at most %d groups are supported, got %d", kMaxGroups, G);
  if (M < 0 || M > kMaxRows) return set_error(GMLP_UNSUPPORTED, "dims: M = %lld rows is out of range", (long long)M);
  if (n < 1 || k < 1 || n >= kMaxLd || k >= kMaxLd)
    return set_error(GMLP_UNSUPPORTED, "dims: n and k must be in [1, 2^20), got %lld and %lld", (long long)n, (long long)k);
  // the smallest tile's launch must fit one grid
  const int64_t tn = (n + 63) / 64, tk = (k + 63) / 64;
  const double tiles = layout == GMLP_GEMM_WGRAD ? (double)G * tn * tk
                                                 : (double)((M + 63 * std::min<int64_t>((int64_t)G + 1, M)) / 64) * tn;
  if (tiles > 2147483647.0) return set_error(GMLP_UNSUPPORTED, "dims: %d groups of %lld x %lld exceed one launch", G, (long long)n, (long long)k);
  return GMLP_OK;
}

}  // namespace

extern "C" gmlp_status gmlp_grouped_matmul_ws_bytes(int32_t layout, int32_t G, int64_t M, int64_t n, int64_t k,
                                                    size_t* bytes) {
  if (!bytes) return set_error(GMLP_INVALID_ARG, "null pointer argument");
  const gmlp_status st = check_mm_sizes(layout, G, M, n, k);
  if (st != GMLP_OK) return st;
  *bytes = kMmFlagBytes + mm_table_bytes(G, M) + sizeof(float) * (size_t)grouped_matmul_part_floats(layout, G, M, n, k);
  return fine();
}

extern "C" gmlp_status gmlp_grouped_matmul(const gmlp_grouped_matmul_args* p, hipStream_t stream) {
  if (!p) return set_error(GMLP_INVALID_ARG, "null pointer argument");
  gmlp_status st = check_dtype(p->dtype);
  if (st != GMLP_OK) return st;
  size_t need = 0;
  if ((st = gmlp_grouped_matmul_ws_bytes(p->layout, p->G, p->M, p->n, p->k, &need)) != GMLP_OK) return st;
  const bool wgrad = p->layout == GMLP_GEMM_WGRAD;
  if (p->out_dtype != 0 && p->out_dtype != GMLP_OUT_FP32 && p->out_dtype != GMLP_OUT_FP32_ACCUMULATE)
    return set_error(GMLP_INVALID_ARG, "out_dtype: unknown value %d", p->out_dtype);
  if (p->out_dtype != 0 && !wgrad)
    return set_error(GMLP_UNSUPPORTED, "out_dtype: fp32 outputs are for weight gradients only");
  if (!p->m_splits || (p->M > 0 && (!p->a || !p->b)) || ((wgrad || p->M > 0) && !p->c))
    return set_error(GMLP_INVALID_ARG, "null pointer argument");
  if (!aligned2(p->a) || !aligned2(p->b) || !aligned4(p->m_splits) || !(p->out_dtype ? aligned4(p->c) : aligned2(p->c)))
    return set_error(GMLP_INVALID_ARG, "a tensor is not aligned to its elements");
  const int64_t acols = wgrad ? p->n : p->k;
  const int64_t bcols = p->layout == GMLP_GEMM_DGRAD ? p->n : p->k;
  const int64_t ccols = wgrad ? p->k : p->n;
  if (p->lda < acols || p->ldb < bcols || p->ldc < ccols || p->lda >= kMaxLd || p->ldb >= kMaxLd || p->ldc >= kMaxLd)
    return set_error(GMLP_INVALID_ARG, "strides: row strides must be at least the row's length and below 2^20");
  const int64_t brows = p->layout == GMLP_GEMM_DGRAD ? p->k : p->n;
  if (!wgrad && p->G > 1 && p->b_stride < (brows - 1) * p->ldb + bcols)
    return set_error(GMLP_INVALID_ARG, "strides: the groups' weights overlap");
  if (wgrad && p->G > 1 && p->c_stride < (p->n - 1) * p->ldc + p->k)
    return set_error(GMLP_INVALID_ARG, "strides: the groups' outputs overlap");
  if (!p->ws || p->ws_bytes < need || !aligned16(p->ws))
    return set_error(GMLP_WORKSPACE, "workspace: %zu bytes, 16-byte aligned, are needed", need);
  MmArgs a{};
  a.layout = p->layout;
  a.type = p->dtype;
  a.out = p->out_dtype;
  a.a = p->a;
  a.b = p->b;
  a.c = p->c;
  a.lda = p->lda;
  a.ldb = p->ldb;
  a.ldc = p->ldc;
  a.b_stride = p->b_stride;
  a.c_stride = p->c_stride;
  a.m_splits = p->m_splits;
  a.G = p->G;
  a.M = p->M;
  a.n = (int)p->n;
  a.k = (int)p->k;
  a.zero_rest = p->zero_rest != 0;
  a.flags = static_cast<uint32_t*>(p->ws);
  a.table = static_cast<uint8_t*>(p->ws) + kMmFlagBytes;
  a.parts = grouped_matmul_parts(p->layout, p->G, p->M, p->n, p->k);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(p->ws) + kMmFlagBytes + mm_table_bytes(p->G, p->M));
  return launched(launch_grouped_matmul(a, stream), "grouped matmul");
}

// ----------------------------------------------------------------------------- expert dispatch
namespace {
gmlp_status check_order(int64_t n, int32_t E) {
  if (E < 1 || E > kOrderMaxGroups)
    return set_error(GMLP_UNSUPPORTED, "dims: 1 to %d experts are supported, got %d", kOrderMaxGroups, E);
  if (n < 0 || n >= kMaxRows) return set_error(GMLP_UNSUPPORTED, "dims: %lld slots are out of range", (long long)n);
  return GMLP_OK;
}
size_t order_ws(int64_t n, int32_t E) {
  const int b = order_blocks(n);
  return b > 1 ? (size_t)b * E * sizeof(int32_t) : 0;
}

enum MoveKind { MOVE_DISPATCH, MOVE_COMBINE, MOVE_DPROBS };
gmlp_status move(const gmlp_move_args* p, MoveKind kind, hipStream_t stream) {
  if (!p) return set_error(GMLP_INVALID_ARG, "null pointer argument");
  gmlp_status st = check_dtype(p->dtype);
  if (st != GMLP_OK) return st;
  if (p->T < 0 || p->k < 1 || p->T * (double)p->k >= (double)kMaxRows)
    return set_error(GMLP_UNSUPPORTED, "dims: %lld tokens of %d slots are out of range", (long long)p->T, p->k);
  if (p->H < 1 || p->H >= kMaxLd) return set_error(GMLP_UNSUPPORTED, "dims: H must be in [1, 2^20), got %lld", (long long)p->H);
  if (p->T == 0) return fine();
  const bool rest = kind == MOVE_DISPATCH && p->zero_rest;
  if (!p->src || !p->rows || (kind == MOVE_DPROBS ? !p->src2 || !p->dprobs : !p->dst) || (rest && !p->m_splits))
    return set_error(GMLP_INVALID_ARG, "null pointer argument");
  if (rest && p->E < 1) return set_error(GMLP_INVALID_ARG, "dims: number of experts must be >= 1, got %d", p->E);
  if (!aligned2(p->src) || !aligned2(p->src2) || !aligned2(p->dst) || !aligned4(p->rows) || !aligned4(p->probs) ||
      !aligned4(p->dprobs) || !aligned4(p->m_splits))
    return set_error(GMLP_INVALID_ARG, "a tensor is not aligned to its elements");
  if (p->ld_src < p->H || (kind == MOVE_DPROBS ? p->ld_src2 : p->ld_dst) < p->H)
    return set_error(GMLP_INVALID_ARG, "strides: row strides must be at least the row's length");
  MoveArgs a{};
  a.type = p->dtype;
  a.src = p->src;
  a.src2 = p->src2;
  a.dst = p->dst;
  a.ld_src = p->ld_src;
  a.ld_src2 = p->ld_src2;
  a.ld_dst = p->ld_dst;
  a.T = p->T;
  a.H = (int)p->H;
  a.k = p->k;
  a.rows = p->rows;
  a.probs = p->probs;
  a.dprobs = p->dprobs;
  a.count = p->m_splits;
  a.E = p->E;
  a.zero_rest = rest;
  if (kind == MOVE_DISPATCH) return launched(launch_dispatch(a, stream), "dispatch");
  if (kind == MOVE_COMBINE) return launched(launch_combine(a, stream), "combine");
  return launched(launch_combine_dprobs(a, stream), "combine dprobs");
}
}  // namespace

extern "C" gmlp_status gmlp_dispatch_plan_ws_bytes(int64_t n, int32_t E, size_t* bytes) {
  if (!bytes) return set_error(GMLP_INVALID_ARG, "null pointer argument");
  const gmlp_status st = check_order(n, E);
  if (st != GMLP_OK) return st;
  *bytes = order_ws(n, E);
  return fine();
}

extern "C" gmlp_status gmlp_dispatch_plan(const int32_t* experts, int64_t n, int32_t E, int32_t* m_splits,
                                          int32_t* rows, int32_t* order, void* ws, size_t ws_bytes,
                                          hipStream_t stream) {
  const gmlp_status st = check_order(n, E);
  if (st != GMLP_OK) return st;
  if (!m_splits || (n > 0 && (!experts || !rows))) return set_error(GMLP_INVALID_ARG, "null pointer argument");
  if (!aligned4(experts) || !aligned4(m_splits) || !aligned4(rows) || !aligned4(order))
    return set_error(GMLP_INVALID_ARG, "a tensor is not aligned to its elements");
  const size_t need = order_ws(n, E);
  if (need && (!ws || ws_bytes < need || !aligned16(ws)))
    return set_error(GMLP_WORKSPACE, "workspace: %zu bytes, 16-byte aligned, are needed", need);
  return launched(launch_group_order(experts, n, E, false, m_splits, rows, order, static_cast<int32_t*>(ws), stream),
                  "dispatch plan");
}

extern "C" gmlp_status gmlp_dispatch(const gmlp_move_args* args, hipStream_t stream) {
  return move(args, MOVE_DISPATCH, stream);
}
extern "C" gmlp_status gmlp_combine(const gmlp_move_args* args, hipStream_t stream) {
  return move(args, MOVE_COMBINE, stream);
}
extern "C" gmlp_status gmlp_combine_dprobs(const gmlp_move_args* args, hipStream_t stream) {
  return move(args, MOVE_DPROBS, stream);
}

// ----------------------------------------------------------------------------- low-rank adapters
namespace {
struct Carve {      // sections of a caller buffer at 256-byte offsets
  uint8_t* base;
  size_t off = 0;
  template <class T>
  T* take(int64_t count) {
    off = (off + 255) & ~size_t(255);
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += (size_t)count * sizeof(T);
    return p;
  }
};
LoraFactor carve_factor(Carve& c, int64_t M, int R) {
  LoraFactor f;
  f.hi = c.take<uint16_t>(M * 2 * lora_rp(R));
  f.inv = c.take<float>(M);
  f.v = c.take<float>(M * R);
  return f;
}
LoraFactor of_type(LoraFactor f, int32_t type) {      // bf16 needs neither scales nor the fp32 values
  if (type == GMLP_BF16) f.inv = f.v = nullptr;
  return f;
}
struct LoraCtx {
  int32_t* count;
  int32_t* order;
  LoraFactor u;
};
LoraCtx carve_lora_ctx(Carve& c, int64_t M, int R, int L) {
  LoraCtx x;
  x.count = c.take<int32_t>(L + 1);
  x.order = c.take<int32_t>(M);
  x.u = carve_factor(c, M, R);
  return x;
}
struct LoraWs {
  uint16_t* at;      // [L, K, ldr]
  uint16_t* bt;      // [L, R, ldn]
  LoraFactor du;
  float* part;
  int64_t ldr, ldn;
};
int64_t up8(int64_t v) { return (v + 7) & ~int64_t(7); }
LoraWs carve_lora_ws(Carve& c, int64_t M, int64_t K, int64_t N, int R, int L) {
  LoraWs w;
  w.ldr = up8(R);
  w.ldn = up8(N);
  w.at = c.take<uint16_t>((int64_t)L * K * w.ldr);
  w.bt = c.take<uint16_t>((int64_t)L * R * w.ldn);
  w.du = carve_factor(c, M, R);
  w.part = c.take<float>(std::max(lora_outer_part_floats(M, K, R, L), lora_outer_part_floats(M, N, R, L)));
  return w;
}
gmlp_status check_lora_sizes(int64_t M, int64_t K, int64_t N, int32_t R, int32_t L) {
  if (M < 0 || M >= kMaxRows) return set_error(GMLP_UNSUPPORTED, "dims: M = %lld rows is out of range", (long long)M);
  if (K < 1 || N < 1 || K >= kMaxLd || N >= kMaxLd)
    return set_error(GMLP_UNSUPPORTED, "dims: K and N must be in [1, 2^20), got %lld and %lld", (long long)K, (long long)N);
  if (R < 1 || R > kLoraMaxRank) return set_error(GMLP_UNSUPPORTED, "dims: ranks 1 to %d are supported, got %d", kLoraMaxRank, R);
  if (L < 1 || L > kLoraMaxAdapters)
    return set_error(GMLP_UNSUPPORTED, "dims: 1 to %d adapters are supported, got %d", kLoraMaxAdapters, L);
  return GMLP_OK;
}
gmlp_status check_lora_weights(const gmlp_lora_weights& w, int64_t K, int64_t N, int R, int L) {
  if (!w.a || !w.b) return set_error(GMLP_INVALID_ARG, "null pointer argument");
  if (!aligned2(w.a) || !aligned2(w.b) || !aligned4(w.scales))
    return set_error(GMLP_INVALID_ARG, "a tensor is not aligned to its elements");
  if (w.lda < K || w.ldb < R || w.lda >= kMaxLd || w.ldb >= kMaxLd)
    return set_error(GMLP_INVALID_ARG, "strides: row strides must be at least the row's length and below 2^20");
  if (L > 1 && (w.a_stride < (R - 1) * w.lda + K || w.b_stride < (N - 1) * w.ldb + R))
    return set_error(GMLP_INVALID_ARG, "strides: the adapters overlap");
  return GMLP_OK;
}
bool bad_ld(int64_t ld, int64_t cols) { return ld < cols; }
}  // namespace

extern "C" gmlp_status gmlp_lora_query_sizes(int64_t M, int64_t K, int64_t N, int32_t R, int32_t L,
                                             gmlp_lora_sizes* out) {
  if (!out) return set_error(GMLP_INVALID_ARG, "null pointer argument");
  const gmlp_status st = check_lora_sizes(M, K, N, R, L);
  if (st != GMLP_OK) return st;
  Carve c{nullptr}, w{nullptr};
  carve_lora_ctx(c, M, R, L);
  carve_lora_ws(w, M, K, N, R, L);
  out->ctx_bytes = c.off + 256;
  out->fwd_ws_bytes = order_ws(M, L + 1);
  out->bwd_ws_bytes = w.off + 256;
  return fine();
}

extern "C" gmlp_status gmlp_lora_forward(const gmlp_lora_fwd_args* p, hipStream_t stream) {
  if (!p) return set_error(GMLP_INVALID_ARG, "null pointer argument");
  gmlp_status st = check_dtype(p->dtype);
  if (st != GMLP_OK) return st;
  gmlp_lora_sizes sz;
  if ((st = gmlp_lora_query_sizes(p->M, p->K, p->N, p->R, p->L, &sz)) != GMLP_OK) return st;
  if ((st = check_lora_weights(p->w, p->K, p->N, p->R, p->L)) != GMLP_OK) return st;
  if (p->M == 0) return fine();
  if (!p->x || !p->ids || !p->y) return set_error(GMLP_INVALID_ARG, "null pointer argument");
  if (!aligned2(p->x) || !aligned2(p->base) || !aligned2(p->y) || !aligned4(p->ids))
    return set_error(GMLP_INVALID_ARG, "a tensor is not aligned to its elements");
  if (bad_ld(p->ldx, p->K) || bad_ld(p->ldy, p->N) || (p->base && bad_ld(p->ldbase, p->N)))
    return set_error(GMLP_INVALID_ARG, "strides: row strides must be at least the row's length");
  if (p->base == p->y && p->ldbase != p->ldy)
    return set_error(GMLP_INVALID_ARG, "strides: base and y are one tensor with two row strides");
  if (!p->ctx || p->ctx_bytes < sz.ctx_bytes || !aligned16(p->ctx))
    return set_error(GMLP_WORKSPACE, "ctx: %zu bytes, 16-byte aligned, are needed", sz.ctx_bytes);
  if (sz.fwd_ws_bytes && (!p->ws || p->ws_bytes < sz.fwd_ws_bytes || !aligned16(p->ws)))
    return set_error(GMLP_WORKSPACE, "workspace: %zu bytes, 16-byte aligned, are needed", sz.fwd_ws_bytes);
  Carve c{static_cast<uint8_t*>(p->ctx)};
  const LoraCtx x = carve_lora_ctx(c, p->M, p->R, p->L);
  const LoraRows rows{x.count, x.order, p->M, p->L};
  hipError_t e = launch_group_order(p->ids, p->M, p->L + 1, true, x.count, nullptr, x.order, static_cast<int32_t*>(p->ws), stream);
  if (e != hipSuccess) return launched(e, "adapter order");
  const LoraFactor u = of_type(x.u, p->dtype);
  LoraShrink s{p->dtype, p->R, rows, p->x, p->ldx, p->w.a, p->w.lda, p->w.a_stride, p->K, nullptr, u};
  if ((e = launch_lora_shrink(s, stream)) != hipSuccess) return launched(e, "lora shrink");
  LoraExpand ex{p->dtype, p->R, rows, u, p->w.b, p->w.ldb, p->w.b_stride, p->N, p->w.scales,
                p->base, p->ldbase, p->y, p->ldy};
  return launched(launch_lora_expand(ex, stream), "lora expand");
}

extern "C" gmlp_status gmlp_lora_backward(const gmlp_lora_bwd_args* p, hipStream_t stream) {
  if (!p) return set_error(GMLP_INVALID_ARG, "null pointer argument");
  gmlp_status st = check_dtype(p->dtype);
  if (st != GMLP_OK) return st;
  gmlp_lora_sizes sz;
  if ((st = gmlp_lora_query_sizes(p->M, p->K, p->N, p->R, p->L, &sz)) != GMLP_OK) return st;
  if ((st = check_lora_weights(p->w, p->K, p->N, p->R, p->L)) != GMLP_OK) return st;
  if (p->M > 0 && (!p->dy || (p->da && !p->x) || !p->ctx)) return set_error(GMLP_INVALID_ARG, "null pointer argument");
  if (!aligned2(p->dy) || !aligned2(p->x) || !aligned2(p->dx) || !aligned2(p->dx_add) || !aligned2(p->da) || !aligned2(p->db))
    return set_error(GMLP_INVALID_ARG, "a tensor is not aligned to its elements");
  if (p->M > 0 && (bad_ld(p->lddy, p->N) || (p->x && bad_ld(p->ldx, p->K)) || (p->dx && bad_ld(p->lddx, p->K)) ||
                   (p->dx_add && bad_ld(p->lddx_add, p->K))))
    return set_error(GMLP_INVALID_ARG, "strides: row strides must be at least the row's length");
  if (p->dx && p->dx == p->dx_add && p->lddx != p->lddx_add)
    return set_error(GMLP_INVALID_ARG, "strides: dx and dx_add are one tensor with two row strides");
  if (p->M > 0 && (p->ctx_bytes < sz.ctx_bytes || !aligned16(p->ctx)))
    return set_error(GMLP_WORKSPACE, "ctx: %zu bytes, 16-byte aligned, are needed", sz.ctx_bytes);
  if (!p->ws || p->ws_bytes < sz.bwd_ws_bytes || !aligned16(p->ws))
    return set_error(GMLP_WORKSPACE, "workspace: %zu bytes, 16-byte aligned, are needed", sz.bwd_ws_bytes);
  hipError_t e;
  const int64_t K = p->K, N = p->N;
  const int R = p->R, L = p->L;
  if (p->M == 0) {
    // no rows: zero gradients
    for (int i = 0; i < 2; ++i) {
      void* d = i ? p->db : p->da;
      if (d && (e = launch_zero16(d, (int64_t)L * R * (i ? N : K), stream)) != hipSuccess) return launched(e, "zero");
    }
    return fine();
  }
  Carve c{const_cast<uint8_t*>(static_cast<const uint8_t*>(p->ctx))}, cw{static_cast<uint8_t*>(p->ws)};
  const LoraCtx x = carve_lora_ctx(c, p->M, R, L);
  const LoraWs w = carve_lora_ws(cw, p->M, K, N, R, L);
  const LoraRows rows{x.count, x.order, p->M, L};
  const LoraFactor u = of_type(x.u, p->dtype), du = of_type(w.du, p->dtype);
  if (p->db) {
    LoraOuter o{p->dtype, R, rows, u, p->dy, p->lddy, N, p->w.scales, p->db, true, w.part};
    if ((e = launch_lora_outer(o, stream)) != hipSuccess) return launched(e, "lora db");
  }
  if (!p->dx && !p->da) return fine();
  // du = scale dy b is the shrink over N with b transposed, dx the expand with a transposed
  const LoraTranspose t[2] = {{p->w.b, p->w.ldb, p->w.b_stride, N, R, w.bt, w.ldn, R * w.ldn},
                              {p->w.a, p->w.lda, p->w.a_stride, R, K, w.at, w.ldr, K * w.ldr}};
  if ((e = launch_lora_transpose(t, p->dx ? 2 : 1, x.count, L, stream)) != hipSuccess) return launched(e, "lora transpose");
  LoraShrink s{p->dtype, R, rows, p->dy, p->lddy, w.bt, w.ldn, R * w.ldn, N, p->w.scales, du};
  if ((e = launch_lora_shrink(s, stream)) != hipSuccess) return launched(e, "lora shrink");
  if (p->dx) {
    LoraExpand ex{p->dtype, R, rows, du, w.at, w.ldr, K * w.ldr, K, nullptr, p->dx_add, p->lddx_add, p->dx, p->lddx};
    if ((e = launch_lora_expand(ex, stream)) != hipSuccess) return launched(e, "lora dx");
  }
  if (p->da) {
    LoraOuter o{p->dtype, R, rows, du, p->x, p->ldx, K, nullptr, p->da, false, w.part};
    if ((e = launch_lora_outer(o, stream)) != hipSuccess) return launched(e, "lora da");
  }
  return fine();
}
