// C ABI of the operators around the experts (routing, norms, products with 4-bit weights): validation and
// launches.
#include "block_ops.h"
#include "block_sizes.h"
#include "gmlp.h"
#include "kernels.h"
#include "planner.h"

#include <math.h>

using namespace gmlp;

namespace {

constexpr int64_t kMaxRows = 1LL << 30;
constexpr int64_t kMaxLd = 1LL << 20;

gmlp_status fine() { return set_error(GMLP_OK, "%s", ""); }
gmlp_status launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return fine();
  return set_error(GMLP_HIP_ERROR, "system: launching %s failed: %s", what, hipGetErrorString(e));
}
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
gmlp_status null_arg() { return set_error(GMLP_INVALID_ARG, "null pointer argument"); }
gmlp_status misaligned() { return set_error(GMLP_INVALID_ARG, "a tensor is not aligned to its elements"); }
gmlp_status short_rows() {
  return set_error(GMLP_INVALID_ARG, "strides: row strides must be at least the row's length");
}
gmlp_status check_rows(int64_t M, const char* name) {
  if (M < 0 || M > kMaxRows) return set_error(GMLP_UNSUPPORTED, "dims: %s = %lld rows is out of range", name, (long long)M);
  return GMLP_OK;
}
gmlp_status check_dtype(int32_t t) {
  if (t != GMLP_BF16 && t != GMLP_FP16) return set_error(GMLP_UNSUPPORTED, "dtype: bf16 or fp16 is required, got %d", t);
  return GMLP_OK;
}

// ----------------------------------------------------------------------------- routing
// What the forward and the backward share.
template <class Args>
gmlp_status check_route(const Args* p) {
  if (p->dtype != GMLP_BF16 && p->dtype != GMLP_FP16 && p->dtype != GMLP_LOGITS_FP32)
    return set_error(GMLP_UNSUPPORTED, "dtype: bf16, fp16 or fp32 logits are required, got %d", p->dtype);
  if (p->score != GMLP_SCORE_SOFTMAX && p->score != GMLP_SCORE_SIGMOID)
    return set_error(GMLP_INVALID_ARG, "score: unknown value %d", p->score);
  const gmlp_status st = check_rows(p->T, "T");
  if (st != GMLP_OK) return st;
  if (p->E < 1 || p->E > kRouteMaxExperts)
    return set_error(GMLP_UNSUPPORTED, "dims: 1 to %d experts are supported, got %d", kRouteMaxExperts, p->E);
  if (p->k < 1 || p->k > kRouteMaxK)
    return set_error(GMLP_UNSUPPORTED, "dims: k must be in [1, %d], got %d", kRouteMaxK, p->k);
  if (!isfinite(p->scale)) return set_error(GMLP_INVALID_ARG, "scale: a finite number is required");
  if (p->T > 0 && (!p->logits || !p->experts)) return null_arg();
  if (!aligned(p->logits, p->dtype == GMLP_LOGITS_FP32 ? 4 : 2) || !aligned(p->experts, 4)) return misaligned();
  if (p->ld < p->E) return short_rows();
  return GMLP_OK;
}
template <class Args>
RouteArgs route_args(const Args* p) {
  RouteArgs a{};
  a.type = p->dtype;
  a.sigmoid = p->score == GMLP_SCORE_SIGMOID;
  a.logits = p->logits;
  a.ld = p->ld;
  a.T = p->T;
  a.E = p->E;
  a.k = p->k;
  a.renormalize = p->renormalize != 0;
  a.scale = p->scale;
  a.experts = const_cast<int32_t*>(p->experts);
  return a;
}
}  // namespace

extern "C" gmlp_status gmlp_route(const gmlp_route_args* p, hipStream_t stream) {
  if (!p) return null_arg();
  const gmlp_status st = check_route(p);
  if (st != GMLP_OK) return st;
  if (p->groups < 1 || p->groups > kRouteMaxGroups || p->E % p->groups)
    return set_error(GMLP_UNSUPPORTED, "groups: 1 to %d groups of equal size are supported, got %d of %d experts", kRouteMaxGroups,
                     p->groups, p->E);
  if (p->top_groups < 1 || p->top_groups > p->groups)
    return set_error(GMLP_INVALID_ARG, "top_groups: must be in [1, %d], got %d", p->groups, p->top_groups);
  if (p->group_best != 1 && p->group_best != 2)
    return set_error(GMLP_UNSUPPORTED, "group_best: 1 or 2 is supported, got %d", p->group_best);
  if (p->k > p->top_groups * (p->E / p->groups))
    return set_error(GMLP_INVALID_ARG, "dims: k = %d exceeds the %d experts that can be chosen", p->k,
                     p->top_groups * (p->E / p->groups));
  if (p->T > 0 && !p->probs) return null_arg();
  if (!aligned(p->probs, 4) || !aligned(p->bias, 4)) return misaligned();
  if (p->T == 0) return fine();
  RouteArgs a = route_args(p);
  a.bias = p->bias;
  a.groups = p->groups;
  a.top_groups = p->top_groups;
  a.group_best = p->group_best;
  a.probs = p->probs;
  return launched(launch_route(a, stream), "route");
}

extern "C" gmlp_status gmlp_route_backward(const gmlp_route_bwd_args* p, hipStream_t stream) {
  if (!p) return null_arg();
  const gmlp_status st = check_route(p);
  if (st != GMLP_OK) return st;
  if (p->T > 0 && (!p->dprobs || !p->dlogits)) return null_arg();
  if (!aligned(p->dprobs, 4) || !aligned(p->dlogits, p->dtype == GMLP_LOGITS_FP32 ? 4 : 2)) return misaligned();
  if (p->ld_dlogits < p->E) return short_rows();
  if (p->T == 0) return fine();
  RouteArgs a = route_args(p);
  a.dprobs = p->dprobs;
  a.dlogits = p->dlogits;
  a.ld_dlogits = p->ld_dlogits;
  return launched(launch_route_backward(a, stream), "route backward");
}

// ----------------------------------------------------------------------------- norms
namespace {
gmlp_status check_norm(const gmlp_norm_inputs& in) {
  gmlp_status st = check_dtype(in.dtype);
  if (st != GMLP_OK) return st;
  if ((st = check_rows(in.T, "T")) != GMLP_OK) return st;
  if (in.H < 1 || in.H > kNormMaxH)
    return set_error(GMLP_UNSUPPORTED, "dims: H must be in [1, %d], got %lld", kNormMaxH, (long long)in.H);
  if (in.gate_kind < GMLP_GATE_NONE || in.gate_kind > GMLP_GATE_FULL)
    return set_error(GMLP_INVALID_ARG, "gate_kind: unknown value %d", in.gate_kind);
  if (!(in.eps >= 0.0f) || !isfinite(in.eps)) return set_error(GMLP_INVALID_ARG, "eps: a finite number >= 0 is required");
  if (!isfinite(in.scale)) return set_error(GMLP_INVALID_ARG, "scale: a finite number is required");
  if (!in.branch && (in.branch_weight || in.gate_kind != GMLP_GATE_NONE || in.scale != 1.0f))
    return set_error(GMLP_INVALID_ARG, "branch: a branch weight, a gate or a scale needs a branch");
  if (!in.branch && !in.weight) return set_error(GMLP_INVALID_ARG, "neither branch nor weight: nothing to compute");
  if (in.T > 0 && !in.x) return null_arg();
  if (in.gate_kind != GMLP_GATE_NONE && (in.T > 0 || in.gate_kind == GMLP_GATE_CHANNEL) && !in.gate) return null_arg();
  if (!aligned(in.x, 2) || !aligned(in.branch, 2) || !aligned(in.weight, in.weight_fp32 ? 4 : 2) ||
      !aligned(in.branch_weight, in.branch_weight_fp32 ? 4 : 2) || !aligned(in.gate, in.gate_fp32 ? 4 : 2))
    return misaligned();
  if (in.ldx < in.H || (in.branch && in.ldbranch < in.H) || (in.gate_kind == GMLP_GATE_FULL && in.ld_gate < in.H) ||
      (in.gate_kind == GMLP_GATE_TOKEN && in.ld_gate < 1))
    return short_rows();
  return GMLP_OK;
}
NormArgs norm_args(const gmlp_norm_inputs& in) {
  NormArgs a{};
  a.type = in.dtype;
  a.gate_kind = in.gate_kind;
  a.weight_fp32 = in.weight_fp32 != 0;
  a.branch_weight_fp32 = in.branch_weight_fp32 != 0;
  a.gate_fp32 = in.gate_fp32 != 0;
  a.eps = in.eps;
  a.scale = in.scale;
  a.T = in.T;
  a.H = (int)in.H;
  a.x = in.x;
  a.branch = in.branch;
  a.weight = in.weight;
  a.branch_weight = in.branch_weight;
  a.gate = in.gate;
  a.ldx = in.ldx;
  a.ldbranch = in.ldbranch;
  a.ld_gate = in.ld_gate;
  return a;
}
}  // namespace

extern "C" gmlp_status gmlp_residual_norm(const gmlp_norm_args* p, hipStream_t stream) {
  if (!p) return null_arg();
  const gmlp_norm_inputs& in = p->in;
  const gmlp_status st = check_norm(in);
  if (st != GMLP_OK) return st;
  if (in.T > 0 && ((in.branch && !p->y) || (in.weight && !p->h))) return null_arg();
  if (!aligned(p->y, 2) || !aligned(p->h, 2) || !aligned(p->stats, 4)) return misaligned();
  if ((in.branch && p->ldy < in.H) || (in.weight && p->ldh < in.H)) return short_rows();
  if (in.branch && p->y && ((p->y == in.x && p->ldy != in.ldx) || (p->y == in.branch && p->ldy != in.ldbranch)))
    return set_error(GMLP_INVALID_ARG, "strides: y and an input are one tensor with two row strides");
  if (in.T == 0) return fine();
  NormArgs a = norm_args(in);
  a.y = p->y;
  a.ldy = p->ldy;
  a.h = p->h;
  a.ldh = p->ldh;
  a.stats = p->stats;
  return launched(launch_norm(a, stream), "residual norm");
}

extern "C" gmlp_status gmlp_residual_norm_bwd_ws_bytes(int64_t T, int64_t H, size_t* bytes) {
  if (!bytes) return null_arg();
  const gmlp_status st = check_rows(T, "T");
  if (st != GMLP_OK) return st;
  if (H < 1 || H > kNormMaxH)
    return set_error(GMLP_UNSUPPORTED, "dims: H must be in [1, %d], got %lld", kNormMaxH, (long long)H);
  *bytes = sizeof(float) * (size_t)sizes::norm_part_floats(T, H);
  return fine();
}

extern "C" gmlp_status gmlp_residual_norm_backward(const gmlp_norm_bwd_args* p, hipStream_t stream) {
  if (!p) return null_arg();
  const gmlp_norm_inputs& in = p->in;
  const gmlp_status st = check_norm(in);
  if (st != GMLP_OK) return st;
  if (in.weight ? (in.T > 0 && !p->dh) : p->dh != nullptr)
    return set_error(GMLP_INVALID_ARG, "dh: goes with a weight");
  if (in.T > 0 && (in.weight || in.branch_weight) && !p->stats) return null_arg();
  if ((p->dbranch && !in.branch) || (p->dgate && in.gate_kind == GMLP_GATE_NONE) || (p->dweight && !in.weight) ||
      (p->dbranch_weight && !in.branch_weight))
    return set_error(GMLP_INVALID_ARG, "a gradient is asked for an input that is not there");
  if (!aligned(p->dy, 2) || !aligned(p->dh, 2) || !aligned(p->stats, 4) || !aligned(p->dx, 2) || !aligned(p->dbranch, 2) ||
      !aligned(p->dgate, in.gate_fp32 ? 4 : 2) || !aligned(p->dweight, in.weight_fp32 ? 4 : 2) ||
      !aligned(p->dbranch_weight, in.branch_weight_fp32 ? 4 : 2))
    return misaligned();
  if ((p->dy && p->lddy < in.H) || (p->dh && p->lddh < in.H) || (p->dx && p->lddx < in.H) ||
      (p->dbranch && p->lddbranch < in.H))
    return short_rows();
  size_t need = 0;
  gmlp_residual_norm_bwd_ws_bytes(in.T, in.H, &need);
  if (!p->ws || p->ws_bytes < need || !aligned(p->ws, 16))
    return set_error(GMLP_WORKSPACE, "workspace: %zu bytes, 16-byte aligned, are needed", need);
  NormArgs a = norm_args(in);
  a.dy = p->dy;
  a.lddy = p->lddy;
  a.dh = p->dh;
  a.lddh = p->lddh;
  a.stats = const_cast<float*>(p->stats);
  a.dx = p->dx;
  a.lddx = p->lddx;
  a.dbranch = p->dbranch;
  a.lddbranch = p->lddbranch;
  a.dgate = p->dgate;
  a.dweight = p->dweight;
  a.dbranch_weight = p->dbranch_weight;
  a.part = static_cast<float*>(p->ws);
  return launched(launch_norm_backward(a, stream), "residual norm backward");
}

// ----------------------------------------------------------------------------- products with 4-bit weights
extern "C" gmlp_status gmlp_grouped_matmul_four_bit(const gmlp_w4_args* p, hipStream_t stream) {
  if (!p) return null_arg();
  gmlp_status st = check_dtype(p->dtype);
  if (st != GMLP_OK) return st;
  if (p->kind != GMLP_W4_INT && p->kind != GMLP_W4_NVFP4) return set_error(GMLP_INVALID_ARG, "kind: unknown value %d", p->kind);
  const bool nv = p->kind == GMLP_W4_NVFP4;
  if (nv ? p->group != 16 : p->group != 32 && p->group != 64 && p->group != 128)
    return set_error(GMLP_UNSUPPORTED, "group: %s, got %d", nv ? "16 is required for NVFP4" : "32, 64 or 128 is required", p->group);
  if ((st = check_rows(p->M, "M")) != GMLP_OK) return st;
  if (p->G < 1 || p->G > 1 << 16) return set_error(GMLP_UNSUPPORTED, "dims: 1 to 65536 groups are supported, got %d", p->G);
  if (p->N < 1 || p->K < 1 || p->N >= kMaxLd || p->K >= kMaxLd)
    return set_error(GMLP_UNSUPPORTED, "dims: N and K must be in [1, 2^20), got %lld and %lld", (long long)p->N, (long long)p->K);
  const int step = nv ? 32 : p->group;
  if (p->K % step) return set_error(GMLP_UNSUPPORTED, "dims: K must be a multiple of %d, got %lld", step, (long long)p->K);
  if (!p->m_splits || !p->codes || !p->scales || (nv && !p->amax) || (p->M > 0 && (!p->x || !p->y))) return null_arg();
  if (nv && p->zeros) return set_error(GMLP_INVALID_ARG, "zeros: NVFP4 weights have none");
  if (!aligned(p->x, 2) || !aligned(p->y, 2) || !aligned(p->codes, 16) || !aligned(p->scales, nv ? 1 : 2) || !aligned(p->amax, 4) ||
      !aligned(p->m_splits, 4))
    return set_error(GMLP_INVALID_ARG, "a tensor is not aligned to its elements, or codes not to 16 bytes");
  if (p->ldx < p->K || p->ldy < p->N || p->ldx >= kMaxLd || p->ldy >= kMaxLd)
    return set_error(GMLP_INVALID_ARG, "strides: row strides must be at least the row's length and below 2^20");
  if (sizes::w4_tiles_bound(p->M, p->G, p->N) > 2147483647LL)
    return set_error(GMLP_UNSUPPORTED, "dims: %lld rows of %lld columns exceed one launch", (long long)p->M, (long long)p->N);
  if (p->M == 0) return fine();
  W4Args a{};
  a.type = p->dtype;
  a.kind = p->kind;
  a.group = p->group;
  a.zero_rest = p->zero_rest != 0;
  a.x = p->x;
  a.ldx = p->ldx;
  a.codes = p->codes;
  a.scales = p->scales;
  a.zeros = p->zeros;
  a.amax = p->amax;
  a.y = p->y;
  a.ldy = p->ldy;
  a.m_splits = p->m_splits;
  a.G = p->G;
  a.M = p->M;
  a.N = (int)p->N;
  a.K = (int)p->K;
  return launched(launch_w4(a, stream), "grouped matmul w4");
}
