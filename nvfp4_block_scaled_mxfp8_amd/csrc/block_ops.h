// Private interface between block_ops.cpp and the kernels of the operators around the experts: routing
// (route.hip), norms (norm.hip) and products with 4-bit weights (w4.hip).
#pragma once
#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace gmlp {

// ----------------------------------------------------------------------------- routing
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxK = 64;
constexpr int kRouteMaxGroups = 64;
enum RouteType { ROUTE_BF16 = 0, ROUTE_FP16 = 1, ROUTE_FP32 = 2 };
struct RouteArgs {
  int type;
  int sigmoid;              // score: else softmax
  const void* logits;
  int64_t ld;
  int64_t T;
  int E, k;
  const float* bias;        // may be null
  int groups, top_groups, group_best;
  int renormalize;
  float scale;
  int32_t* experts;         // [T, k]; read by the backward
  float* probs;
  const float* dprobs;      // backward
  void* dlogits;
  int64_t ld_dlogits;
  uint32_t row_blocks;      // workgroups along x, set by the launcher
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_route_backward(const RouteArgs& a, hipStream_t s);

// ----------------------------------------------------------------------------- norms
constexpr int kNormMaxH = 32768;
enum NormGate { GATE_NONE = 0, GATE_CHANNEL = 1, GATE_TOKEN = 2, GATE_FULL = 3 };
struct NormArgs {
  int type;                 // MmType
  int gate_kind;
  int weight_fp32, branch_weight_fp32, gate_fp32;
  float eps, scale;
  int64_t T;
  int H;
  const void* x;
  const void* branch;       // null: y = x
  const void* weight;       // null: no h
  const void* branch_weight;
  const void* gate;
  int64_t ldx, ldbranch, ld_gate;
  void* y;
  void* h;
  int64_t ldy, ldh;
  float* stats;             // [2][T]: the factors of branch and of y; null: not kept
  // backward
  const void* dy;           // null: zeros
  const void* dh;
  int64_t lddy, lddh;
  void* dx;
  void* dbranch;
  int64_t lddx, lddbranch;
  void* dgate;
  void* dweight;
  void* dbranch_weight;
  float* part;              // column sums of the workgroups
  uint32_t row_blocks;      // workgroups along x, set by the launcher
};
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s);

// ----------------------------------------------------------------------------- products with 4-bit weights
enum W4Kind { W4_INT = 0, W4_NVFP4 = 1 };
struct W4Args {
  int type;                 // MmType
  int kind;
  int group;
  int zero_rest;
  const void* x;
  int64_t ldx;
  const uint8_t* codes;     // [G][N][K / 2]
  const void* scales;       // [G][N][K / group]: of x's type, NVFP4: E4M3 bytes
  const uint8_t* zeros;     // [G][N][K / group] or null (8)
  const float* amax;        // [G], NVFP4
  void* y;
  int64_t ldy;
  const int32_t* m_splits;
  int G;
  int64_t M;
  int N, K;
  uint32_t row_blocks;      // workgroups along x, set by the launcher
};
hipError_t launch_w4(const W4Args& a, hipStream_t s);

}  // namespace gmlp
