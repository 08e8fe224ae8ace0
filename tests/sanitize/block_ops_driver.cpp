// Drives the entry points of the operators around the experts through a sanitizer build of block_ops.cpp: the
// launchers here are stand-ins that write every byte that their kernels may write, so that the sizes the library reports are
// checked against the buffers; and checks block_sizes.h against counts.  Test code only.
#include "block_ops.h"
#include "block_sizes.h"
#include "gmlp.h"

#include <cstdio>
#include <cstdlib>
#include <cstring>

namespace gmlp {
static int64_t launches = 0;
hipError_t launch_route(const RouteArgs& a, hipStream_t) {
  memset(a.experts, 1, 4 * (size_t)(a.T * a.k));
  memset(a.probs, 1, 4 * (size_t)(a.T * a.k));
  ++launches;
  return hipSuccess;
}
hipError_t launch_route_backward(const RouteArgs& a, hipStream_t) {
  memset(a.dlogits, 1, (a.type == ROUTE_FP32 ? 4 : 2) * (size_t)((a.T - 1) * a.ld_dlogits + a.E));
  ++launches;
  return hipSuccess;
}
hipError_t launch_norm(const NormArgs& a, hipStream_t) {
  if (a.stats) memset(a.stats, 1, 8 * (size_t)a.T);
  ++launches;
  return hipSuccess;
}
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t) {
  memset(a.part, 1, sizeof(float) * (size_t)sizes::norm_part_floats(a.T, a.H));
  ++launches;
  return hipSuccess;
}
hipError_t launch_w4(const W4Args&, hipStream_t) {
  ++launches;
  return hipSuccess;
}
}  // namespace gmlp

using namespace gmlp;

static int bad = 0;
static void expect(const char* what, gmlp_status got, gmlp_status want) {
  if (got != want) {
    printf("%s: status %d, expected %d (%s)\n", what, got, want, gmlp_last_error());
    ++bad;
  }
}
struct Buf {
  void* p;
  explicit Buf(size_t n) : p(aligned_alloc(16, n ? (n + 15) / 16 * 16 : 16)) { memset(p, 0, n); }
  ~Buf() { free(p); }
};

static void route(int64_t T, int E, int k, int dtype) {
  Buf l(4 * T * E), e(4 * T * k), pr(4 * T * k), d(4 * T * E);
  gmlp_route_args a;
  memset(&a, 0, sizeof(a));
  a.dtype = dtype;
  a.logits = l.p;
  a.ld = a.E = E;
  a.T = T;
  a.k = k;
  a.groups = a.top_groups = a.group_best = 1;
  a.scale = 1.0f;
  a.experts = static_cast<int32_t*>(e.p);
  a.probs = static_cast<float*>(pr.p);
  expect("route", gmlp_route(&a, nullptr), GMLP_OK);
  gmlp_route_bwd_args b;
  memset(&b, 0, sizeof(b));
  b.dtype = dtype;
  b.logits = l.p;
  b.ld = b.E = b.ld_dlogits = E;
  b.T = T;
  b.k = k;
  b.scale = 1.0f;
  b.experts = a.experts;
  b.dprobs = a.probs;
  b.dlogits = d.p;
  expect("route backward", gmlp_route_backward(&b, nullptr), GMLP_OK);
}

static void norm(int64_t T, int64_t H) {
  size_t need = 0;
  expect("norm ws", gmlp_residual_norm_bwd_ws_bytes(T, H, &need), GMLP_OK);
  Buf t(64), stats(8 * T), ws(need);
  gmlp_norm_inputs in;
  memset(&in, 0, sizeof(in));
  in.gate_kind = GMLP_GATE_CHANNEL;
  in.scale = 0.5f;
  in.T = T;
  in.H = in.ldx = in.ldbranch = H;
  in.x = in.branch = in.weight = in.branch_weight = in.gate = t.p;
  gmlp_norm_args a{in, t.p, H, t.p, H, static_cast<float*>(stats.p)};
  expect("norm", gmlp_residual_norm(&a, nullptr), GMLP_OK);
  gmlp_norm_bwd_args b{in, t.p, H, t.p, H, static_cast<float*>(stats.p), t.p, H, t.p, H, t.p, t.p, t.p, ws.p, need};
  expect("norm backward", gmlp_residual_norm_backward(&b, nullptr), GMLP_OK);
  b.ws_bytes = need - 1;
  expect("norm short ws", gmlp_residual_norm_backward(&b, nullptr), GMLP_WORKSPACE);
}

static void w4(int64_t M, int64_t N, int64_t K, int kind, int group) {
  Buf t(64);
  gmlp_w4_args a;
  memset(&a, 0, sizeof(a));
  a.kind = kind;
  a.group = group;
  a.x = a.codes = static_cast<uint8_t*>(t.p);
  a.scales = a.y = t.p;
  a.amax = static_cast<float*>(t.p);
  a.m_splits = static_cast<int32_t*>(t.p);
  a.G = 3;
  a.M = M;
  a.N = a.ldy = N;
  a.K = a.ldx = K;
  expect("w4", gmlp_grouped_matmul_four_bit(&a, nullptr), GMLP_OK);
}

// A row's threads cover it in eights, with less than a wave of them to spare, and fit a workgroup.
static void norm_sizes() {
  for (int64_t H = 1; H <= kNormMaxH; ++H)
    for (int C : {1, 2, 4}) {
      const int64_t n = sizes::norm_threads(H, C);
      if (n % 64 || n * C * 8 < H || (n - 64) * C * 8 >= H || (C == 4 && n > 1024)) {
        printf("norm threads of %lld in %d: %lld\n", (long long)H, C, (long long)n);
        ++bad;
      }
    }
}

int main() {
  for (int dtype = 0; dtype < 3; ++dtype) {
    route(1, 1, 1, dtype);
    route(37, 130, 8, dtype);
    route(0, 8, 2, dtype);
  }
  for (int64_t T : {0, 1, 37, 600, 5000})
    for (int64_t H : {1, 9, 1001, 32768}) norm(T, H);
  w4(1, 1, 32, GMLP_W4_INT, 32);
  w4(37, 50, 256, GMLP_W4_INT, 128);
  w4(37, 50, 96, GMLP_W4_NVFP4, 16);
  w4(0, 50, 96, GMLP_W4_NVFP4, 16);
  norm_sizes();
  if (launches != 2 * 6 + 16 + 20 + 3) {
    printf("%lld launches\n", (long long)launches);
    ++bad;
  }
  if (bad) return 1;
  printf("all statuses as expected\n");
  return 0;
}
