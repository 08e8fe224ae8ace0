// Drives every entry point of the bf16 / fp16 operators through the sanitizer build (ops.cpp with the
// launchers of ops_stubs.cpp): calls at exactly the reported sizes must succeed and write inside their
// buffers, calls one byte short must be refused.
#include "gmlp.h"

#include <cstdio>
#include <cstdlib>
#include <cstring>

static int bad = 0;
static void expect(const char* what, gmlp_status got, gmlp_status want) {
  if (got != want) {
    printf("%s: status %d, expected %d (%s)\n", what, got, want, gmlp_last_error());
    ++bad;
  }
}
// 16-byte aligned buffer of exactly n bytes (at least 1)
struct Buf {
  void* p;
  explicit Buf(size_t n) : p(aligned_alloc(16, n ? (n + 15) / 16 * 16 : 16)) { memset(p, 0, n); }
  ~Buf() { free(p); }
};

static void matmul(int layout, int G, int64_t M, int64_t n, int64_t k) {
  size_t need = 0;
  expect("matmul ws", gmlp_grouped_matmul_ws_bytes(layout, G, M, n, k, &need), GMLP_OK);
  Buf ws(need), m(4 * G), t(64);
  gmlp_grouped_matmul_args a;
  memset(&a, 0, sizeof(a));
  a.layout = layout;
  a.a = a.b = t.p;
  a.c = t.p;
  a.lda = layout == GMLP_GEMM_WGRAD ? n : k;
  a.ldb = layout == GMLP_GEMM_DGRAD ? n : k;
  a.ldc = layout == GMLP_GEMM_WGRAD ? k : n;
  a.b_stride = a.c_stride = n * k;
  a.m_splits = static_cast<int32_t*>(m.p);
  a.G = G;
  a.M = M;
  a.n = n;
  a.k = k;
  a.ws = ws.p;
  a.ws_bytes = need;
  expect("matmul", gmlp_grouped_matmul(&a, nullptr), GMLP_OK);
  a.ws_bytes = need - 1;
  expect("matmul short ws", gmlp_grouped_matmul(&a, nullptr), GMLP_WORKSPACE);
  a.ws_bytes = need;
  a.dtype = 9;
  expect("matmul dtype", gmlp_grouped_matmul(&a, nullptr), GMLP_UNSUPPORTED);
}

static void plan(int64_t n, int E) {
  size_t need = 0;
  expect("plan ws", gmlp_dispatch_plan_ws_bytes(n, E, &need), GMLP_OK);
  Buf ws(need), ids(4 * n), m(4 * E), rows(4 * n), order(4 * n);
  int32_t *i = static_cast<int32_t*>(ids.p), *s = static_cast<int32_t*>(m.p), *r = static_cast<int32_t*>(rows.p),
          *o = static_cast<int32_t*>(order.p);
  expect("plan", gmlp_dispatch_plan(i, n, E, s, r, o, ws.p, need, nullptr), GMLP_OK);
  expect("plan without order", gmlp_dispatch_plan(i, n, E, s, r, nullptr, ws.p, need, nullptr), GMLP_OK);
  if (need) expect("plan short ws", gmlp_dispatch_plan(i, n, E, s, r, o, ws.p, need - 1, nullptr), GMLP_WORKSPACE);
}

static void moves() {
  Buf t(4096), w(4096);
  gmlp_move_args a;
  memset(&a, 0, sizeof(a));
  a.src = a.src2 = t.p;
  a.dst = w.p;
  a.ld_src = a.ld_src2 = a.ld_dst = 8;
  a.T = 4;
  a.H = 8;
  a.k = 2;
  a.E = 3;
  a.rows = a.m_splits = static_cast<int32_t*>(t.p);
  a.probs = static_cast<float*>(t.p);
  a.dprobs = static_cast<float*>(w.p);
  a.zero_rest = 1;
  expect("dispatch", gmlp_dispatch(&a, nullptr), GMLP_OK);
  expect("combine", gmlp_combine(&a, nullptr), GMLP_OK);
  expect("dprobs", gmlp_combine_dprobs(&a, nullptr), GMLP_OK);
  a.H = 9;
  expect("dispatch stride", gmlp_dispatch(&a, nullptr), GMLP_INVALID_ARG);
  a.T = 0;
  expect("dispatch nothing", gmlp_dispatch(&a, nullptr), GMLP_OK);
}

static void lora(int dtype, int64_t M, int64_t K, int64_t N, int R, int L) {
  gmlp_lora_sizes sz;
  expect("lora sizes", gmlp_lora_query_sizes(M, K, N, R, L, &sz), GMLP_OK);
  Buf ctx(sz.ctx_bytes), fws(sz.fwd_ws_bytes), bws(sz.bwd_ws_bytes), t(64), ids(4 * M + 4), da(2 * L * R * K), db(2 * L * R * N);
  gmlp_lora_weights w = {t.p, K, R * K, t.p, R, N * R, nullptr};
  gmlp_lora_fwd_args f;
  memset(&f, 0, sizeof(f));
  f.dtype = dtype;
  f.R = R;
  f.L = L;
  f.M = M;
  f.K = K;
  f.N = N;
  f.x = t.p;
  f.ldx = K;
  f.w = w;
  f.ids = static_cast<int32_t*>(ids.p);
  f.y = t.p;
  f.ldy = N;
  f.ctx = ctx.p;
  f.ctx_bytes = sz.ctx_bytes;
  f.ws = fws.p;
  f.ws_bytes = sz.fwd_ws_bytes;
  expect("lora forward", gmlp_lora_forward(&f, nullptr), GMLP_OK);
  f.ctx_bytes -= 1;
  if (M) expect("lora short ctx", gmlp_lora_forward(&f, nullptr), GMLP_WORKSPACE);
  gmlp_lora_bwd_args b;
  memset(&b, 0, sizeof(b));
  b.dtype = dtype;
  b.R = R;
  b.L = L;
  b.M = M;
  b.K = K;
  b.N = N;
  b.dy = b.x = t.p;
  b.lddy = N;
  b.ldx = b.lddx = K;
  b.w = w;
  b.dx = t.p;
  b.da = da.p;
  b.db = db.p;
  b.ctx = ctx.p;
  b.ctx_bytes = sz.ctx_bytes;
  b.ws = bws.p;
  b.ws_bytes = sz.bwd_ws_bytes;
  expect("lora backward", gmlp_lora_backward(&b, nullptr), GMLP_OK);
  b.dx = nullptr;
  expect("lora backward without dx", gmlp_lora_backward(&b, nullptr), GMLP_OK);
  b.da = nullptr;
  expect("lora backward db only", gmlp_lora_backward(&b, nullptr), GMLP_OK);
  b.ws_bytes -= 1;
  expect("lora short ws", gmlp_lora_backward(&b, nullptr), GMLP_WORKSPACE);
}

int main() {
  for (int layout = 0; layout < 3; ++layout) {
    matmul(layout, 1, 1, 1, 1);
    matmul(layout, 7, 300, 40, 24);
    matmul(layout, 3, 1000, 16, 600);
    matmul(layout, 5, 0, 8, 8);
  }
  plan(0, 1);
  plan(5, 1024);
  plan(1025, 3);
  plan(300000, 64);
  moves();
  for (int dtype = 0; dtype < 2; ++dtype) {
    lora(dtype, 1, 8, 8, 1, 1);
    lora(dtype, 37, 65, 50, 3, 4);
    lora(dtype, 3000, 33, 17, 128, 9);
    lora(dtype, 0, 16, 24, 8, 2);
  }
  if (bad) return 1;
  printf("all statuses as expected\n");
  return 0;
}
