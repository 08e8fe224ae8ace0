// Host-only stand-ins for the kernel launchers of the bf16 / fp16 operators, for the sanitizer build of
// ops.cpp: each writes every byte of scratch and saved state that its kernels may write, so that
// AddressSanitizer checks the sizes the library reports against the layout it carves.  Test code only.
#include "kernels.h"

#include <algorithm>
#include <cstring>

namespace gmlp {

// the sizes, as the kernel files report them in order of magnitude (any consistent values do)
size_t grouped_matmul_table_bytes(int G, int64_t M) { return 32 * (size_t)(1 + std::max<int64_t>(M / 256 + G + 1, G)); }
int grouped_matmul_parts(int, int, int64_t M, int64_t, int64_t k) { return M > 0 && k >= 512 ? 3 : 1; }
int64_t grouped_matmul_part_floats(int layout, int G, int64_t M, int64_t n, int64_t k) {
  const int p = grouped_matmul_parts(layout, G, M, n, k);
  return p > 1 ? p * (layout == MM_WGRAD ? G * n * k : M * n) : 0;
}
hipError_t launch_grouped_matmul(const MmArgs& a, hipStream_t) {
  *a.flags = 0;
  memset(a.table, 1, grouped_matmul_table_bytes(a.G, a.M));
  memset(a.part, 1, sizeof(float) * (size_t)grouped_matmul_part_floats(a.layout, a.G, a.M, a.n, a.k));
  return hipSuccess;
}
int order_blocks(int64_t n) { return (int)std::max<int64_t>(1, std::min<int64_t>(256, (n + 1023) / 1024)); }
hipError_t launch_group_order(const int32_t*, int64_t n, int G, bool, int32_t* count, int32_t* rows, int32_t* order,
                              int32_t* ws, hipStream_t) {
  memset(count, 0, sizeof(int32_t) * G);
  if (rows) memset(rows, 0, sizeof(int32_t) * n);
  if (order) memset(order, 0, sizeof(int32_t) * n);
  if (order_blocks(n) > 1) memset(ws, 0, sizeof(int32_t) * G * order_blocks(n));
  return hipSuccess;
}
hipError_t launch_dispatch(const MoveArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_combine(const MoveArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_combine_dprobs(const MoveArgs&, hipStream_t) { return hipSuccess; }
static void touch(const LoraFactor& f, int64_t M, int R) {
  memset(f.hi, 1, sizeof(uint16_t) * M * 2 * lora_rp(R));
  if (f.inv) memset(f.inv, 1, sizeof(float) * M);
  if (f.v) memset(f.v, 1, sizeof(float) * M * R);
}
hipError_t launch_lora_shrink(const LoraShrink& a, hipStream_t) {
  touch(a.out, a.rows.M, a.R);
  return hipSuccess;
}
hipError_t launch_lora_expand(const LoraExpand&, hipStream_t) { return hipSuccess; }
int64_t lora_outer_part_floats(int64_t M, int64_t C, int R, int L) { return (M / 256 + std::min<int64_t>(L, M)) * R * C; }
hipError_t launch_lora_outer(const LoraOuter& a, hipStream_t) {
  memset(a.part, 1, sizeof(float) * (size_t)lora_outer_part_floats(a.rows.M, a.C, a.R, a.rows.L));
  return hipSuccess;
}
hipError_t launch_zero16(void* p, int64_t n, hipStream_t) {
  memset(p, 0, 2 * n);
  return hipSuccess;
}
hipError_t launch_lora_transpose(const LoraTranspose* t, int n, const int32_t*, int L, hipStream_t) {
  for (int i = 0; i < n; ++i) memset(t[i].dst, 1, 2 * (size_t)((L - 1) * t[i].dst_stride + t[i].C * t[i].ldd));
  return hipSuccess;
}

}  // namespace gmlp
