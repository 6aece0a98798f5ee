// grouped_gemm.cu -- which kernel a product grouped by expert runs on.
#include "grouped_gemm.h"

namespace moe {

size_t grouped_gemm_workspace_bytes(const moe_shape& s, const moe_layout& l, int64_t N, int64_t Kd) {
  return 256;
}

cudaError_t launch_grouped_gemm(GemmDir dir, const GroupedGemm& g, cudaStream_t st) {
  return grouped_gemm_tc_takes(dir, g) ? launch_grouped_gemm_tc(dir, g, st) : launch_grouped_gemm_any(dir, g, st);
}

}  // namespace moe
