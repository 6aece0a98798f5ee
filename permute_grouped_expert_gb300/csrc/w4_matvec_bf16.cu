// w4_matvec_bf16.cu -- the bf16 kernels of w4_matvec.cuh for aligned groups of scales.
#include "w4_matvec.cuh"

namespace moe {
namespace w4 {

template cudaError_t run<__nv_bfloat16, true>(const Params&, int, int64_t, int64_t, cudaStream_t);

}  // namespace w4
}  // namespace moe
