// w4_matvec_bf16_ragged.cu -- the bf16 kernels of w4_matvec.cuh for groups of scales at any place.
#include "w4_matvec.cuh"

namespace moe {
namespace w4 {

template cudaError_t run<__nv_bfloat16, false>(const Params&, int, int64_t, int64_t, cudaStream_t);

}  // namespace w4
}  // namespace moe
