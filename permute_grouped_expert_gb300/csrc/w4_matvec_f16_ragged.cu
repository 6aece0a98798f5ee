// w4_matvec_f16_ragged.cu -- the f16 kernels of w4_matvec.cuh for groups of scales at any place.
#include "w4_matvec.cuh"

namespace moe {
namespace w4 {

template cudaError_t run<__half, false>(const Params&, int, int64_t, int64_t, cudaStream_t);

}  // namespace w4
}  // namespace moe
