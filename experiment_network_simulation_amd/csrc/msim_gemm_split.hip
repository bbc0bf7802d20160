/* The products of numbers that are the sum of two f16. */
#include "msim_gemm_kernel.h"

namespace msim {

template hipError_t launch_gemm<M_SPLIT, false>(GemmP, const Plan &, hipStream_t);
template hipError_t launch_gemm<M_SPLIT, true>(GemmP, const Plan &, hipStream_t);

} // namespace msim
