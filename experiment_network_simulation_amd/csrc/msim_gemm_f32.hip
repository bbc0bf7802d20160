/* The products of 32-bit numbers. */
#include "msim_gemm_kernel.h"

namespace msim {

template hipError_t launch_gemm<M_F32, false>(GemmP, const Plan &, hipStream_t);
template hipError_t launch_pair<M_F32>(GemmP, const Plan &, GemmP, const Plan &, const Columns &, hipStream_t);

} // namespace msim
