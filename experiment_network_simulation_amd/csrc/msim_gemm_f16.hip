/* The products of f16. */
#include "msim_gemm_kernel.h"

namespace msim {

template hipError_t launch_gemm<M_F16, false>(GemmP, const Plan &, hipStream_t);
template hipError_t launch_pair<M_F16>(GemmP, const Plan &, GemmP, const Plan &, const Columns &, hipStream_t);

} // namespace msim
