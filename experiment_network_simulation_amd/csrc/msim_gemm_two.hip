/* The products of numbers that are the sum of two bf16, with results in f16. */
#include "msim_gemm_kernel.h"

namespace msim {

template hipError_t launch_pair<M_TWO>(GemmP, const Plan &, GemmP, const Plan &, const Columns &, hipStream_t);

} // namespace msim
