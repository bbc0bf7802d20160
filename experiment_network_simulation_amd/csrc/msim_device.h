/* What the kernels of the calls without a context share: element types and how a
 * call launches and reports. */
#ifndef MSIM_DEVICE_H
#define MSIM_DEVICE_H

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "msim.h"
#include "msim_error.h"

/* What is wrong with a router (and the code for it), or NULL; msim_route makes the same checks. */
__attribute__((visibility("hidden"))) const char *msim_check_route(const msim_route_spec *s, bool backward, int *code) noexcept;

namespace {

constexpr int WAVE = 64;

struct F32 {
    typedef float raw;
    static __device__ float get(raw v) { return v; }
    static __device__ raw put(float v) { return v; }
};
struct F16 {
    typedef uint16_t raw;
    static __device__ float get(raw v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ raw put(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};
struct BF16 {
    typedef uint16_t raw;
    static __device__ float get(raw v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
    /* to nearest, ties to even; a NaN stays one */
    static __device__ raw put(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};

/* what the wavefront's lanes wrote to LDS is there for its other lanes */
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

[[maybe_unused]] inline int fail(int code, const char *what) { msim_set_error(what); return code; }

/* Enqueues a kernel.  The result is the launch's own: an error that another call
 * left pending on this thread neither fails it nor is taken from its owner. */
template <typename... P, typename... A>
hipError_t launch(void (*kernel)(P...), uint32_t grid, uint32_t block, size_t lds, hipStream_t st, A... args)
{
    return [&](P... p) {
        void *at[] = {&p...};
        return hipLaunchKernel((const void *)kernel, dim3(grid), dim3(block), at, lds, st);
    }(args...);
}

/* Enqueues `blocks` workgroups by f(first, how many), in as many launches as the runtime needs, which takes less than
 * 2^32 work-items in one; `first` is a multiple of 8. */
template <typename F> hipError_t in_turns(uint64_t blocks, uint32_t threads, F f)
{
    if (blocks >> 32) return hipErrorInvalidConfiguration;
    const uint64_t most = 0xFFFFFFFFu / threads & ~7u;
    hipError_t e = hipSuccess;
    for (uint64_t first = 0; first < blocks && e == hipSuccess; first += most)
        e = f((uint32_t)first, (uint32_t)(blocks - first < most ? blocks - first : most));
    return e;
}

[[maybe_unused]] inline int launched(hipError_t e, const char *what)
{
    if (e == hipSuccess) return MSIM_OK;
    (void)hipGetLastError();               /* it is reported here */
    msim_set_error2(what, hipGetErrorString(e));
    return MSIM_E_HIP;
}

/* an answer for a workspace that the call cannot use, or MSIM_OK */
[[maybe_unused]] inline int check_workspace(const void *ws, uint64_t have, uint64_t need, const char *what)
{
    if (!need) return MSIM_OK;
    if (!ws || have < need || (uintptr_t)ws % 256) return fail(MSIM_E_WORKSPACE, what);
    return MSIM_OK;
}

} // namespace

#endif
