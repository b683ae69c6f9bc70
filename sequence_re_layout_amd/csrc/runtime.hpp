// runtime.hpp -- what every HIP source of libbasp shares at a launch: the
// timing events of basp_time_next_call, the launch itself, and the frame of
// an entry point.
#pragma once

#include <hip/hip_runtime.h>

#include <hip/hip_ext.h>

#include "plan_internal.hpp"

namespace basp {

// Events set by basp_time_next_call for the next call of this thread.
struct Timing {
    hipEvent_t start = nullptr, stop = nullptr;
};
inline thread_local Timing t_timing;

// The launch's own status (not the thread's sticky last error, which other
// code in the process may have left set).  first/last: this launch opens or
// closes the current entry-point call, for the timing events.  lds: bytes of
// dynamic shared memory.
template <typename Desc>
inline basp_status launch_kernel(const void *fn, dim3 grid, int block, const Desc &D, void *stream,
                                 bool first, bool last, size_t lds = 0)
{
    void *args[] = {const_cast<Desc *>(&D)};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (t_timing.start || t_timing.stop)
        e = hipExtLaunchKernel(fn, grid, dim3(block), args, lds, st,
                               first ? t_timing.start : nullptr, last ? t_timing.stop : nullptr, 0);
    else
        e = hipLaunchKernel(fn, grid, dim3(block), args, lds, st);
    return e == hipSuccess ? BASP_OK : BASP_ERR_HIP;
}

// Runs f, the body of an entry point, and clears the timing request after it.
template <typename F>
inline basp_status timed_call(F f)
{
    const basp_status s = f();
    t_timing = Timing();
    return record(s);
}

}  // namespace basp
