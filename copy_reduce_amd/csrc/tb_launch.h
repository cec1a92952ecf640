// tb_launch.h -- how libtb launches a kernel, with the events that the timing
// hook (tb_time_next_launch) hands to it.  Included by the kernel sources.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

namespace tbk {

// Events the next launch made by this host thread records as part of the
// launch itself (set by tb_time_next_launch; consumed by that launch).
inline thread_local hipEvent_t t_next_start = nullptr;
inline thread_local hipEvent_t t_next_stop = nullptr;

// Every kernel of the library is launched here.  With events (the timing hook,
// or `done` from the caller), the launch carries them as its own start / stop
// events, so no separate event command sits between kernels.  A launch has
// one stop event: when `done` takes it (a ring slot's completion event) and
// the timing hook also set one, the hook's is recorded right after the launch
// as a command of its own, so it too fires when the kernel has completed.
template <typename... KArgs, typename... Args>
static hipError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, hipStream_t s, hipEvent_t done,
                         Args... args) {
    const hipEvent_t start = t_next_start;
    const hipEvent_t hook_stop = t_next_stop;
    const hipEvent_t stop = done != nullptr ? done : hook_stop;
    t_next_start = t_next_stop = nullptr;
    if (start != nullptr || stop != nullptr)
        hipExtLaunchKernelGGL(kernel, grid, block, 0, s, start, stop, 0u, args...);
    else
        hipLaunchKernelGGL(kernel, grid, block, 0, s, args...);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && done != nullptr && hook_stop != nullptr)
        e = hipEventRecord(hook_stop, s);
    return e;
}

// A call of several kernels: between them the hook's stop event is held back,
// so that the start event rides on the first launch and the stop event on the
// last.  Usage: LaunchSeq seq; launch(...); ...; seq.last(); launch(...).
class LaunchSeq {
public:
    LaunchSeq() : stop_(t_next_stop) { t_next_stop = nullptr; }
    void last() { t_next_stop = stop_; }

private:
    hipEvent_t stop_;
};

}  // namespace tbk
