// Set-up that a kernel needs once on each device: function attributes belong to the device
// that was current when they were set, and contexts of one process may be on several, used
// by several threads.
#pragma once
#include <atomic>
#include <cstdint>
#include <driver_types.h>

namespace lora {

// The device that the calling thread's present call has made current (api.cpp, use_device):
// asking the runtime again would cost a decode call 2 % of its time.
int launch_device();

class OncePerDevice {
public:
    // Runs `work` unless it has succeeded on the launch's device before.  Threads that come
    // first together may all run it; it has to bear that.
    template <typename F>
    cudaError_t operator()(F &&work)
    {
        const unsigned device = unsigned(launch_device());
        const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;   // another: every time
        if (done_.load(std::memory_order_acquire) & bit)
            return cudaSuccess;
        const cudaError_t e = work();
        if (e == cudaSuccess)
            done_.fetch_or(bit, std::memory_order_release);
        return e;
    }

private:
    std::atomic<uint64_t> done_{0};
};

}  // namespace lora
