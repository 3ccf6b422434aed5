// Two host threads raise one kernel's shared-memory limit at the same time,
// the smaller request in the runtime's hands when the larger one comes.  The
// runtime's two calls are fakes, so no GPU is needed.  Prints "ok" if the
// limit is the larger one in the end, which later calls rely on.
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

namespace {

std::atomic<int> limit{-1}, calls{0}, entered{0};

cudaError_t fake_device(int* dev) {
    *dev = 0;
    return cudaSuccess;
}

cudaError_t fake_attribute(const void*, cudaFuncAttribute, int bytes) {
    ++entered;
    if (bytes < 65536) std::this_thread::sleep_for(std::chrono::milliseconds(300));
    limit = bytes;
    ++calls;
    return cudaSuccess;
}

}  // namespace

#define cudaGetDevice fake_device
#define cudaFuncSetAttribute fake_attribute
#include "hisa_kernels.cuh"

int main() {
    static const int kernel = 0;
    std::thread small([] { hisa::smem_limit(&kernel, 1024); });
    while (entered.load() == 0) std::this_thread::yield();
    std::thread large([] { hisa::smem_limit(&kernel, 131072); });
    small.join();
    large.join();
    if (hisa::smem_limit(&kernel, 131072) != cudaSuccess || hisa::smem_limit(&kernel, 512) != cudaSuccess) return 1;
    if (limit.load() != 131072 || calls.load() != 2) {
        std::printf("limit %d after %d calls\n", limit.load(), calls.load());
        return 1;
    }
    std::puts("ok");
    return 0;
}
