// Host-side helpers shared by the operators beside the WTConv layer (gated scan, AdamW, norm).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include <map>
#include <mutex>
#include <utility>

#include "wtconv.h"

namespace wtconv {

inline int elem_bytes_of(int dtype) { return dtype == WTCONV_F32 ? 4 : 2; }
// (n > 0, up to the largest int)
inline int ceil_div(int n, int d) { return (n - 1) / d + 1; }
inline bool dtype_ok(int dtype) { return dtype == WTCONV_F32 || dtype == WTCONV_BF16 || dtype == WTCONV_F16; }
inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool fault_injected() {
    const char *e = getenv("WTCONV_INJECT_FAULT");
    return e != nullptr && e[0] == '1';
}
inline int status_of(cudaError_t e) { return e == cudaSuccess ? WTCONV_OK : WTCONV_ERR_CUDA; }

// Strides of an activation [B][rows][inner] whose innermost axis is contiguous: >= 0, offsets far from
// 2^63, and for an output no two elements at one place (the axis of smaller stride must end before the
// other's next step).
inline bool activation_ok(const void *p, long long batch, long long row, long long B, long long rows, long long inner, int dtype,
                          bool output) {
    const long long limit = 1ll << 59;
    if (p == nullptr || !aligned_to(p, elem_bytes_of(dtype)) || batch < 0 || row < 0) return false;
    if ((B > 1 && batch > limit / B) || (rows > 1 && row > limit / rows)) return false;
    if (!output) return true;
    const bool by_row = rows > 1, by_batch = B > 1;
    if (by_row && by_batch) {
        const bool row_first = row <= batch;
        const long long small = row_first ? row : batch, large = row_first ? batch : row;
        const long long count = row_first ? rows : B;
        return small >= inner && large >= small * (count - 1) + inner;
    }
    return (!by_row || row >= inner) && (!by_batch || batch >= inner);
}
inline bool f32_ok(const void *p, bool optional) { return (p != nullptr || optional) && aligned_to(p, 4); }

// SMs of the current device (148 if it cannot be asked: a plan is then only less balanced)
inline int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
        cudaGetLastError();
        return 148;
    }
    return sms;
}

// Lets a kernel have `shared` bytes of dynamic shared memory on the current device.  Asked of the
// runtime once per kernel and device: it takes a microsecond.
template <typename... P> cudaError_t allow_shared(void (*kernel)(P...), size_t shared) noexcept {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    try {
        static std::mutex lock;
        static std::map<std::pair<void (*)(P...), int>, size_t> allowed;
        std::lock_guard<std::mutex> guard(lock);
        size_t &have = allowed[{kernel, dev}];
        if (have >= shared) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
        if (e == cudaSuccess) have = shared;
        return e;
    } catch (...) {  // no memory for the entry: nothing leaves through the C entry point
        return cudaErrorMemoryAllocation;
    }
}

// CTAs of a kernel that an SM of the current device holds at once (1 if it cannot be asked).  Asked of the runtime
// once per kernel and device.
template <typename... P> int resident_ctas(void (*kernel)(P...), int threads) noexcept {
    int dev = 0, ctas = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    try {
        static std::mutex lock;
        static std::map<std::pair<void (*)(P...), int>, int> known;
        std::lock_guard<std::mutex> guard(lock);
        int &have = known[{kernel, dev}];
        if (have == 0 && cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, kernel, threads, 0) == cudaSuccess) have = ctas;
        if (have > 0) return have;
    } catch (...) {  // no memory for the entry
    }
    cudaGetLastError();
    return 1;
}

// Launches a kernel that may be set up while the one before it on the stream still runs: every kernel
// of these operators waits for that one's end by itself (begin_kernel in train_device.cuh).  Between
// the two kernels of a short call that is most of the gap.  cluster: CTAs that share a cluster.
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), unsigned grid, unsigned threads, size_t shared, cudaStream_t st, unsigned cluster,
                          const A &...args) {
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(grid);
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = shared;
    config.stream = st;
    cudaLaunchAttribute attrs[2] = {};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster, attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    config.attrs = attrs;
    config.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&config, kernel, args...);
}

}  // namespace wtconv
