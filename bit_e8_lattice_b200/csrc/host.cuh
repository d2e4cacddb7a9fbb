// Host-side helpers of the entry points: alignment, status codes, launches.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/e8q.h"

namespace e8q {

inline e8q_status cuda_ok(cudaError_t e) { return e == cudaSuccess ? E8Q_OK : E8Q_ERR_CUDA; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

// Launch with programmatic stream serialisation: the kernel may start while
// the previous kernel on the stream is finishing; it waits for that
// kernel's results with griddepcontrol.wait.
// The first kernel of a call is launched without it (`overlaps` false).
template <typename P>
e8q_status launch_pdl(void (*kernel)(P), dim3 grid, int threads, size_t smem, cudaStream_t s, const P& params,
                      bool overlaps = true) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = overlaps ? 1 : 0;
    return cuda_ok(cudaLaunchKernelEx(&cfg, kernel, params));
}
template <typename P>
e8q_status launch_pdl(void (*kernel)(P), int grid, int threads, size_t smem, cudaStream_t s, const P& params) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), threads, smem, s, params);
}

}  // namespace e8q
