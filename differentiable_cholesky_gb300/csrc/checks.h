// Host-side argument checks shared by the C entry points.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "chol.h"

namespace chol {

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

inline Range range_of(const void* p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + bytes};
}

// Device (or managed) memory only: a host pointer handed to a kernel would
// fault or, where the GPU can reach host memory, silently run over the link.
inline bool is_device_pointer(const void* p) {
    cudaPointerAttributes attr;
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();  // clear the non-sticky error
        return false;
    }
    return attr.type == cudaMemoryTypeDevice || attr.type == cudaMemoryTypeManaged;
}

inline bool aligned(const void* p, size_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline int to_code(cudaError_t e) { return e == cudaSuccess ? CHOL_OK : CHOL_ECUDA; }

}  // namespace chol
