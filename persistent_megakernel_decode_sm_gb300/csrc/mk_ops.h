// Shared by the prompt operators' translation units: host-side helpers of their C entry points.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "mk_internal.h"

namespace mk {

inline mk_status op_cuda_fail(cudaError_t e, const char* what) {
    return fail(MK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}
#define MK_CK(call)                                               \
    do {                                                          \
        cudaError_t e_ = (call);                                  \
        if (e_ != cudaSuccess) return op_cuda_fail(e_, #call);    \
    } while (0)

inline bool op_aligned(const void* p, unsigned a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Whether two sets of rows share a byte: `rows` rows of `width` bytes, `stride` bytes apart.  Rows
// of the same stride may lie beside one another (column slices of one buffer); of two different
// strides the whole ranges are compared.
struct RowSpan {
    const void* p;
    int64_t rows, width, stride;
};
inline bool spans_overlap(const RowSpan& a, const RowSpan& b) {
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
    const auto lo = [](const RowSpan& s) { return int64_t(reinterpret_cast<uintptr_t>(s.p)); };
    const auto hi = [&](const RowSpan& s) { return lo(s) + (s.rows - 1) * s.stride + s.width; };
    if (hi(a) <= lo(b) || hi(b) <= lo(a)) return false;
    if (a.stride != b.stride || a.stride < a.width || b.stride < b.width) return true;
    const int64_t s = a.stride, off = ((lo(b) - lo(a)) % s + s) % s;   // b's columns within a's rows
    return off < a.width || off + b.width > s;
}

}  // namespace mk
