// Shared by the prompt operators' translation units: host-side helpers of their C entry points.
#pragma once

#include <cuda.h>   // tensor-map types (the encoder itself is fetched through the runtime)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
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

// bf16 tensor map: `rank` extents, the byte strides of all but the innermost, the box; 128-byte
// swizzle (64 bytes for boxes of 64-byte rows); what lies outside the extents reads as zeros
inline mk_status op_tensor_map(CUtensorMap* out, const void* base, int rank, const cuuint64_t* dim, const cuuint64_t* stride,
                               const cuuint32_t* box) {
    typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                               const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<Encode> cached{nullptr};
    Encode enc = cached.load();
    if (!enc) {
        cudaDriverEntryPointQueryResult q{};
        void* fn = nullptr;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn)
            return fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
        enc = reinterpret_cast<Encode>(fn);
        cached.store(enc);
    }
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    const CUresult r = enc(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank), const_cast<void*>(base), dim, stride, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, box[0] == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MK_OK : fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", int(r));
}

// SMs of the current device, and its ordinal (both looked up once per device)
inline mk_status op_device(int* device, int* sms) {
    static std::atomic<int> count[64];
    MK_CK(cudaGetDevice(device));
    if (*device >= 64) return fail(MK_ERR_ARG, "device ordinal %d out of range", *device);
    int n = count[*device].load();
    if (!n) {
        MK_CK(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *device));
        count[*device].store(n);
    }
    *sms = n;
    return MK_OK;
}

// Lets a kernel use `bytes` of dynamic shared memory on this device; `done` is the kernel's own
// mask of the devices it is set on already.
inline mk_status op_smem(const void* fn, int bytes, int device, std::atomic<uint64_t>* done) {
    if (done->load() >> device & 1) return MK_OK;
    MK_CK(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    done->fetch_or(uint64_t(1) << device);
    return MK_OK;
}

// The checks of mk_attend that need no pointers, and its workspace bytes
mk_status mk_attend_plan(const mk_attend_args* a, size_t* workspace_bytes);

// ---- the prompt path's small kernels (mk_prefill.cu) ----------------------------------------------
struct PrefillRows {
    int32_t batch, nq, nkv, d;
    int32_t first[kMaxBatch], pos[kMaxBatch];   // per sequence: its first token of the call, that token's position
    const float2* rope;                         // [max_seq][d / 2] (cos, sin)
    __nv_bfloat16* k;                           // the layer's cache
    __nv_bfloat16* v;
    int64_t batch_stride, head_stride;
    const int32_t* table;                       // paged: [batch][max_blocks]
    int32_t block, max_blocks, n_blocks;
    int32_t* status;
};
mk_status prefill_tokens(const int32_t* tokens, int64_t n, int32_t* out, cudaStream_t stream);   // (HOST tokens, read before it returns)
mk_status prefill_norm(float* x, const int32_t* tokens, const void* embed, const void* gain, void* y, int64_t rows, int H,
                       float eps, cudaStream_t stream);
mk_status prefill_rope_append(const float* qkv, void* q, const PrefillRows& rows, int64_t tokens, cudaStream_t stream);

}  // namespace mk
