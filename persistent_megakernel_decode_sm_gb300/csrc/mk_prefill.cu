// The small kernels of the prompt path (mk_prefill): host tokens to the device, token embedding, RMSNorm, and
// the rotation of q and k with the append of k and v to the cache.  Each reads and writes its rows once: bytes bound them.
#include <algorithm>
#include <cstring>

#include "mk_ops.h"
#include "mk_sm103.cuh"

namespace mk {

// A piece of the call's host tokens, read by the launch itself, whatever memory the caller keeps them in (a copy
// from page-locked memory would read them after the call has returned).  4 KB a launch: the size that every launch
// may have; 5 of them for 4096 tokens.
struct TokenPiece {
    int32_t n;
    int32_t token[1000];
};
constexpr int kTokenPiece = int(sizeof(TokenPiece::token) / sizeof(int32_t));
__global__ void __launch_bounds__(256) tokens_kernel(int32_t* out, const __grid_constant__ TokenPiece p) {
    sm::pdl_trigger();
    sm::pdl_wait();
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < p.n) out[i] = p.token[i];
}

constexpr int kNormThreads = 256;

__device__ __forceinline__ float block_sum(float v) {   // the same in every thread
    __shared__ float part[kNormThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kNormThreads / 32; ++w) s += part[w];
    return s;
}

// y = x / sqrt(mean(x^2) + eps) * gain, in fp32, rounded once to bf16; a block per token.  With tokens given
// x is first taken from the embedding rows.  (H is a multiple of 8 and at most kMaxK: 8 vectors a thread.)
__global__ void __launch_bounds__(kNormThreads) norm_kernel(float* x, const int32_t* tokens, const __nv_bfloat16* embed,
                                                            const __nv_bfloat16* gain, __nv_bfloat16* y, int H, float eps) {
    sm::pdl_trigger();
    sm::pdl_wait();
    const int64_t row = blockIdx.x;
    float* xr = x + row * H;
    constexpr int kVec = kMaxK / 8 / kNormThreads;
    float v[kVec][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int c = (threadIdx.x + i * kNormThreads) * 8;
        if (c >= H) break;
        if (tokens) {
            const uint4 u = *reinterpret_cast<const uint4*>(embed + int64_t(tokens[row]) * H + c);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[i][2 * k] = __uint_as_float(w[k] << 16);
                v[i][2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
            *reinterpret_cast<float4*>(xr + c) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
            *reinterpret_cast<float4*>(xr + c + 4) = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
        } else {
            const float4 a = *reinterpret_cast<const float4*>(xr + c), b = *reinterpret_cast<const float4*>(xr + c + 4);
            v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
            v[i][4] = b.x; v[i][5] = b.y; v[i][6] = b.z; v[i][7] = b.w;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(v[i][k], v[i][k], ss);
    }
    const float r = 1.f / sqrtf(block_sum(ss) / float(H) + eps);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int c = (threadIdx.x + i * kNormThreads) * 8;
        if (c >= H) break;
        const uint4 u = *reinterpret_cast<const uint4*>(gain + c);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t out[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float a = v[i][2 * k] * r * __uint_as_float(w[k] << 16);
            const float b = v[i][2 * k + 1] * r * __uint_as_float(w[k] & 0xFFFF0000u);
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[k]) : "f"(b), "f"(a));
        }
        *reinterpret_cast<uint4*>(y + row * H + c) = make_uint4(out[0], out[1], out[2], out[3]);
    }
}

// Pairs (i, i + d/2) of q and k rotated by their position's angles (the bind's table), rounded once; q to its
// own buffer, k and v to the cache row of their position.  A block per token, four pairs or four values of v a thread
// (d is 32, 64 or 128: shifts; rows and cache are 16-byte aligned).
__global__ void __launch_bounds__(256) rope_append_kernel(const float* qkv, __nv_bfloat16* q, const __grid_constant__ PrefillRows p) {
    sm::pdl_trigger();
    sm::pdl_wait();
    const int tok = blockIdx.x;
    int b = 0;
    while (b + 1 < p.batch && tok >= p.first[b + 1]) ++b;
    const int pos = p.pos[b] + (tok - p.first[b]), half = p.d / 2;
    const float2* cs = p.rope + int64_t(pos) * half;
    const float* src = qkv + int64_t(tok) * (p.nq + 2 * p.nkv) * p.d;
    int64_t base = int64_t(b) * p.batch_stride, slot = pos;
    bool good = true;
    if (p.table) {
        const int blk = __ldg(p.table + int64_t(b) * p.max_blocks + pos / p.block);
        good = unsigned(blk) < unsigned(p.n_blocks);
        if (!good && threadIdx.x == 0) *p.status = MK_ERR_BOUNDS;   // (nothing is written there)
        base = 0;
        slot = int64_t(blk) * p.block + pos % p.block;
    }
    const int heads = p.nq + p.nkv, quads = half / 4, log2_quads = __ffs(quads) - 1;
    auto pack4 = [](const float (&x)[4]) {
        uint2 r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.x) : "f"(x[1]), "f"(x[0]));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.y) : "f"(x[3]), "f"(x[2]));
        return r;
    };
    for (int i = threadIdx.x; i < heads << log2_quads; i += blockDim.x) {
        const int h = i >> log2_quads, e = (i & (quads - 1)) * 4;
        const float4 a4 = *reinterpret_cast<const float4*>(src + h * p.d + e), c4 = *reinterpret_cast<const float4*>(src + h * p.d + e + half);
        const float4 t01 = *reinterpret_cast<const float4*>(cs + e), t23 = *reinterpret_cast<const float4*>(cs + e + 2);
        const float a[4] = {a4.x, a4.y, a4.z, a4.w}, c[4] = {c4.x, c4.y, c4.z, c4.w};
        const float co[4] = {t01.x, t01.z, t23.x, t23.z}, si[4] = {t01.y, t01.w, t23.y, t23.w};
        float r0[4], r1[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            r0[k] = a[k] * co[k] - c[k] * si[k];
            r1[k] = a[k] * si[k] + c[k] * co[k];
        }
        __nv_bfloat16* dst = h < p.nq ? q + (int64_t(tok) * p.nq + h) * p.d
                                      : p.k + base + (h - p.nq) * p.head_stride + slot * p.d;
        if (h < p.nq || good) {
            *reinterpret_cast<uint2*>(dst + e) = pack4(r0);
            *reinterpret_cast<uint2*>(dst + e + half) = pack4(r1);
        }
    }
    if (good)
        for (int i = threadIdx.x; i < p.nkv << (log2_quads + 1); i += blockDim.x) {
            const int h = i >> (log2_quads + 1), e = (i & (2 * quads - 1)) * 4;
            const float4 v = *reinterpret_cast<const float4*>(src + (heads + h) * p.d + e);
            const float x[4] = {v.x, v.y, v.z, v.w};
            *reinterpret_cast<uint2*>(p.v + base + h * p.head_stride + slot * p.d + e) = pack4(x);
        }
}

template <typename... Args, typename... Given>
static mk_status prefill_launch(void (*fn)(Args...), int64_t blocks, cudaStream_t stream, Given... given) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    MK_CK(cudaLaunchKernelEx(&cfg, fn, given...));
    return MK_OK;
}

mk_status prefill_tokens(const int32_t* tokens, int64_t n, int32_t* out, cudaStream_t stream) {
    for (int64_t at = 0; at < n; at += kTokenPiece) {
        TokenPiece p{};
        p.n = int32_t(std::min<int64_t>(kTokenPiece, n - at));
        std::memcpy(p.token, tokens + at, size_t(p.n) * sizeof(int32_t));
        const mk_status st = prefill_launch(&tokens_kernel, (p.n + 255) / 256, stream, out + at, p);
        if (st != MK_OK) return st;
    }
    return MK_OK;
}
mk_status prefill_norm(float* x, const int32_t* tokens, const void* embed, const void* gain, void* y, int64_t rows, int H,
                       float eps, cudaStream_t stream) {
    return prefill_launch(&norm_kernel, rows, stream, x, tokens, static_cast<const __nv_bfloat16*>(embed),
                          static_cast<const __nv_bfloat16*>(gain), static_cast<__nv_bfloat16*>(y), H, eps);
}
mk_status prefill_rope_append(const float* qkv, void* q, const PrefillRows& rows, int64_t tokens, cudaStream_t stream) {
    return prefill_launch(&rope_append_kernel, tokens, stream, qkv, static_cast<__nv_bfloat16*>(q), rows);
}

}  // namespace mk
