// The linear map of the prompt path: out = act(x w^T + bias) + residual (mk_linear).
#include "mk_ops.h"

#include <cuda_bf16.h>

namespace mk {

struct LinearParams {
    int rows, n, k, act;
    const __nv_bfloat16* x;
    int64_t x_stride;
    const __nv_bfloat16* w;
    const __nv_bfloat16* bias;
    const void* residual;
    int64_t residual_stride;
    int residual_f32, out_f32;
    void* out;
    int64_t out_stride;
};

// bias, activation and residual of one output, in fp32; rounded once by the store
__device__ __forceinline__ float linear_act(int act, float y, float up) {
    switch (act) {
        case MK_ACT_SILU: return y / (1.f + expf(-y));
        case MK_ACT_GELU: return 0.5f * y * (1.f + erff(y * 0.70710678118654752f));
        case MK_ACT_SWIGLU: return y / (1.f + expf(-y)) * up;
        default: return y;
    }
}

// One thread per output; 16 x 16 outputs a block, their rows staged 16 inputs at a time.
__global__ void __launch_bounds__(256) linear_simple_kernel(const LinearParams p) {
    __shared__ float sx[16][17], sw[16][17], su[16][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int j = blockIdx.x * 16 + tx, r = blockIdx.y * 16 + ty;
    const bool gated = p.act == MK_ACT_SWIGLU;
    float y = 0.f, u = 0.f;
    for (int k0 = 0; k0 < p.k; k0 += 16) {
        const int jl = blockIdx.x * 16 + ty, kk = k0 + tx;
        sx[ty][tx] = r < p.rows && kk < p.k ? __bfloat162float(p.x[r * p.x_stride + kk]) : 0.f;
        sw[ty][tx] = jl < p.n && kk < p.k ? __bfloat162float(p.w[int64_t(jl) * p.k + kk]) : 0.f;
        su[ty][tx] = gated && jl < p.n && kk < p.k ? __bfloat162float(p.w[(int64_t(p.n) + jl) * p.k + kk]) : 0.f;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            y = fmaf(sx[ty][i], sw[tx][i], y);
            if (gated) u = fmaf(sx[ty][i], su[tx][i], u);
        }
        __syncthreads();
    }
    if (r >= p.rows || j >= p.n) return;
    if (p.bias) {
        y += __bfloat162float(p.bias[j]);
        if (gated) u += __bfloat162float(p.bias[p.n + j]);
    }
    y = linear_act(p.act, y, u);
    if (p.residual) {
        const int64_t at = r * p.residual_stride + j;
        y += p.residual_f32 ? static_cast<const float*>(p.residual)[at]
                            : __bfloat162float(static_cast<const __nv_bfloat16*>(p.residual)[at]);
    }
    const int64_t at = r * p.out_stride + j;
    if (p.out_f32) static_cast<float*>(p.out)[at] = y;
    else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
}

static mk_status linear_check(const mk_linear_args* a) {
    if (!a) return fail(MK_ERR_ARG, "null argument");
    if (a->rows < 0 || a->n < 1 || a->k < 8 || a->k % 8)
        return fail(MK_ERR_ARG, "linear: rows %d, n %d, k %d (rows >= 0, n >= 1, k a multiple of 8)", a->rows, a->n, a->k);
    if (a->activation < MK_ACT_NONE || a->activation > MK_ACT_SWIGLU)
        return fail(MK_ERR_ARG, "linear: unknown activation %d", a->activation);
    if ((a->out_dtype != MK_BF16 && a->out_dtype != MK_F32) ||
        (a->residual && a->residual_dtype != MK_BF16 && a->residual_dtype != MK_F32))
        return fail(MK_ERR_ARG, "linear: unknown data type");
    const bool gated = a->activation == MK_ACT_SWIGLU;
    if (gated && a->n > (1 << 30)) return fail(MK_ERR_ARG, "linear: n %d too large", a->n);
    if (a->rows == 0) return MK_OK;
    const int64_t os = a->out_dtype == MK_F32 ? 4 : 2, rs = a->residual_dtype == MK_F32 ? 4 : 2;
    if (!a->x || !a->w || !a->out) return fail(MK_ERR_ARG, "linear: null pointer");
    if (!op_aligned(a->x, 16) || !op_aligned(a->w, 16)) return fail(MK_ERR_ARG, "linear: x and w must be 16-byte aligned");
    if (!op_aligned(a->out, unsigned(os)) || !op_aligned(a->bias, 2) || (a->residual && !op_aligned(a->residual, unsigned(rs))) ||
        !op_aligned(a->status, 4))
        return fail(MK_ERR_ARG, "linear: bias, residual, out or status not aligned to its element");
    if (a->rows > 1 && (a->x_stride < a->k || a->x_stride % 8 || a->out_stride < a->n ||
                        (a->residual && a->residual_stride != 0 && a->residual_stride < a->n)))
        return fail(MK_ERR_ARG, "linear: strides must cover their rows, x_stride be a multiple of 8");
    const RowSpan out{a->out, a->rows, a->n * os, a->out_stride * os};
    const int64_t f = gated ? 2 : 1;
    const bool same = a->residual == a->out && a->residual_dtype == a->out_dtype &&
                      (a->rows == 1 || a->residual_stride == a->out_stride);
    if (spans_overlap(out, {a->x, a->rows, int64_t(a->k) * 2, a->x_stride * 2}) ||
        spans_overlap(out, {a->w, 1, f * a->n * a->k * 2, 0}) || spans_overlap(out, {a->bias, 1, f * a->n * 2, 0}) ||
        (!same && spans_overlap(out, {a->residual, a->rows, a->n * rs, a->residual_stride * rs})))
        return fail(MK_ERR_ARG, "linear: out overlaps an input");
    return MK_OK;
}

}  // namespace mk

using namespace mk;

extern "C" mk_status mk_linear(const mk_linear_args* a, void* stream) {
    const mk_status st = linear_check(a);
    if (st != MK_OK || a->rows == 0) return st;
    LinearParams p{};
    p.rows = a->rows; p.n = a->n; p.k = a->k; p.act = a->activation;
    p.x = static_cast<const __nv_bfloat16*>(a->x);
    p.x_stride = a->rows == 1 ? a->k : a->x_stride;
    p.w = static_cast<const __nv_bfloat16*>(a->w);
    p.bias = static_cast<const __nv_bfloat16*>(a->bias);
    p.residual = a->residual;
    p.residual_stride = a->residual_stride;
    p.residual_f32 = a->residual_dtype == MK_F32;
    p.out_f32 = a->out_dtype == MK_F32;
    p.out = a->out;
    p.out_stride = a->out_stride;
    linear_simple_kernel<<<dim3((a->n + 15) / 16, (a->rows + 15) / 16), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    MK_CK(cudaGetLastError());
    return MK_OK;
}
