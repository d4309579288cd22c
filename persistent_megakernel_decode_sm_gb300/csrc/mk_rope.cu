// Norms of q and k, rotation by the tokens' positions, q to its buffer, k and v to the cache (mk_rope_append).
#include <algorithm>
#include <climits>
#include <cmath>

#include "mk_ops.h"
#include "mk_sm103.cuh"

namespace mk {

constexpr int kRopePairs = 128;     // of the widest head
constexpr int kRopeThreads = 128;

struct RopeParams {
    int tokens, nq, nkv, heads;     // heads: nq + 2 nkv
    int units, turned;              // 16 elements each: of a head, of its rotated part
    int rounds, per;                // of a token: rounds of the heads that a warp takes at a time; rounds of one warp
    int parts;                      // warps of a token
    const void* qkv;
    int64_t qkv_stride;
    const __nv_bfloat16* q_gain;
    const __nv_bfloat16* k_gain;
    float eps, inv_d;
    const int32_t* positions;
    int64_t position_stride;
    const int32_t* slots;
    __nv_bfloat16* k;
    __nv_bfloat16* v;
    int64_t batch_stride, head_stride;
    int max_seq, limit;             // slots of a sequence, of the cache
    __nv_bfloat16* q;
    int64_t q_stride;
    int32_t* status;
    uint8_t axis[kRopePairs];
    uint64_t turn[kRopePairs];      // turns per position, 64 bits behind the point (whole turns left out)
};

// cos and sin of position * rate: the product wraps at whole turns, so the angle is reduced exactly for every 32-bit
// position (an angle in fp32 radians would be off by 2^-24 of itself); 31 bits of it become an fp32 in [-1, 1) half turns.
__device__ __forceinline__ float2 rope_angle(int position, uint64_t rate) {
    const uint64_t turns = uint64_t(int64_t(position)) * rate;
    float2 cs;
    sincospif(float(int32_t(turns >> 32)) * 0x1p-31f, &cs.y, &cs.x);
    return cs;
}

// 8 elements at `at` in fp32
template <bool F32>
__device__ __forceinline__ void rope_load(const void* row, int at, uint4 (&raw)[F32 ? 2 : 1]) {
    if constexpr (F32) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(row) + at);
        raw[0] = __ldcs(p);
        raw[1] = __ldcs(p + 1);
    } else {
        raw[0] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(row) + at));
    }
}
__device__ __forceinline__ void rope_widen(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
}
template <bool F32>
__device__ __forceinline__ void rope_values(const uint4 (&raw)[F32 ? 2 : 1], float* x) {
    if constexpr (F32) {
        *reinterpret_cast<uint4*>(x) = raw[0];
        *reinterpret_cast<uint4*>(x + 4) = raw[1];
    } else {
        rope_widen(raw[0], x);
    }
}
__device__ __forceinline__ uint4 rope_pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(x[2 * k + 1]), "f"(x[2 * k]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp takes `per` rounds of a token's heads; a round is 32 / GROUP heads of GROUP lanes, a lane holds 16 elements (two
// 16-byte pieces of bf16): the pairs 8 u .. 8 u + 7, whose elements lie rotary / 2 apart or side by side, or 16 elements that
// only pass.  A head's sum of squares is a shuffle over its lanes; a token's cosines and sines are worked out once by the warp.
template <int GROUP, bool F32, bool NEIGHBOURS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float4 angles[kRopeThreads / 32][kRopePairs / 2];
    sm::pdl_trigger();
    sm::pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t job = int64_t(blockIdx.x) * (kRopeThreads / 32) + warp;
    const int t = int(job / p.parts), r0 = int(job % p.parts) * p.per, r1 = min(r0 + p.per, p.rounds);
    if (t >= p.tokens) return;
    float2* mine = reinterpret_cast<float2*>(angles[warp]);
    for (int i = lane; i < 8 * p.turned; i += 32) mine[i] = rope_angle(p.positions[p.axis[i] * p.position_stride + t], p.turn[i]);
    const int slot = p.slots[t];
    const bool stored = slot >= 0 && slot < p.limit;
    if (slot >= p.limit && p.status) *p.status = MK_ERR_BOUNDS;
    const int sequence = stored ? slot / p.max_seq : 0;
    const int d = 16 * p.units;
    const int64_t cache = int64_t(sequence) * p.batch_stride + (int64_t(slot) - int64_t(sequence) * p.max_seq) * d;
    __syncwarp();

    const int u = lane % GROUP, sub = lane / GROUP;
    const bool live = u < p.units, turns = u < p.turned;
    const int lo = turns && !NEIGHBOURS ? 8 * u : 16 * u, hi = turns && !NEIGHBOURS ? 8 * (p.turned + u) : 16 * u + 8;
    float cs[16];   // the lane's 8 pairs: cosine, sine
    if (turns)
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(cs + 4 * i) = angles[warp][4 * u + i];
    const int64_t row = int64_t(t) * p.qkv_stride;
    const void* src = F32 ? static_cast<const void*>(static_cast<const float*>(p.qkv) + row)
                          : static_cast<const void*>(static_cast<const __nv_bfloat16*>(p.qkv) + row);
    constexpr int kAhead = F32 ? 2 : 4;   // rounds whose loads are in flight together
    for (int r = r0; r < r1; r += kAhead) {
        uint4 raw[kAhead][2][F32 ? 2 : 1];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int h = (r + i) * (32 / GROUP) + sub;
            if (r + i < r1 && h < p.heads && live) {
                rope_load<F32>(src, h * d + lo, raw[i][0]);
                rope_load<F32>(src, h * d + hi, raw[i][1]);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (r + i >= r1) break;
            const int h = (r + i) * (32 / GROUP) + sub;
            const bool here = h < p.heads && live;
            float x[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = 0.f;
            if (here) {
                rope_values<F32>(raw[i][0], x);
                rope_values<F32>(raw[i][1], x + 8);
            }
            const __nv_bfloat16* gain = h < p.nq ? p.q_gain : h < p.nq + p.nkv ? p.k_gain : nullptr;
            if (p.q_gain || p.k_gain) {   // (uniform: every lane of the warp takes part in the sums)
                float ss = 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
                for (int o = GROUP / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                if (gain && here) {
                    const float scale = 1.f / sqrtf(fmaf(ss, p.inv_d, p.eps));
                    float g[16];
                    rope_widen(__ldg(reinterpret_cast<const uint4*>(gain + lo)), g);
                    rope_widen(__ldg(reinterpret_cast<const uint4*>(gain + hi)), g + 8);
#pragma unroll
                    for (int k = 0; k < 16; ++k) x[k] *= scale * g[k];
                }
            }
            if (!here) continue;
            if (turns && h < p.nq + p.nkv) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float &a = NEIGHBOURS ? x[2 * k] : x[k], &b = NEIGHBOURS ? x[2 * k + 1] : x[k + 8];
                    const float c = cs[2 * k], s = cs[2 * k + 1], a0 = a;
                    a = a0 * c - b * s;
                    b = a0 * s + b * c;
                }
            }
            __nv_bfloat16* dst;
            if (h < p.nq) dst = p.q + int64_t(t) * p.q_stride + h * d;
            else {
                if (!stored) continue;
                const bool is_k = h < p.nq + p.nkv;
                dst = (is_k ? p.k : p.v) + cache + int64_t(h - p.nq - (is_k ? 0 : p.nkv)) * p.head_stride;
            }
            *reinterpret_cast<uint4*>(dst + lo) = rope_pack(x);
            *reinterpret_cast<uint4*>(dst + hi) = rope_pack(x + 8);
        }
    }
}

template <int GROUP, bool F32>
static mk_status rope_launch(const RopeParams& p, bool neighbours, int64_t blocks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kRopeThreads);
    MK_CK(neighbours ? cudaLaunchKernelEx(&cfg, &rope_kernel<GROUP, F32, true>, p) : cudaLaunchKernelEx(&cfg, &rope_kernel<GROUP, F32, false>, p));
    return MK_OK;
}
template <int GROUP>
static mk_status rope_launch(RopeParams& p, bool f32, bool neighbours, int sms, cudaStream_t stream) {
    p.rounds = (p.heads + 32 / GROUP - 1) / (32 / GROUP);
    // few tokens: a warp for every round; many: a warp takes a token
    p.per = int64_t(p.tokens) * p.rounds <= 16 * int64_t(sms) ? 1 : p.rounds;
    p.parts = (p.rounds + p.per - 1) / p.per;
    const int64_t warps = int64_t(p.tokens) * p.parts, blocks = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    return f32 ? rope_launch<GROUP, true>(p, neighbours, blocks, stream) : rope_launch<GROUP, false>(p, neighbours, blocks, stream);
}

static mk_status rope_check(const mk_rope_args* a) {
    if (!a) return fail(MK_ERR_ARG, "null argument");
    if (a->tokens < 0 || a->tokens > (1 << 30)) return fail(MK_ERR_ARG, "rope_append: %d tokens", a->tokens);
    const int d = a->head_dim;
    if (d < 16 || d > 256 || d % 16) return fail(MK_ERR_ARG, "rope_append: head_dim %d (a multiple of 16, at most 256)", d);
    if (a->n_q_heads < 1 || a->n_kv_heads < 1 || a->n_q_heads > 4096 || a->n_kv_heads > 4096 || a->n_q_heads + 2 * a->n_kv_heads > 4096)
        return fail(MK_ERR_ARG, "rope_append: %d q heads, %d kv heads", a->n_q_heads, a->n_kv_heads);
    if (a->rotary < 0 || a->rotary > d || a->rotary % 16)
        return fail(MK_ERR_ARG, "rope_append: %d rotated elements (a multiple of 16, at most head_dim)", a->rotary);
    if (a->neighbours != 0 && a->neighbours != 1) return fail(MK_ERR_ARG, "rope_append: neighbours %d", a->neighbours);
    if (a->qkv_dtype != MK_BF16 && a->qkv_dtype != MK_F32) return fail(MK_ERR_ARG, "rope_append: unknown data type");
    if (!(a->eps >= 0.f) || std::isinf(a->eps)) return fail(MK_ERR_ARG, "rope_append: eps must be finite and not negative");
    if (a->n_axes < 1 || a->n_axes > 4 || (a->n_axes > 1 && !a->sections)) return fail(MK_ERR_ARG, "rope_append: %d position axes", a->n_axes);
    if (a->sections) {
        int64_t sum = 0;
        for (int i = 0; i < a->n_axes; ++i) {
            if (a->sections[i] < 0) return fail(MK_ERR_ARG, "rope_append: a section of %d pairs", a->sections[i]);
            sum += a->sections[i];
        }
        if (sum != a->rotary / 2) return fail(MK_ERR_ARG, "rope_append: sections add up to %lld pairs of %d", static_cast<long long>(sum), a->rotary / 2);
    }
    if (a->rotary > 0) {
        if (!a->freqs) return fail(MK_ERR_ARG, "rope_append: null pointer");
        for (int i = 0; i < a->rotary / 2; ++i)
            if (!std::isfinite(a->freqs[i])) return fail(MK_ERR_ARG, "rope_append: frequencies must be finite");
    }
    if (a->max_seq < 1 || a->sequences < 1 || int64_t(a->max_seq) * a->sequences > INT_MAX)
        return fail(MK_ERR_ARG, "rope_append: %d sequences of %d positions (at most 2^31 - 1 slots)", a->sequences, a->max_seq);
    if (a->layer < 0) return fail(MK_ERR_ARG, "rope_append: layer %d", a->layer);
    if (a->tokens == 0) return MK_OK;
    if (!a->qkv || !a->q || !a->kv || !a->kv->k || !a->kv->v || !a->slots || (a->rotary > 0 && !a->positions))
        return fail(MK_ERR_ARG, "rope_append: null pointer");
    const int64_t es = a->qkv_dtype == MK_F32 ? 4 : 2, q_width = int64_t(a->n_q_heads) * d,
                  width = q_width + 2 * int64_t(a->n_kv_heads) * d;
    if (!op_aligned(a->qkv, 16) || !op_aligned(a->q, 16) || !op_aligned(a->kv->k, 16) || !op_aligned(a->kv->v, 16) ||
        !op_aligned(a->q_gain, 16) || !op_aligned(a->k_gain, 16))
        return fail(MK_ERR_ARG, "rope_append: qkv, gains, q and the cache must be 16-byte aligned");
    if (!op_aligned(a->positions, 4) || !op_aligned(a->slots, 4) || !op_aligned(a->status, 4))
        return fail(MK_ERR_ARG, "rope_append: positions, slots or status not 4-byte aligned");
    if (a->tokens > 1 && (a->qkv_stride < width || a->qkv_stride % (16 / es) || a->q_stride < q_width || a->q_stride % 8))
        return fail(MK_ERR_ARG, "rope_append: strides must cover their rows, in steps of 16 bytes");
    if (a->n_axes > 1 && a->rotary > 0 && a->position_stride < a->tokens)
        return fail(MK_ERR_ARG, "rope_append: a position_stride of %lld for %d tokens", static_cast<long long>(a->position_stride), a->tokens);
    const mk_kv& kv = *a->kv;
    const int64_t rows = int64_t(a->max_seq) * d;
    if ((a->n_kv_heads > 1 && (kv.head_stride < rows || kv.head_stride % 8)) ||
        (a->sequences > 1 && (kv.batch_stride < (a->n_kv_heads - 1) * (a->n_kv_heads > 1 ? kv.head_stride : 0) + rows || kv.batch_stride % 8)) ||
        (a->layer > 0 && (kv.layer_stride < (a->n_kv_heads - 1) * (a->n_kv_heads > 1 ? kv.head_stride : 0) + rows || kv.layer_stride % 8)))
        return fail(MK_ERR_ARG, "rope_append: the cache's strides must cover max_seq positions of every head, in multiples of 8");
    const int64_t heads = (a->n_kv_heads - 1) * (a->n_kv_heads > 1 ? kv.head_stride : 0) + rows,
                  span = ((a->sequences > 1 ? (a->sequences - 1) * kv.batch_stride : 0) + heads) * 2, off = a->layer * kv.layer_stride * 2;
    const RowSpan q{a->q, a->tokens, q_width * 2, a->q_stride * 2}, in{a->qkv, a->tokens, width * es, a->qkv_stride * es};
    const RowSpan cache[2] = {{static_cast<const uint8_t*>(kv.k) + (a->layer ? off : 0), 1, span, 0},
                              {static_cast<const uint8_t*>(kv.v) + (a->layer ? off : 0), 1, span, 0}};
    const bool same = a->q == a->qkv && a->qkv_dtype == MK_BF16 && (a->tokens == 1 || a->q_stride == a->qkv_stride);
    const int64_t at = a->n_axes > 1 ? (a->n_axes - 1) * a->position_stride + a->tokens : a->tokens;
    const RowSpan others[4] = {{a->q_gain, 1, d * 2, 0}, {a->k_gain, 1, d * 2, 0}, {a->rotary > 0 ? a->positions : nullptr, 1, at * 4, 0},
                               {a->slots, 1, int64_t(a->tokens) * 4, 0}};
    bool clash = !same && spans_overlap(q, in);
    for (const RowSpan& c : cache) {
        clash = clash || spans_overlap(c, q) || spans_overlap(c, in);
        for (const RowSpan& o : others) clash = clash || spans_overlap(c, o);
    }
    for (const RowSpan& o : others) clash = clash || spans_overlap(q, o);
    // (one interleaved buffer may hold both caches: then only equal addresses are refused)
    if (clash || kv.k == kv.v) return fail(MK_ERR_ARG, "rope_append: q or the cache overlaps an input, or one another");
    return MK_OK;
}

}  // namespace mk

using namespace mk;

extern "C" mk_status mk_rope_append(const mk_rope_args* a, void* stream) {
    mk_status st = rope_check(a);
    if (st != MK_OK || a->tokens == 0) return st;
    int device = 0, sms = 0;
    if ((st = op_device(&device, &sms)) != MK_OK) return st;
    RopeParams p{};
    const int d = a->head_dim;
    p.tokens = a->tokens; p.nq = a->n_q_heads; p.nkv = a->n_kv_heads; p.heads = p.nq + 2 * p.nkv;
    p.units = d / 16; p.turned = a->rotary / 16;
    p.qkv = a->qkv; p.qkv_stride = a->qkv_stride;
    p.q_gain = static_cast<const __nv_bfloat16*>(a->q_gain);
    p.k_gain = static_cast<const __nv_bfloat16*>(a->k_gain);
    p.eps = a->eps; p.inv_d = 1.f / float(d);
    p.positions = a->positions; p.position_stride = a->n_axes > 1 ? a->position_stride : 0;
    p.slots = a->slots;
    const int64_t off = a->layer ? a->layer * a->kv->layer_stride : 0;
    p.k = static_cast<__nv_bfloat16*>(a->kv->k) + off;
    p.v = static_cast<__nv_bfloat16*>(a->kv->v) + off;
    p.batch_stride = a->sequences > 1 ? a->kv->batch_stride : 0;
    p.head_stride = p.nkv > 1 ? a->kv->head_stride : 0;
    p.max_seq = a->max_seq; p.limit = a->max_seq * a->sequences;
    p.q = static_cast<__nv_bfloat16*>(a->q); p.q_stride = a->q_stride;
    p.status = a->status;
    int axis = 0, left = a->sections ? a->sections[0] : a->rotary / 2;
    for (int i = 0; i < a->rotary / 2; ++i) {
        while (left == 0) left = a->sections[++axis];   // (the sections add up to every pair)
        --left;
        p.axis[i] = uint8_t(axis);
        // the rate in turns, less its whole turns (fmod is exact), to 64 bits behind the point: off by 2^-53 of the
        // rate, 3e-10 radians at position 2^20 and a radian per position
        double turns = std::fmod(a->freqs[i] * 0.15915494309189535, 1.0);
        if (turns < 0.0) turns += 1.0;
        p.turn[i] = turns < 1.0 ? uint64_t(turns * 0x1p64) : 0;
    }
    const bool f32 = a->qkv_dtype == MK_F32, nb = a->neighbours != 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.units <= 1) return rope_launch<1>(p, f32, nb, sms, s);
    if (p.units <= 2) return rope_launch<2>(p, f32, nb, sms, s);
    if (p.units <= 4) return rope_launch<4>(p, f32, nb, sms, s);
    if (p.units <= 8) return rope_launch<8>(p, f32, nb, sms, s);
    return rope_launch<16>(p, f32, nb, sms, s);
}
