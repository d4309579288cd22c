// The linear map of the prompt path: out = act(x w^T + bias) + residual (mk_linear), and the same with low-rank
// adapters in front of the activation (mk_linear_adapted): kernels, plans and checks of both entry points' units.
#pragma once

#include "mk_ops.h"
#include "mk_sm103.cuh"

#include <algorithm>
#include <type_traits>

namespace mk {

struct LinearParams {
    int rows, n, k, act;
    int tiles_n, tiles_m, split;   // feature tiles, token tiles; CTAs (one cluster) that share a tile's contraction
    const __nv_bfloat16* bias;
    const void* residual;
    int64_t residual_stride;
    int residual_f32, out_f32;
    void* out;
    int64_t out_stride;
    int32_t* status;
};

// Adapters.  Their part of a tile's sums is a longer contraction: behind the blocks of w and x come blocks of the `up` rows of
// every adapter that a token of the tile names, against the tokens' low-rank rows scale x down^T, zero for the
// tokens of other adapters (mk_adapt.cu works them out, and lists each tile's adapters).  So the weights of an adapter are
// read once per tile of tokens, whoever names it, and the sums meet in the accumulators in front of the activation.
// The low-rank rows are cut into bf16 parts, two (16 of fp32's 24 bits: off by 2^-18 of the adapter's share, far below a bf16
// output's own rounding) or, for an fp32 output, three.  An adapter takes 16 columns of the rank, 32, or a multiple of 64; a piece is
// up to 64 of them.  A block is 64 columns of up (four, two or one adapter's pieces, rows of 32, 64 or 128 bytes) in one
// stage beside the first part of the terms' 64 columns, and the other parts in the stage after it: up is copied once for all parts,
// and what a block costs by itself (waits, commits) is shared by 8 or 12 products.  A CTA pair, whose tiles name few adapters, takes
// blocks of 32 columns in one stage each (4096 tokens through 2 x 8192 x 2048 165 us, with blocks over two stages 2.5% more).
template <bool ADAPT>
struct LinearExtra {
    static constexpr int32_t width = 0;
};
template <>
struct LinearExtra<true> {
    CUtensorMap up, terms;     // terms: [rows][part][blocks][64]
    const int32_t* index;      // [rows], -1 or n_adapters and more: none
    const int32_t* count;      // [tiles of tokens]: adapters of the tile
    const int32_t* list;       // [tiles of tokens][slots]: which, in the order in which its tokens name them
    int32_t slots, width;      // columns of an adapter
    int32_t part;              // columns of a part
    int32_t n_adapters, rank;
    const __nv_bfloat16 *x, *w, *up_rows, *term_rows;   // what linear_alone reads
    int64_t x_stride;
};
constexpr int kAdaptCols = 64;   // of a block
constexpr int kPairCols = 32, kPairBytes = 128 * kPairCols * 2;   // of a CTA pair's, all in one stage: columns, bytes of 128 rows
__device__ __forceinline__ int adapt_piece(int width) { return min(width, kAdaptCols); }
// This CTA's share [b0, b1) of the adapters' blocks of a token tile, for the role that asks, and the adapters of its
// columns: in shared memory for the CTA's first tile, in global memory for the others (behind the wait for the kernel that lists them)
struct LinearShare {
    const volatile int32_t* list;
    int adapters, pieces, b0, b1;
    __device__ __forceinline__ void cut(int width, int cols, int rank, int split) {   // (cols: of a block)
        pieces = width < cols ? adapters : adapters * (width / cols);
        const int blocks = (adapters * width + cols - 1) / cols;
        b0 = int(int64_t(blocks) * rank / split);
        b1 = int(int64_t(blocks) * (rank + 1) / split);
    }
};
struct LinearFirst {   // the first tile's adapters; stages given to a block of adapters, whose terms may be copied
    int32_t list[256], count;
    uint64_t ready, granted[10];
};
// What the linear kernel with adapters reads before its own wait is whole: the kernel in front starts it behind its wait for
// everything before.  But that wait orders the other kernel's reads, not this one's; read at the L2 (L2 true), where every
// earlier kernel's writes have arrived, such a value cannot be one that an SM's L1 still holds.
template <bool L2, typename T>
__device__ __forceinline__ T linear_get(const T* at) {
    if constexpr (L2) return __ldcg(at);
    else return *at;
}
// By one warp: the adapters that tokens [m0, m0 + tokens) name, in order
__device__ __forceinline__ void linear_list(const LinearExtra<true>& e, int m0, int tokens, LinearFirst& first) {
    const int lane = threadIdx.x & 31;
    int count = 0;
    for (int t = 0; t < tokens; t += 32) {
        int name = t + lane < tokens ? linear_get<true>(e.index + m0 + t + lane) : -1;
        if (name >= e.n_adapters) name = -1;
        bool is_new = (__match_any_sync(0xFFFFFFFFu, name) & ((1u << lane) - 1)) == 0 && name >= 0;
        for (int i = 0; i < count; ++i) is_new = is_new && first.list[i] != name;
        const uint32_t all = __ballot_sync(0xFFFFFFFFu, is_new);
        if (is_new) first.list[count + __popc(all & ((1u << lane) - 1))] = name;
        count += __popc(all);
        __syncwarp();
    }
    if (lane == 0) first.count = count;
}
// The adapter and its column of consecutive pieces of a tile's columns, for one lane: the next adapter's name is read ahead
struct LinearColumns {
    const volatile int32_t* list;
    int adapters, width, at, column, name, ahead;
    __device__ __forceinline__ LinearColumns(const LinearShare& s, int w, int first)
        : list(s.list), adapters(s.adapters), width(w), at(first / w), column(first - at * w), name(read(at)), ahead(read(at + 1)) {}
    __device__ __forceinline__ int read(int i) const { return i < adapters ? list[i] : 0; }
    __device__ __forceinline__ void step(int by) {   // (never beyond an adapter's last column but to the next one's first)
        if ((column += by) < width) return;
        column = 0;
        name = ahead;
        ahead = read(++at + 1);
    }
};

// y Phi(y) by the lower tail Q(a) = Phi(-a), a = |y|: y Q for y < 0, y (1 - Q) else, so nothing cancels (1 + erf does,
// below -1; erfcf takes 1.2 us more for 333 x 1001 outputs than this and erff).  Q = exp(-a^2 / 2) t P(t) with
// t = 1 / (1 + 0.34 a): exp(a^2 / 2) Q(a) falls like 1 / a, so P is smooth over all of it.  P is the least-squares fit of
// degree 8 over a in [0, 14], its points reweighted towards equal errors: off by 3e-8 of the value, 4e-7 evaluated in fp32.
__device__ __forceinline__ float linear_gelu(float y) {
    const float a = fabsf(y);
    float t, e;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(a, 0.34f, 1.f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a * a * -0.72134752f));   // (log2(e) / 2)
    float q = -0.0261204801f;
    q = fmaf(q, t, 0.139499515f);
    q = fmaf(q, t, -0.273132801f);
    q = fmaf(q, t, 0.202182725f);
    q = fmaf(q, t, -0.0447184853f);
    q = fmaf(q, t, 0.115359172f);
    q = fmaf(q, t, 0.115197659f);
    q = fmaf(q, t, 0.136112198f);
    q = fmaf(q, t, 0.135620505f);
    q = q * t * e;
    return y * (y < 0.f ? q : 1.f - q);
}
// y and the up factor of one output, bias included, to the value before the residual, in fp32
__device__ __forceinline__ float linear_act(int act, float y, float up) {
    if (act == MK_ACT_NONE) return y;
    if (act == MK_ACT_GELU) return linear_gelu(y);
    const float s = y / (1.f + expf(-y));
    return act == MK_ACT_SWIGLU ? s * up : s;
}
// The residuals of the tokens r, r + 1, .. of feature j, of which `left` exist (zeros where not wanted)
template <bool L2, int N>
__device__ __forceinline__ void linear_residuals(const LinearParams& p, bool wanted, int r, int j, int left, float (&res)[N], int step = 1) {
    const int64_t at = r * p.residual_stride + j, by = p.residual_stride * step;
#pragma unroll
    for (int i = 0; i < N; ++i) res[i] = 0.f;
    if (!p.residual || !wanted) return;
    if (p.residual_f32) {
        const float* src = static_cast<const float*>(p.residual) + at;
#pragma unroll
        for (int i = 0; i < N; ++i, src += by)
            if (i * step < left) res[i] = linear_get<L2>(src);
    } else {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.residual) + at;
#pragma unroll
        for (int i = 0; i < N; ++i, src += by)
            if (i * step < left) res[i] = __bfloat162float(linear_get<L2>(src));
    }
}
// What the sums of a thread's columns start from: the bias and, where no activation comes between,
// the residual (in one of the CTAs that share the contraction)
template <bool L2, int N>
__device__ __forceinline__ void linear_begin(const LinearParams& p, int r, int j, int left, bool mine, bool plain, float bias, float (&v)[N]) {
    linear_residuals<L2>(p, mine && plain, r, j, left, v);
    if (mine)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += bias;
}
template <bool F32>
__device__ __forceinline__ void linear_stores(const LinearParams& p, int r, int j, int left, const float (&y)[8], int step = 1) {
    using Out = std::conditional_t<F32, float, __nv_bfloat16>;
    Out* dst = static_cast<Out*>(p.out) + (r * p.out_stride + j);
    const int64_t by = p.out_stride * step;
#pragma unroll
    for (int i = 0; i < 8; ++i, dst += by)
        if (i * step < left) {
            if constexpr (F32) *dst = y[i];
            else *dst = __float2bfloat16_rn(y[i]);
        }
}
// The same but for sums that came to NaN: a bit for each of these.  Behind a call: as a branch of every step of the epilogue it slowed
// 4096 tokens through 2048 x 8192 from 119 to 132 us (fp32; bf16 87 to 92) that hold no NaN.
template <bool F32>
__device__ __noinline__ uint32_t linear_stores_sound_of(const LinearParams& p, int r, int j, int left, float y0, float y1, float y2, float y3, float y4,
                                                        float y5, float y6, float y7, int step) {
    const float y[8] = {y0, y1, y2, y3, y4, y5, y6, y7};
    using Out = std::conditional_t<F32, float, __nv_bfloat16>;
    Out* dst = static_cast<Out*>(p.out) + (r * p.out_stride + j);
    const int64_t by = p.out_stride * step;
    uint32_t nan = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i, dst += by)
        if (i * step < left) {
            if (y[i] != y[i]) nan |= 1u << i;
            else if constexpr (F32) *dst = y[i];
            else *dst = __float2bfloat16_rn(y[i]);
        }
    return nan;
}
template <bool F32>
__device__ __forceinline__ uint32_t linear_stores_sound(const LinearParams& p, int r, int j, int left, const float (&y)[8], int step = 1) {
    return linear_stores_sound_of<F32>(p, r, j, left, y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7], step);
}
__device__ __forceinline__ void linear_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 linear_load(const __nv_bfloat16* p, bool wanted) {
    return wanted ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void linear_widen(const uint4& u, float (&x)[8], bool add = false) {   // 8 bf16
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = (add ? x[2 * i] : 0.f) + __uint_as_float(w[i] << 16);
        x[2 * i + 1] = (add ? x[2 * i + 1] : 0.f) + __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
// Whether 8 bf16 are all finite
__device__ __forceinline__ bool linear_finite(const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    bool ok = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) ok = ok && (w[i] & 0x7F80u) != 0x7F80u && (w[i] & 0x7F800000u) != 0x7F800000u;
    return ok;
}
// What a lane has found out about its feature: the tile's adapters whose up rows of it are not finite (how many, the last of them),
// and the adapter that it last looked up among the tile's
struct LinearSuspects {
    int bad = -1, last = -1;
    int name = -1, slot = -1;
};
// Of the tokens m + i step (bits i of `nan`) whose outputs of feature j came to NaN, those that have to be taken again: another
// token's adapter is not finite there, or the token's own makes an infinity in a part.  The others are NaN in their own right.
template <bool GATED, bool F32>
__device__ __noinline__ uint32_t linear_suspects(const LinearParams& p, const LinearExtra<true>& e, const volatile int32_t* list, int adapters,
                                                 int m, int step, int j, uint32_t nan, LinearSuspects& s) {
    constexpr int kRows = GATED ? 2 : 1;
    const int64_t next = int64_t(p.n) * e.rank;   // from gate to up rows
    auto row = [&](int adapter) { return e.up_rows + (int64_t(adapter) * kRows * p.n + j) * e.rank; };
    if (s.bad < 0) {
        s.bad = 0;
        for (int i = 0; i < adapters; ++i) {
            const __nv_bfloat16* u = row(list[i]);
            bool ok = true;
#pragma unroll 2
            for (int c = 0; c < e.rank; c += 8)
#pragma unroll
                for (int part = 0; part < kRows; ++part) ok = linear_finite(__ldg(reinterpret_cast<const uint4*>(u + part * next + c))) && ok;
            if (!ok) {
                ++s.bad;
                s.last = i;
            }
        }
    }
    uint32_t again = 0;
    for (uint32_t left = nan; left; left &= left - 1) {
        const int i = __ffs(left) - 1, token = m + i * step, own = e.index[token];
        if (own != s.name) {
            s.name = own;
            s.slot = -1;
            for (int at = 0; at < adapters && own >= 0; ++at)
                if (list[at] == own) s.slot = at;
        }
        bool redo = s.bad > 1 || (s.bad == 1 && s.last != s.slot), in_parts = false;
        if (s.slot >= 0) {   // (most often a token whose x is not finite, and its first sum NaN)
            const __nv_bfloat16 *t = e.term_rows + int64_t(token) * (F32 ? 3 : 2) * e.part + s.slot * e.width, *u = row(own);
            float sum[kRows], parts[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) sum[r] = parts[r] = 0.f;
            bool is_nan = false;
#pragma unroll 1
            for (int c = 0; c < e.rank && !is_nan; c += 8) {
                float h[F32 ? 3 : 2][8], b[8];
#pragma unroll
                for (int k = 0; k < (F32 ? 3 : 2); ++k) linear_widen(*reinterpret_cast<const uint4*>(t + k * e.part + c), h[k]);
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    linear_widen(*reinterpret_cast<const uint4*>(u + r * next + c), b);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        sum[r] = fmaf(F32 ? h[0][k] + h[1][k] + h[F32 ? 2 : 1][k] : h[0][k] + h[1][k], b[k], sum[r]);
#pragma unroll
                        for (int q = 0; q < (F32 ? 3 : 2); ++q) parts[r] += fabsf(h[q][k] * b[k]);
                    }
                    is_nan = is_nan || sum[r] != sum[r];
                }
            }
            if (is_nan) continue;
#pragma unroll
            for (int r = 0; r < kRows; ++r) in_parts = in_parts || !isfinite(parts[r]);
        }
        if (redo || in_parts) again |= 1u << i;
    }
    return again;
}
// An adapter's infinity or NaN times a zero of another token's low-rank row is NaN: a tensor core cannot leave the product out.
// Sums that came to NaN so are taken again here, with no adapter but the token's own (and as that one's parts may
// be infinities of both signs, its value in one piece); what is NaN by itself is stored as that.  By a whole warp: the tokens
// m + i step (bits i of a lane's `nan`, of 8 that are the same of every lane, `left` from m on) of the lanes' features j, j + 1, ...
// x and w are read straight into m16n8k16 products (a thread's 16 bytes of a row are the elements 2 i, 2 i + 1 of two products),
// summed 512 elements at a time; 16 features of 8 tokens take 3 loads a lane per 32 of the contraction.
// Where no sum is NaN this is one comparison an output (0.1 to 0.3 us a call, 1.3 of 4096 tokens through 2 x 8192 x 2048).  Where some
// are in their own right, finding that out reads the up rows of the tile's adapters: 512 of those 4096 tokens of NaN 370 us for 165,
// all of them 920, 64 tokens of 64 adapters of rank 64 (4096 x 6144) 208 for 46 (with all of these taken again 2.9 ms, 9.2 ms and
// 340 us).  Taking a tile again is bound by the latencies of x's and w's loads: one adapter of NaN among those 64 515 us, among those of
// the 4096 tokens, 60 of which name it, 3.1 ms.
template <bool GATED, bool F32>
__device__ __noinline__ void linear_alone(const LinearParams& p, const LinearExtra<true>& e, const volatile int32_t* list, int adapters,
                                          int m, int step, int j, int left, uint32_t nan, LinearSuspects& suspects) {
    using Out = std::conditional_t<F32, float, __nv_bfloat16>;
    constexpr unsigned kAll = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    if (!__any_sync(kAll, nan != 0)) return;
    sm::pdl_wait();   // (the terms)
    uint32_t mine = 0;
    if (nan) {
        mine = linear_suspects<GATED, F32>(p, e, list, adapters, m, step, j, nan, suspects);
        for (uint32_t stays = nan & ~mine; stays; stays &= stays - 1)
            static_cast<Out*>(p.out)[(m + (__ffs(stays) - 1) * step) * p.out_stride + j] = Out(__uint_as_float(0x7FFFFFFFu));
    }
    const unsigned all = __ballot_sync(kAll, mine != 0);   // (a lane without a feature has stored nothing, and has no bits)
    if (!all) return;
    const int most = __shfl_sync(kAll, left, __ffs(all) - 1), j0 = __shfl_sync(kAll, j, 0);
    // a product's column is token g (behind the last: the last one's again), its sums are of tokens 2 q and 2 q + 1
    const __nv_bfloat16* x = e.x + int64_t(m + min(g, (most - 1) / step) * step) * e.x_stride + q * 8;
    int own[2], slot[2];   // their adapters, and where these are among the tile's
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        own[h] = (2 * q + h) * step < most ? e.index[m + (2 * q + h) * step] : -1;
        slot[h] = -1;
        if (own[h] >= 0)
            for (int i = 0; i < adapters; ++i)
                if (list[i] == own[h]) slot[h] = i;
    }
#pragma unroll 1
    for (int half = 0; half < 32; half += 16) {
        if (!(all >> half & 0xFFFFu)) continue;
        int row[2];   // of w, less the gate rows
#pragma unroll
        for (int r = 0; r < 2; ++r) row[r] = min(j0 + half + g + 8 * r, p.n - 1);
        float y[GATED ? 2 : 1][4];
#pragma unroll
        for (int part = 0; part < (GATED ? 2 : 1); ++part) {
            const __nv_bfloat16 *w0 = e.w + (int64_t(part) * p.n + row[0]) * p.k + q * 8, *w1 = e.w + (int64_t(part) * p.n + row[1]) * p.k + q * 8;
#pragma unroll
            for (int v = 0; v < 4; ++v) y[part][v] = 0.f;
#pragma unroll 1
            for (int k0 = 0; k0 < p.k; k0 += 512) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                for (int c = k0; c < min(k0 + 512, p.k); c += 32) {
                    const bool in = c + q * 8 < p.k;
                    const uint4 a = linear_load(w0 + c, in), b = linear_load(w1 + c, in), t = linear_load(x + c, in);
                    linear_mma(acc, a.x, b.x, a.y, b.y, t.x, t.y);
                    linear_mma(acc, a.z, b.z, a.w, b.w, t.z, t.w);
                }
#pragma unroll
                for (int v = 0; v < 4; ++v) y[part][v] += acc[v];
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {   // (feature g + 8 (v / 2), token 2 q + v % 2)
                if (slot[v & 1] >= 0) {
                    const __nv_bfloat16* t = e.term_rows + int64_t(m + (2 * q + (v & 1)) * step) * (F32 ? 3 : 2) * e.part + slot[v & 1] * e.width;
                    const __nv_bfloat16* u = e.up_rows + ((int64_t(own[v & 1]) * (GATED ? 2 : 1) + part) * p.n + row[v / 2]) * e.rank;
#pragma unroll 1
                    for (int c = 0; c < e.rank; c += 8) {
                        float a[8], b[8];
                        linear_widen(*reinterpret_cast<const uint4*>(t + c), a);
                        linear_widen(*reinterpret_cast<const uint4*>(t + e.part + c), a, true);
                        if (F32) linear_widen(*reinterpret_cast<const uint4*>(t + 2 * e.part + c), a, true);
                        linear_widen(*reinterpret_cast<const uint4*>(u + c), b);
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[part][v] = fmaf(a[i], b[i], y[part][v]);
                    }
                }
                if (p.bias) y[part][v] += __bfloat162float(linear_get<true>(p.bias + part * p.n + row[v / 2]));
            }
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int i = (2 * q + (v & 1)) * step, of = half + g + 8 * (v / 2);   // token, the lane whose feature it is
            if (!(__shfl_sync(kAll, mine, of) >> (2 * q + (v & 1)) & 1u)) continue;
            float res[1];
            linear_residuals<true>(p, true, m + i, j0 + of, 1, res);
            const float out = linear_act(GATED ? MK_ACT_SWIGLU : p.act, y[0][v], GATED ? y[GATED ? 1 : 0][v] : 0.f) + res[0];
            static_cast<Out*>(p.out)[(m + i) * p.out_stride + j0 + of] = Out(out);
        }
    }
}
__device__ __forceinline__ bool linear_nan(const float (&y)[8]) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) nan = nan || y[i] != y[i];
    return nan;
}

// 8 columns c, c + STEP, .. (below c1) of a split tile: the partial sums of `split` CTAs (ranks
// by * s + at), staged as [column][128 rows], added in order; the up sums lie `up_bytes` further
template <int STEP, bool GATED, bool F32, bool ADAPT>
__device__ __forceinline__ void linear_join(const LinearParams& p, const LinearExtra<ADAPT>& e, const std::conditional_t<ADAPT, LinearFirst, char>& tile, uint32_t stage0,
                                            uint32_t up_bytes, int split, int by, int at, int m0, int c, int c1, int row, int j,
                                            [[maybe_unused]] LinearSuspects& suspects) {
    float y[8], u[8], res[8];
    const int left = !ADAPT || j < p.n ? c1 - c : 0;   // (with adapters lanes without a feature come here too)
    linear_residuals<ADAPT>(p, GATED || p.act != MK_ACT_NONE, m0 + c, j, left, res, STEP);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = u[i] = 0.f;
    for (int s = 0; s < split; ++s) {
        const uint32_t peer = sm::cluster_addr(stage0, uint32_t(by * s + at));
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // (a column past c1 reads one below it: every address is inside the stages)
            const uint32_t src = peer + uint32_t((min(c + i * STEP, c1 - 1) * 128 + row) * 4);
            y[i] += sm::cluster_ld(src);
            if (GATED) u[i] += sm::cluster_ld(src + up_bytes);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = linear_act(GATED ? MK_ACT_SWIGLU : p.act, y[i], u[i]) + res[i];
    if constexpr (ADAPT) {
        if (__any_sync(0xFFFFFFFFu, linear_nan(y))) {
            const uint32_t nan = linear_stores_sound<F32>(p, m0 + c, j, left, y, STEP);
            linear_alone<GATED, F32>(p, e, tile.list, tile.count, m0 + c, STEP, j, left, nan, suspects);
            return;
        }
    }
    linear_stores<F32>(p, m0 + c, j, left, y, STEP);
}

// A tile is 128 output features (the MMA's M: rows of w, one per tensor-memory lane) by BN tokens
// (its N: one accumulator column each), so few tokens cost few columns, a bias belongs to a lane,
// and a warp's store of one column is 32 neighbouring outputs of a token's row.  SwiGLU holds the
// gate rows and the up rows of the same features as two accumulators, multiplied in the epilogue.
// The contraction runs in blocks of 64 through a ring of shared-memory stages.
//
// The tensor core truncates as it accumulates, an error that grows with the length of the sum
// (measured at k = 8192 with an fp32 output: 1.5e-6 of its norm, against 7e-7 for plain fp32 sums).  fp32
// outputs are therefore summed in pieces of kPromote blocks that the epilogue warps add up in registers
// (3.4e-7); a bf16 output rounds a thousand times coarser and takes the whole contraction in one piece.
constexpr int kLinK = 64;
constexpr int kPromote = 8;
constexpr int kAdaptPromote = 3;   // (blocks of adapters, of 12 products each, where those of w and x have 4)
template <int BN, bool GATED>
struct LinearTile {
    static constexpr int kAccs = GATED ? 2 : 1;
    static constexpr int kABytes = 128 * kLinK * 2, kBBytes = BN * kLinK * 2;
    static constexpr int kStageBytes = kAccs * kABytes + kBBytes;
    static constexpr int kStages = 200 * 1024 / kStageBytes < 10 ? 200 * 1024 / kStageBytes : 10;
    static constexpr int kBufCols = BN * kAccs;                    // columns of one tile's accumulators
    static constexpr int kCols = 2 * kBufCols < 32 ? 32 : 2 * kBufCols;   // two tiles: one is written out while the next is summed
    static constexpr int kSmem = kStages * kStageBytes + 1024;    // (+ alignment of the first stage)
    static constexpr int kWarps = BN >= 64 ? 8 : 4;               // epilogue warps: 32 lanes by kWidth columns each
    static constexpr int kWidth = BN / (kWarps / 4);
    static_assert(kCols <= 512 && (kCols & (kCols - 1)) == 0);
    static_assert(kStages * kStageBytes >= kBufCols * 128 * 4);   // a split tile's partial sums are staged there
};

// Warp 0: TMA producer.  Warp 1: tensor memory and MMA issue.  The others: epilogue; with adapters the last: copies of their terms.
//
// With adapters the kernel starts once every CTA of the kernel in front of it (mk_adapt.cu's, whose first act is to wait for the
// kernels before it) has started: every kernel before that one is done, so x, w and the residual are read and sums taken at once,
// beside that kernel, and only who copies its results waits for its end.
template <int BN, bool GATED, bool F32, bool ADAPT>
__global__ void __launch_bounds__(64 + 32 * LinearTile<BN, GATED>::kWarps + (ADAPT ? 32 : 0), 1)
linear_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
              const __grid_constant__ LinearParams p, const __grid_constant__ LinearExtra<ADAPT> e) {
    using T = LinearTile<BN, GATED>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * T::kStages + 5];
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
    __shared__ std::conditional_t<ADAPT, LinearFirst, char> first_tile;
    volatile int* abort_word = &abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stage0 = (sm::smem(raw) + 1023u) & ~1023u;
    const uint32_t bar0 = sm::smem(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (T::kStages + s); };
    auto acc_full = [&](int s) { return bar0 + 8u * (2 * T::kStages + s); };
    auto acc_empty = [&](int s) { return bar0 + 8u * (2 * T::kStages + 2 + s); };
    const uint32_t drained = bar0 + 8u * (2 * T::kStages + 4);
    if (threadIdx.x == 0) {
        for (int s = 0; s < T::kStages; ++s) { sm::bar_init(full(s), 1); sm::bar_init(empty(s), 1); }
        for (int s = 0; s < 2; ++s) { sm::bar_init(acc_full(s), 1); sm::bar_init(acc_empty(s), T::kWarps); }
        sm::bar_init(drained, 1);
        if constexpr (ADAPT) {
            static_assert(T::kStages <= 10);
            sm::bar_init(sm::smem(&first_tile.ready), 1);
            for (int s = 0; s < T::kStages; ++s) sm::bar_init(sm::smem(&first_tile.granted[s]), 1);
        }
        abort_flag = 0;
        sm::bar_fence_init();
        sm::tma_prefetch_map(&map_w);
        sm::tma_prefetch_map(&map_x);
    }
    if (warp == 1) sm::tmem_alloc(sm::smem(&tmem_at), T::kCols);
    sm::tc_fence_before();
    __syncthreads();
    sm::tc_fence_after();
    const uint32_t tmem = tmem_at;
    sm::pdl_trigger();
    if constexpr (!ADAPT) sm::pdl_wait();

    // this CTA's tiles, and its share [kb0, kb1) of their contraction blocks
    const int rank = p.split > 1 ? int(sm::cluster_rank()) : 0;
    const int first = int(blockIdx.x) / p.split, step = int(gridDim.x) / p.split;
    const int tiles = p.tiles_n * p.tiles_m;
    const int blocks = (p.k + kLinK - 1) / kLinK;
    const int kb0 = int(int64_t(blocks) * rank / p.split), kb1 = int(int64_t(blocks) * (rank + 1) / p.split);
    const int piece = F32 ? kPromote : kb1 - kb0;   // blocks summed in tensor memory at a time
    auto place = [&](int tile, int& n0, int& m0) {
        n0 = tile / p.tiles_m * 128;
        m0 = tile % p.tiles_m * BN;
    };
    // (fails only as its wait does)
    [[maybe_unused]] auto share = [&](int tile, LinearShare& s) {
        if constexpr (ADAPT) {
            const int m = tile % p.tiles_m;
            if (tile == first) {
                if (!sm::bar_wait_warp(sm::smem(&first_tile.ready), 0, abort_word, p.status)) return false;
                s.list = first_tile.list;
                s.adapters = *reinterpret_cast<const volatile int32_t*>(&first_tile.count);
            } else {
                sm::pdl_wait();
                s.list = e.list + int64_t(m) * e.slots;
                s.adapters = *reinterpret_cast<const volatile int32_t*>(e.count + m);
            }
            s.cut(e.width, kAdaptCols, rank, p.split);
        }
        return true;
    };

    if (warp == 0) {
        const bool issuer = sm::elect_one();
        int it = 0, s = 0;
        uint32_t phase = 1;   // (the first round finds every stage empty)
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
            int n0, m0;
            place(tile, n0, m0);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                if (!(ok = sm::bar_wait_warp(empty(s), phase, abort_word, p.status))) break;
                const uint32_t at = stage0 + s * T::kStageBytes;
                if (issuer) {
                    sm::bar_expect(full(s), T::kStageBytes);
                    sm::tma_load_2d(at, &map_w, full(s), kb * kLinK, n0);
                    if (GATED) sm::tma_load_2d(at + T::kABytes, &map_w, full(s), kb * kLinK, p.n + n0);
                    sm::tma_load_2d(at + T::kAccs * T::kABytes, &map_x, full(s), kb * kLinK, m0);
                }
                __syncwarp();
                if (++s == T::kStages) { s = 0; phase ^= 1u; }
            }
            if constexpr (ADAPT) {
                LinearShare sh{};
                if (!ok || !(ok = share(tile, sh))) break;
                // (up does not depend on the kernel in front: its copies are made as soon as there are stages; the last warp adds the terms)
                const int span = adapt_piece(e.width), most = kAdaptCols / span;
                const uint32_t bytes = uint32_t(span) * 256u;   // of a piece, 128 rows
                LinearColumns col(sh, e.width, sh.b0 * kAdaptCols);
                auto next_stage = [&] {
                    ++it;
                    if (++s == T::kStages) { s = 0; phase ^= 1u; }
                };
                for (int b = sh.b0; b < sh.b1; ++b) {
                    if (!(ok = sm::bar_wait_warp(empty(s), phase, abort_word, p.status))) break;
                    if (issuer) {
                        const int items = min(most, sh.pieces - b * most);
                        sm::bar_expect(full(s), uint32_t(items * T::kAccs) * bytes + T::kBBytes);
                        sm::bar_arrive(sm::smem(&first_tile.granted[s]));
                        uint32_t at = stage0 + s * T::kStageBytes;
                        for (int i = 0; i < items; ++i, at += bytes) {
                            sm::tma_load_3d(at, &e.up, full(s), col.column, n0, col.name);
                            if (GATED) sm::tma_load_3d(at + T::kABytes, &e.up, full(s), col.column, p.n + n0, col.name);
                            col.step(span);
                        }
                    }
                    __syncwarp();
                    next_stage();
                    if (!(ok = sm::bar_wait_warp(empty(s), phase, abort_word, p.status))) break;
                    if (issuer) {
                        sm::bar_expect(full(s), T::kBBytes * (F32 ? 2 : 1));
                        sm::bar_arrive(sm::smem(&first_tile.granted[s]));
                    }
                    __syncwarp();
                    next_stage();
                }
            }
        }
        if (*abort_word && issuer)   // the copies in flight land before the CTA gives its shared memory back
            for (int i = max(0, it - T::kStages); i < it; ++i) sm::bar_drain(full(i % T::kStages), uint32_t(i / T::kStages) & 1u);
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t idesc = sm::mma_idesc(128, BN);
        const bool leader = sm::elect_one();
        const uint64_t a0 = sm::desc_k_sw128(stage0), b0 = sm::desc_k_sw128(stage0 + T::kAccs * T::kABytes);
        int s = 0, n = 0;
        uint32_t phase = 0;
        bool ok = true;
        // the adapters' blocks [x0, x1) into accumulators d: an item's products with each of its terms
        const int span = adapt_piece(e.width);
        const uint64_t up0 = span == 16 ? sm::desc_k_sw32(stage0) : span == 32 ? sm::desc_k_sw64(stage0) : a0;
        const uint64_t odd = span == 16 ? 4096 >> 4 : 2, even = span == 64 ? 4 : 8192 >> 4;   // 16 columns further, 32
        [[maybe_unused]] auto adapters = [&](uint32_t d, const LinearShare& sh, int x0, int x1, bool fresh) {
            for (int b = x0; b < x1; ++b) {
                const int s1 = s + 1 == T::kStages ? 0 : s + 1;
                if (!(ok = sm::bar_wait_warp(full(s), phase, abort_word, p.status)) ||
                    !(ok = sm::bar_wait_warp(full(s1), phase ^ uint32_t(s1 == 0), abort_word, p.status)))
                    break;
                sm::tc_fence_after();
                const uint64_t at = uint64_t(s * (T::kStageBytes >> 4)), at1 = uint64_t(s1 * (T::kStageBytes >> 4));
                const uint64_t x[3] = {b0 + at, b0 + at1, a0 + at1};   // the parts
                const int steps = min(kAdaptCols, sh.pieces * span - b * kAdaptCols) / 16;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kAdaptCols / 16; ++kk) {
                        if (kk >= steps) break;
                        const uint64_t up = up0 + at + kk / 2 * even + kk % 2 * odd;
#pragma unroll
                        for (int part = 0; part < (F32 ? 3 : 2); ++part) {
                            sm::mma_ss(d, up, x[part] + 2 * kk, idesc, !fresh || b > x0 || kk > 0 || part > 0);
                            if (GATED) sm::mma_ss(d + BN, up + (T::kABytes >> 4), x[part] + 2 * kk, idesc, !fresh || b > x0 || kk > 0 || part > 0);
                        }
                    }
                    sm::mma_commit(empty(s));
                    sm::mma_commit(empty(s1));
                }
                __syncwarp();
                for (int i = 0; i < 2; ++i)
                    if (++s == T::kStages) { s = 0; phase ^= 1u; }
            }
        };
        for (int tile = first; tile < tiles && ok; tile += step) {
            for (int k0 = kb0; k0 < kb1 && ok; k0 += piece, ++n) {
                const int buf = n & 1;
                if (n >= 2 && !(ok = sm::bar_wait_warp(acc_empty(buf), uint32_t(n / 2 - 1) & 1u, abort_word, p.status))) break;
                const uint32_t d = tmem + buf * T::kBufCols;
                const int k1 = min(k0 + piece, kb1);
                for (int kb = k0; kb < k1; ++kb) {
                    if (!(ok = sm::bar_wait_warp(full(s), phase, abort_word, p.status))) break;
                    sm::tc_fence_after();
                    const uint64_t a = a0 + uint64_t(s * (T::kStageBytes >> 4)), b = b0 + uint64_t(s * (T::kStageBytes >> 4));
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < kLinK / 16; ++kk) {   // (32 bytes along the row: 2 in the descriptor's units)
                            sm::mma_ss(d, a + 2 * kk, b + 2 * kk, idesc, kb > k0 || kk > 0);
                            if (GATED) sm::mma_ss(d + BN, a + (T::kABytes >> 4) + 2 * kk, b + 2 * kk, idesc, kb > k0 || kk > 0);
                        }
                        sm::mma_commit(empty(s));
                    }
                    __syncwarp();
                    if (++s == T::kStages) { s = 0; phase ^= 1u; }
                }
                if constexpr (ADAPT && !F32) {   // (the tile's only piece)
                    LinearShare sh{};
                    if (ok && (ok = share(tile, sh))) adapters(d, sh, sh.b0, sh.b1, false);
                }
                if (ok && leader) sm::mma_commit(acc_full(buf));
                __syncwarp();
            }
            if constexpr (ADAPT && F32) {
                LinearShare sh{};
                ok = ok && share(tile, sh);
                for (int x0 = sh.b0; x0 < sh.b1 && ok; x0 += kAdaptPromote, ++n) {
                    const int buf = n & 1;
                    if (n >= 2 && !(ok = sm::bar_wait_warp(acc_empty(buf), uint32_t(n / 2 - 1) & 1u, abort_word, p.status))) break;
                    adapters(tmem + buf * T::kBufCols, sh, x0, min(x0 + kAdaptPromote, sh.b1), true);
                    if (ok && leader) sm::mma_commit(acc_full(buf));
                    __syncwarp();
                }
            }
        }
        if (*abort_word && leader) { sm::mma_commit(drained); sm::bar_drain(drained, 0); }
        __syncwarp();
    } else if (ADAPT && warp == 2 + T::kWarps) {
        if constexpr (ADAPT) {   // the first tile's adapters, then the terms
            const bool issuer = sm::elect_one();
            int n0, m0, s = 0;
            place(first, n0, m0);
            linear_list(e, m0, min(BN, p.rows - m0), first_tile);
            __syncwarp();
            if (issuer) sm::bar_arrive(sm::smem(&first_tile.ready));
            __syncwarp();
            sm::pdl_wait();
            uint32_t phases = 0;   // of the grants of each stage
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                LinearShare sh{};
                if (!(ok = share(tile, sh))) break;
                place(tile, n0, m0);
                s = (s + kb1 - kb0) % T::kStages;
                for (int i = 2 * sh.b0; i < 2 * sh.b1; ++i) {
                    if (!(ok = sm::bar_wait_warp(sm::smem(&first_tile.granted[s]), phases >> s & 1u, abort_word, p.status))) break;
                    phases ^= 1u << s;
                    const uint32_t at = stage0 + s * T::kStageBytes;
                    const int c = i / 2 * kAdaptCols;
                    if (issuer) {
                        sm::tma_load_2d(at + T::kAccs * T::kABytes, &e.terms, full(s), c + (i % 2 ? e.part : 0), m0);
                        if (F32 && i % 2) sm::tma_load_2d(at, &e.terms, full(s), c + 2 * e.part, m0);
                    }
                    __syncwarp();
                    if (++s == T::kStages) s = 0;
                }
            }
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, row = quarter * 32 + lane, cols = (warp - 2) / 4 * T::kWidth;
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        const bool plain = !GATED && p.act == MK_ACT_NONE;
        float v[T::kWidth], u[GATED ? T::kWidth : 1];   // the thread's feature, its columns
        int n = 0;
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
            int n0, m0;
            place(tile, n0, m0);
            const int j = n0 + row, left = j < p.n ? p.rows - m0 - cols : 0;
            // bias, and without an activation the residual, enter the sums first: their loads are hidden
            linear_begin<ADAPT>(p, m0 + cols, j, left, rank == 0, plain, p.bias && j < p.n ? __bfloat162float(linear_get<ADAPT>(p.bias + j)) : 0.f, v);
            if (GATED) {
                const float b = rank == 0 && p.bias && j < p.n ? __bfloat162float(linear_get<ADAPT>(p.bias + p.n + j)) : 0.f;
#pragma unroll
                for (int i = 0; i < T::kWidth; ++i) u[GATED ? i : 0] = b;
            }
            int end = kb1;   // (of the loop over pieces: further by those of the adapters)
            if constexpr (ADAPT && F32) {
                LinearShare sh{};
                if (!(ok = share(tile, sh))) break;
                end = kb0 + ((kb1 - kb0 + piece - 1) / piece + (sh.b1 - sh.b0 + kAdaptPromote - 1) / kAdaptPromote) * piece;
            }
#pragma unroll 1
            for (int k0 = kb0; k0 < end; k0 += piece, ++n) {
                const int buf = n & 1;
                if (!(ok = sm::bar_wait_warp(acc_full(buf), uint32_t(n / 2) & 1u, abort_word, p.status))) break;
                sm::tc_fence_after();
                const uint32_t acc = tmem + buf * T::kBufCols + cols + lanes;
#pragma unroll
                for (int c = 0; c < T::kWidth; c += 16) {
                    uint32_t t[16];
                    sm::tmem_ld16(acc + c, t);
                    sm::tmem_wait_ld(t);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[c + i] += __uint_as_float(t[i]);
                    if (GATED) {
                        sm::tmem_ld16(acc + BN + c, t);
                        sm::tmem_wait_ld(t);
#pragma unroll
                        for (int i = 0; i < 16; ++i) u[GATED ? c + i : 0] += __uint_as_float(t[i]);
                    }
                }
                sm::tc_fence_before();
                __syncwarp();
                if (lane == 0) sm::bar_arrive(acc_empty(buf));
            }
            if (!ok) break;
            if (p.split > 1) {
                // partial sums to this CTA's stages (free: every product has read them): [column][feature]
#pragma unroll
                for (int i = 0; i < T::kWidth; ++i) {
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage0 + uint32_t(((cols + i) * 128 + row) * 4)), "f"(v[i]) : "memory");
                    if (GATED)
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage0 + uint32_t(((BN + cols + i) * 128 + row) * 4)),
                                     "f"(u[GATED ? i : 0]) : "memory");
                }
                break;
            }
            [[maybe_unused]] uint32_t nan[(T::kWidth + 31) / 32] = {};   // (a bit for each token)
#pragma unroll
            for (int c = 0; c < T::kWidth; c += 8) {
                if (c >= p.rows - m0 - cols) break;
                float y[8], res[8];
                linear_residuals<ADAPT>(p, !plain, m0 + cols + c, j, left - c, res);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = linear_act(GATED ? MK_ACT_SWIGLU : p.act, v[c + i], GATED ? u[GATED ? c + i : 0] : 0.f) + res[i];
                if (ADAPT && __builtin_expect(linear_nan(y), 0)) nan[c / 32] |= linear_stores_sound<F32>(p, m0 + cols + c, j, left - c, y) << (c % 32);
                else linear_stores<F32>(p, m0 + cols + c, j, left - c, y);
            }
            if constexpr (ADAPT) {
                bool any = false;
#pragma unroll
                for (uint32_t word : nan) any = any || word != 0;
                LinearShare sh{};
                if (__any_sync(0xFFFFFFFFu, any) && share(tile, sh)) {
                    LinearSuspects suspects;
#pragma unroll
                    for (int c = 0; c < T::kWidth; c += 32)
#pragma unroll 1
                        for (int i = 0; i < min(32, T::kWidth); i += 8)
                            linear_alone<GATED, F32>(p, e, sh.list, sh.adapters, m0 + cols + c + i, 1, j, left - c - i, nan[c / 32] >> i & 0xFFu, suspects);
                }
            }
        }
    }
    if (p.split > 1) {
        // the tile's columns are shared out over the cluster; each is summed over the CTAs in rank order
        __syncwarp();
        sm::cluster_sync();
        if (warp >= 2 && warp < 2 + T::kWarps && !(ADAPT ? __any_sync(0xFFFFFFFFu, *abort_word) : *abort_word)) {
            int n0, m0;
            place(first, n0, m0);
            const int t = threadIdx.x - 64, row = t & 127, j = n0 + row;
            constexpr int kGroups = T::kWarps / 4;
            const int c1 = min(BN * (rank + 1) / p.split, p.rows - m0);
            LinearSuspects suspects;
            if (ADAPT ? n0 + (row & ~31) < p.n : j < p.n)
                for (int c = BN * rank / p.split + t / 128; c < c1; c += 8 * kGroups)
                    linear_join<kGroups, GATED, F32, ADAPT>(p, e, first_tile, stage0, BN * 128 * 4, p.split, 1, 0, m0, c, c1, row, j, suspects);
        }
        __syncwarp();
        sm::cluster_sync();   // no CTA leaves while a peer reads its partial sums
    }
    sm::tc_fence_before();
    __syncthreads();
    sm::tc_fence_after();
    if (warp == 1) sm::tmem_free(tmem, T::kCols);
}

// ---- many tokens: CTA pairs ------------------------------------------------------------------
// A pair of CTAs makes a tile of 256 rows of w by 256 tokens: each CTA stages its 128 rows of w and 128
// of the tokens, 32 KB for 512 cycles of products.  What limits a CTA by itself is shared
// memory (128 bytes a cycle for the tiles written and the operands read): 128 x 256 moves 96 + 96
// bytes a cycle at the full product rate, the pair 64 + 64.  SwiGLU puts 64 gate rows and the same
// 64 features' up rows into a CTA's 128; their accumulators sit 64 lanes apart and meet in the epilogue
// through shared memory.
template <bool GATED>
struct PairTile {
    static constexpr int kRows = GATED ? 64 : 128;          // features of one CTA
    static constexpr int kHalfBytes = 128 * kLinK * 2;      // a CTA's part of w, and of the tokens
    static constexpr int kStageBytes = 2 * kHalfBytes;
    static constexpr int kStages = 6;
    static constexpr int kExchange = GATED ? 2 * 2 * 8 * 128 * 4 : 0;   // [buffer][column half][8][128] fp32
    static constexpr int kSmem = kStages * kStageBytes + kExchange + 1024;
    static_assert(kStages * kStageBytes >= 128 * 256 * 4);  // a split tile's partial sums are staged there
};

// Warp 0: TMA producer.  Warp 1: tensor memory, MMA issue (even CTA).  Warps 2-9: epilogue, each 32 lanes
// by 128 of the 256 columns, held in registers.
template <bool GATED, bool F32, bool ADAPT>
__global__ void __launch_bounds__(320, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                   const __grid_constant__ LinearParams p, const __grid_constant__ LinearExtra<ADAPT> e) {
    using T = PairTile<GATED>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * T::kStages + 4];
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
    __shared__ std::conditional_t<ADAPT, LinearFirst, char> first_tile;
    volatile int* abort_word = &abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stage0 = (sm::smem(raw) + 1023u) & ~1023u;
    const uint32_t bar0 = sm::smem(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (T::kStages + s); };
    auto acc_full = [&](int s) { return bar0 + 8u * (2 * T::kStages + s); };
    auto acc_empty = [&](int s) { return bar0 + 8u * (2 * T::kStages + 2 + s); };
    const int rank = int(sm::cluster_rank()), half = rank & 1, part = rank >> 1;
    const uint32_t leader = uint32_t(rank & ~1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < T::kStages; ++s) { sm::bar_init(full(s), 1); sm::bar_init(empty(s), 1); }
        for (int s = 0; s < 2; ++s) { sm::bar_init(acc_full(s), 1); sm::bar_init(acc_empty(s), 16); }
        if constexpr (ADAPT) sm::bar_init(sm::smem(&first_tile.ready), 1);
        abort_flag = 0;
        sm::bar_fence_init();
        sm::tma_prefetch_map(&map_w);
        sm::tma_prefetch_map(&map_x);
    }
    if (warp == 1) sm::tmem_alloc_pair(sm::smem(&tmem_at), 512);
    sm::tc_fence_before();
    __syncthreads();
    sm::cluster_sync();   // both CTAs' barriers and tensor memory are there
    sm::tc_fence_after();
    const uint32_t tmem = tmem_at;
    sm::pdl_trigger();
    if constexpr (!ADAPT) sm::pdl_wait();

    const int cluster = 2 * p.split;
    const int first = int(blockIdx.x) / cluster, step = int(gridDim.x) / cluster;
    const int tiles = p.tiles_n * p.tiles_m;
    const int blocks = (p.k + kLinK - 1) / kLinK;
    const int kb0 = int(int64_t(blocks) * part / p.split), kb1 = int(int64_t(blocks) * (part + 1) / p.split);
    const int piece = F32 ? kPromote : kb1 - kb0;   // blocks summed in tensor memory at a time
    auto place = [&](int tile, int& n0, int& m0) {
        const int group = tile / (8 * p.tiles_n), in = tile - group * 8 * p.tiles_n;
        const int width = min(8, p.tiles_m - group * 8);
        m0 = (group * 8 + in % width) * 256;
        n0 = in / width * (2 * T::kRows) + half * T::kRows;
    };
    // (fails only as its wait does)
    [[maybe_unused]] auto share = [&](int tile, LinearShare& s) {
        if constexpr (ADAPT) {
            int n0, m0;
            place(tile, n0, m0);
            if (tile == first) {
                if (!sm::bar_wait_warp(sm::smem(&first_tile.ready), 0, abort_word, p.status)) return false;
                s.list = first_tile.list;
                s.adapters = *reinterpret_cast<const volatile int32_t*>(&first_tile.count);
            } else {
                sm::pdl_wait();
                s.list = e.list + int64_t(m0 / 256) * e.slots;
                s.adapters = *reinterpret_cast<const volatile int32_t*>(e.count + m0 / 256);
            }
            s.cut(e.width, kPairCols, part, p.split);
        }
        return true;
    };

    if (warp == 0) {
        const bool issuer = sm::elect_one();
        int it = 0, s = 0;
        uint32_t phase = 1;   // (the first round finds every stage empty)
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
            int n0, m0;
            place(tile, n0, m0);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                if (!(ok = sm::bar_wait_warp(empty(s), phase, abort_word, p.status))) break;
                const uint32_t at = stage0 + s * T::kStageBytes, bar = sm::cluster_addr(full(s), leader);
                if (issuer) {
                    if (half == 0) sm::bar_expect(full(s), 2 * T::kStageBytes);   // both CTAs' copies
                    sm::tma_load_2d_pair(at, &map_w, bar, kb * kLinK, n0);
                    if (GATED) sm::tma_load_2d_pair(at + T::kHalfBytes / 2, &map_w, bar, kb * kLinK, p.n + n0);
                    sm::tma_load_2d_pair(at + T::kHalfBytes, &map_x, bar, kb * kLinK, m0 + half * 128);
                }
                __syncwarp();
                if (++s == T::kStages) { s = 0; phase ^= 1u; }
            }
            if constexpr (ADAPT) {
                LinearShare sh{};
                if (!ok || !(ok = share(tile, sh))) break;
                // up first, as far as the stages go: it does not depend on the kernel in front, as the terms do
                int given_s = s, given = sh.b0;   // (of the terms)
                auto terms = [&](int upto) {
                    for (; given < upto; ++given) {
                        const uint32_t at = stage0 + given_s * T::kStageBytes, bar = sm::cluster_addr(full(given_s), leader);
                        const int c = given * kPairCols;
                        if (issuer) {
                            sm::tma_load_2d_pair(at + T::kHalfBytes, &e.terms, bar, c, m0 + half * 128);
                            sm::tma_load_2d_pair(at + T::kHalfBytes + kPairBytes, &e.terms, bar, c + e.part, m0 + half * 128);
                            if (F32) sm::tma_load_2d_pair(at + kPairBytes, &e.terms, bar, c + 2 * e.part, m0 + half * 128);
                        }
                        if (++given_s == T::kStages) given_s = 0;
                    }
                };
                const bool two = e.width == 16;
                const int last = two && sh.adapters % 2 ? sh.adapters / 2 : -1;   // a block of one adapter's 16 columns
                constexpr uint32_t kTerms = T::kHalfBytes + (F32 ? T::kHalfBytes / 2 : 0);
                const uint32_t up_rows = GATED ? (two ? kPairBytes / 4 : kPairBytes / 2) : 0;   // (behind the gate rows)
                LinearColumns col(sh, e.width, sh.b0 * kPairCols);
                int b = sh.b0;
                for (; b < sh.b1; ++b, ++it) {
                    if (b - sh.b0 >= T::kStages) {
                        if (b - sh.b0 == T::kStages) sm::pdl_wait();
                        terms(b);
                    }
                    if (!(ok = sm::bar_wait_warp(empty(s), phase, abort_word, p.status))) break;
                    if (issuer) {
                        const uint32_t at = stage0 + s * T::kStageBytes, bar = sm::cluster_addr(full(s), leader);
                        if (half == 0) sm::bar_expect(full(s), 2 * ((b == last ? kPairBytes / 2 : kPairBytes) + kTerms));
                        sm::tma_load_3d_pair(at, &e.up, bar, col.column, n0, col.name);
                        if (GATED) sm::tma_load_3d_pair(at + up_rows, &e.up, bar, col.column, p.n + n0, col.name);
                        if (two) {
                            col.step(16);
                            if (b != last) {
                                sm::tma_load_3d_pair(at + kPairBytes / 2, &e.up, bar, 0, n0, col.name);
                                if (GATED) sm::tma_load_3d_pair(at + kPairBytes / 2 + up_rows, &e.up, bar, 0, p.n + n0, col.name);
                                col.step(16);
                            }
                        } else {
                            col.step(kPairCols);
                        }
                    }
                    __syncwarp();
                    if (++s == T::kStages) { s = 0; phase ^= 1u; }
                }
                sm::pdl_wait();
                terms(b);   // (after a wait that ran out too: every copy that a barrier expects is made)
                __syncwarp();
            }
        }
        // the products' last arrivals on this CTA's barriers come before it leaves
        for (int i = max(0, it - T::kStages); i < it && ok; ++i)
            ok = sm::bar_wait_warp(empty(i % T::kStages), uint32_t(i / T::kStages) & 1u, abort_word, p.status);
        if (*abort_word) {   // the copies in flight land (microseconds) before the CTA leaves
            const uint64_t t0 = sm::timer_ns();
            while (sm::timer_ns() - t0 < 10000000ull) {}
        }
        __syncwarp();
    } else if (warp == 1) {
        if (half == 0) {
            constexpr uint32_t idesc = sm::mma_idesc(256, 256);
            const uint16_t both = uint16_t(3u << leader);
            const bool issuer = sm::elect_one();
            const uint64_t a0 = sm::desc_k_sw128(stage0), b0 = sm::desc_k_sw128(stage0 + T::kHalfBytes);
            int s = 0, n = 0;
            uint32_t phase = 0;
            bool ok = true;
            const bool two = e.width == 16;
            const uint64_t up0 = two ? sm::desc_k_sw32(stage0) : sm::desc_k_sw64(stage0);
            const uint64_t part0[3] = {sm::desc_k_sw64(stage0 + T::kHalfBytes), sm::desc_k_sw64(stage0 + T::kHalfBytes + kPairBytes), sm::desc_k_sw64(stage0 + kPairBytes)};
            const uint64_t step16 = two ? kPairBytes / 2 >> 4 : 2;
            [[maybe_unused]] auto adapters = [&](uint32_t d, const LinearShare& sh, int x0, int x1, bool fresh) {
                for (int b = x0; b < x1; ++b) {
                    if (!(ok = sm::bar_wait_warp(full(s), phase, abort_word, p.status))) break;
                    sm::tc_fence_after();
                    const uint64_t at = uint64_t(s * (T::kStageBytes >> 4)), a = up0 + at;
                    const int steps = two && 2 * b + 1 == sh.adapters ? 1 : 2;   // of 16 columns
                    if (issuer) {
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk) {
                            if (kk >= steps) break;
#pragma unroll
                            for (int term = 0; term < (F32 ? 3 : 2); ++term)
                                sm::mma_ss_pair(d, a + kk * step16, part0[term] + at + 2 * kk, idesc,
                                                !fresh || b > x0 || kk > 0 || term > 0);
                        }
                        sm::mma_commit_pair(empty(s), both);
                    }
                    __syncwarp();
                    if (++s == T::kStages) { s = 0; phase ^= 1u; }
                }
            };
            for (int tile = first; tile < tiles && ok; tile += step) {
                for (int k0 = kb0; k0 < kb1 && ok; k0 += piece, ++n) {
                    const int buf = n & 1;
                    if (n >= 2 && !(ok = sm::bar_wait_warp(acc_empty(buf), uint32_t(n / 2 - 1) & 1u, abort_word, p.status))) break;
                    const uint32_t d = tmem + buf * 256;
                    const int k1 = min(k0 + piece, kb1);
                    for (int kb = k0; kb < k1; ++kb) {
                        if (!(ok = sm::bar_wait_warp(full(s), phase, abort_word, p.status))) break;
                        sm::tc_fence_after();
                        const uint64_t a = a0 + uint64_t(s * (T::kStageBytes >> 4)), b = b0 + uint64_t(s * (T::kStageBytes >> 4));
                        if (issuer) {
#pragma unroll
                            for (int kk = 0; kk < kLinK / 16; ++kk)
                                sm::mma_ss_pair(d, a + 2 * kk, b + 2 * kk, idesc, kb > k0 || kk > 0);
                            sm::mma_commit_pair(empty(s), both);
                        }
                        __syncwarp();
                        if (++s == T::kStages) { s = 0; phase ^= 1u; }
                    }
                    if constexpr (ADAPT && !F32) {   // (the tile's only piece)
                        LinearShare sh{};
                        if (ok && (ok = share(tile, sh))) adapters(d, sh, sh.b0, sh.b1, false);
                    }
                    if (ok && issuer) sm::mma_commit_pair(acc_full(buf), both);
                    __syncwarp();
                }
                if constexpr (ADAPT && F32) {
                    LinearShare sh{};
                    ok = ok && share(tile, sh);
                    for (int x0 = sh.b0; x0 < sh.b1 && ok; x0 += kAdaptPromote, ++n) {
                        const int buf = n & 1;
                        if (n >= 2 && !(ok = sm::bar_wait_warp(acc_empty(buf), uint32_t(n / 2 - 1) & 1u, abort_word, p.status))) break;
                        adapters(tmem + buf * 256, sh, x0, min(x0 + kAdaptPromote, sh.b1), true);
                        if (ok && issuer) sm::mma_commit_pair(acc_full(buf), both);
                        __syncwarp();
                    }
                }
            }
            if (*abort_word) {   // products in flight end before the tensor memory is freed
                const uint64_t t0 = sm::timer_ns();
                while (sm::timer_ns() - t0 < 10000000ull) {}
            }
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, row = quarter * 32 + lane, cols = (warp - 2) / 4 * 128;
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        const bool up_row = GATED && row >= 64, plain = !GATED && p.act == MK_ACT_NONE;
        if constexpr (ADAPT) {
            if (warp == 2 && first < tiles) {
                int n0, m0;
                place(first, n0, m0);
                linear_list(e, m0, min(256, p.rows - m0), first_tile);
                __syncwarp();
                if (lane == 0) sm::bar_arrive(sm::smem(&first_tile.ready));
            }
        }
        float v[128];   // the thread's row of the tile, its 128 columns
        int n = 0;
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
            int n0, m0;
            place(tile, n0, m0);
            const int j = n0 + (GATED ? row & 63 : row);
            const bool live = j < p.n;
            const int jb = up_row ? p.n + j : j;   // (bias rows: gate rows, then up rows)
            linear_begin<ADAPT>(p, m0 + cols, j, live ? p.rows - m0 - cols : 0, part == 0, plain,
                              p.bias && live ? __bfloat162float(linear_get<ADAPT>(p.bias + jb)) : 0.f, v);
            int end = kb1;   // (of the loop over pieces: further by those of the adapters)
            if constexpr (ADAPT && F32) {
                LinearShare sh{};
                ok = share(tile, sh);
                end = ok ? kb0 + ((kb1 - kb0 + piece - 1) / piece + (sh.b1 - sh.b0 + kAdaptPromote - 1) / kAdaptPromote) * piece : kb0;
            }
#pragma unroll 1
            for (int k0 = kb0; k0 < end; k0 += piece, ++n) {
                const int buf = n & 1;
                if (!(ok = sm::bar_wait_warp(acc_full(buf), uint32_t(n / 2) & 1u, abort_word, p.status))) break;
                sm::tc_fence_after();
                const uint32_t acc = tmem + buf * 256 + cols + lanes;
#pragma unroll
                for (int c = 0; c < 128; c += 16) {
                    uint32_t t[16];
                    sm::tmem_ld16(acc + c, t);
                    sm::tmem_wait_ld(t);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[c + i] += __uint_as_float(t[i]);
                }
                sm::tc_fence_before();
                __syncwarp();
                if (lane == 0) sm::bar_arrive_cluster(sm::cluster_addr(acc_empty(buf), leader));
            }
            if (GATED) ok = sm::pair_sync(1 + cols / 128 * 2 + (quarter & 1), ok);   // (the warps that exchange leave together)
            if (!ok) break;
            if (p.split > 1) {   // partial sums to this CTA's stages (every product has read them): [column][row]
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage0 + uint32_t(((cols + i) * 128 + row) * 4)), "f"(v[i]) : "memory");
                break;
            }
            // 8 columns a step.  SwiGLU: 16 columns, of which the gate row keeps 0-7 and receives their up
            // values from its up row, which keeps 8-15 and receives their gate values; two buffers take turns
            constexpr int kStep = GATED ? 16 : 8;
            // a bit for each step of which a token is NaN, and a byte of one for each of its tokens, in local memory (four registers for
            // them are too many: another 8 us there)
            [[maybe_unused]] uint32_t again = 0;
            [[maybe_unused]] uint8_t nan[128 / kStep];
#pragma unroll
            for (int c = 0; c < 128; c += kStep) {
                const int m = m0 + cols + c + (up_row ? 8 : 0), left = live ? p.rows - m : 0;
                if (m0 + cols + c >= p.rows) break;   // (the same for both warps of an exchange: they share cols)
                float y[8], res[8];
                linear_residuals<ADAPT>(p, !plain, m, j, left, res);
                if constexpr (GATED) {
                    const uint32_t at = stage0 + T::kStages * T::kStageBytes + uint32_t(((c / 16 & 1) * 2 + cols / 128) * (8 * 128 * 4));
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + uint32_t((i * 128 + row) * 4)),
                                     "f"(up_row ? v[c + i] : v[c + 8 + i]) : "memory");
                    asm volatile("bar.sync %0, 64;" ::"r"(1 + cols / 128 * 2 + (quarter & 1)) : "memory");
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float got;
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(got) : "r"(at + uint32_t((i * 128 + (row ^ 64)) * 4)) : "memory");
                        const float own = up_row ? v[c + 8 + i] : v[c + i];
                        y[i] = linear_act(MK_ACT_SWIGLU, up_row ? got : own, up_row ? own : got) + res[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = linear_act(p.act, v[c + i], 0.f) + res[i];
                }
                if (ADAPT && __builtin_expect(linear_nan(y), 0)) {
                    again |= 1u << (c / kStep);
                    nan[c / kStep] = uint8_t(linear_stores_sound<F32>(p, m, j, left, y));
                } else linear_stores<F32>(p, m, j, left, y);
            }
            if constexpr (ADAPT) {
                LinearShare sh{};
                if (__any_sync(0xFFFFFFFFu, again != 0) && share(tile, sh)) {
                    LinearSuspects suspects;
#pragma unroll 1
                    for (int i = 0; i < 128 / kStep; ++i) {
                        const int m = m0 + cols + i * kStep + (up_row ? 8 : 0);
                        linear_alone<GATED, F32>(p, e, sh.list, sh.adapters, m, 1, j, live ? p.rows - m : 0, again >> i & 1u ? nan[i] : 0u, suspects);
                    }
                }
            }
        }
    }
    if (p.split > 1) {
        // the tile's columns are shared out over the pairs; each is summed in order of the contraction
        __syncwarp();
        sm::cluster_sync();
        if (warp >= 2 && !(ADAPT ? __any_sync(0xFFFFFFFFu, *abort_word) : *abort_word)) {
            int n0, m0;
            place(first, n0, m0);
            const int t = threadIdx.x - 64, row = t % T::kRows, j = n0 + row;
            constexpr int kGroups = 256 / T::kRows;
            const int width0 = 256 * part / p.split, c1 = min(256 * (part + 1) / p.split, p.rows - m0);
            LinearSuspects suspects;
            if (ADAPT ? n0 + (row & ~31) < p.n : j < p.n)
                for (int c = width0 + t / T::kRows; c < c1; c += 8 * kGroups)
                    linear_join<kGroups, GATED, F32, ADAPT>(p, e, first_tile, stage0, 64 * 4, p.split, 2, half, m0, c, c1, row, j, suspects);
        }
        __syncwarp();
    }
    sm::tc_fence_before();
    __syncthreads();
    sm::cluster_sync();   // no CTA leaves while a peer may still reach its shared memory
    sm::tc_fence_after();
    if (warp == 1) sm::tmem_free_pair(tmem, 512);
}

// A launch: clusters of one shape, dependent on the kernel before it only from pdl_wait on
struct LinearLaunch {
    cudaLaunchConfig_t c{};
    cudaLaunchAttribute attr[2];
    LinearLaunch(int threads, int bytes, cudaStream_t stream) {
        c.blockDim = dim3(unsigned(threads));
        c.dynamicSmemBytes = size_t(bytes);
        c.stream = stream;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        c.attrs = attr;
        c.numAttrs = 2;
        shape(1, 1);
    }
    LinearLaunch(const LinearLaunch&) = delete;
    void shape(int cluster, int64_t clusters) {
        attr[0].val.clusterDim.x = unsigned(cluster);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        c.gridDim = dim3(unsigned(cluster * clusters));
    }
};

// How a call is cut: tiles, CTAs or pairs that share a tile's contraction, and what that costs
struct LinearPlan {
    int tiles_n, tiles_m, split;
    int64_t clusters;   // of the grid
    int64_t cost;       // estimated cycles
};
// With adapters a tile counts more blocks, 1.6 for each 64 columns of the adapters that its tokens name (8 or 12 products, where a
// block of w and x has 4).  Who names which is not known here: each of up to 512 tokens is taken to have its own adapter, of
// more rows / 512 neighbours share one.  The low-rank kernel in front is seen more of by pairs, which need an SM's whole shared memory, and
// by split tiles, whose parts all end behind it: kAdaptPair and kAdaptSplit cycles.  us as planned so, and without the two and with four adapters
// a tile whatever its width: tokens with an adapter each of 256 (4096 x 4096), 128 of rank 64 45.5 and 51.0, 256 73 and 80, 512 of rank 16
// 56 and 81, of rank 64 132 and 153, fp32 153 and 193; 2048 of rank 64, fp32 (2048 x 2048) 306 and 382; 100 tokens of 8 adapters in
// runs, 1024 x 8192, SwiGLU 14.7 and 18.1.  Runs of 128 of 512 tokens, 128 adapters loaded, take 31 either way, with tiles of 128 28.
constexpr int kAdaptPair = 6000, kAdaptSplit = 2000;
struct LinearNamed {
    int adapters = 0, width = 0;   // loaded; columns of each
    int blocks(int tokens, int rows) const {
        const int each = (rows + 511) / 512, named = std::min({(tokens + each - 1) / each, adapters, rows});
        return (named * width + kAdaptCols - 1) / kAdaptCols * 8 / 5;
    }
};
// Times by rounds of the clusters that run at once: a round's blocks of the contraction at `cycles` each, a fixed
// part (set-up, the first copies' way, the epilogue) and, where the contraction is cut over `split` units of `unit`
// CTAs, the exchange of partial sums (`join`).  Unsplit tiles go to a persistent grid whose fixed part shows once.
// Clusters of 8 leave SMs out (15 run at once on 152 SMs, 36 of 4, 76 of 2): 16 tiles over 8 CTAs each took two
// rounds, 46.7 us against 38.8 with 4 (512 x 2048 x 8192).
static mk_status linear_split(const void* fn, LinearLaunch& cfg, std::atomic<int> (&resident)[8], int unit, int most, int blocks, int extra,
                              int cycles, int fixed, int join, int more, LinearPlan& pl) {
    const int64_t tiles = int64_t(pl.tiles_n) * pl.tiles_m;
    if (tiles > (1 << 28)) return fail(MK_ERR_ARG, "linear: %lld tiles", static_cast<long long>(tiles));
    pl.cost = INT64_MAX;
    for (int s = 1; s <= most && unit * s <= 8 && (s == 1 || blocks >= 2 * s); ++s) {
        int fit = resident[s - 1].load();
        if (!fit) {
            cfg.shape(unit * s, 1);
            MK_CK(cudaOccupancyMaxActiveClusters(&fit, fn, &cfg.c));
            if (fit < 1 && s == 1) return fail(MK_ERR_RESOURCES, "linear: its CTAs cannot be resident");
            resident[s - 1].store(fit < 1 ? -1 : fit);
        }
        if (fit < 1) break;
        const int64_t rounds = (tiles + fit - 1) / fit, part = int64_t((blocks + extra + s - 1) / s) * cycles;
        const bool even = (s & (s - 1)) == 0;   // (else the shares of a tile's columns come out uneven)
        const int64_t t = s == 1 ? rounds * part + fixed : rounds * (part + fixed + more + (even ? join : 2 * join));
        if (t < pl.cost) { pl.cost = t; pl.split = s; pl.clusters = s > 1 || tiles < fit ? tiles : fit; }
    }
    return MK_OK;
}
static mk_status linear_maps(const mk_linear_args* a, const LinearParams& p, int64_t w_rows, uint32_t w_box, uint32_t x_box,
                             CUtensorMap* map_w, CUtensorMap* map_x) {
    const int64_t xs = p.rows == 1 ? p.k : a->x_stride;
    const cuuint64_t wd[2] = {cuuint64_t(p.k), cuuint64_t(w_rows)}, ws[1] = {cuuint64_t(p.k) * 2};
    const cuuint64_t xd[2] = {cuuint64_t(p.k), cuuint64_t(p.rows)}, xst[1] = {cuuint64_t(xs) * 2};
    const cuuint32_t wb[2] = {kLinK, w_box}, xb[2] = {kLinK, x_box};
    const mk_status st = op_tensor_map(map_w, a->w, 2, wd, ws, wb);
    return st != MK_OK ? st : op_tensor_map(map_x, a->x, 2, xd, xst, xb);
}

// The two kernels behind one face: plan(), then launch() with its plan.  A call with adapters counts `extra` blocks more
template <int BN, bool GATED, bool F32, bool ADAPT>
struct LinearOne {
    using T = LinearTile<BN, GATED>;
    static constexpr int kTokens = BN, kFeatures = 128, kUnit = 1;
    // cycles as fitted to 96 to 768 tokens by 688 or 2048 inputs by 1001 to 2048 outputs, splits 1 to 4 (1.87 GHz)
    static constexpr int kCycles = GATED ? (BN < 128 ? 750 : 900) : BN <= 32 ? 355 : BN == 64 ? 374 : 450;
    static constexpr int kFixed = BN < 128 ? 7800 : 8400, kJoin = BN == 128 ? 3400 : 500 + 32 * BN;
    static mk_status plan(const LinearParams& p, int extra, int device, LinearPlan& pl) {
        static std::atomic<uint64_t> set{0};
        static std::atomic<int> resident[64][8];
        const void* fn = reinterpret_cast<const void*>(&linear_kernel<BN, GATED, F32, ADAPT>);
        const mk_status st = op_smem(fn, T::kSmem, device, &set);
        if (st != MK_OK) return st;
        pl.tiles_n = (p.n + 127) / 128;
        pl.tiles_m = (p.rows + BN - 1) / BN;
        LinearLaunch cfg(64 + 32 * T::kWarps + (ADAPT ? 32 : 0), T::kSmem, nullptr);
        return linear_split(fn, cfg, resident[device], 1, 8, (p.k + kLinK - 1) / kLinK, extra, kCycles, kFixed, kJoin, ADAPT ? kAdaptSplit : 0, pl);
    }
    static mk_status launch(const mk_linear_args* a, LinearParams& p, const LinearExtra<ADAPT>& e, const LinearPlan& pl, cudaStream_t stream) {
        CUtensorMap map_w, map_x;
        const mk_status st = linear_maps(a, p, int64_t(p.n) * T::kAccs, 128, BN, &map_w, &map_x);
        if (st != MK_OK) return st;
        p.tiles_n = pl.tiles_n; p.tiles_m = pl.tiles_m; p.split = pl.split;
        LinearLaunch cfg(64 + 32 * T::kWarps + (ADAPT ? 32 : 0), T::kSmem, stream);
        cfg.shape(pl.split, pl.clusters);
        MK_CK(cudaLaunchKernelEx(&cfg.c, &linear_kernel<BN, GATED, F32, ADAPT>, map_w, map_x, p, e));
        return MK_OK;
    }
};
template <bool GATED, bool F32, bool ADAPT>
struct LinearPair {
    using T = PairTile<GATED>;
    static constexpr int kTokens = 256, kFeatures = 2 * T::kRows, kUnit = 2;
    static mk_status plan(const LinearParams& p, int extra, int device, LinearPlan& pl) {
        static std::atomic<uint64_t> set{0};
        static std::atomic<int> resident[64][8];
        const void* fn = reinterpret_cast<const void*>(&linear_pair_kernel<GATED, F32, ADAPT>);
        const mk_status st = op_smem(fn, T::kSmem, device, &set);
        if (st != MK_OK) return st;
        pl.tiles_n = (p.n + 2 * T::kRows - 1) / (2 * T::kRows);
        pl.tiles_m = (p.rows + 255) / 256;
        LinearLaunch cfg(320, T::kSmem, nullptr);
        return linear_split(fn, cfg, resident[device], 2, 4, (p.k + kLinK - 1) / kLinK, extra, 515, (GATED ? 20000 : 15000) + (ADAPT ? kAdaptPair : 0), 2500,
                            ADAPT ? kAdaptSplit : 0, pl);
    }
    static mk_status launch(const mk_linear_args* a, LinearParams& p, const LinearExtra<ADAPT>& e, const LinearPlan& pl, cudaStream_t stream) {
        CUtensorMap map_w, map_x;
        const mk_status st = linear_maps(a, p, int64_t(p.n) * (GATED ? 2 : 1), T::kRows, 128, &map_w, &map_x);
        if (st != MK_OK) return st;
        p.tiles_n = pl.tiles_n; p.tiles_m = pl.tiles_m; p.split = pl.split;
        LinearLaunch cfg(320, T::kSmem, stream);
        cfg.shape(2 * pl.split, pl.clusters);
        MK_CK(cudaLaunchKernelEx(&cfg.c, &linear_pair_kernel<GATED, F32, ADAPT>, map_w, map_x, p, e));
        return MK_OK;
    }
};
// The tile width (or the pairs) whose plan costs least: wide tiles read w fewer times and pairs make twice the products a
// cycle, narrow tiles fill the device (2048 x 2048 weights, us: 96 tokens 7.2 with 64 columns over 4 CTAs each, 7.8
// with 32 over 2, 8.4 with 128 over 4, 11.0 in pairs; 768 tokens 24.4 with 32, 13.3 with 128, 15.1 in pairs; 2048
// tokens and more: pairs).
template <bool ADAPT>
struct LinearChoice {
    LinearPlan plan;
    int tokens, features, unit;   // of a tile; CTAs of a unit (2: a pair)
    mk_status (*launch)(const mk_linear_args*, LinearParams&, const LinearExtra<ADAPT>&, const LinearPlan&, cudaStream_t);
};
template <bool GATED, bool F32, bool ADAPT>
static mk_status linear_choose(const LinearParams& p, const LinearNamed& named, int device, LinearChoice<ADAPT>& best) {
    LinearPlan pl{};
    best = LinearChoice<ADAPT>{};
    mk_status st = MK_OK;
    auto offer = [&](auto kernel, bool wanted) {
        using K = decltype(kernel);
        if (st != MK_OK || !wanted || (st = K::plan(p, named.blocks(K::kTokens, p.rows), device, pl)) != MK_OK) return;
        if (!best.launch || pl.cost < best.plan.cost) best = {pl, K::kTokens, K::kFeatures, K::kUnit, &K::launch};
    };
    offer(LinearOne<16, GATED, F32, ADAPT>{}, p.rows <= 64);
    offer(LinearOne<32, GATED, F32, ADAPT>{}, p.rows > 16 && p.rows <= 768);
    offer(LinearOne<64, GATED, F32, ADAPT>{}, p.rows > 32 && p.rows <= 1536);
    offer(LinearOne<128, GATED, F32, ADAPT>{}, p.rows > 64);
    offer(LinearPair<GATED, F32, ADAPT>{}, p.rows > 128);
    return st;
}

// What a plan depends on: sizes, activation, types
static mk_status linear_check_shape(const mk_linear_args* a) {
    if (!a) return fail(MK_ERR_ARG, "null argument");
    if (a->rows < 0 || a->rows > (1 << 30) || a->n < 1 || a->n > (1 << 30) || a->k < 8 || a->k % 8)
        return fail(MK_ERR_ARG, "linear: rows %d, n %d, k %d (rows in [0, 2^30], n in [1, 2^30], k a multiple of 8)", a->rows, a->n, a->k);
    if (a->activation < MK_ACT_NONE || a->activation > MK_ACT_SWIGLU)
        return fail(MK_ERR_ARG, "linear: unknown activation %d", a->activation);
    if ((a->out_dtype != MK_BF16 && a->out_dtype != MK_F32) ||
        (a->residual && a->residual_dtype != MK_BF16 && a->residual_dtype != MK_F32))
        return fail(MK_ERR_ARG, "linear: unknown data type");
    return MK_OK;
}
static mk_status linear_check(const mk_linear_args* a) {
    const mk_status st = linear_check_shape(a);
    if (st != MK_OK || a->rows == 0) return st;
    const bool gated = a->activation == MK_ACT_SWIGLU;
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

// The parameters of a checked call, and its plan on the current device
template <bool ADAPT>
static mk_status linear_plan(const mk_linear_args* a, const LinearNamed& named, LinearParams& p, LinearChoice<ADAPT>& choice) {
    p.rows = a->rows; p.n = a->n; p.k = a->k; p.act = a->activation;
    p.bias = static_cast<const __nv_bfloat16*>(a->bias);
    p.residual = a->residual;
    p.residual_stride = a->residual_stride;
    p.residual_f32 = a->residual_dtype == MK_F32;
    p.out_f32 = a->out_dtype == MK_F32;
    p.out = a->out;
    p.out_stride = a->out_stride;
    p.status = a->status;
    int device = 0, sms = 0;
    const mk_status st = op_device(&device, &sms);
    if (st != MK_OK) return st;
    if (a->activation == MK_ACT_SWIGLU)
        return p.out_f32 ? linear_choose<true, true, ADAPT>(p, named, device, choice) : linear_choose<true, false, ADAPT>(p, named, device, choice);
    return p.out_f32 ? linear_choose<false, true, ADAPT>(p, named, device, choice) : linear_choose<false, false, ADAPT>(p, named, device, choice);
}

}  // namespace mk
