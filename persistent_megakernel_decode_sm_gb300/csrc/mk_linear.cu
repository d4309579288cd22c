// The linear map of the prompt path: out = act(x w^T + bias) + residual (mk_linear).
#include "mk_ops.h"
#include "mk_sm103.cuh"

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
template <int N>
__device__ __forceinline__ void linear_residuals(const LinearParams& p, bool wanted, int r, int j, int left, float (&res)[N], int step = 1) {
    const int64_t at = r * p.residual_stride + j, by = p.residual_stride * step;
#pragma unroll
    for (int i = 0; i < N; ++i) res[i] = 0.f;
    if (!p.residual || !wanted) return;
    if (p.residual_f32) {
        const float* src = static_cast<const float*>(p.residual) + at;
#pragma unroll
        for (int i = 0; i < N; ++i, src += by)
            if (i * step < left) res[i] = *src;
    } else {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.residual) + at;
#pragma unroll
        for (int i = 0; i < N; ++i, src += by)
            if (i * step < left) res[i] = __bfloat162float(*src);
    }
}
// What the sums of a thread's columns start from: the bias and, where no activation comes between,
// the residual (in one of the CTAs that share the contraction)
template <int N>
__device__ __forceinline__ void linear_begin(const LinearParams& p, int r, int j, int left, bool mine, bool plain, float bias, float (&v)[N]) {
    linear_residuals<N>(p, mine && plain, r, j, left, v);
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
// 8 columns c, c + STEP, .. (below c1) of a split tile: the partial sums of `split` CTAs (ranks
// by * s + at), staged as [column][128 rows], added in order; the up sums lie `up_bytes` further
template <int STEP, bool GATED, bool F32>
__device__ __forceinline__ void linear_join(const LinearParams& p, uint32_t stage0, uint32_t up_bytes, int split, int by, int at,
                                            int m0, int c, int c1, int row, int j) {
    float y[8], u[8], res[8];
    linear_residuals<8>(p, GATED || p.act != MK_ACT_NONE, m0 + c, j, c1 - c, res, STEP);
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
    linear_stores<F32>(p, m0 + c, j, c1 - c, y, STEP);
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

// Warp 0: TMA producer.  Warp 1: tensor memory and MMA issue.  The others: epilogue.
template <int BN, bool GATED, bool F32>
__global__ void __launch_bounds__(64 + 32 * LinearTile<BN, GATED>::kWarps, 1)
linear_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
              const __grid_constant__ LinearParams p) {
    using T = LinearTile<BN, GATED>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * T::kStages + 5];
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
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
    sm::pdl_wait();

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
        for (int tile = first; tile < tiles && ok; tile += step)
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
                if (ok && leader) sm::mma_commit(acc_full(buf));
                __syncwarp();
            }
        if (*abort_word && leader) { sm::mma_commit(drained); sm::bar_drain(drained, 0); }
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
            linear_begin<T::kWidth>(p, m0 + cols, j, left, rank == 0, plain, p.bias && j < p.n ? __bfloat162float(p.bias[j]) : 0.f, v);
            if (GATED) {
                const float b = rank == 0 && p.bias && j < p.n ? __bfloat162float(p.bias[p.n + j]) : 0.f;
#pragma unroll
                for (int i = 0; i < T::kWidth; ++i) u[GATED ? i : 0] = b;
            }
#pragma unroll 1
            for (int k0 = kb0; k0 < kb1; k0 += piece, ++n) {
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
#pragma unroll
            for (int c = 0; c < T::kWidth; c += 8) {
                if (c >= p.rows - m0 - cols) break;
                float y[8], res[8];
                linear_residuals(p, !plain, m0 + cols + c, j, left - c, res);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = linear_act(GATED ? MK_ACT_SWIGLU : p.act, v[c + i], GATED ? u[GATED ? c + i : 0] : 0.f) + res[i];
                linear_stores<F32>(p, m0 + cols + c, j, left - c, y);
            }
        }
    }
    if (p.split > 1) {
        // the tile's columns are shared out over the cluster; each is summed over the CTAs in rank order
        __syncwarp();
        sm::cluster_sync();
        if (warp >= 2 && !*abort_word) {
            int n0, m0;
            place(first, n0, m0);
            const int t = threadIdx.x - 64, row = t & 127, j = n0 + row;
            constexpr int kGroups = T::kWarps / 4;
            const int c1 = min(BN * (rank + 1) / p.split, p.rows - m0);
            if (j < p.n)
                for (int c = BN * rank / p.split + t / 128; c < c1; c += 8 * kGroups)
                    linear_join<kGroups, GATED, F32>(p, stage0, BN * 128 * 4, p.split, 1, 0, m0, c, c1, row, j);
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
template <bool GATED, bool F32>
__global__ void __launch_bounds__(320, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                   const __grid_constant__ LinearParams p) {
    using T = PairTile<GATED>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * T::kStages + 4];
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
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
    sm::pdl_wait();

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
            for (int tile = first; tile < tiles && ok; tile += step)
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
                    if (ok && issuer) sm::mma_commit_pair(acc_full(buf), both);
                    __syncwarp();
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
        float v[128];   // the thread's row of the tile, its 128 columns
        int n = 0;
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
            int n0, m0;
            place(tile, n0, m0);
            const int j = n0 + (GATED ? row & 63 : row);
            const bool live = j < p.n;
            const int jb = up_row ? p.n + j : j;   // (bias rows: gate rows, then up rows)
            linear_begin<128>(p, m0 + cols, j, live ? p.rows - m0 - cols : 0, part == 0, plain,
                              p.bias && live ? __bfloat162float(p.bias[jb]) : 0.f, v);
#pragma unroll 1
            for (int k0 = kb0; k0 < kb1; k0 += piece, ++n) {
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
#pragma unroll
            for (int c = 0; c < 128; c += kStep) {
                const int m = m0 + cols + c + (up_row ? 8 : 0), left = live ? p.rows - m : 0;
                if (m0 + cols + c >= p.rows) break;   // (the same for both warps of an exchange: they share cols)
                float y[8], res[8];
                linear_residuals<8>(p, !plain, m, j, left, res);
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
                linear_stores<F32>(p, m, j, left, y);
            }
        }
    }
    if (p.split > 1) {
        // the tile's columns are shared out over the pairs; each is summed in order of the contraction
        __syncwarp();
        sm::cluster_sync();
        if (warp >= 2 && !*abort_word) {
            int n0, m0;
            place(first, n0, m0);
            const int t = threadIdx.x - 64, row = t % T::kRows, j = n0 + row;
            constexpr int kGroups = 256 / T::kRows;
            const int width0 = 256 * part / p.split, c1 = min(256 * (part + 1) / p.split, p.rows - m0);
            if (j < p.n)
                for (int c = width0 + t / T::kRows; c < c1; c += 8 * kGroups)
                    linear_join<kGroups, GATED, F32>(p, stage0, 64 * 4, p.split, 2, half, m0, c, c1, row, j);
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
// Times by rounds of the clusters that run at once: a round's blocks of the contraction at `cycles` each, a fixed
// part (set-up, the first copies' way, the epilogue) and, where the contraction is cut over `split` units of `unit`
// CTAs, the exchange of partial sums (`join`).  Unsplit tiles go to a persistent grid whose fixed part shows once.
// Clusters of 8 leave SMs out (15 run at once on 152 SMs, 36 of 4, 76 of 2): 16 tiles over 8 CTAs each took two
// rounds, 46.7 us against 38.8 with 4 (512 x 2048 x 8192).
static mk_status linear_split(const void* fn, LinearLaunch& cfg, std::atomic<int> (&resident)[8], int unit, int most, int blocks,
                              int cycles, int fixed, int join, LinearPlan& pl) {
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
        const int64_t rounds = (tiles + fit - 1) / fit, part = int64_t((blocks + s - 1) / s) * cycles;
        const bool even = (s & (s - 1)) == 0;   // (else the shares of a tile's columns come out uneven)
        const int64_t t = s == 1 ? rounds * part + fixed : rounds * (part + fixed + (even ? join : 2 * join));
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

// The two kernels behind one face: plan(), then launch() with its plan
template <int BN, bool GATED, bool F32>
struct LinearOne {
    using T = LinearTile<BN, GATED>;
    static constexpr int kTokens = BN, kFeatures = 128, kUnit = 1;
    // cycles as fitted to 96 to 768 tokens by 688 or 2048 inputs by 1001 to 2048 outputs, splits 1 to 4 (1.87 GHz)
    static constexpr int kCycles = GATED ? (BN < 128 ? 750 : 900) : BN <= 32 ? 355 : BN == 64 ? 374 : 450;
    static constexpr int kFixed = BN < 128 ? 7800 : 8400, kJoin = BN == 128 ? 3400 : 500 + 32 * BN;
    static mk_status plan(const LinearParams& p, int device, LinearPlan& pl) {
        static std::atomic<uint64_t> set{0};
        static std::atomic<int> resident[64][8];
        const void* fn = reinterpret_cast<const void*>(&linear_kernel<BN, GATED, F32>);
        const mk_status st = op_smem(fn, T::kSmem, device, &set);
        if (st != MK_OK) return st;
        pl.tiles_n = (p.n + 127) / 128;
        pl.tiles_m = (p.rows + BN - 1) / BN;
        LinearLaunch cfg(64 + 32 * T::kWarps, T::kSmem, nullptr);
        return linear_split(fn, cfg, resident[device], 1, 8, (p.k + kLinK - 1) / kLinK, kCycles, kFixed, kJoin, pl);
    }
    static mk_status launch(const mk_linear_args* a, LinearParams& p, const LinearPlan& pl, cudaStream_t stream) {
        CUtensorMap map_w, map_x;
        const mk_status st = linear_maps(a, p, int64_t(p.n) * T::kAccs, 128, BN, &map_w, &map_x);
        if (st != MK_OK) return st;
        p.tiles_n = pl.tiles_n; p.tiles_m = pl.tiles_m; p.split = pl.split;
        LinearLaunch cfg(64 + 32 * T::kWarps, T::kSmem, stream);
        cfg.shape(pl.split, pl.clusters);
        MK_CK(cudaLaunchKernelEx(&cfg.c, &linear_kernel<BN, GATED, F32>, map_w, map_x, p));
        return MK_OK;
    }
};
template <bool GATED, bool F32>
struct LinearPair {
    using T = PairTile<GATED>;
    static constexpr int kTokens = 256, kFeatures = 2 * T::kRows, kUnit = 2;
    static mk_status plan(const LinearParams& p, int device, LinearPlan& pl) {
        static std::atomic<uint64_t> set{0};
        static std::atomic<int> resident[64][8];
        const void* fn = reinterpret_cast<const void*>(&linear_pair_kernel<GATED, F32>);
        const mk_status st = op_smem(fn, T::kSmem, device, &set);
        if (st != MK_OK) return st;
        pl.tiles_n = (p.n + 2 * T::kRows - 1) / (2 * T::kRows);
        pl.tiles_m = (p.rows + 255) / 256;
        LinearLaunch cfg(320, T::kSmem, nullptr);
        return linear_split(fn, cfg, resident[device], 2, 4, (p.k + kLinK - 1) / kLinK, 515, GATED ? 20000 : 15000, 2500, pl);
    }
    static mk_status launch(const mk_linear_args* a, LinearParams& p, const LinearPlan& pl, cudaStream_t stream) {
        CUtensorMap map_w, map_x;
        const mk_status st = linear_maps(a, p, int64_t(p.n) * (GATED ? 2 : 1), T::kRows, 128, &map_w, &map_x);
        if (st != MK_OK) return st;
        p.tiles_n = pl.tiles_n; p.tiles_m = pl.tiles_m; p.split = pl.split;
        LinearLaunch cfg(320, T::kSmem, stream);
        cfg.shape(2 * pl.split, pl.clusters);
        MK_CK(cudaLaunchKernelEx(&cfg.c, &linear_pair_kernel<GATED, F32>, map_w, map_x, p));
        return MK_OK;
    }
};
// The tile width (or the pairs) whose plan costs least: wide tiles read w fewer times and pairs make twice the products a
// cycle, narrow tiles fill the device (2048 x 2048 weights, us: 96 tokens 7.2 with 64 columns over 4 CTAs each, 7.8
// with 32 over 2, 8.4 with 128 over 4, 11.0 in pairs; 768 tokens 24.4 with 32, 13.3 with 128, 15.1 in pairs; 2048
// tokens and more: pairs).
struct LinearChoice {
    LinearPlan plan;
    int tokens, features, unit;   // of a tile; CTAs of a unit (2: a pair)
    mk_status (*launch)(const mk_linear_args*, LinearParams&, const LinearPlan&, cudaStream_t);
};
template <bool GATED, bool F32>
static mk_status linear_choose(const LinearParams& p, int device, LinearChoice& best) {
    LinearPlan pl{};
    best = LinearChoice{};
    mk_status st = MK_OK;
    auto offer = [&](auto kernel, bool wanted) {
        using K = decltype(kernel);
        if (st != MK_OK || !wanted || (st = K::plan(p, device, pl)) != MK_OK) return;
        if (!best.launch || pl.cost < best.plan.cost) best = {pl, K::kTokens, K::kFeatures, K::kUnit, &K::launch};
    };
    offer(LinearOne<16, GATED, F32>{}, p.rows <= 64);
    offer(LinearOne<32, GATED, F32>{}, p.rows > 16 && p.rows <= 768);
    offer(LinearOne<64, GATED, F32>{}, p.rows > 32 && p.rows <= 1536);
    offer(LinearOne<128, GATED, F32>{}, p.rows > 64);
    offer(LinearPair<GATED, F32>{}, p.rows > 128);
    return st;
}

static mk_status linear_check(const mk_linear_args* a) {
    if (!a) return fail(MK_ERR_ARG, "null argument");
    if (a->rows < 0 || a->rows > (1 << 30) || a->n < 1 || a->n > (1 << 30) || a->k < 8 || a->k % 8)
        return fail(MK_ERR_ARG, "linear: rows %d, n %d, k %d (rows in [0, 2^30], n in [1, 2^30], k a multiple of 8)", a->rows, a->n, a->k);
    if (a->activation < MK_ACT_NONE || a->activation > MK_ACT_SWIGLU)
        return fail(MK_ERR_ARG, "linear: unknown activation %d", a->activation);
    if ((a->out_dtype != MK_BF16 && a->out_dtype != MK_F32) ||
        (a->residual && a->residual_dtype != MK_BF16 && a->residual_dtype != MK_F32))
        return fail(MK_ERR_ARG, "linear: unknown data type");
    const bool gated = a->activation == MK_ACT_SWIGLU;
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

// The parameters of a checked call, and its plan on the current device
static mk_status linear_plan(const mk_linear_args* a, LinearParams& p, LinearChoice& choice) {
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
        return p.out_f32 ? linear_choose<true, true>(p, device, choice) : linear_choose<true, false>(p, device, choice);
    return p.out_f32 ? linear_choose<false, true>(p, device, choice) : linear_choose<false, false>(p, device, choice);
}

extern "C" mk_status mk_linear(const mk_linear_args* a, void* stream) {
    mk_status st = linear_check(a);
    if (st != MK_OK || a->rows == 0) return st;
    LinearParams p{};
    LinearChoice c;
    if ((st = linear_plan(a, p, c)) != MK_OK) return st;
    return c.launch(a, p, c.plan, static_cast<cudaStream_t>(stream));
}

extern "C" mk_status mk_linear_plan(const mk_linear_args* a, int32_t* plan) {
    if (!plan) return fail(MK_ERR_ARG, "null argument");
    mk_status st = linear_check(a);
    if (st != MK_OK) return st;
    if (a->rows == 0) return fail(MK_ERR_ARG, "linear: no rows, no plan");
    LinearParams p{};
    LinearChoice c;
    if ((st = linear_plan(a, p, c)) != MK_OK) return st;
    const int32_t out[6] = {c.unit, c.features, c.tokens, c.plan.split, c.plan.tiles_n * c.plan.tiles_m, int32_t(c.plan.clusters)};
    for (int i = 0; i < 6; ++i) plan[i] = out[i];
    return MK_OK;
}
