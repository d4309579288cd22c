// Norms of q and k, rotation by the tokens' positions, q to its buffer, k and v to the cache (mk_rope_append).
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "mk_ops.h"
#include "mk_sm103.cuh"

namespace mk {

constexpr int kRopePairs = 128;     // of the widest head
constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 4;        // of an SM

struct RopeParams {
    int tokens, nq, nkv;
    int units, turned;              // 16 elements each: of a head, of its rotated part
    int rounds_q, rounds_k, rounds; // of a token: rounds of heads that a warp takes at a time, for q, k and in all
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
// position (an angle in fp32 radians would be off by 2^-24 of itself); 32 bits of it become radians in [-pi, pi), where the
// special-function unit's sine and cosine are off by at most 2^-20.9: their precise forms cost 50 instructions a pair, a quarter of a token's,
// and an output keeps 2^-9 of its value.
__device__ __forceinline__ float2 rope_angle(int position, uint64_t rate) {
    const uint64_t turns = uint64_t(int64_t(position)) * rate;
    const float angle = float(int32_t(turns >> 32)) * 1.46291807926715968e-9f;   // pi / 2^31
    return make_float2(__cosf(angle), __sinf(angle));
}
__device__ __forceinline__ void rope_widen(const uint4& u, float2* x) {   // 8 bf16
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 rope_pack(const float2* x) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(x[k].y), "f"(x[k].x));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A round is 32 / GROUP heads of one kind (q, k or v) of GROUP lanes each; a lane holds 16 elements, two pieces of 8: pairs of
// elements between the pieces (rotary / 2 apart) or within them, or elements that only pass.  A head's sum of squares is a shuffle
// over its lanes; a token's cosines and sines are worked out once by the warp, and a kind's gains are multiplied into them once.
//
// The rounds of all tokens in order are shared out evenly over the warps.  A warp's heads come as bulk copies of up to kRounds
// rounds into places of its own, kDepth of them in flight, through the next tokens: what is in flight takes neither registers nor
// instructions.
// What bounds it: 16384 tokens of 48 heads of 128, bf16, normed, three axes 69 us (5.8 TB/s, 86% of a copy's rate), 4096 of fp32 26.5
// (5.7 TB/s; 2 us of it the launch and the first copies' way): the chain sums - shuffles - root - products of a round, with 16
// warps an SM (a lane's 32 factors take 112 registers; 20 warps with 96 take as long) and issue slots half used.  Loads
// straight into registers took 88 and 29.7; 16-byte copies by every lane (cp.async) 72 and 42; whole tokens to the warps in turn 74 and 28.9
// (their last round fills the device unevenly); copies of 4 KB, three in flight, 72 and 26.8; two rounds side by side 73.
template <bool F32>
struct RopeTile {
    static constexpr int kPlace = 2048, kRounds = kPlace / (F32 ? 2048 : 1024), kDepth = 4;   // (a round is at most 512 elements)
    static constexpr int kSmem = kRopeThreads / 32 * kDepth * kPlace;
};
template <int GROUP, bool F32, bool NEIGHBOURS>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const __grid_constant__ RopeParams p) {
    using T = RopeTile<F32>;
    constexpr int kHeads = 32 / GROUP, kSize = F32 ? 4 : 2;
    extern __shared__ __align__(16) uint8_t places[];
    __shared__ __align__(16) float angles[kRopeThreads / 32][2][kRopePairs];   // cosines, sines
    __shared__ uint64_t bars[kRopeThreads / 32][T::kDepth];
    __shared__ int abort_flag;
    volatile int* abort_word = &abort_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t place0 = sm::smem(places) + uint32_t(warp * T::kDepth * T::kPlace), bar0 = sm::smem(bars[warp]);
    if (threadIdx.x == 0) abort_flag = 0;
    if (lane == 0) {
        for (int i = 0; i < T::kDepth; ++i) sm::bar_init(bar0 + 8u * i, 1);
        sm::bar_fence_init();
    }
    __syncthreads();
    sm::pdl_trigger();
    sm::pdl_wait();
    const int d = 16 * p.units;
    const int64_t all = int64_t(p.tokens) * p.rounds, warps = int64_t(gridDim.x) * (kRopeThreads / 32),
                  self = int64_t(blockIdx.x) * (kRopeThreads / 32) + warp, begin = all * self / warps;
    const int count = int(all * (self + 1) / warps - begin);   // this warp's rounds, from a token and a round of it
    const int t0 = int(begin / p.rounds), round0 = int(begin - int64_t(t0) * p.rounds);
    const int round_k = p.rounds_q, round_v = p.rounds_q + p.rounds_k;

    // the next copy: rounds [r, r + n) of the token of `row`, whose heads lie one behind the other whatever their kinds
    auto head_of = [&](int r) {   // the first head of a round (of the one behind the last: all)
        return r <= round_k ? min(r * kHeads, p.nq) : r <= round_v ? p.nq + min((r - round_k) * kHeads, p.nkv) : p.nq + p.nkv + min((r - round_v) * kHeads, p.nkv);
    };
    int next_left = count, next_r = round0, next_at = 0;
    const char* row = static_cast<const char*>(p.qkv) + int64_t(t0) * p.qkv_stride * kSize;
    auto fetch = [&] {
        if (next_left <= 0) return;
        const int n = min(min(p.rounds - next_r, T::kRounds), next_left);
        if (lane == 0) {
            const int from = head_of(next_r);
            const uint32_t bytes = uint32_t((head_of(next_r + n) - from) * d * kSize), bar = bar0 + 8u * next_at;
            sm::bar_expect(bar, bytes);
            sm::bulk_load(place0 + uint32_t(next_at * T::kPlace), row + int64_t(from) * d * kSize, bytes, bar);
        }
        next_left -= n;
        next_r += n;
        if (next_r == p.rounds) {
            next_r = 0;
            row += p.qkv_stride * kSize;
        }
        next_at = next_at + 1 == T::kDepth ? 0 : next_at + 1;
    };
#pragma unroll 1
    for (int i = 0; i < T::kDepth; ++i) fetch();

    const int u = lane % GROUP, sub = lane / GROUP;
    const bool live = u < p.units;
    // where the lane's pieces start in a head: of q and k, and of v (neighbouring lanes' pieces lie side by side)
    const int from = u < p.turned ? 0 : p.turned, lo_qk = 16 * from + 8 * (u - from),
              hi_qk = lo_qk + 8 * (u < p.turned ? p.turned : p.units - p.turned);
    int at = 0, have = 0, chunk_head = 0;   // rounds left of the copy being read, its first head
    uint32_t phase = 0;
    bool ok = true;
#pragma unroll 1
    for (int t = t0, left = count, first = round0; left > 0 && ok; ++t, first = 0) {
        const int last = min(first + left, p.rounds);
        left -= last - first;
        __syncwarp();
        if (first < round_v)
            for (int i = lane; i < 8 * p.turned; i += 32) {
                const float2 cs = rope_angle(p.positions[p.axis[i] * p.position_stride + t], p.turn[i]);
                angles[warp][0][i] = cs.x;
                angles[warp][1][i] = cs.y;
            }
        const int slot = p.slots[t];
        const bool stored = slot >= 0 && slot < p.limit;
        if (slot >= p.limit && p.status) *p.status = MK_ERR_BOUNDS;
        const int sequence = stored ? slot / p.max_seq : 0;
        const int64_t cache = int64_t(sequence) * p.batch_stride + (int64_t(slot) - int64_t(sequence) * p.max_seq) * d;
        __syncwarp();
        int r = first;
#pragma unroll 1
        for (int kind = 0; kind < 3 && ok; ++kind) {
            const int heads = kind == 0 ? p.nq : p.nkv, r0 = kind == 0 ? 0 : kind == 1 ? round_k : round_v,
                      r1 = min(last, kind == 0 ? round_k : kind == 1 ? round_v : p.rounds);
            if (r >= r1) continue;
            const bool turn = u < p.turned && kind < 2;
            const int lo = kind < 2 ? lo_qk : 8 * u, hi = kind < 2 ? hi_qk : 8 * (p.units + u);
            __nv_bfloat16* const out = kind == 0 ? p.q + int64_t(t) * p.q_stride : (kind == 1 ? p.k : p.v) + cache;
            const int64_t out_stride = kind == 0 ? d : p.head_stride;
            const bool writes = live && (kind == 0 || stored);
            const __nv_bfloat16* gain = kind == 0 ? p.q_gain : kind == 1 ? p.k_gain : nullptr;
            // an element's own factor, and that of the other one of its pair: (a, b) -> (a g c - b h s, b h c + a g s)
            float2 own[8], across[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) own[k] = make_float2(1.f, 1.f);
            if (gain && live) {
                rope_widen(__ldg(reinterpret_cast<const uint4*>(gain + lo)), own);
                rope_widen(__ldg(reinterpret_cast<const uint4*>(gain + hi)), own + 4);
            }
            if (turn) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {   // two pairs a step
                    const int pair = NEIGHBOURS ? 4 * u + 2 * (k & 1) + (k < 2 ? 0 : 4 * p.turned) : 8 * u + 2 * k;
                    const float2 c = *reinterpret_cast<const float2*>(&angles[warp][0][pair]), s = *reinterpret_cast<const float2*>(&angles[warp][1][pair]);
                    if (NEIGHBOURS) {
                        float2 &g0 = own[2 * k], &g1 = own[2 * k + 1];
                        across[2 * k] = make_float2(-g0.y * s.x, g0.x * s.x);
                        across[2 * k + 1] = make_float2(-g1.y * s.y, g1.x * s.y);
                        g0 = sm::mul2(g0, make_float2(c.x, c.x));
                        g1 = sm::mul2(g1, make_float2(c.y, c.y));
                    } else {
                        across[k] = sm::mul2(own[k + 4], make_float2(-s.x, -s.y));
                        across[k + 4] = sm::mul2(own[k], s);
                        own[k] = sm::mul2(own[k], c);
                        own[k + 4] = sm::mul2(own[k + 4], c);
                    }
                }
            }
            const int apart = (hi - lo) * kSize;
#pragma unroll 1
            while (r < r1) {
                if (have == 0) {   // the next copy
                    if (!(ok = sm::bar_wait_warp(bar0 + 8u * at, phase, abort_word, p.status))) break;
                    have = min(last - r, T::kRounds);
                    chunk_head = head_of(r);
                }
                const int n = min(r1 - r, have);
                const uint8_t* src = places + (warp * T::kDepth + at) * T::kPlace + ((head_of(r) - chunk_head + sub) * d + lo) * kSize;
#pragma unroll 1
                for (int i = 0; i < n; ++i, src += kHeads * d * kSize) {
                    // (lanes without a head or a piece read their round's place, whatever is there, and store nothing)
                    const int h = (r - r0 + i) * kHeads + sub;
                    const bool here = live && h < heads;
                    float2 x[8];
                    if constexpr (F32) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            *reinterpret_cast<float4*>(x + 2 * k) = *reinterpret_cast<const float4*>(src + 16 * k);
                            *reinterpret_cast<float4*>(x + 4 + 2 * k) = *reinterpret_cast<const float4*>(src + apart + 16 * k);
                        }
                    } else {
                        rope_widen(*reinterpret_cast<const uint4*>(src), x);
                        rope_widen(*reinterpret_cast<const uint4*>(src + apart), x + 4);
                    }
                    if (gain) {
                        float2 s2 = make_float2(0.f, 0.f), s3 = s2;
#pragma unroll
                        for (int k = 0; k < 8; k += 2) {
                            s2 = sm::fma2(x[k], x[k], s2);
                            s3 = sm::fma2(x[k + 1], x[k + 1], s3);
                        }
                        float ss = here ? (s2.x + s3.x) + (s2.y + s3.y) : 0.f;
#pragma unroll
                        for (int o = GROUP / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                        const float scale = rsqrtf(fmaf(ss, p.inv_d, p.eps));
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = sm::mul2(x[k], make_float2(scale, scale));
                    }
                    if (turn) {
                        float2 y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            y[k] = sm::fma2(NEIGHBOURS ? make_float2(x[k].y, x[k].x) : x[k ^ 4], across[k], sm::mul2(x[k], own[k]));
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = y[k];
                    } else if (gain) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = sm::mul2(x[k], own[k]);
                    }
                    if (here && writes) {
                        __nv_bfloat16* dst = out + h * out_stride;
                        *reinterpret_cast<uint4*>(dst + lo) = rope_pack(x);
                        *reinterpret_cast<uint4*>(dst + hi) = rope_pack(x + 4);
                    }
                }
                r += n;
                have -= n;
                if (have == 0) {
                    if (++at == T::kDepth) { at = 0; phase ^= 1u; }
                    __syncwarp();
                    fetch();   // (into the place that was just read)
                }
            }
        }
    }
    if (!ok && lane == 0) {   // a wait ran out: the copies still in flight end before the CTA does
        const uint64_t t1 = sm::timer_ns();
        while (sm::timer_ns() - t1 < 10000000ull) {}
    }
}

template <int GROUP, bool F32, bool NEIGHBOURS>
static mk_status rope_launch(const RopeParams& p, int device, int sms, cudaStream_t stream) {
    static std::atomic<uint64_t> set{0};
    const mk_status st = op_smem(reinterpret_cast<const void*>(&rope_kernel<GROUP, F32, NEIGHBOURS>), RopeTile<F32>::kSmem, device, &set);
    if (st != MK_OK) return st;
    constexpr int kWarps = kRopeThreads / 32;
    const int64_t rounds = int64_t(p.tokens) * p.rounds;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(unsigned(std::min<int64_t>((rounds + kWarps - 1) / kWarps, int64_t(sms) * kRopeCtas)));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.dynamicSmemBytes = RopeTile<F32>::kSmem;
    MK_CK(cudaLaunchKernelEx(&cfg, &rope_kernel<GROUP, F32, NEIGHBOURS>, p));
    return MK_OK;
}
template <int GROUP>
static mk_status rope_launch(RopeParams& p, bool f32, bool neighbours, int device, int sms, cudaStream_t stream) {
    p.rounds_q = (p.nq + 32 / GROUP - 1) / (32 / GROUP);
    p.rounds_k = (p.nkv + 32 / GROUP - 1) / (32 / GROUP);
    p.rounds = p.rounds_q + 2 * p.rounds_k;
    if (f32)
        return neighbours ? rope_launch<GROUP, true, true>(p, device, sms, stream) : rope_launch<GROUP, true, false>(p, device, sms, stream);
    return neighbours ? rope_launch<GROUP, false, true>(p, device, sms, stream) : rope_launch<GROUP, false, false>(p, device, sms, stream);
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
    p.tokens = a->tokens; p.nq = a->n_q_heads; p.nkv = a->n_kv_heads;
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
    if (p.units <= 1) return rope_launch<1>(p, f32, nb, device, sms, s);
    if (p.units <= 2) return rope_launch<2>(p, f32, nb, device, sms, s);
    if (p.units <= 4) return rope_launch<4>(p, f32, nb, device, sms, s);
    if (p.units <= 8) return rope_launch<8>(p, f32, nb, device, sms, s);
    return rope_launch<16>(p, f32, nb, device, sms, s);
}
