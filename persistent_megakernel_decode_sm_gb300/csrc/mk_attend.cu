// Attention of query tokens over one layer of the decode KV cache (mk_attend): causal, an optional
// sliding window with sinks, an optional prefix shared by the batch.
#include "mk_ops.h"
#include "mk_sm103.cuh"

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

namespace mk {

// ---- work -----------------------------------------------------------------------------------------
// A segment is a run of query tokens over a range of positions: one sequence, or (the shared prefix)
// every token over sequence 0's first positions.  It is cut into items: a block of at most 128 rows --
// neighbouring tokens by the query heads of one KV head, so grouped heads share the K/V they read --
// times a share of the key tiles the block sees (`splits` shares).  An output row whose tokens have one share
// is written by its item; else the items leave (o, m, l) in the workspace and attend_merge_kernel joins them.
struct AttendSeg {
    int32_t q0, n;         // first query token, tokens
    int32_t pos0;          // position of the first token; kNoCausal: every token sees every key of the segment
    int32_t key0, key1;    // positions [key0, key1)
    int32_t cache;         // the sequence whose cache rows (or table row) are read
    int32_t splits, item0; // shares of the key tiles; items of the segments before
    int32_t part0;         // first row group of its parts in the workspace (units of n_q_heads rows)
    int32_t merge0;        // tokens with parts to join in the segments before (a sequence's, not the prefix's)
};
constexpr int32_t kNoCausal = INT_MIN;
// m of a part that sees no key, and of one whose scores are all -infinity (both have l = 0): a row of such
// parts alone is zeros, or 0 / 0 with one of the second kind
constexpr float kNoKeys = -INFINITY, kNoWeight = -FLT_MAX;
constexpr int kBlockRows = 128;
constexpr int attend_keys(int d) { return d == 128 ? 64 : 128; }   // keys of a tile

struct AttendCommon {
    int32_t nq, nkv, group, block_tokens;   // block_tokens: query tokens of a block, 128 / group
    int32_t segs, prefix_seg;               // prefix_seg: 1 where segment 0 is the shared prefix
    int32_t merge_tokens;                   // tokens with parts to join
    int32_t window, sinks;
    float scale_log2;                       // scale / ln 2
    const int32_t* table;                   // paged: [batch][max_blocks]
    int32_t block, max_blocks, n_blocks, box_log2;   // positions one copy takes: a power of two that divides block
    // pos / block as pos * block_inv >> block_shift, exact for pos < 2^30: with 2^(L-1) < block <= 2^L and
    // block_inv = ceil(2^(30 + L) / block), block_inv * block - 2^(30 + L) < block <= 2^L, so the quotient is off by
    // less than pos 2^L / (2^(30 + L) block) < 1 / block
    uint32_t block_inv;
    int32_t block_shift;
    __nv_bfloat16* out;
    int64_t out_stride;
    float* part_o;                          // [row][d], then per row (m, l)
    float2* part_ml;
    int32_t* status;
};
template <int SEGS>
struct AttendParams : AttendCommon {
    AttendSeg seg[SEGS];
};

// The key tiles a block of queries at positions [t0, t1] of a segment sees, in two ranges of positions:
// [0, sink_end) and [low, end)
template <int kKeys>
struct KeyRange {
    int sink_end, low, end;
    int sink_tiles, first, count;   // tiles of the sinks, first tile of the window, tiles in all
    __device__ __forceinline__ KeyRange(const AttendSeg& s, int t0, int t1, int window, int sinks) {
        const bool causal = s.pos0 != kNoCausal;
        end = causal ? min(t1 + 1, s.key1) : s.key1;
        low = window ? max(t0 - window + 1, s.key0) : s.key0;
        sink_end = window ? min(sinks, end) : 0;
        if (sink_end >= low) { sink_end = 0; low = s.key0; }   // they meet: one range
        sink_tiles = (sink_end + kKeys - 1) / kKeys;
        first = max(low / kKeys, sink_tiles);
        count = end > low ? sink_tiles + max(0, (end + kKeys - 1) / kKeys - first) : 0;
    }
    __device__ __forceinline__ int tile(int i) const { return i < sink_tiles ? i : first + i - sink_tiles; }
    __device__ __forceinline__ bool whole(int k0, int n) const {   // every position of [k0, k0 + n) is seen by some query
        return (k0 >= low && k0 + n <= end) || k0 + n <= sink_end;
    }
    __device__ __forceinline__ bool any(int k0, int n) const { return k0 < sink_end || (k0 + n > low && k0 < end); }
    __device__ __forceinline__ bool has(int k) const { return k < sink_end || (k >= low && k < end); }
};

template <int D>
struct AttendTile {
    static constexpr int kSub = D < 64 ? D : 64;                // elements of a swizzled row
    static constexpr int kSubs = D / kSub;
    static constexpr int kRowBytes = kSub * 2;
    static constexpr int kKeys = attend_keys(D);
    static constexpr int kQBytes = kBlockRows * D * 2, kTileBytes = kKeys * D * 2;   // the queries; a tile of K or V
    static constexpr int kKStages = 3, kVStages = 2;
    static constexpr int kBars = 1 + 2 * kKStages + 2 * kVStages + 8, kFlags = 8;   // kFlags: ring of the copies' skip masks
    static constexpr int kTiles = kQBytes + kTileBytes * (kKStages + kVStages);
    static constexpr int kSmem = kTiles + kBars * 8 + kFlags * 4 + 8;   // (two CTAs to an SM: 114 KB each at most)
    static_assert(kSmem + 1024 <= 228 * 512);
    // tensor memory: scores, output, softmax weights (two bf16 a column).  At D = 128, where the output takes half of the
    // CTA's columns, there are two places for a tile's scores in turn, and its weights go over them.
    static constexpr bool kShareSP = D == 128;
    static constexpr int kPlaces = kShareSP ? 2 : 1;
    static constexpr int kS = 0, kO = 128, kP = kShareSP ? 0 : 192;
    // rows are divided by the sum of their weights as rounded, which cancels the rounding of a weight that
    // outweighs the others -- but at D = 64, where that took 9% (97 us against 89; 4096 tokens, causal, 1B heads).  There
    // such a weight is 1 where its key is the maximum of the reference's tile; in a later tile it can be anything up to
    // 2^8, and its rounding, half a bf16 step at most, stays in the row beside the output's own.
    static constexpr bool kRoundedSum = D != 64;
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
// The first 16 of 32 registers to 16 columns of tensor memory
__device__ __forceinline__ void tmem_st16_head(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
                 "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
// The low n bits set (none for n <= 0, all for n >= 32)
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }

// One pass over the key tiles: S = q K^T on the tensor cores into tensor memory, one thread per row turns its 128
// scores into weights exp2(scale_log2 (s - m)) with a reference m (below), writes them back as bf16, and
// O += P V runs with P read from tensor memory.  Two CTAs share an SM, so one's products run while the
// other's threads are at their exponentials.
// What bounds it with many rows at widths up to 64 is the chain of one warp's instructions per tile, two such warps to a
// scheduler (4096 causal tokens of 32 / 8 heads by 64: 80 us, 855 TFLOP/s; tensor pipe 39% and special functions 39%
// busy).  Measured against: two threads per row at 80 or 96 registers 107 us; tiles of 64 keys with three or four CTAs 107
// and 161; registers moved between warps (setmaxnreg) 98; the exponentials taken out left the time as it was.
// At width 128 a tile has 64 keys, so that two tiles' scores have a place and the products of one run beside the weights
// of the other: 1170 TFLOP/s for 4096 causal tokens (1097 with 128 keys and one place), 1410 for 16384, although a product
// of 128 x 64 scores takes 48 cycles where half of a 128 x 128 one takes 32 (its operands' way out of shared memory).
// Reading a row's scores while the tensor cores write others takes 400 cycles, alone 92.
// With few rows the cache's bytes bound it (8 tokens with windows of 4096, 8 heads by 128: 27 us, 5.0 TB/s; 31 with
// tiles of 128 keys and one place each for K and V).
// Warps 0-3: softmax, a row per thread.  Warp 4: TMA producer.  Warp 5: tensor memory and MMA issue.
template <int D, int SEGS>
__global__ void __launch_bounds__(192, 2)
attend_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v, const __grid_constant__ AttendParams<SEGS> p) {
    using T = AttendTile<D>;
    constexpr int kKeys = T::kKeys;
    extern __shared__ __align__(1024) uint8_t raw[];   // tiles, barriers, skip masks, tensor memory's place, abort word
    uint64_t* bars = reinterpret_cast<uint64_t*>(raw + T::kTiles);
    uint32_t* skips = reinterpret_cast<uint32_t*>(bars + T::kBars);
    uint32_t& tmem_at = skips[T::kFlags];
    volatile int* abort_word = reinterpret_cast<volatile int*>(skips + T::kFlags + 1);
    if (sm::smem(raw) & 1023u) {   // (the swizzled tiles need it; there is no static shared memory to displace them)
        if (threadIdx.x == 0 && p.status) *p.status = MK_ERR_RESOURCES;
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = sm::smem(raw);
    const uint32_t q_at = base, k_at = base + T::kQBytes, v_at = k_at + T::kKStages * T::kTileBytes;
    const uint32_t bar0 = sm::smem(bars);
    const uint32_t q_full = bar0;
    auto k_full = [&](int s) { return bar0 + 8u * (1 + s); };
    auto k_empty = [&](int s) { return bar0 + 8u * (1 + T::kKStages + s); };
    auto v_full = [&](int s) { return bar0 + 8u * (1 + 2 * T::kKStages + s); };
    auto v_empty = [&](int s) { return bar0 + 8u * (1 + 2 * T::kKStages + T::kVStages + s); };
    constexpr int kMore = 1 + 2 * T::kKStages + 2 * T::kVStages;
    auto s_full = [&](int j) { return bar0 + 8u * (kMore + j % T::kPlaces); };          // (of tile j's place)
    auto p_ready = [&](int j) { return bar0 + 8u * (kMore + 2 + j % T::kPlaces); };
    auto turn = [&](int j) { return uint32_t(j / T::kPlaces) & 1u; };
    auto pv_done = [&](int j) { return bar0 + 8u * (kMore + 4 + j % T::kPlaces); };
    const uint32_t drained = bar0 + 8u * (kMore + 6), s_free = drained + 8u;

    // the item: (segment, block of queries -- the last ones, which see most, first --, KV head, share)
    int si = 0;
    {
        int lo = 0, hi = p.segs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (int(blockIdx.x) >= p.seg[mid].item0) lo = mid;
            else hi = mid - 1;
        }
        si = lo;
    }
    const AttendSeg seg = p.seg[si];
    const int item = int(blockIdx.x) - seg.item0;
    const int share = item % seg.splits, g = item / seg.splits % p.nkv;
    const int blocks = (seg.n + p.block_tokens - 1) / p.block_tokens;
    const int tok0 = (blocks - 1 - item / (seg.splits * p.nkv)) * p.block_tokens;   // within the segment
    const int toks = min(p.block_tokens, seg.n - tok0), rows = toks * p.group;
    const bool causal = seg.pos0 != kNoCausal;
    const int t0 = causal ? seg.pos0 + tok0 : 0, t1 = t0 + toks - 1;
    const KeyRange<kKeys> range(seg, t0, t1, p.window, p.sinks);
    int first = 0, n = range.count;
    if (seg.splits > 1) {   // (at most 2^24 tiles by 255 shares: 32 bits hold the products)
        first = int(uint32_t(range.count) * uint32_t(share) / uint32_t(seg.splits));
        n = int(uint32_t(range.count) * uint32_t(share + 1) / uint32_t(seg.splits)) - first;
    }
    const int warps = (rows + 31) / 32;   // softmax warps with a row

    if (threadIdx.x == 0) {
        sm::bar_init(q_full, 1);
        for (int s = 0; s < T::kKStages; ++s) { sm::bar_init(k_full(s), 1); sm::bar_init(k_empty(s), 1); }
        for (int s = 0; s < T::kVStages; ++s) { sm::bar_init(v_full(s), 1); sm::bar_init(v_empty(s), 1); }
        for (int i = 0; i < T::kPlaces; ++i) {
            sm::bar_init(s_full(i), 1);
            sm::bar_init(p_ready(i), uint32_t(warps));
            sm::bar_init(pv_done(i), 1);
        }
        sm::bar_init(s_free, uint32_t(warps));
        sm::bar_init(drained, 1);
        *abort_word = 0;
        sm::bar_fence_init();
        sm::tma_prefetch_map(&map_q);
        sm::tma_prefetch_map(&map_k);
        sm::tma_prefetch_map(&map_v);
    }
    if (warp == 5) sm::tmem_alloc(sm::smem(&tmem_at), 256);
    sm::tc_fence_before();
    __syncthreads();
    sm::tc_fence_after();
    const uint32_t tmem = tmem_at;
    sm::pdl_trigger();
    sm::pdl_wait();

    if (warp == 4) {
        if (n > 0) {
            if (lane == 0) {
                sm::bar_expect(q_full, uint32_t(p.block_tokens * p.group * D * 2));
                for (int c = 0; c < T::kSubs; ++c)
                    sm::tma_load_3d(q_at + c * kBlockRows * T::kRowBytes, &map_q, q_full, c * T::kSub, g * p.group, seg.q0 + tok0);
            }
            // a key tile is one copy, or one for each part of it that lies in one block: a lane's each
            const int box = p.table ? 1 << p.box_log2 : kKeys, parts = kKeys / box;
            const int32_t* table = p.table + int64_t(seg.cache) * p.max_blocks;
            const int cache = p.table ? 0 : seg.cache;
            // The K of a tile goes ahead of the V of the tile before it, in the order of their use.
            int jk = 0, jv = 0;   // tiles whose K, whose V copies are on their way
            int at = 0, v_pos = 0;          // the lane's part of the tile in the cache; of the tile before
            bool good = false, v_good = false;
            uint32_t bytes = 0, v_bytes = 0;
            auto copy = [&](const CUtensorMap* map, uint32_t dst, uint32_t full, uint32_t empty, int i, int stages) {
                int ok = 1;
                if (lane == 0) {
                    if (i >= stages) ok = sm::bar_wait(empty, uint32_t(i / stages - 1) & 1u, abort_word, p.status);
                    if (ok) sm::bar_expect(full, bytes);
                }
                if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) return false;
                if (good)
                    for (int c = 0; c < T::kSubs; ++c)
                        sm::tma_load_4d(dst + (c * kKeys + lane * box) * T::kRowBytes, map, full, c * T::kSub, at, g, cache);
                return true;
            };
            int pos = 0, blk = 0, entry = 0;   // of the next tile, its table entry read a tile ahead
            bool want = false;
            auto look = [&](int j) {
                pos = range.tile(first + j) * kKeys + lane * box;
                want = lane < parts && range.any(pos, box);
                if (p.table && want) {
                    blk = int(uint64_t(uint32_t(pos)) * p.block_inv >> p.block_shift);   // pos / p.block
                    entry = __ldg(table + blk);
                }
            };
            look(0);
            for (int j = 0; j <= n; ++j) {
                v_pos = at; v_good = good; v_bytes = bytes;
                if (j < n) {
                    at = pos;
                    good = want;
                    if (p.table && want) {
                        good = unsigned(entry) < unsigned(p.n_blocks);
                        if (!good && p.status) *p.status = MK_ERR_BOUNDS;
                        at = entry * p.block + (pos - blk * p.block);
                    }
                    const uint32_t copied = __ballot_sync(0xFFFFFFFFu, good);
                    if (lane == 0) skips[j % T::kFlags] = ~copied & ((1u << parts) - 1u);
                    bytes = uint32_t(__popc(copied) * box * D * 2);
                    const int ks = j % T::kKStages;
                    if (!copy(&map_k, k_at + ks * T::kTileBytes, k_full(ks), k_empty(ks), j, T::kKStages)) break;
                    jk = j + 1;
                    if (j + 1 < n) look(j + 1);   // (on its way while the V copy waits for its place)
                }
                if (j > 0) {
                    const int vs = (j - 1) % T::kVStages;
                    const int k_pos = at;
                    const bool k_good = good;
                    const uint32_t k_bytes = bytes;
                    at = v_pos; good = v_good; bytes = v_bytes;
                    if (!copy(&map_v, v_at + vs * T::kTileBytes, v_full(vs), v_empty(vs), j - 1, T::kVStages)) break;
                    jv = j;
                    at = k_pos; good = k_good; bytes = k_bytes;
                }
            }
            if (lane == 0 && *abort_word) {   // the copies in flight land before the CTA gives its shared memory back
                sm::bar_drain(q_full, 0);
                for (int i = max(0, jk - T::kKStages); i < jk; ++i) sm::bar_drain(k_full(i % T::kKStages), uint32_t(i / T::kKStages) & 1u);
                for (int i = max(0, jv - T::kVStages); i < jv; ++i) sm::bar_drain(v_full(i % T::kVStages), uint32_t(i / T::kVStages) & 1u);
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        if (n > 0) {
            constexpr uint32_t idesc_s = sm::mma_idesc(128, kKeys), idesc_o = sm::mma_idesc(128, D, true);
            const bool leader = sm::elect_one();
            const uint64_t q_desc = D == 32 ? sm::desc_k_sw64(q_at) : sm::desc_k_sw128(q_at);
            const uint64_t k_desc = D == 32 ? sm::desc_k_sw64(k_at) : sm::desc_k_sw128(k_at);
            const uint64_t v_desc = D == 32 ? sm::desc_mn_sw64(v_at) : sm::desc_mn_sw128(v_at, kKeys * T::kRowBytes);
            auto k_there = [&](int j) { return sm::bar_wait_warp(k_full(j % T::kKStages), uint32_t(j / T::kKStages) & 1u, abort_word, p.status); };
            auto v_there = [&](int j) { return sm::bar_wait_warp(v_full(j % T::kVStages), uint32_t(j / T::kVStages) & 1u, abort_word, p.status); };
            auto scores = [&](int j) {
                const int s = j % T::kKStages;
                const uint64_t k = k_desc + uint64_t(s * (T::kTileBytes >> 4));
                sm::tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {   // 16 elements of the head dimension
                        const int sub = i * 16 / T::kSub, at = i * 16 % T::kSub * 2;
                        sm::mma_ss(tmem + T::kS + j % T::kPlaces * kKeys, q_desc + ((sub * kBlockRows * T::kRowBytes + at) >> 4),
                                   k + ((sub * kKeys * T::kRowBytes + at) >> 4), idesc_s, i > 0);
                    }
                    sm::mma_commit(s_full(j));
                    sm::mma_commit(k_empty(s));
                }
                __syncwarp();
            };
            // (the copies are waited for ahead of the barriers that the softmax is behind: a wait that is over still costs
            // 100 cycles, and there it would be in the tile's chain)
            bool ok = sm::bar_wait_warp(q_full, 0, abort_word, p.status) && k_there(0);
            if (ok) scores(0);
            if (T::kShareSP && ok && n > 1 && (ok = k_there(1))) scores(1);
            for (int j = 0; j < n && ok; ++j) {
                if (!T::kShareSP && j + 1 < n) {   // the next scores as soon as these are in registers
                    if (!(ok = k_there(j + 1) && sm::bar_wait_warp(s_free, uint32_t(j) & 1u, abort_word, p.status))) break;
                    scores(j + 1);
                }
                if (!(ok = v_there(j) && sm::bar_wait_warp(p_ready(j), turn(j), abort_word, p.status))) break;
                sm::tc_fence_after();
                const int s = j % T::kVStages;
                const uint64_t v = v_desc + uint64_t(s * (T::kTileBytes >> 4));
                if (leader) {
#pragma unroll
                    for (int i = 0; i < kKeys / 16; ++i)   // 16 keys: 8 columns of P, two groups of 8 rows of V
                        sm::mma_ts(tmem + T::kO, tmem + T::kP + j % T::kPlaces * kKeys + i * 8, v + (i * 16 * T::kRowBytes >> 4), idesc_o, j > 0 || i > 0);
                    sm::mma_commit(pv_done(j));
                    sm::mma_commit(v_empty(s));
                }
                __syncwarp();
                if (T::kShareSP && j + 2 < n) {   // the next scores of this place, once its weights are read
                    if (!(ok = k_there(j + 2) && sm::bar_wait_warp(pv_done(j), turn(j), abort_word, p.status))) break;
                    scores(j + 2);
                }
            }
            if (*abort_word && leader) { sm::mma_commit(drained); sm::bar_drain(drained, 0); }
        }
        __syncwarp();
    } else if (warp < warps) {
        const int row = threadIdx.x;
        const bool live = row < rows;
        const int tok = tok0 + row / p.group, head = g * p.group + row % p.group;
        const int t = causal ? seg.pos0 + tok : seg.key1 - 1;
        const int low = p.window ? max(t - p.window + 1, seg.key0) : seg.key0;
        const int sinks = p.window ? p.sinks : 0;
        const uint32_t lanes = uint32_t(warp * 32) << 16;
        const float c = p.scale_log2;
        // The reference m of a row's weights exp2((s - m) c) need not be the maximum so far: the formats of weights and
        // sums have fp32's exponents.  D < 128: it is the maximum of the first tile in which the row sees a key, and
        // moves only to one more than 2^8 above it (O is rescaled then).  D = 128: it starts at 0, which holds for
        // scores of ordinary size, and no maximum is taken; a tile whose sum of weights exceeds 2^20, or, while none
        // counted, falls below 2^-20, is read again and its maximum becomes the reference.
        float m = 0.f, l = 0.f;
        bool set = false;   // some tile of this row counted
        bool keys = false;  // the row sees a key of this share (its scores may all be -infinity)
        float high = live ? -INFINITY : INFINITY;   // (D < 128) a maximum above it is the new reference
        bool ok = true;     // (a wait that ran out shows at the vote of its tile: until then the lanes stay together)
        const int seen_end = causal ? t0 + 1 : seg.key1;   // keys that every row of the block sees: [seen_low, seen_end), the sinks
        const int seen_low = p.window ? max(t1 - p.window + 1, seg.key0) : seg.key0;
        constexpr int kQ = kKeys / 32;
        uint32_t s[kQ][32];   // scores, then in the low half of each 32 registers their weights
        auto place = [&](int j) { return tmem + lanes + j % T::kPlaces * kKeys; };   // of the scores, at D = 128 of the weights too
        auto load = [&](int j) {
            ok = sm::bar_wait_sync(s_full(j), turn(j), abort_word, p.status) && ok;
            sm::tc_fence_after();
#pragma unroll
            for (int q = 0; q < kQ; ++q) sm::tmem_ld32(place(j) + q * 32, s[q]);
        };
        for (int j = 0; j < n; ++j) {
            const int k0 = range.tile(first + j) * kKeys;
            load(j);
            const uint32_t skip = p.table ? skips[j % T::kFlags] : 0u;
            const bool seen = skip == 0 && k0 + kKeys <= seen_end && (k0 >= seen_low || k0 + kKeys <= sinks);
            keys = keys || seen;
            auto sees = [&](int at) {   // a bit for each of 32 keys from k0 + at: whether this row sees it
                uint32_t see = low_bits(t - k0 - at + 1) & (~low_bits(low - k0 - at) | low_bits(sinks - k0 - at));
                if (skip)
                    for (int i = 0; i < 4; ++i)
                        if (skip >> ((at + 8 * i) >> p.box_log2) & 1u) see &= ~(0xFFu << (8 * i));
                return see;
            };
            float total;
            // the tile's weights, their sum, and (store) the weights to tensor memory from halfway on, where `middle` has
            // waited for the place (a pair of weights takes the place of a pair of scores in registers)
            auto weights = [&](bool store, auto&& middle) {
                const float b = m * c;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int q = 0; q < kQ; ++q) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 x = make_float2(__uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1]));
                        x = fma2(x, make_float2(c, c), make_float2(-b, -b));
                        x = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                        const uint32_t w = pack_bf16(x.x, x.y);
                        if (T::kRoundedSum) x = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
                        sum[i & 1] = add2(sum[i & 1], x);
                        s[q][i] = w;
                    }
                    if (q == 1) middle();
                    if (store && q >= 1) tmem_st16_head(tmem + T::kP + lanes + q * 16, s[q]);
                    if (store && q == 1) tmem_st16_head(tmem + T::kP + lanes, s[0]);
                }
                total = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            };
            auto rescale = [&](float f) {
                l *= f;
#pragma unroll 1
                for (int i = 0; i < D; i += 16) {
                    uint32_t o[16];
                    sm::tmem_ld16(tmem + T::kO + lanes + i, o);
                    sm::tmem_wait_ld(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    sm::tmem_st16(tmem + T::kO + lanes + i, o);
                }
            };
            if constexpr (!T::kShareSP) {
#pragma unroll
                for (int q = 0; q < kQ; ++q) sm::tmem_wait_ld(s[q]);
                sm::tc_fence_before();   // the scores are in registers: the next may come
                __syncwarp();
                if (lane == 0) sm::bar_arrive(s_free);
                if (!seen)
#pragma unroll
                    for (int q = 0; q < kQ; ++q) {
                        const uint32_t see = sees(q * 32);
                        keys = keys || see != 0;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(see >> i & 1u)) s[q][i] = 0xFF800000u;
                    }
                float mx[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint32_t* x = &s[q / 2][q % 2 * 16];
                    mx[q] = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
                    for (int i = 2; i < 16; i += 2) mx[q] = max3(mx[q], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                }
                const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                const bool rise = top > high;
                if (__any_sync(0xFFFFFFFFu, rise || !ok)) {
                    // the products that wrote O are done before it is touched
                    if (j > 0) ok = sm::bar_wait_sync(pv_done(j - 1), turn(j - 1), abort_word, p.status) && ok;
                    sm::tc_fence_after();
                    if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
                    const float f = rise && set ? exp2_approx((m - top) * c) : 1.f;
                    if (rise) { m = top; high = m + 8.f / c; }
                    if (j > 0) rescale(f);
                }
                const bool was_done = j == 0 || sm::bar_test(pv_done(j - 1), turn(j - 1));   // (asked ahead of its use)
                // (halfway through them the products that read the last weights are mostly done: waiting for them before
                // the maximum or behind all weights took 3% and 5% more)
                weights(true, [&] {
                    if (!__all_sync(0xFFFFFFFFu, was_done)) ok = sm::bar_wait_warp(pv_done(j - 1), turn(j - 1), abort_word, p.status);
                    sm::tc_fence_after();
                });
            } else
            for (int pass = 0;; ++pass) {
                if (pass == 1)
#pragma unroll
                    for (int q = 0; q < kQ; ++q) sm::tmem_ld32(place(j) + q * 32, s[q]);
#pragma unroll
                for (int q = 0; q < kQ; ++q) sm::tmem_wait_ld(s[q]);
                if (!seen)
#pragma unroll
                    for (int q = 0; q < kQ; ++q) {
                        const uint32_t see = sees(q * 32);
                        keys = keys || see != 0;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(see >> i & 1u)) s[q][i] = 0xFF800000u;
                    }
                weights(false, [] {});
                const bool off = live && (!(total <= 1048576.f) || (!set && total < 9.5367431640625e-7f));
                if (pass == 1 || !__any_sync(0xFFFFFFFFu, off || !ok)) break;
                if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
                float top = -INFINITY;
#pragma unroll 1
                for (int q = 0; q < kQ; ++q) {
                    uint32_t v[32];
                    sm::tmem_ld32(place(j) + q * 32, v);
                    sm::tmem_wait_ld(v);
                    const uint32_t see = seen ? 0xFFFFFFFFu : sees(q * 32);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (see >> i & 1u) top = fmaxf(top, __uint_as_float(v[i]));
                }
                float f = 1.f;
                if (off && top > -INFINITY && (!set || top > m)) {
                    if (set) f = exp2_approx((m - top) * c);
                    m = top;
                }
                if (j > 0) {   // the products that wrote O are done before it is touched
                    ok = sm::bar_wait_sync(pv_done(j - 1), turn(j - 1), abort_word, p.status);
                    if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
                    sm::tc_fence_after();
                    rescale(f);
                }
            }
            if (!ok) break;
            if (T::kShareSP)
#pragma unroll
                for (int q = 0; q < kQ; ++q) tmem_st16_head(place(j) + q * 16, s[q]);
            set = set || total > 0.f;
            l += total;
            if (!seen && (skip != 0 || !range.whole(k0, kKeys))) {
                // rows of V that no query of the block sees may hold anything, and 0 x NaN is NaN: zero them
                const int vs = j % T::kVStages;
                ok = sm::bar_wait_warp(v_full(vs), uint32_t(j / T::kVStages) & 1u, abort_word, p.status);
                for (int r = threadIdx.x; ok && r < kKeys; r += warps * 32)
                    if (!range.has(k0 + r) || (skip >> (r >> p.box_log2) & 1u))
                        for (int q = 0; q < T::kSubs; ++q)
                            for (int i = 0; i < T::kRowBytes; i += 16)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                    v_at + vs * T::kTileBytes + (q * kKeys + r) * T::kRowBytes + i), "r"(0) : "memory");
                sm::fence_async_smem();
            }
            sm::tmem_wait_st();
            sm::tc_fence_before();
            __syncwarp();
            if (lane == 0) sm::bar_arrive(p_ready(j));
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok && n > 0) ok = sm::bar_wait_warp(pv_done(n - 1), turn(n - 1), abort_word, p.status);
        if (ok) {
            sm::tc_fence_after();
            const bool whole = seg.splits == 1 && !p.prefix_seg;   // no other item adds to this row
            const int64_t at = (int64_t(seg.part0) + int64_t(share) * seg.n + tok) * p.nq + head;
            // a row without a key is zeros; one whose scores hold a NaN, or are all -infinity, is 0 / 0 as the formula has it
            const float inv = 1.f / l;
            if (!whole && live) p.part_ml[at] = make_float2(!keys ? kNoKeys : l == 0.f ? kNoWeight : m * c, l);
#pragma unroll
            for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                if (n > 0) {
                    sm::tmem_ld32(tmem + T::kO + lanes + i, o);
                    sm::tmem_wait_ld(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                if (!live) continue;
                if (whole) {
                    uint4* dst = reinterpret_cast<uint4*>(p.out + (seg.q0 + tok) * p.out_stride + head * D + i);
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float x[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = keys ? __uint_as_float(o[e + k]) * inv : 0.f;
                        dst[e / 8] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
                    }
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(p.part_o + at * D + i);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) dst[e / 4] = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
        }
    }
    sm::tc_fence_before();
    __syncthreads();
    sm::tc_fence_after();
    if (warp == 5) sm::tmem_free(tmem, 256);
}

// Joins the parts of a row: with M = max m, out = sum 2^(m - M) o / sum 2^(m - M) l; parts with l = 0 add nothing.
// l is NaN where a score of the part is, and so is out then.  WARPS warps per row (token,
// head): they load the rows' (m, l), then D / 4 threads a part's o, several parts at a time, and add their sums in a
// fixed order.  A chain of memory latencies: many parts take four warps, which halve it against one, and the first parts' o is
// on its way while the weights are made (one token over 8192 positions, both kernels: 8.8 us, 10.1 with o behind them).
template <int D, int SEGS, int WARPS>
__global__ void __launch_bounds__(128) attend_merge_kernel(const __grid_constant__ AttendParams<SEGS> p) {
    sm::pdl_trigger();
    constexpr int kThreads = WARPS * 32, kLanes = D / 4, kGroups = kThreads / kLanes, kRows = 4 / WARPS;
    constexpr int kMaxParts = 512;   // a sequence's and the prefix's shares, 255 each at most
    __shared__ float weight[kRows][WARPS == 1 ? 64 : kMaxParts];
    __shared__ float4 sums[kRows][kThreads];
    __shared__ float red[kRows][2][WARPS];
    const int r = threadIdx.x / kThreads, t = threadIdx.x % kThreads;
    const int64_t item = int64_t(blockIdx.x) * kRows + r;
    const bool live = item < int64_t(p.merge_tokens) * p.nq;
    const int at_token = live ? int(item / p.nq) : 0, head = live ? int(item % p.nq) : 0;
    int si = p.prefix_seg;
    {
        int lo = p.prefix_seg, hi = p.segs - 1;   // the segment of this token: the last that starts at or before it
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (at_token >= p.seg[mid].merge0) lo = mid;
            else hi = mid - 1;
        }
        si = lo;
    }
    const AttendSeg& seg = p.seg[si];
    const int local = at_token - seg.merge0, tok = seg.q0 + local;
    const int np = p.prefix_seg ? p.seg[0].splits : 0, n = live ? np + seg.splits : 0;
    auto at = [&](int s) {
        const int64_t row = s < np ? int64_t(p.seg[0].part0) + int64_t(s) * p.seg[0].n + tok
                                   : int64_t(seg.part0) + int64_t(s - np) * seg.n + local;
        return row * p.nq + head;
    };
    auto sync = [&]() { if (WARPS == 1) __syncwarp(); else __syncthreads(); };
    const int e = t % kLanes * 4;
    auto part = [&](int s) { return *reinterpret_cast<const float4*>(p.part_o + at(s) * D + e); };
    sm::pdl_wait();
    constexpr int kAhead = 4;   // parts of o on their way while the weights are made
    float4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (t / kLanes + i * kGroups < n) ahead[i] = part(t / kLanes + i * kGroups);
    const float2 own = t < n ? p.part_ml[at(t)] : make_float2(kNoKeys, 0.f);
    float M = own.x;
    for (int s = t + kThreads; s < n; s += kThreads) M = fmaxf(M, p.part_ml[at(s)].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, x));
    if (WARPS > 1) {
        if ((t & 31) == 0) red[r][0][t >> 5] = M;
        sync();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) M = fmaxf(M, red[r][0][w]);
    }
    float L = 0.f;
    for (int s = t; s < n; s += kThreads) {
        const float2 ml = s == t ? own : p.part_ml[at(s)];
        const float w = ml.y != 0.f ? exp2_approx(ml.x - M) : 0.f;   // (a part without a key: its o may hold anything)
        weight[r][s] = w;
        if (ml.y != 0.f) L = fmaf(w, ml.y, L);   // (NaN also where w is 0)
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, x);
    if (WARPS > 1 && (t & 31) == 0) red[r][1][t >> 5] = L;
    sync();
    if (WARPS > 1) {
        L = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) L += red[r][1][w];
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto join = [&](int s, const float4& o) {
        const float w = weight[r][s];
        if (w != 0.f) {
            acc.x = fmaf(w, o.x, acc.x);
            acc.y = fmaf(w, o.y, acc.y);
            acc.z = fmaf(w, o.z, acc.z);
            acc.w = fmaf(w, o.w, acc.w);
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (t / kLanes + i * kGroups < n) join(t / kLanes + i * kGroups, ahead[i]);
#pragma unroll 4
    for (int s = t / kLanes + kAhead * kGroups; s < n; s += kGroups) join(s, part(s));
    sums[r][t] = acc;
    sync();
    if (!live || t >= kLanes) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) {
        const float4 o = sums[r][g * kLanes + t];
        acc.x += o.x; acc.y += o.y; acc.z += o.z; acc.w += o.w;
    }
    const float inv = M > kNoKeys ? 1.f / L : 0.f;
    uint2* dst = reinterpret_cast<uint2*>(p.out + tok * p.out_stride + head * D + e);
    *dst = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

// Checks the arguments that the workspace's size depends on.
static mk_status attend_check_shape(const mk_attend_args* a) {
    if (!a) return fail(MK_ERR_ARG, "null argument");
    if (a->head_dim != 32 && a->head_dim != 64 && a->head_dim != 128)
        return fail(MK_ERR_ARG, "attend: head_dim must be 32, 64 or 128");
    if (a->n_kv_heads < 1 || a->n_q_heads < 1 || a->n_q_heads % a->n_kv_heads || a->n_q_heads / a->n_kv_heads > kMaxHpg ||
        a->n_q_heads > 4096)
        return fail(MK_ERR_ARG, "attend: %d query heads over %d KV heads (a multiple of at most %d)", a->n_q_heads,
                    a->n_kv_heads, kMaxHpg);
    if (a->batch < 1 || a->batch > MK_ATTEND_MAX_BATCH)
        return fail(MK_ERR_ARG, "attend: batch must be in [1, %d]", MK_ATTEND_MAX_BATCH);
    if (!a->q_lens || !a->kv_lens) return fail(MK_ERR_ARG, "attend: null lengths");
    if (a->max_seq < 1 || a->max_seq > (1 << 30) || a->layer < 0 || a->window < 0 || a->sinks < 0 || a->shared_prefix < 0)
        return fail(MK_ERR_ARG, "attend: max_seq must be in [1, 2^30]; layer, window, sinks and shared_prefix not negative");
    if (a->shared_prefix && a->window) return fail(MK_ERR_ARG, "attend: a shared prefix needs window 0");
    if (!(a->scale >= 0.f) || std::isinf(a->scale)) return fail(MK_ERR_ARG, "attend: scale must be finite and not negative");
    int64_t tokens = 0;
    for (int b = 0; b < a->batch; ++b) {
        if (a->q_lens[b] < 0 || a->kv_lens[b] < 0 || a->kv_lens[b] > a->max_seq)
            return fail(MK_ERR_ARG, "attend: sequence %d: %d query tokens, %d positions of %d", b, a->q_lens[b],
                        a->kv_lens[b], a->max_seq);
        if (a->shared_prefix && a->q_lens[b] > 0 && a->shared_prefix > a->kv_lens[b] - a->q_lens[b])
            return fail(MK_ERR_ARG, "attend: sequence %d: its query tokens start inside the shared prefix", b);
        tokens += a->q_lens[b];
    }
    if (tokens > (1 << 24)) return fail(MK_ERR_ARG, "attend: more than 2^24 query tokens");
    if (a->shared_prefix > a->max_seq) return fail(MK_ERR_ARG, "attend: the shared prefix is longer than max_seq");
    return MK_OK;
}

// Positions of a head in the cache, and the elements from one head to the next
static int64_t attend_positions(const mk_attend_args* a) {
    return a->pages ? int64_t(a->pages->n_blocks) * a->pages->block_size : a->max_seq;
}
static int64_t attend_head_stride(const mk_attend_args* a) {
    return a->n_kv_heads > 1 ? a->kv->head_stride : attend_positions(a) * a->head_dim;
}

static mk_status attend_check(const mk_attend_args* a) {
    const mk_status st = attend_check_shape(a);
    if (st != MK_OK) return st;
    int64_t tokens = 0;
    for (int b = 0; b < a->batch; ++b) tokens += a->q_lens[b];
    if (!a->kv || !a->kv->k || !a->kv->v) return fail(MK_ERR_ARG, "attend: null KV cache");
    if (!op_aligned(a->kv->k, 16) || !op_aligned(a->kv->v, 16)) return fail(MK_ERR_ARG, "attend: KV pointers must be 16-byte aligned");
    const int64_t d = a->head_dim, ql = int64_t(a->n_q_heads) * d;
    const mk_kv& kv = *a->kv;
    // (a stride counts where there is a second head, sequence or layer to reach)
    const bool batched = !a->pages && a->batch > 1;
    if ((a->n_kv_heads > 1 && kv.head_stride % 8) || (a->layer > 0 && (kv.layer_stride % 8 || kv.layer_stride < 0)) ||
        (batched && kv.batch_stride % 8))
        return fail(MK_ERR_ARG, "attend: KV strides must be multiples of 8 elements");
    if (a->pages) {
        const mk_kv_pages& pg = *a->pages;
        if (!pg.block_table || !op_aligned(pg.block_table, 4)) return fail(MK_ERR_ARG, "attend: block table null or not 4-byte aligned");
        if (pg.block_size < 8 || pg.block_size % 8 || pg.n_blocks < 1 || pg.max_blocks < 1 ||
            int64_t(pg.n_blocks) * pg.block_size > INT_MAX || int64_t(pg.max_blocks) * pg.block_size < a->max_seq)
            return fail(MK_ERR_ARG, "attend: blocks of a multiple of 8 positions, a table that covers max_seq");
    }
    const int64_t rows = attend_positions(a) * d, heads = attend_head_stride(a) * (a->n_kv_heads - 1) + rows;   // elements of a head, of a layer
    if (attend_head_stride(a) < rows || (batched && kv.batch_stride < heads) || (!a->pages && a->layer > 0 && kv.layer_stride < heads))
        return fail(MK_ERR_ARG, "attend: KV strides must cover a head's positions, its sequence's and its layer's heads");
    if (tokens == 0) return MK_OK;
    if (!a->q || !a->out || !op_aligned(a->q, 16) || !op_aligned(a->out, 16) || !op_aligned(a->status, 4))
        return fail(MK_ERR_ARG, "attend: q and out must be 16-byte aligned");
    if (tokens > 1 && (a->q_stride < ql || a->out_stride < ql || a->q_stride % 8 || a->out_stride % 8))
        return fail(MK_ERR_ARG, "attend: q and out strides must be multiples of 8 and cover the heads");
    const RowSpan out{a->out, tokens, ql * 2, a->out_stride * 2};
    if (spans_overlap(out, {a->q, tokens, ql * 2, a->q_stride * 2})) return fail(MK_ERR_ARG, "attend: out overlaps q");
    const int64_t cached = (a->layer > 0 ? a->layer * kv.layer_stride : 0) + (batched ? (a->batch - 1) * kv.batch_stride : 0) + heads;
    if (spans_overlap(out, {kv.k, 1, cached * 2, 0}) || spans_overlap(out, {kv.v, 1, cached * 2, 0}))
        return fail(MK_ERR_ARG, "attend: out overlaps the cache");
    return MK_OK;
}

// The segments, items and workspace of a call
struct AttendPlan {
    int64_t tokens = 0, items = 0, part_rows = 0;   // part_rows: rows of parts in the workspace
    int64_t merge_tokens = 0;
    int segs = 0, prefix_seg = 0, parts = 0;   // parts: of a row, at most
    AttendSeg seg[MK_ATTEND_MAX_BATCH + 1];
};
static int64_t attend_tiles(const AttendSeg& s, int t0, int t1, int window, int sinks, int kKeys) {   // key tiles of a block (as KeyRange)
    const int64_t end = s.pos0 == kNoCausal ? s.key1 : std::min(t1 + 1, s.key1);
    int64_t low = window ? std::max<int64_t>(int64_t(t0) - window + 1, s.key0) : s.key0;
    int64_t sink = window ? std::min<int64_t>(sinks, end) : 0;
    if (sink >= low) { sink = 0; low = s.key0; }
    const int64_t st = (sink + kKeys - 1) / kKeys;
    return end > low ? st + std::max<int64_t>(0, (end + kKeys - 1) / kKeys - std::max(low / kKeys, st)) : 0;
}
static mk_status attend_plan(const mk_attend_args* a, int sms, AttendPlan& pl) {
    const int group = a->n_q_heads / a->n_kv_heads, bt = kBlockRows / group, keys = attend_keys(a->head_dim);
    const uint32_t slots = 2 * uint32_t(sms);   // (two CTAs to an SM)
    // of each segment: the key tiles of its last block of queries (the most) and of its middle one; blocks by heads
    uint32_t tiles[MK_ATTEND_MAX_BATCH + 1] = {}, middle[MK_ATTEND_MAX_BATCH + 1] = {}, blocks[MK_ATTEND_MAX_BATCH + 1] = {};
    for (int b = 0; b < a->batch; ++b) pl.tokens += a->q_lens[b];
    auto add = [&](const AttendSeg& s) {
        auto seen = [&](int t) {
            const bool causal = s.pos0 != kNoCausal;
            return uint32_t(attend_tiles(s, causal ? s.pos0 + t : 0, causal ? s.pos0 + std::min(t + bt, s.n) - 1 : 0, a->window, a->sinks, keys));
        };
        const int n = (s.n + bt - 1) / bt;
        const uint32_t k = seen((n - 1) * bt);
        int at = pl.segs++;   // longest first, behind the prefix: what starts last is short
        for (; at > pl.prefix_seg && tiles[at - 1] < k; --at) {
            pl.seg[at] = pl.seg[at - 1];
            tiles[at] = tiles[at - 1];
            middle[at] = middle[at - 1];
            blocks[at] = blocks[at - 1];
        }
        pl.seg[at] = s;
        tiles[at] = k;
        middle[at] = std::max(seen(n / 2 * bt < s.n ? n / 2 * bt : 0), (k + 1) / 2);   // (0 with more tokens than positions)
        blocks[at] = uint32_t(n) * uint32_t(a->n_kv_heads);   // (2^24 tokens by 4096 heads at most, 4096 / 8 of them: fits)
    };
    if (a->shared_prefix && pl.tokens) {
        add({0, int32_t(pl.tokens), kNoCausal, 0, a->shared_prefix, 0, 1, 0, 0, 0});
        pl.prefix_seg = 1;
    }
    int64_t q0 = 0, work = 0;
    uint32_t longest = 1;
    for (int b = 0; b < a->batch; ++b) {
        const int n = a->q_lens[b];
        if (n) add({int32_t(q0), n, a->kv_lens[b] - n, a->shared_prefix, a->kv_lens[b], b, 1, 0, 0, 0});
        q0 += n;
    }
    for (int i = 0; i < pl.segs; ++i) {
        work += int64_t(blocks[i]) * middle[i];
        longest = std::max(longest, tiles[i]);
    }
    // A share of the key tiles: the one with the least time, in tiles, by this estimate: an item costs its tiles and
    // kItem more; long items of one length run in whole rounds of `slots`, the others (a causal prompt's blocks, of every
    // length) fill what these leave; joining costs kMerge.  (Eight single tokens with windows of 4096: shares of
    // 8 tiles made 320 items for 304 places and so two rounds, 43 us against 32 with shares of 9.)
    const uint32_t kItem = 256 / keys, kMerge = 384 / keys;
    auto splits = [](uint32_t t, uint32_t share) { return std::min(std::max(1u, (t + share - 1) / share), 255u); };
    auto cost = [&](uint32_t share) {
        uint32_t top = 0, each[MK_ATTEND_MAX_BATCH + 1];
        int64_t all = 0, many = 0;
        bool merge = pl.prefix_seg != 0;
        for (int i = 0; i < pl.segs; ++i) {
            const uint32_t n = splits(tiles[i], share);
            each[i] = (tiles[i] + n - 1) / n + kItem;
            top = std::max(top, each[i]);
            all += int64_t(blocks[i]) * (middle[i] + n * kItem);
            merge = merge || n > 1;
        }
        for (int i = 0; i < pl.segs; ++i)
            if (2 * each[i] > top && 4 * middle[i] > 3 * tiles[i]) many += int64_t(blocks[i]) * splits(tiles[i], share);
        return std::max({(many + slots - 1) / slots * top, (all + slots - 1) / slots, int64_t(top)}) + (merge ? kMerge : 0);
    };
    uint32_t share = longest;
    if (work < int64_t(slots) * longest * 4) {   // (else the blocks alone fill the device for rounds)
        int64_t best = cost(longest);
        for (uint32_t k : {1u, 2u, 4u})
            for (uint32_t s = std::max<uint32_t>(2, uint32_t(work / (slots * k))), end = 2 * s; s <= end && s < longest; s += std::max(1u, s / 4)) {
                const int64_t c = cost(s);
                if (c < best) { best = c; share = s; }
            }
    }
    int64_t part = 0;
    for (int i = 0; i < pl.segs; ++i) {
        AttendSeg& s = pl.seg[i];
        s.splits = int32_t(splits(tiles[i], share));
        s.item0 = int32_t(pl.items);
        s.merge0 = int32_t(pl.merge_tokens);
        pl.items += int64_t(blocks[i]) * s.splits;
        if (s.splits > 1 || pl.prefix_seg) {
            s.part0 = int32_t(part);
            part += int64_t(s.splits) * s.n;
            if (i >= pl.prefix_seg) pl.merge_tokens += s.n;
            pl.parts = std::max(pl.parts, s.splits + (pl.prefix_seg ? pl.seg[0].splits : 0));
        }
        if (pl.items > INT_MAX || part > INT_MAX) return fail(MK_ERR_ARG, "attend: too many query tokens");
    }
    pl.part_rows = part * a->n_q_heads;
    return MK_OK;
}
static size_t attend_bytes(const AttendPlan& pl, int d) {
    return align256(size_t(pl.part_rows) * d * 4) + align256(size_t(pl.part_rows) * 8);
}

template <int D, int SEGS>
static mk_status attend_launch(const mk_attend_args* a, const AttendCommon& common, const AttendPlan& pl, int device, cudaStream_t stream) {
    using T = AttendTile<D>;
    static std::atomic<uint64_t> set{0};
    mk_status st = op_smem(reinterpret_cast<const void*>(&attend_kernel<D, SEGS>), T::kSmem, device, &set);
    if (st != MK_OK) return st;
    AttendParams<SEGS> p;
    static_cast<AttendCommon&>(p) = common;
    for (int i = 0; i < pl.segs; ++i) p.seg[i] = pl.seg[i];
    const mk_kv& kv = *a->kv;
    CUtensorMap mq, mk_, mv;
    const int64_t qs = pl.tokens == 1 ? int64_t(p.nq) * D : a->q_stride;
    const cuuint64_t qd[3] = {cuuint64_t(D), cuuint64_t(p.nq), cuuint64_t(pl.tokens)}, qst[2] = {cuuint64_t(D) * 2, cuuint64_t(qs) * 2};
    const cuuint32_t qb[3] = {T::kSub, cuuint32_t(p.group), cuuint32_t(p.block_tokens)};
    const int64_t seqs = a->pages ? 1 : a->batch, hs = attend_head_stride(a), bs = seqs > 1 ? kv.batch_stride : hs;
    const cuuint64_t kd[4] = {cuuint64_t(D), cuuint64_t(attend_positions(a)), cuuint64_t(p.nkv), cuuint64_t(seqs)};
    const cuuint64_t kst[3] = {cuuint64_t(D) * 2, cuuint64_t(hs) * 2, cuuint64_t(bs) * 2};
    const cuuint32_t kb[4] = {T::kSub, cuuint32_t(p.table ? 1 << p.box_log2 : T::kKeys), 1, 1};
    const int64_t off = int64_t(a->layer) * kv.layer_stride;
    if ((st = op_tensor_map(&mq, a->q, 3, qd, qst, qb)) != MK_OK) return st;
    if ((st = op_tensor_map(&mk_, static_cast<const uint16_t*>(kv.k) + off, 4, kd, kst, kb)) != MK_OK) return st;
    if ((st = op_tensor_map(&mv, static_cast<const uint16_t*>(kv.v) + off, 4, kd, kst, kb)) != MK_OK) return st;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(unsigned(pl.items));
    cfg.blockDim = dim3(192);
    cfg.dynamicSmemBytes = T::kSmem;
    MK_CK(cudaLaunchKernelEx(&cfg, &attend_kernel<D, SEGS>, mq, mk_, mv, p));
    if (pl.merge_tokens) {
        const int64_t rows = pl.merge_tokens * p.nq;
        const bool wide = pl.parts > 8;
        if ((wide ? rows : (rows + 3) / 4) > INT_MAX) return fail(MK_ERR_ARG, "attend: too many query tokens");
        cfg.gridDim = dim3(unsigned(wide ? rows : (rows + 3) / 4));
        cfg.blockDim = dim3(128);
        cfg.dynamicSmemBytes = 0;
        MK_CK(wide ? cudaLaunchKernelEx(&cfg, &attend_merge_kernel<D, SEGS, 4>, p) : cudaLaunchKernelEx(&cfg, &attend_merge_kernel<D, SEGS, 1>, p));
    }
    return MK_OK;
}
template <int D>
static mk_status attend_launch_segs(const mk_attend_args* a, const AttendCommon& c, const AttendPlan& pl, int device, cudaStream_t stream) {
    return pl.segs <= 16 ? attend_launch<D, 16>(a, c, pl, device, stream)
                         : attend_launch<D, MK_ATTEND_MAX_BATCH + 1>(a, c, pl, device, stream);
}

}  // namespace mk

using namespace mk;

mk_status mk::mk_attend_plan(const mk_attend_args* a, size_t* workspace_bytes) {
    *workspace_bytes = 0;
    mk_status st = attend_check_shape(a);
    if (st != MK_OK) return st;
    bool any = false;
    for (int b = 0; b < a->batch; ++b) any = any || a->q_lens[b] > 0;
    if (!any) return MK_OK;
    int device = 0, sms = 0;
    AttendPlan pl;
    if ((st = op_device(&device, &sms)) != MK_OK || (st = attend_plan(a, sms, pl)) != MK_OK) return st;
    *workspace_bytes = attend_bytes(pl, a->head_dim);
    return MK_OK;
}

extern "C" size_t mk_attend_workspace(const mk_attend_args* a) {
    size_t bytes = 0;
    return mk_attend_plan(a, &bytes) == MK_OK ? bytes : 0;
}

extern "C" mk_status mk_attend(const mk_attend_args* a, void* workspace, size_t workspace_bytes, void* stream) {
    mk_status st = attend_check(a);
    if (st != MK_OK) return st;
    bool any = false;
    for (int b = 0; b < a->batch; ++b) any = any || a->q_lens[b] > 0;
    if (!any) return MK_OK;
    int device = 0, sms = 0;
    AttendPlan pl;
    if ((st = op_device(&device, &sms)) != MK_OK || (st = attend_plan(a, sms, pl)) != MK_OK) return st;
    const size_t need = attend_bytes(pl, a->head_dim);
    if (need > 0 && (!workspace || !op_aligned(workspace, 256))) return fail(MK_ERR_ARG, "attend: workspace null or not 256-byte aligned");
    if (need > workspace_bytes)
        return fail(MK_ERR_CAPACITY, "attend: workspace of %zu bytes, %zu needed (mk_attend_workspace)", workspace_bytes, need);
    AttendCommon p{};
    p.nq = a->n_q_heads; p.nkv = a->n_kv_heads; p.group = p.nq / p.nkv; p.block_tokens = kBlockRows / p.group;
    p.segs = pl.segs; p.prefix_seg = pl.prefix_seg; p.merge_tokens = int32_t(pl.merge_tokens);
    p.window = std::min(a->window, 1 << 30); p.sinks = std::min(a->sinks, 1 << 30);   // (positions stay below 2^30)
    p.scale_log2 = float((a->scale != 0.f ? double(a->scale) : 1.0 / std::sqrt(double(a->head_dim))) * 1.4426950408889634);
    if (a->pages) {
        p.table = a->pages->block_table; p.block = a->pages->block_size;
        p.max_blocks = a->pages->max_blocks; p.n_blocks = a->pages->n_blocks;
        p.block_shift = 30;
        while ((int64_t(1) << (p.block_shift - 30)) < p.block) ++p.block_shift;
        p.block_inv = uint32_t(((uint64_t(1) << p.block_shift) + uint32_t(p.block) - 1) / uint32_t(p.block));
        p.box_log2 = 3;
        while ((1 << p.box_log2) < attend_keys(a->head_dim) && p.block % (2 << p.box_log2) == 0) ++p.box_log2;
    }
    p.out = static_cast<__nv_bfloat16*>(a->out);
    p.out_stride = a->out_stride;
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + align256(size_t(pl.part_rows) * a->head_dim * 4));
    p.status = a->status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->head_dim == 32) return attend_launch_segs<32>(a, p, pl, device, s);
    if (a->head_dim == 64) return attend_launch_segs<64>(a, p, pl, device, s);
    return attend_launch_segs<128>(a, p, pl, device, s);
}
