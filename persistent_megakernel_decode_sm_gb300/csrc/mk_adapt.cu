// The linear map with low-rank adapters of many requests (mk_linear_adapted): the low-rank rows t = scale x down^T of every
// token with its own adapter, then the linear map with the adapters' part as a longer contraction (mk_linear.cuh).
#include <algorithm>

#include "mk_linear.cuh"

namespace mk {

constexpr int kLowThreads = 256, kLowTokens = 16, kLowWarps = kLowThreads / 32;
constexpr int kLowTile = 256;       // most tokens of a tile of the linear map
constexpr int kLowFew = 512;        // tokens that are few: the work is in their adapters' rows, not in theirs

struct LowParams {
    int rows, k, rank, n_adapters;
    int tile, subs;                 // tokens of a tile of the linear map, blocks of kLowTokens tokens in it
    int slots, width, f32;          // as LinearExtra; whether the output is fp32: three parts
    const __nv_bfloat16* x;
    int64_t x_stride;
    const __nv_bfloat16* down;
    const float* scale;
    const int32_t* index;
    int32_t* count;
    int32_t* list;
    __nv_bfloat16* terms;           // [rows][parts][part columns]
    int64_t part;
    int32_t* status;
};

// Two low-rank values' next bf16 part, and what it leaves.  A part that is not the last stays finite: a value that would round to
// an infinity takes bf16's largest, and so do infinities and NaN, which are then in every rest and become the last part.
__device__ __forceinline__ __nv_bfloat162 low_part(float (&v)[2], bool last) {
    constexpr float kMost = 3.3895313892515355e38f;   // (2 - 2^-7) 2^127
    __nv_bfloat162 h;
    h.x = __float2bfloat16_rn(last ? v[0] : fminf(fmaxf(v[0], -kMost), kMost));
    h.y = __float2bfloat16_rn(last ? v[1] : fminf(fmaxf(v[1], -kMost), kMost));
    v[0] -= __bfloat162float(h.x);
    v[1] -= __bfloat162float(h.y);
    return h;
}

// A cluster works on 16 neighbouring tokens of one tile of the linear map, for the tile's adapters y, y + gridDim.y, ..: those of
// its tokens that name the adapter get their low-rank row, the others zeros.  8 NT columns of the rank at a time; x and down are
// read from global memory straight into the operands of m16n8k16 products (a thread's 16 bytes of a row are the elements 2 i, 2 i + 1
// of two products: the contraction may take its elements in any order as long as both operands do), only rows that count.  The
// contraction is shared out over the warps and the CTAs of the cluster in blocks of 32; the sums meet in shared memory, in a
// fixed order, once for all columns of the rank.
// These products need no more than the reading of x and down does (they are 1/8 to 1/100 of the linear map's), so they stay on
// mma.sync, with registers for operands and no staging.
template <int NT>
__global__ void __launch_bounds__(kLowThreads, 2) low_rank_kernel(const __grid_constant__ LowParams p) {
    constexpr int kCols = 8 * NT;
    extern __shared__ float all_sums[];                 // [2][16][width], in turn for the adapters
    __shared__ __align__(16) int name[kLowTile];
    __shared__ int list[kLowTile], warp_heads[kLowWarps];
    __shared__ float part[kLowWarps][16][kCols];
    // every kernel before this one is done when the next one may start: it reads x beside this one
    sm::pdl_wait();
    sm::pdl_trigger();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int split = int(gridDim.z), rank_z = int(blockIdx.z);
    const int m = int(blockIdx.x) / p.subs, sub = int(blockIdx.x) % p.subs, m0 = m * p.tile, tokens = min(p.tile, p.rows - m0);
    // the tile's adapters in the order in which its tokens name them
#pragma unroll
    for (int i = t; i < kLowTile; i += kLowThreads) {
        int mine = -1;
        if (i < tokens) {
            mine = p.index[m0 + i];
            if (mine >= p.n_adapters) {
                if (p.status) *p.status = MK_ERR_BOUNDS;
                mine = -1;
            }
        }
        name[i] = mine;
    }
    __syncthreads();
    int count = 0;
    for (int from = 0; from < tokens; from += kLowThreads) {
        const int i = from + t, mine = i < tokens ? name[i] : -1;
        bool head = mine >= 0 && (i == 0 || name[i - 1] != mine);
        if (head) {
            bool seen = false;   // (four names a step, no step waiting for another)
#pragma unroll 4
            for (int j = 0; j < i; j += 4) {
                const int4 n = *reinterpret_cast<const int4*>(name + j);
                seen = seen || n.x == mine || (j + 1 < i && n.y == mine) || (j + 2 < i && n.z == mine) || (j + 3 < i && n.w == mine);
            }
            head = !seen;
        }
        const uint32_t heads = __ballot_sync(0xFFFFFFFFu, head);
        if (lane == 0) warp_heads[warp] = __popc(heads);
        __syncthreads();
        int before = count + __popc(heads & ((1u << lane) - 1));
#pragma unroll
        for (int w = 0; w < kLowWarps; ++w) {
            if (w < warp) before += warp_heads[w];
            count += warp_heads[w];
        }
        if (head) list[before] = mine;
        __syncthreads();
    }
    if (sub == 0 && blockIdx.y == 0 && rank_z == 0) {
        if (t == 0) p.count[m] = count;
        for (int i = t; i < count; i += kLowThreads) p.list[int64_t(m) * p.slots + i] = list[i];
    }

    const int row0 = sub * kLowTokens;                  // in the tile
    if (row0 >= tokens) return;                         // (all CTAs of the cluster)
    const int g = lane >> 2, q = lane & 3;              // a product's row, and its quarter of 32 elements
    const int blocks = (p.k + 31) / 32, width = p.width;
    const __nv_bfloat16* x0 = p.x + int64_t(m0 + row0 + g) * p.x_stride + q * 8;
    float* sums = all_sums;
    // A warp's blocks in turn, from another one on in every cluster: neighbours mostly share an adapter, and with all of them at the same
    // rows of down at the same time these come from few places of the L2
    const int mine = max(0, (blocks - rank_z * kLowWarps - warp + split * kLowWarps - 1) / (split * kLowWarps));
    const int first = mine > 0 ? int(blockIdx.x + blockIdx.y) % mine : 0;
    bool reached = false;                               // whether a peer may still read this CTA's sums
    for (int slot = int(blockIdx.y); slot < count; slot += int(gridDim.y)) {
        const int adapter = list[slot];
        const bool use[2] = {name[row0 + g] == adapter, name[row0 + 8 + g] == adapter};   // (names behind the last token are -1)
        const bool any = __any_sync(0xFFFFFFFFu, use[0] || use[1]);                       // (every warp looks at every token)
        if (any) {
            const __nv_bfloat16* down0 = p.down + (int64_t(adapter) * p.rank + g) * p.k + q * 8;
            for (int c0 = 0; c0 < width; c0 += kCols) {
                const __nv_bfloat16* down = down0 + int64_t(c0) * p.k;
                float acc[NT][4];
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[j][v] = 0.f;
#pragma unroll NT == 8 ? 2 : 4
                for (int i = 0; i < mine; ++i) {
                    const int turn = i + first < mine ? i + first : i + first - mine, b = rank_z * kLowWarps + warp + turn * split * kLowWarps;
                    const bool in = b * 32 + q * 8 < p.k;
                    uint4 xs[2], ds[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) ds[j] = linear_load(down + int64_t(8 * j) * p.k + b * 32, in && c0 + 8 * j + g < p.rank);
#pragma unroll
                    for (int h = 0; h < 2; ++h) xs[h] = linear_load(x0 + 8 * h * p.x_stride + b * 32, in && use[h]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        linear_mma(acc[j], xs[0].x, xs[1].x, xs[0].y, xs[1].y, ds[j].x, ds[j].y);
                        linear_mma(acc[j], xs[0].z, xs[1].z, xs[0].w, xs[1].w, ds[j].z, ds[j].w);
                    }
                }
                __syncthreads();                        // (the warps' sums of the columns before are read)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<float2*>(&part[warp][g + 8 * h][8 * j + 2 * q]) = make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
                __syncthreads();
                for (int e = t; e < 16 * kCols; e += kLowThreads) {
                    float s = 0.f;
#pragma unroll
                    for (int w = 0; w < kLowWarps; ++w) s += part[w][e / kCols][e % kCols];
                    if (c0 + e % kCols < width) sums[e / kCols * width + c0 + e % kCols] = s;
                }
            }
            __syncwarp();
            if (split > 1) sm::cluster_sync();
            else __syncthreads();
            reached = true;
        }
        // the cluster's CTAs share out the pairs of columns
        const float scale = any && p.scale ? p.scale[adapter] : 1.f;
        for (int e = rank_z * kLowThreads + t; e < kLowTokens * width / 2; e += split * kLowThreads) {
            const int r = 2 * e / width, c = 2 * e - r * width;
            if (row0 + r >= tokens) break;
            float v[2] = {0.f, 0.f};
            if (any && name[row0 + r] == adapter && c < p.rank) {   // (columns behind the rank stay zero whatever x and the scale are)
                const uint32_t src = sm::smem(sums + r * width + c);
                float2 got[8];   // (of all CTAs together: their way takes longer than everything else here)
#pragma unroll
                for (int z = 0; z < 8; ++z) got[z] = z < split ? sm::cluster_ld2(sm::cluster_addr(src, uint32_t(z))) : make_float2(0.f, 0.f);
#pragma unroll
                for (int z = 0; z < 8; ++z) {
                    v[0] += got[z].x;
                    v[1] += got[z].y;
                }
                v[0] *= scale;
                v[1] *= scale;
            }
            __nv_bfloat16* dst = p.terms + int64_t(m0 + row0 + r) * (p.f32 ? 3 : 2) * p.part + slot * width + c;
            *reinterpret_cast<__nv_bfloat162*>(dst) = low_part(v, false);
            if (p.f32) *reinterpret_cast<__nv_bfloat162*>(dst += p.part) = low_part(v, false);
            *reinterpret_cast<__nv_bfloat162*>(dst + p.part) = low_part(v, true);
        }
        // the next adapter's sums go to the other half; they are in this one again when every CTA has passed the next barrier
        if (any) sums = sums == all_sums ? all_sums + 16 * width : all_sums;
    }
    __syncwarp();
    if (split > 1 && reached) sm::cluster_sync();
}

// A call is made in pieces of rows whose terms fit this; each at least a tile
constexpr int64_t kAdaptTermsBytes = 256ll << 20;

struct AdaptPlan {
    LinearChoice<true> choice;
    int slots, width, tiles;        // of a piece
    int64_t rows, part;             // tokens of a piece, columns of a part of their terms
    size_t list, terms, bytes;      // offsets of what lies behind the counts; all
};

static mk_status adapt_check(const mk_linear_args* a, const mk_adapters* ad, bool pointers) {
    if (!a || !ad) return fail(MK_ERR_ARG, "null argument");
    if (ad->n_adapters < 1 || ad->n_adapters > 65536) return fail(MK_ERR_ARG, "linear_adapted: %d adapters (1 to 65536)", ad->n_adapters);
    if (ad->rank < 8 || ad->rank > MK_ADAPTERS_MAX_RANK || ad->rank % 8)
        return fail(MK_ERR_ARG, "linear_adapted: rank %d (a multiple of 8, at most %d)", ad->rank, MK_ADAPTERS_MAX_RANK);
    if (!pointers) return MK_OK;
    if (!ad->down || !ad->up || !ad->index) return fail(MK_ERR_ARG, "linear_adapted: null pointer");
    if (!op_aligned(ad->down, 16) || !op_aligned(ad->up, 16) || !op_aligned(ad->scale, 4) || !op_aligned(ad->index, 4))
        return fail(MK_ERR_ARG, "linear_adapted: down and up must be 16-byte aligned, scale and index 4-byte aligned");
    const int64_t os = a->out_dtype == MK_F32 ? 4 : 2, f = a->activation == MK_ACT_SWIGLU ? 2 : 1;
    const RowSpan out{a->out, a->rows, a->n * os, a->out_stride * os};
    const int64_t per = int64_t(ad->n_adapters) * ad->rank * 2;
    if (spans_overlap(out, {ad->down, 1, per * a->k, 0}) || spans_overlap(out, {ad->up, 1, per * f * a->n, 0}) ||
        spans_overlap(out, {ad->scale, 1, int64_t(ad->n_adapters) * 4, 0}) || spans_overlap(out, {ad->index, 1, int64_t(a->rows) * 4, 0}))
        return fail(MK_ERR_ARG, "linear_adapted: out overlaps an input");
    return MK_OK;
}

static mk_status adapt_plan(const mk_linear_args* a, const mk_adapters* ad, AdaptPlan& pl) {
    LinearParams p{};
    const bool f32 = a->out_dtype == MK_F32;
    pl.width = ad->rank <= 16 ? 16 : ad->rank <= 32 ? 32 : (ad->rank + kAdaptCols - 1) / kAdaptCols * kAdaptCols;
    const mk_status st = linear_plan(a, LinearNamed{ad->n_adapters, pl.width}, p, pl.choice);
    if (st != MK_OK) return st;
    const int tile = pl.choice.tokens;
    pl.slots = std::min({tile, ad->n_adapters, a->rows});
    pl.part = (int64_t(pl.slots) * pl.width + kAdaptCols - 1) / kAdaptCols * kAdaptCols;
    const int64_t all = (int64_t(a->rows) + tile - 1) / tile, row = pl.part * (f32 ? 3 : 2) * 2;   // bytes of a token's terms
    pl.tiles = int(std::min(all, std::max<int64_t>(1, kAdaptTermsBytes / (row * tile))));
    pl.rows = std::min<int64_t>(a->rows, int64_t(pl.tiles) * tile);
    pl.list = align256(size_t(pl.tiles) * 4);
    pl.terms = pl.list + align256(size_t(pl.tiles) * size_t(pl.slots) * 4);
    pl.bytes = pl.terms + align256(size_t(pl.rows * row));
    return MK_OK;
}

template <int NT>
static mk_status low_launch(LowParams& p, int device, int sms, cudaStream_t stream) {
    static std::atomic<uint64_t> set{0};
    const mk_status st = op_smem(reinterpret_cast<const void*>(&low_rank_kernel<NT>), 2 * kLowTokens * MK_ADAPTERS_MAX_RANK * 4, device, &set);
    if (st != MK_OK) return st;
    p.subs = (p.tile + kLowTokens - 1) / kLowTokens;
    const int64_t subs = int64_t((p.rows + p.tile - 1) / p.tile) * p.subs;
    // Adapters of a tile side by side where there are few tokens, then the contraction over clusters of 2, 4 or 8 while two CTAs an SM
    // (what is resident) are not exceeded and each warp keeps a block of 32.  64 tokens with an adapter of rank 64 each (4096 x 6144): the
    // whole call 45.6 us, with at most one CTA an SM 16% more, with four, which come in rounds, 14%
    const int lanes = p.rows <= kLowFew ? std::min({p.slots, 16}) : 1;
    int split = 1;
    while (split < 8 && 2 * subs * lanes * split <= 2 * sms && 2 * split * kLowWarps * 32 <= p.k) split *= 2;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = unsigned(split);
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(unsigned(subs), unsigned(lanes), unsigned(split));
    cfg.blockDim = dim3(kLowThreads);
    cfg.dynamicSmemBytes = size_t(2 * kLowTokens * p.width) * 4;
    MK_CK(cudaLaunchKernelEx(&cfg, &low_rank_kernel<NT>, p));
    return MK_OK;
}

}  // namespace mk

using namespace mk;

extern "C" size_t mk_linear_adapted_workspace(const mk_linear_args* a, const mk_adapters* ad) {
    AdaptPlan pl{};
    if (linear_check_shape(a) != MK_OK || adapt_check(a, ad, false) != MK_OK || a->rows == 0 || adapt_plan(a, ad, pl) != MK_OK) return 0;
    return pl.bytes;
}

extern "C" mk_status mk_linear_adapted(const mk_linear_args* a, const mk_adapters* ad, void* workspace, size_t workspace_bytes,
                                       void* stream) {
    mk_status st = linear_check(a);
    if (st != MK_OK || (st = adapt_check(a, ad, a && a->rows > 0)) != MK_OK || a->rows == 0) return st;
    AdaptPlan pl{};
    int device = 0, sms = 0;
    if ((st = op_device(&device, &sms)) != MK_OK || (st = adapt_plan(a, ad, pl)) != MK_OK) return st;
    if (!workspace || !op_aligned(workspace, 256)) return fail(MK_ERR_ARG, "linear_adapted: workspace null or not 256-byte aligned");
    if (workspace_bytes < pl.bytes)
        return fail(MK_ERR_CAPACITY, "linear_adapted: workspace of %zu bytes, %zu needed (mk_linear_adapted_workspace)", workspace_bytes, pl.bytes);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f32 = a->out_dtype == MK_F32;
    for (int64_t r0 = 0; r0 < a->rows; r0 += pl.rows) {
        mk_linear_args c = *a;   // this piece's rows
        c.rows = int32_t(std::min<int64_t>(pl.rows, a->rows - r0));
        c.x = static_cast<const uint16_t*>(a->x) + r0 * a->x_stride;
        c.out = static_cast<uint8_t*>(a->out) + r0 * a->out_stride * (f32 ? 4 : 2);
        if (a->residual) c.residual = static_cast<const uint8_t*>(a->residual) + r0 * a->residual_stride * (a->residual_dtype == MK_F32 ? 4 : 2);
        LowParams low{};
        low.rows = c.rows; low.k = c.k; low.rank = ad->rank; low.n_adapters = ad->n_adapters;
        low.tile = pl.choice.tokens; low.slots = pl.slots; low.width = pl.width; low.f32 = f32;
        low.x = static_cast<const __nv_bfloat16*>(c.x);
        low.x_stride = c.rows == 1 ? c.k : c.x_stride;
        low.down = static_cast<const __nv_bfloat16*>(ad->down);
        low.scale = ad->scale;
        low.index = ad->index + r0;
        low.count = reinterpret_cast<int32_t*>(ws);
        low.list = reinterpret_cast<int32_t*>(ws + pl.list);
        low.terms = reinterpret_cast<__nv_bfloat16*>(ws + pl.terms);
        low.part = pl.part;
        low.status = a->status;
        if ((st = pl.width > 32 && c.rows <= kLowFew ? low_launch<8>(low, device, sms, s)
                  : pl.width > 16 ? low_launch<4>(low, device, sms, s)
                                  : low_launch<2>(low, device, sms, s)) != MK_OK) return st;
        LinearExtra<true> e{};
        e.index = low.index;
        e.n_adapters = ad->n_adapters;
        e.rank = ad->rank;
        e.x = low.x;
        e.x_stride = low.x_stride;
        e.w = static_cast<const __nv_bfloat16*>(c.w);
        e.up_rows = static_cast<const __nv_bfloat16*>(ad->up);
        e.term_rows = low.terms;
        e.count = low.count;
        e.list = low.list;
        e.slots = pl.slots;
        e.width = pl.width;
        e.part = int32_t(pl.part);
        const int64_t w_rows = int64_t(c.n) * (c.activation == MK_ACT_SWIGLU ? 2 : 1);
        const cuuint64_t ud[3] = {cuuint64_t(ad->rank), cuuint64_t(w_rows), cuuint64_t(ad->n_adapters)};
        const cuuint64_t us[2] = {cuuint64_t(ad->rank) * 2, cuuint64_t(w_rows) * cuuint64_t(ad->rank) * 2};
        const bool pair = pl.choice.unit == 2;
        const int block = pair ? kPairCols : kAdaptCols;
        const cuuint32_t ub[3] = {cuuint32_t(std::min(pl.width, block)), cuuint32_t(pair ? pl.choice.features / 2 : 128), 1};
        if ((st = op_tensor_map(&e.up, ad->up, 3, ud, us, ub)) != MK_OK) return st;
        const cuuint32_t tile = cuuint32_t(pair ? 128 : pl.choice.tokens);
        const cuuint64_t cols = cuuint64_t(pl.part) * (f32 ? 3 : 2), td[2] = {cols, cuuint64_t(c.rows)}, ts[1] = {cols * 2};
        const cuuint32_t tb[2] = {cuuint32_t(block), tile};
        if ((st = op_tensor_map(&e.terms, low.terms, 2, td, ts, tb)) != MK_OK) return st;
        // (the piece's own tiles: pieces are whole tiles but for the last)
        LinearParams p{};
        LinearPlan plan = pl.choice.plan;
        p.rows = c.rows; p.n = c.n; p.k = c.k; p.act = c.activation;
        p.bias = static_cast<const __nv_bfloat16*>(c.bias);
        p.residual = c.residual; p.residual_stride = c.residual_stride; p.residual_f32 = c.residual_dtype == MK_F32;
        p.out_f32 = f32; p.out = c.out; p.out_stride = c.out_stride; p.status = c.status;
        plan.tiles_m = (c.rows + pl.choice.tokens - 1) / pl.choice.tokens;
        const int64_t tiles = int64_t(plan.tiles_n) * plan.tiles_m;
        plan.clusters = plan.split > 1 ? tiles : std::min(tiles, plan.clusters);
        if ((st = pl.choice.launch(&c, p, e, plan, s)) != MK_OK) return st;
    }
    return MK_OK;
}
