// Attention of query tokens over one layer of the decode KV cache (mk_attend): causal, an optional
// sliding window with sinks, an optional prefix shared by the batch.
#include "mk_ops.h"

#include <cuda_bf16.h>

#include <climits>
#include <cmath>

namespace mk {

struct AttendSeq {
    int32_t q0, n, len, pad;   // first query token, query tokens, positions
};

struct AttendParams {
    int nq, nkv, group, d, batch, tokens;
    const __nv_bfloat16* q;
    int64_t q_stride;
    __nv_bfloat16* out;
    int64_t out_stride;
    const __nv_bfloat16* k;   // the layer's cache
    const __nv_bfloat16* v;
    int64_t batch_stride, head_stride;
    const int32_t* table;     // paged: [batch][max_blocks]
    int block, max_blocks, n_blocks;
    int window, sinks, prefix;
    float scale;
    int32_t* status;
    AttendSeq seq[MK_ATTEND_MAX_BATCH];
};

// One warp per (token, head): one pass over the visible positions with a running maximum and sum.
__global__ void __launch_bounds__(128) attend_simple_kernel(const __grid_constant__ AttendParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t item = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (item >= int64_t(p.tokens) * p.nq) return;
    const int tok = int(item / p.nq), h = int(item % p.nq), g = h / p.group;
    int b = 0;
    while (tok >= p.seq[b].q0 + p.seq[b].n) ++b;
    const int t = p.seq[b].len - p.seq[b].n + (tok - p.seq[b].q0);
    const int e = p.d / 32;
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    const __nv_bfloat16* qr = p.q + tok * p.q_stride + int64_t(h) * p.d + lane * e;
    for (int i = 0; i < 4; ++i) q[i] = i < e ? __bfloat162float(qr[i]) * p.scale : 0.f;
    for (int pos = 0; pos <= t; ++pos) {
        if (p.window && pos >= p.sinks) pos = max(pos, t - p.window + 1);
        const int sb = pos < p.prefix ? 0 : b;
        int64_t at;
        if (p.table) {
            const int blk = p.table[int64_t(sb) * p.max_blocks + pos / p.block];
            if (unsigned(blk) >= unsigned(p.n_blocks)) {
                if (p.status && lane == 0) *p.status = MK_ERR_BOUNDS;
                continue;
            }
            at = g * p.head_stride + (int64_t(blk) * p.block + pos % p.block) * p.d;
        } else {
            at = sb * p.batch_stride + g * p.head_stride + int64_t(pos) * p.d;
        }
        float s = 0.f;
        for (int i = 0; i < e; ++i) s = fmaf(q[i], __bfloat162float(p.k[at + lane * e + i]), s);
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
        const float mn = fmaxf(m, s), c = expf(m - mn), w = expf(s - mn);
        l = l * c + w;
        for (int i = 0; i < e; ++i) o[i] = o[i] * c + w * __bfloat162float(p.v[at + lane * e + i]);
        m = mn;
    }
    __nv_bfloat16* orow = p.out + tok * p.out_stride + int64_t(h) * p.d + lane * e;
    for (int i = 0; i < e; ++i) orow[i] = __float2bfloat16_rn(l > 0.f ? o[i] / l : 0.f);
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
    if (a->max_seq < 1 || a->layer < 0 || a->window < 0 || a->sinks < 0 || a->shared_prefix < 0)
        return fail(MK_ERR_ARG, "attend: max_seq must be positive; layer, window, sinks and shared_prefix not negative");
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

static mk_status attend_check(const mk_attend_args* a) {
    const mk_status st = attend_check_shape(a);
    if (st != MK_OK) return st;
    int64_t tokens = 0;
    for (int b = 0; b < a->batch; ++b) tokens += a->q_lens[b];
    if (!a->kv || !a->kv->k || !a->kv->v) return fail(MK_ERR_ARG, "attend: null KV cache");
    if (!op_aligned(a->kv->k, 16) || !op_aligned(a->kv->v, 16)) return fail(MK_ERR_ARG, "attend: KV pointers must be 16-byte aligned");
    const int64_t d = a->head_dim, ql = int64_t(a->n_q_heads) * d;
    const mk_kv& kv = *a->kv;
    if (kv.head_stride % 8 || kv.layer_stride % 8 || kv.batch_stride % 8 || kv.layer_stride < 0)
        return fail(MK_ERR_ARG, "attend: KV strides must be multiples of 8 elements");
    if (a->pages) {
        const mk_kv_pages& pg = *a->pages;
        if (!pg.block_table || !op_aligned(pg.block_table, 4)) return fail(MK_ERR_ARG, "attend: block table null or not 4-byte aligned");
        if (pg.block_size < 8 || pg.block_size % 8 || pg.n_blocks < 1 || pg.max_blocks < 1 ||
            int64_t(pg.n_blocks) * pg.block_size > INT_MAX || int64_t(pg.max_blocks) * pg.block_size < a->max_seq)
            return fail(MK_ERR_ARG, "attend: blocks of a multiple of 8 positions, a table that covers max_seq");
        if (kv.head_stride < int64_t(pg.n_blocks) * pg.block_size * d)
            return fail(MK_ERR_ARG, "attend: KV strides must cover the pool per head");
    } else if (kv.head_stride < a->max_seq * d || (a->batch > 1 && kv.batch_stride < kv.head_stride * a->n_kv_heads)) {
        return fail(MK_ERR_ARG, "attend: KV strides must cover [max_seq, head_dim] per head");
    }
    if (tokens == 0) return MK_OK;
    if (!a->q || !a->out || !op_aligned(a->q, 16) || !op_aligned(a->out, 16) || !op_aligned(a->status, 4))
        return fail(MK_ERR_ARG, "attend: q and out must be 16-byte aligned");
    if (tokens > 1 && (a->q_stride < ql || a->out_stride < ql || a->q_stride % 8 || a->out_stride % 8))
        return fail(MK_ERR_ARG, "attend: q and out strides must be multiples of 8 and cover the heads");
    if (spans_overlap({a->out, tokens, ql * 2, a->out_stride * 2}, {a->q, tokens, ql * 2, a->q_stride * 2}))
        return fail(MK_ERR_ARG, "attend: out overlaps q");
    return MK_OK;
}

}  // namespace mk

using namespace mk;

extern "C" size_t mk_attend_workspace(const mk_attend_args* a) {
    if (attend_check_shape(a) != MK_OK) return 0;
    return 0;
}

extern "C" mk_status mk_attend(const mk_attend_args* a, void* workspace, size_t workspace_bytes, void* stream) {
    const mk_status st = attend_check(a);
    if (st != MK_OK) return st;
    (void)workspace; (void)workspace_bytes;
    AttendParams p{};
    p.nq = a->n_q_heads; p.nkv = a->n_kv_heads; p.group = p.nq / p.nkv; p.d = a->head_dim; p.batch = a->batch;
    for (int b = 0; b < a->batch; ++b) {
        p.seq[b] = {p.tokens, a->q_lens[b], a->kv_lens[b], 0};
        p.tokens += a->q_lens[b];
    }
    if (p.tokens == 0) return MK_OK;
    p.q = static_cast<const __nv_bfloat16*>(a->q);
    p.out = static_cast<__nv_bfloat16*>(a->out);
    p.q_stride = a->q_stride; p.out_stride = a->out_stride;
    p.k = static_cast<const __nv_bfloat16*>(a->kv->k) + a->layer * a->kv->layer_stride;
    p.v = static_cast<const __nv_bfloat16*>(a->kv->v) + a->layer * a->kv->layer_stride;
    p.batch_stride = a->kv->batch_stride; p.head_stride = a->kv->head_stride;
    if (a->pages) {
        p.table = a->pages->block_table; p.block = a->pages->block_size;
        p.max_blocks = a->pages->max_blocks; p.n_blocks = a->pages->n_blocks;
    }
    p.window = a->window; p.sinks = a->sinks; p.prefix = a->shared_prefix;
    p.scale = a->scale != 0.f ? a->scale : float(1.0 / std::sqrt(double(p.d)));
    p.status = a->status;
    const int64_t warps = int64_t(p.tokens) * p.nq;
    attend_simple_kernel<<<unsigned((warps + 3) / 4), 128, 0, static_cast<cudaStream_t>(stream)>>>(p);
    MK_CK(cudaGetLastError());
    return MK_OK;
}
