// Block tables and slot maps of a paged cache, built on the device from the requests' lengths (mk_assign_pages).
#include <algorithm>
#include <climits>

#include "mk_ops.h"
#include "mk_sm103.cuh"

namespace mk {

constexpr int kPagesThreads = 256;
constexpr int kPagesEach = MK_PAGES_MAX_BATCH / kPagesThreads;   // requests of a thread in the scan

struct PagesParams {
    mk_pages_args a;
    int shared;      // whole blocks of the shared prefix
    int vector;      // slots, positions and sequences take 16-byte stores
};

// What every CTA works out for itself from the lengths: three prefix sums over the requests
struct PagesScan {
    int tokens[MK_PAGES_MAX_BATCH + 1], taken[MK_PAGES_MAX_BATCH + 1], returned[MK_PAGES_MAX_BATCH + 1];   // of the requests before
    int len[MK_PAGES_MAX_BATCH], held[MK_PAGES_MAX_BATCH];                                                 // positions and blocks before the call
};

// The last of the n + 1 ascending `sums` that is at most i (sums[0] = 0 <= i < sums[n]): whose i is
__device__ __forceinline__ int pages_owner(const int* sums, int n, int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (sums[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// One launch.  Nothing in it waits for another CTA: each repeats the scan over the lengths (at most 4 requests a thread), reads only
// ring places and table entries that no CTA writes, and takes its share of the moved blocks and of the tokens.  A block taken from
// those that this call returns is looked up in the table row it is returned from, not in the ring.  Where the ends are
// updated in place the CTA that is last to have read them writes them.
__global__ void __launch_bounds__(kPagesThreads) pages_kernel(const __grid_constant__ PagesParams p) {
    __shared__ PagesScan s;
    __shared__ long long part[kPagesThreads / 32][3];
    __shared__ int bad_length, front_free[2];
    sm::pdl_trigger();
    sm::pdl_wait();
    const mk_pages_args& a = p.a;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    if (t == 0) {
        bad_length = 0;
        front_free[0] = *reinterpret_cast<const volatile int*>(a.ends);
        front_free[1] = *reinterpret_cast<const volatile int*>(a.ends + 1);
    }
    __syncthreads();
    const long long most = (long long)(a.max_blocks) * a.block_size;
    long long sum[3] = {0, 0, 0};
    int each[kPagesEach][3];
#pragma unroll
    for (int i = 0; i < kPagesEach; ++i) {
        const int b = t * kPagesEach + i;
        each[i][0] = each[i][1] = each[i][2] = 0;
        if (b >= a.batch) continue;
        const int len = a.lens[b], wanted = a.new_lens[b];
        if (len < 0 || wanted < 0 || len > most || wanted > most) {
            bad_length = 1;
            continue;
        }
        const int held = max(p.shared, int((len + (long long)(a.block_size) - 1) / a.block_size));
        const int need = max(p.shared, int((wanted + (long long)(a.block_size) - 1) / a.block_size));
        s.len[b] = len;
        s.held[b] = held;
        each[i][0] = max(wanted - len, 0);
        each[i][1] = max(need - held, 0);
        each[i][2] = max(held - need, 0);
#pragma unroll
        for (int k = 0; k < 3; ++k) sum[k] += each[i][k];
    }
    long long before[3];   // of the threads before this one, first in its warp, then in the CTA
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        long long v = sum[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) part[warp][k] = v;
        before[k] = v - sum[k];
    }
    __syncthreads();
    long long total[3] = {0, 0, 0};
#pragma unroll
    for (int w = 0; w < kPagesThreads / 32; ++w)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (w == warp) before[k] += total[k];
            total[k] += part[w][k];
        }
    const int front = front_free[0], free = front_free[1];
    mk_status st = MK_OK;
    if (bad_length || front < 0 || front >= a.n_blocks || free < 0 || free + total[2] > a.n_blocks) st = MK_ERR_BOUNDS;
    else if (total[1] > free + total[2] || total[0] > a.max_tokens) st = MK_ERR_CAPACITY;
    const int tokens = st == MK_OK ? int(total[0]) : 0, taken = st == MK_OK ? int(total[1]) : 0,
              returned = st == MK_OK ? int(total[2]) : 0;
    if (st == MK_OK) {   // (the sums fit 32 bits now)
#pragma unroll
        for (int i = 0; i < kPagesEach; ++i) {
            const int b = t * kPagesEach + i;
            if (b <= a.batch) {
                s.tokens[b] = int(before[0]);
                s.taken[b] = int(before[1]);
                s.returned[b] = int(before[2]);
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) before[k] += each[i][k];
        }
        if (t == kPagesThreads - 1 && a.batch == MK_PAGES_MAX_BATCH) {
            s.tokens[a.batch] = tokens;
            s.taken[a.batch] = taken;
            s.returned[a.batch] = returned;
        }
    }
    __syncthreads();
    if (st != MK_OK && a.status && blockIdx.x == 0 && t == 0) *a.status = st;

    auto wrap = [&](long long i) { return int(i >= a.n_blocks ? i - a.n_blocks : i); };   // (i below 2 n_blocks)
    auto given_back = [&](int j) {   // the j-th returned block
        const int b = pages_owner(s.returned, a.batch, j), count = s.returned[b + 1] - s.returned[b];
        return a.table[int64_t(b) * a.max_blocks + s.held[b] - count + (j - s.returned[b])];
    };
    auto new_block = [&](int k) { return k < free ? a.ring[wrap((long long)(front) + k)] : given_back(k - free); };
    const int self = int(blockIdx.x) * kPagesThreads + t, threads = int(gridDim.x) * kPagesThreads;
    for (int j = self; j < returned; j += threads) {
        const int at = wrap((long long)(front) + free);
        a.ring[wrap((long long)(at) + j)] = given_back(j);
    }
    for (int k = self; k < taken; k += threads) {
        const int b = pages_owner(s.taken, a.batch, k);
        a.table[int64_t(b) * a.max_blocks + s.held[b] + (k - s.taken[b])] = new_block(k);
    }
    if (a.first)
        for (int b = self; b <= a.batch; b += threads) a.first[b] = st == MK_OK ? s.tokens[b] : 0;

    // four neighbouring tokens a thread: one search, then steps to the next block or request
    for (long long at = 4ll * self; at < a.max_tokens; at += 4ll * threads) {
        int slot[4] = {-1, -1, -1, -1}, pos[4] = {0, 0, 0, 0}, seq[4] = {-1, -1, -1, -1};
        const int i0 = int(at);
        if (i0 < tokens) {
            int b = pages_owner(s.tokens, a.batch, i0), x = s.len[b] + (i0 - s.tokens[b]);
            int j = x / a.block_size, off = x - j * a.block_size, id = INT_MIN;
            bool have = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i0 + i >= tokens) break;
                if (i0 + i >= s.tokens[b + 1]) {
                    do ++b;
                    while (i0 + i >= s.tokens[b + 1]);   // (ends: i0 + i < tokens = the last sum)
                    x = s.len[b];
                    j = x / a.block_size;
                    off = x - j * a.block_size;
                    have = false;
                }
                if (off == a.block_size) {
                    ++j;
                    off = 0;
                    have = false;
                }
                if (!have) {
                    id = j < s.held[b] ? a.table[int64_t(b) * a.max_blocks + j] : new_block(s.taken[b] + (j - s.held[b]));
                    have = true;
                }
                const bool good = unsigned(id) < unsigned(a.n_blocks);
                if (!good && a.status) *a.status = MK_ERR_BOUNDS;
                slot[i] = good ? id * a.block_size + off : -1;
                pos[i] = x;
                seq[i] = b;
                ++x;
                ++off;
            }
        }
        auto put = [&](int* dst, const int (&v)[4]) {
            if (!dst) return;
            if (p.vector && at + 4 <= a.max_tokens) *reinterpret_cast<int4*>(dst + at) = make_int4(v[0], v[1], v[2], v[3]);
            else
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at + i < a.max_tokens) dst[at + i] = v[i];
        };
        put(a.slots, slot);
        put(a.positions, pos);
        put(a.sequences, seq);
    }

    // the ends, by the only CTA, by the first (of another buffer), or in place by the last one to come here
    bool writer = t == 0 && blockIdx.x == 0;
    if (gridDim.x > 1 && a.ends_out == a.ends) {
        writer = false;
        if (t == 0) {
            __threadfence();
            writer = atomicAdd(a.ends_out + 2, 1) == int(gridDim.x) - 1;
        }
    }
    if (writer) {
        a.ends_out[0] = st == MK_OK ? wrap((long long)(front) + taken) : front;
        a.ends_out[1] = st == MK_OK ? free + returned - taken : free;
        a.ends_out[2] = 0;
    }
}

static mk_status pages_check(const mk_pages_args* a) {
    if (!a) return fail(MK_ERR_ARG, "null argument");
    if (a->batch < 1 || a->batch > MK_PAGES_MAX_BATCH)
        return fail(MK_ERR_ARG, "assign_pages: batch %d (1 to %d)", a->batch, MK_PAGES_MAX_BATCH);
    if (a->block_size < 1 || a->max_blocks < 1 || a->n_blocks < 1 || int64_t(a->n_blocks) * a->block_size > INT_MAX ||
        int64_t(a->max_blocks) * a->block_size > INT_MAX)
        return fail(MK_ERR_ARG, "assign_pages: block_size %d, max_blocks %d, n_blocks %d (each positive, at most 2^31 - 1 positions)",
                    a->block_size, a->max_blocks, a->n_blocks);
    if (a->shared_prefix < 0 || a->shared_prefix / a->block_size > a->max_blocks)
        return fail(MK_ERR_ARG, "assign_pages: shared prefix of %d positions", a->shared_prefix);
    if (a->max_tokens < 0) return fail(MK_ERR_ARG, "assign_pages: max_tokens %d", a->max_tokens);
    if (!a->ring || !a->ends || !a->ends_out || !a->table || !a->lens || !a->new_lens || (!a->slots && a->max_tokens > 0))
        return fail(MK_ERR_ARG, "assign_pages: null pointer");
    const int64_t rows = a->batch, tokens = a->max_tokens;
    const struct { const void* p; int64_t words; bool written; } use[] = {
        {a->ring, a->n_blocks, true}, {a->ends, 3, false}, {a->ends_out, 3, true}, {a->table, rows * a->max_blocks, true},
        {a->lens, rows, false}, {a->new_lens, rows, false}, {a->slots, tokens, true}, {a->positions, tokens, true},
        {a->sequences, tokens, true}, {a->first, rows + 1, true}, {a->status, 1, true}};
    constexpr int n = sizeof use / sizeof use[0];
    for (int i = 0; i < n; ++i) {
        if (!op_aligned(use[i].p, 4)) return fail(MK_ERR_ARG, "assign_pages: a pointer is not 4-byte aligned");
        for (int j = 0; j < i; ++j)
            if ((use[i].written || use[j].written) && !(use[i].p == a->ends_out && use[j].p == a->ends && a->ends == a->ends_out) &&
                spans_overlap({use[i].p, 1, use[i].words * 4, 0}, {use[j].p, 1, use[j].words * 4, 0}))
                return fail(MK_ERR_ARG, "assign_pages: two buffers overlap");
    }
    return MK_OK;
}

}  // namespace mk

using namespace mk;

extern "C" mk_status mk_assign_pages(const mk_pages_args* a, void* stream) {
    mk_status st = pages_check(a);
    if (st != MK_OK) return st;
    int device = 0, sms = 0;
    if ((st = op_device(&device, &sms)) != MK_OK) return st;
    PagesParams p{};
    p.a = *a;
    p.shared = a->shared_prefix / a->block_size;
    p.vector = op_aligned(a->slots, 16) && op_aligned(a->positions, 16) && op_aligned(a->sequences, 16);
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.blockDim = dim3(kPagesThreads);
    // a token or four a thread, two CTAs an SM at most: each repeats the scan
    const int64_t wanted = (int64_t(a->max_tokens) + 4 * kPagesThreads - 1) / (4 * kPagesThreads);
    cfg.gridDim = dim3(unsigned(std::max<int64_t>(1, std::min<int64_t>(wanted, 2 * sms))));
    MK_CK(cudaLaunchKernelEx(&cfg, &pages_kernel, p));
    return MK_OK;
}
