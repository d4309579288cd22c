// Block tables and slot maps of a paged cache, built on the device from the requests' lengths (mk_assign_pages).
#include <algorithm>
#include <climits>

#include "mk_ops.h"
#include "mk_sm103.cuh"

namespace mk {

constexpr int kPagesThreads = 256;
constexpr int kRun = 128;   // tokens of a warp
constexpr int kPagesEach = MK_PAGES_MAX_BATCH / kPagesThreads;   // requests of a thread in the scan

struct PagesParams {
    mk_pages_args a;
    int shared;      // whole blocks of the shared prefix
    int vector;                // slots, positions and sequences take 16-byte stores
    uint32_t inverse, shift;   // x / block_size = x * inverse >> shift for x below 2^31
};

// What every CTA works out for itself from the lengths: three prefix sums over the requests
struct PagesScan {
    int tokens[MK_PAGES_MAX_BATCH + 1], taken[MK_PAGES_MAX_BATCH + 1], returned[MK_PAGES_MAX_BATCH + 1];   // of the requests before
    int len[MK_PAGES_MAX_BATCH], held[MK_PAGES_MAX_BATCH];                                                 // positions and blocks before the call
};

// The last of the ascending sums[lo .. hi - 1] that is at most i (sums[lo] <= i): whose i is
__device__ __forceinline__ int pages_owner(const int* sums, int lo, int hi, int i) {
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (sums[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ uint32_t pages_add(uint32_t a, uint32_t b) { return a + b < a ? ~0u : a + b; }
__device__ __forceinline__ int pages_divide(const PagesParams& p, int x) { return int(uint64_t(x) * p.inverse >> p.shift); }
__device__ __forceinline__ int pages_blocks(const PagesParams& p, int positions) {
    const int n = pages_divide(p, positions);
    return n + (n * p.a.block_size < positions);
}

// The same over all n requests for a whole warp's i: 32 sums at a time
__device__ __forceinline__ int pages_warp_owner(const int* sums, int n, int i) {
    const int lane = threadIdx.x & 31;
    const int part = 32 * (__popc(__ballot_sync(0xFFFFFFFFu, 32 * lane < n && sums[min(32 * lane, n)] <= i)) - 1), b = part + lane;
    return part + __popc(__ballot_sync(0xFFFFFFFFu, b < n && sums[min(b, n)] <= i)) - 1;
}

// One launch.  Nothing in it waits for another CTA: each repeats the scan over the lengths (at most 4 requests a thread), reads only
// ring places and table entries that no CTA writes, and takes its share of the moved blocks and of the tokens.  A block taken from
// those that this call returns is looked up in the table row it is returned from, not in the ring.  Where the ends are
// updated in place the CTA that is last to have read them writes them.
// What bounds it: latencies in a row (lengths, the scan, a search, a table entry; 3.5 us for a step of 8 requests, 5.1 for 36000
// tokens of 200) and for a million tokens the instructions of scan and searches (8.3 us, 1.5 TB/s; with one CTA an SM 15, two 8.9,
// four 11.2, whose last runs fall on fewer SMs).
__global__ void __launch_bounds__(kPagesThreads) pages_kernel(const __grid_constant__ PagesParams p) {
    __shared__ PagesScan s;
    __shared__ uint32_t part[kPagesThreads / 32][3];
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
    const int most = a.max_blocks * a.block_size;
    // (sums stop at 2^32 - 1, above all that can be served; so the order of their additions does not matter)
    uint32_t sum[3] = {0, 0, 0}, each[kPagesEach][3];
    const int mine = (a.batch + kPagesThreads - 1) / kPagesThreads;   // requests of a thread
#pragma unroll
    for (int i = 0; i < kPagesEach; ++i) {
        const int b = t * mine + i;
        each[i][0] = each[i][1] = each[i][2] = 0;
        if (i >= mine || b >= a.batch) continue;
        const int len = a.lens[b], wanted = a.new_lens[b];
        if (len < 0 || wanted < 0 || len > most || wanted > most) {
            bad_length = 1;
            continue;
        }
        const int held = max(p.shared, pages_blocks(p, len)), need = max(p.shared, pages_blocks(p, wanted));
        s.len[b] = len;
        s.held[b] = held;
        each[i][0] = uint32_t(max(wanted - len, 0));
        each[i][1] = uint32_t(max(need - held, 0));
        each[i][2] = uint32_t(max(held - need, 0));
#pragma unroll
        for (int k = 0; k < 3; ++k) sum[k] = pages_add(sum[k], each[i][k]);
    }
    uint32_t before[3];   // of the threads before this one, first in its warp, then in the CTA
#pragma unroll
    for (int k = 0; k < 3; ++k) before[k] = sum[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, before[k], o);
            if (lane >= o) before[k] = pages_add(before[k], v);
        }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (lane == 31) part[warp][k] = before[k];
        before[k] = __shfl_up_sync(0xFFFFFFFFu, before[k], 1);
        if (lane == 0) before[k] = 0;
    }
    __syncthreads();
    uint32_t total[3] = {0, 0, 0};
#pragma unroll
    for (int w = 0; w < kPagesThreads / 32; ++w)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (w == warp) before[k] = pages_add(before[k], total[k]);
            total[k] = pages_add(total[k], part[w][k]);
        }
    const int front = front_free[0], free = front_free[1];
    mk_status st = MK_OK;
    if (bad_length || front < 0 || front >= a.n_blocks || free < 0 || (long long)(free) + total[2] > a.n_blocks) st = MK_ERR_BOUNDS;
    else if (total[1] > uint32_t(free) + total[2] || total[0] > uint32_t(a.max_tokens)) st = MK_ERR_CAPACITY;
    const int tokens = st == MK_OK ? int(total[0]) : 0, taken = st == MK_OK ? int(total[1]) : 0,
              returned = st == MK_OK ? int(total[2]) : 0;
    if (st == MK_OK) {   // (the sums fit 32 bits now)
#pragma unroll
        for (int i = 0; i < kPagesEach; ++i) {
            const int b = t * mine + i;
            if (i < mine && b < a.batch) {
                s.tokens[b] = int(before[0]);
                s.taken[b] = int(before[1]);
                s.returned[b] = int(before[2]);
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) before[k] += each[i][k];
        }
        if (t == 0) {
            s.tokens[a.batch] = tokens;
            s.taken[a.batch] = taken;
            s.returned[a.batch] = returned;
        }
    }
    __syncthreads();
    if (st != MK_OK && a.status && blockIdx.x == 0 && t == 0) *a.status = st;

    auto wrap = [&](long long i) { return int(i >= a.n_blocks ? i - a.n_blocks : i); };   // (i below 2 n_blocks)
    auto given_back = [&](int j) {   // where the j-th returned block stands
        const int b = pages_owner(s.returned, 0, a.batch, j), count = s.returned[b + 1] - s.returned[b];
        return a.table + int64_t(b) * a.max_blocks + s.held[b] - count + (j - s.returned[b]);
    };
    auto new_block = [&](int k) -> const int* { return k < free ? a.ring + wrap((long long)(front) + k) : given_back(k - free); };
    const int self = int(blockIdx.x) * kPagesThreads + t, threads = int(gridDim.x) * kPagesThreads;
    // (there may be 2^31 - 1 tokens and as many moved blocks: bounds are taken as differences, steps in 64 bits)
    // a warp takes 128 neighbouring tokens, a lane four of them: mostly of one request and one block, else one after the other
    auto block_of = [&](int b, int j) -> const int* {
        return j < s.held[b] ? a.table + int64_t(b) * a.max_blocks + j : new_block(s.taken[b] + (j - s.held[b]));
    };
    for (long long run = (long long)(self / 32) * kRun; run < a.max_tokens; run += (long long)(threads / 32) * kRun) {
        const long long at = run + 4 * lane;
        int slot[4] = {-1, -1, -1, -1}, pos[4] = {0, 0, 0, 0}, seq[4] = {-1, -1, -1, -1};
        if (run < tokens) {
            const int b0 = pages_warp_owner(s.tokens, a.batch, int(run)), b1 = pages_warp_owner(s.tokens, a.batch, int(run) + min(kRun, tokens - int(run)) - 1);
            if (at < tokens) {
                const int token = int(at);
                int b = pages_owner(s.tokens, b0, b1 + 1, token), x = s.len[b] + (token - s.tokens[b]);
                int j = pages_divide(p, x), off = x - j * a.block_size;
                if (s.tokens[b + 1] - token >= 4 && a.block_size - off >= 4) {
                    const int id = *block_of(b, j);
                    const bool good = unsigned(id) < unsigned(a.n_blocks);
                    if (!good && a.status) *a.status = MK_ERR_BOUNDS;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        slot[i] = good ? id * a.block_size + off + i : -1;
                        pos[i] = x + i;
                        seq[i] = b;
                    }
                } else {
                    int id[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {   // (the loads of all four are in flight together)
                        if (i >= tokens - token) break;
                        while (token + i >= s.tokens[b + 1]) ++b;   // (ends: token + i < tokens, the last sum)
                        x = s.len[b] + (token + i - s.tokens[b]);
                        j = pages_divide(p, x);
                        slot[i] = x - j * a.block_size;
                        id[i] = *block_of(b, j);
                        pos[i] = x;
                        seq[i] = b;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (seq[i] < 0) continue;
                        const bool good = unsigned(id[i]) < unsigned(a.n_blocks);
                        if (!good && a.status) *a.status = MK_ERR_BOUNDS;
                        slot[i] = good ? id[i] * a.block_size + slot[i] : -1;
                    }
                }
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
    // the moved blocks, from the last thread on (which has no tokens where the first ones suffice)
    const int back = threads - 1 - self;
    for (long long j = back; j < returned; j += threads) {
        const int at = wrap((long long)(front) + free);
        a.ring[wrap(at + j)] = *given_back(int(j));
    }
    for (long long k = back; k < taken; k += threads) {
        const int b = pages_owner(s.taken, 0, a.batch, int(k));
        a.table[int64_t(b) * a.max_blocks + s.held[b] + (k - s.taken[b])] = *new_block(int(k));
    }
    if (a.first)
        for (int b = back; b <= a.batch; b += threads) a.first[b] = st == MK_OK ? s.tokens[b] : 0;

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
            if ((use[i].written || use[j].written) && !(i == 2 && j == 1 && a->ends == a->ends_out) &&   // (ends, updated in place)
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
    p.shift = 31;
    while ((int64_t(1) << (p.shift - 31)) < a->block_size) ++p.shift;
    p.inverse = uint32_t(((uint64_t(1) << p.shift) + uint32_t(a->block_size) - 1) / uint32_t(a->block_size));
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.blockDim = dim3(kPagesThreads);
    // (each CTA repeats the scan over the lengths: no more than are resident)
    const int64_t wanted = (int64_t(a->max_tokens) + kRun * (kPagesThreads / 32) - 1) / (kRun * (kPagesThreads / 32));
    cfg.gridDim = dim3(unsigned(std::max<int64_t>(1, std::min<int64_t>(wanted, 3 * sms))));
    MK_CK(cudaLaunchKernelEx(&cfg, &pages_kernel, p));
    return MK_OK;
}
