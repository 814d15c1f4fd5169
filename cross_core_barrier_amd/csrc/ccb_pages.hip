// ccb_pages.hip -- pages of a paged cache handed out and taken back on the GPU
// (include/ccb_pages.h): kernels and C entry points.
//
// Both calls are a prefix sum over the sequences, then work on tokens or pages
// that are numbered through.  One kernel does it: every workgroup computes the
// whole prefix sum for itself (a few loads a thread, from the caches), takes its
// share of the tokens or pages, and finds their sequences by bisection in LDS.
// What the call changes of its own inputs (lens, count) is written by the
// workgroup that ends last, when all others have read them: it is the one that
// finds the counters of `state` full, and leaves them at 0.  A grow's grid goes by the
// room for tokens (up to 2048 are one workgroup), a trim's by the table's capacity, since
// the host knows no lengths: 64 sequences of up to 126 pages are 4 workgroups, and a
// wide table starts up to 512 to take back a few pages.
//
// What bounds it: latency.  A step of 64 sequences takes 3.6 us (trim) and 6.4
// (grow), of which 2.5 is the start and the rest a chain of loads: lengths, two
// sums, a token's sequence, its page.  A million tokens of 1000 sequences take
// 13.7 us for 17 MB written (3.3 at a copy's rate), 256 prompts of 243,000 tokens
// 8.7; so many tokens a workgroup that its sums are worth their while, 2048: with
// 1024 (256 threads) the million took 16.3, with 4096 (1024 threads) 16.6.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccb_kv8_device.h"
#include "ccb_kv8_internal.h"
#include "ccb_pages.h"

namespace {

using kv8::report;

constexpr uint32_t kMost = 1u << 30;  // sums stop here: above every size there is
constexpr int32_t kShortBatch = 1024;
constexpr int32_t kTeam = 32, kMostGroups = 512;  // workgroups to a counter, and in all
constexpr int32_t kLineWords = CCB_LINE_BYTES / 4;
static_assert((1 + kMostGroups / kTeam) * CCB_LINE_BYTES == CCB_PAGES_STATE_BYTES, "a line for each counter");

// a + b for sums that stop at kMost.
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return min(a + b, kMost); }

// x summed over the lanes up to this one (without exchanges through LDS, whose
// latency six times over is a third of a microsecond).
__device__ __forceinline__ uint32_t scan(uint32_t x)
{
    x = add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xf, 0xf, true));  // 1, 2, 4, 8 lanes before,
    x = add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xf, 0xf, true));  // in rows of 16
    x = add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xf, 0xf, true));
    x = add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xf, 0xf, true));
    x = add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xa, 0xf, false));  // the last of a row, to the
    x = add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xc, 0xf, false));  // next; of two, to two
    return x;
}

// x's sum over the threads before this one, and over all.
template <int THREADS>
__device__ __forceinline__ uint32_t sum_before(uint32_t x, uint32_t* scratch, uint32_t& all)
{
    constexpr int W = THREADS / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t sum = scan(x);
    __syncthreads();  // the scratch of the sum before
    if (lane == 63) scratch[wave] = sum;
    uint32_t own = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sum, 0x138, 0xf, 0xf, true);  // the lane before's
    __syncthreads();
    uint32_t before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w < wave) before = add(before, scratch[w]);
        all = add(all, scratch[w]);
    }
    return add(before, own);
}

// The last b in [0, batch) with at[b] <= i (at[0] is 0).
__device__ __forceinline__ int32_t find(const uint32_t* at, int32_t batch, uint32_t i)
{
    int32_t lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (at[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

// Whether this workgroup is the last to come here; all of its reads are done.  In
// two steps, 32 workgroups to a counter: one address takes 11 ns an arrival, so
// that 512 at one would take 6 us.
__device__ __forceinline__ bool last_of_all(int32_t* state, int32_t* flag)
{
    const int32_t grid = (int32_t)gridDim.x, me = (int32_t)blockIdx.x;
    if (grid == 1) return true;
    __syncthreads();
    if (threadIdx.x == 0) {
        auto last = [](int32_t* word, int32_t of) {
            if (__hip_atomic_fetch_add(word, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != of - 1) return false;
            __hip_atomic_store(word, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            return true;
        };
        const int32_t teams = (grid + kTeam - 1) / kTeam, team = me % teams;
        *flag = last(state + (1 + team) * kLineWords, (grid - team + teams - 1) / teams) && last(state, teams);
    }
    __syncthreads();
    return *flag != 0;
}

struct Pool {
    ccbPagePool p;
    ccbPageTable t;
    int32_t* err;
    int32_t shift;  // log2 of pageSize
};

__device__ __forceinline__ int32_t pages_of(const Pool& a, int32_t tokens)
{
    return (tokens + a.p.pageSize - 1) >> a.shift;
}

template <int CAP, int THREADS>
__global__ __launch_bounds__(THREADS) void pages_k_trim(Pool a, const int32_t* keep)
{
    constexpr int MINE = CAP / THREADS;  // sequences of a thread, at most
    __shared__ uint32_t at[CAP];         // pages given back before sequence b
    __shared__ int32_t low[CAP];         // its first page that goes
    __shared__ uint32_t scratch[THREADS / 64];
    __shared__ int32_t flag;
    const int32_t batch = a.t.batch, room = a.t.maxPages << a.shift;
    const int32_t each = (batch + THREADS - 1) / THREADS, b0 = threadIdx.x * each;
    int32_t len[MINE], stay[MINE];
    uint32_t mine = 0;
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
        const int32_t b = b0 + k;
        len[k] = 0, stay[k] = 0;
        if (k >= each || b >= batch) continue;
        len[k] = a.t.lens[b];
        stay[k] = keep[b];
    }
    int32_t have = *a.p.count;
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
        if (len[k] < 0 || len[k] > room) {
            report(a.err);
            stay[k] = -1;  // left alone
            len[k] = 0;
        }
        stay[k] = stay[k] < 0 || stay[k] > len[k] ? len[k] : stay[k];
        mine = add(mine, (uint32_t)(pages_of(a, len[k]) - pages_of(a, stay[k])));
    }
    uint32_t all;
    uint32_t before = sum_before<THREADS>(mine, scratch, all);
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
        const int32_t b = b0 + k;
        if (k >= each || b >= batch) continue;
        at[b] = before;
        low[b] = pages_of(a, stay[k]);
        before = add(before, (uint32_t)(pages_of(a, len[k]) - low[b]));
    }
    __syncthreads();
    const bool fits = have >= 0 && (int64_t)have + all <= a.p.numPages;
    if (!fits && (all > 0 || have < 0 || have > a.p.numPages) && threadIdx.x == 0) report(a.err);
    if (fits) {
        for (uint32_t i = blockIdx.x * THREADS + threadIdx.x; i < all; i += gridDim.x * THREADS) {
            const int32_t b = find(at, batch, i);
            int32_t page = a.t.pages[b * a.t.stride + low[b] + (int32_t)(i - at[b])];
            if (page < 0 || page >= a.p.numPages) {
                report(a.err);
                page = -1;
            }
            a.p.free[have + (int32_t)(all - 1 - i)] = page;
        }
    }
    if (!last_of_all(a.p.state, &flag) || !fits) return;
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
        const int32_t b = b0 + k;
        if (k < each && b < batch && stay[k] < len[k]) a.t.lens[b] = stay[k];
    }
    if (threadIdx.x == 0) *a.p.count = have + (int32_t)all;
}

typedef int32_t i4 __attribute__((ext_vector_type(4)));
typedef int64_t l2 __attribute__((ext_vector_type(2)));

template <int CAP, int THREADS>
__global__ __launch_bounds__(THREADS) void pages_k_grow(Pool a, const int32_t* counts, ccbSlotMaps m)
{
    constexpr int MINE = CAP / THREADS;
    __shared__ uint32_t start[CAP + 1];  // tokens before sequence b
    __shared__ uint32_t taken[CAP];      // pages handed out before it
    __shared__ int32_t held[CAP];        // its tokens so far, or -1 where it gets no room
    __shared__ uint32_t scratch[THREADS / 64];
    __shared__ uint32_t used;
    __shared__ int32_t flag;
    const int32_t batch = a.t.batch, room = a.t.maxPages << a.shift;
    const int32_t each = (batch + THREADS - 1) / THREADS, b0 = threadIdx.x * each;
    const uint32_t tokens = (uint32_t)m.tokens;
    int32_t len[MINE], count[MINE];
    uint32_t need[MINE], mine = 0;
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
        const int32_t b = b0 + k;
        len[k] = 0, count[k] = 0;
        if (k >= each || b >= batch) continue;
        len[k] = a.t.lens[b];
        count[k] = counts[b];
    }
    int32_t have = *a.p.count;
    const bool bad = have < 0 || have > a.p.numPages;
    if (bad) have = 0;
    if (threadIdx.x == 0) {
        used = 0;
        if (bad) report(a.err);
    }
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
        if (count[k] < 0) report(a.err);
        mine = add(mine, min((uint32_t)max(count[k], 0), kMost));
    }
    uint32_t all, pages;
    uint32_t before = sum_before<THREADS>(mine, scratch, all);
    mine = 0;
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
        const int32_t b = b0 + k;
        need[k] = 0;
        if (k >= each || b >= batch) continue;
        const uint32_t c = min((uint32_t)max(count[k], 0), kMost), end = add(before, c);
        start[b] = min(before, tokens);
        const bool ok = count[k] >= 0 && len[k] >= 0 && len[k] <= room && c <= (uint32_t)(room - len[k]) &&
                        end <= tokens;
        if (!ok) {
            report(a.err);
            len[k] = -1;
        } else {
            need[k] = (uint32_t)(pages_of(a, len[k] + count[k]) - pages_of(a, len[k]));
        }
        mine = add(mine, need[k]);
        before = end;
    }
    before = sum_before<THREADS>(mine, scratch, pages);
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
        const int32_t b = b0 + k;
        if (k >= each || b >= batch) continue;
        const uint32_t after = add(before, need[k]);
        if (after <= (uint32_t)have) most = after;  // (sums only grow)
        if (need[k] > 0 && after > (uint32_t)have) len[k] = -1;
        taken[b] = before;
        held[b] = len[k];
        before = after;
    }
    if (most > 0) atomicMax(&used, most);
    if (threadIdx.x == 0) start[batch] = min(all, tokens);
    __syncthreads();

    // four tokens of a thread
    const uint32_t total = start[batch];
    for (uint32_t i0 = (blockIdx.x * THREADS + threadIdx.x) * 4; i0 < tokens; i0 += gridDim.x * THREADS * 4) {
        int64_t slot[4];
        int32_t position[4], sequence[4];
        int32_t b = -1, page = -1, number = -1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t i = i0 + e;
            slot[e] = -1, position[e] = -1, sequence[e] = -1;
            if (i >= total) continue;
            if (b < 0 || start[b + 1] <= i) b = find(start, batch, i), number = -1;
            sequence[e] = b;
            const int32_t n = held[b];
            if (n < 0) continue;
            const int32_t t = n + (int32_t)(i - start[b]), j = t >> a.shift;
            if (j != number) {
                number = j;
                const int32_t low = pages_of(a, n);
                int32_t* entry = a.t.pages + b * a.t.stride + j;
                if (j < low) {
                    page = *entry;
                } else {
                    page = a.p.free[have - 1 - (int32_t)(taken[b] + (uint32_t)(j - low))];
                    if ((t & (a.p.pageSize - 1)) == 0) *entry = page;  // by its first token
                }
                if (page < 0 || page >= a.p.numPages) {
                    report(a.err);
                    page = -1;
                }
            }
            position[e] = t;
            if (page >= 0) slot[e] = ((int64_t)page << a.shift) + (t & (a.p.pageSize - 1));
        }
        if (i0 + 4 <= tokens) {
            if (m.slots != nullptr) {
                *(l2*)(m.slots + i0) = l2{slot[0], slot[1]};
                *(l2*)(m.slots + i0 + 2) = l2{slot[2], slot[3]};
            }
            if (m.positions != nullptr) *(i4*)(m.positions + i0) = i4{position[0], position[1], position[2], position[3]};
            if (m.sequences != nullptr) *(i4*)(m.sequences + i0) = i4{sequence[0], sequence[1], sequence[2], sequence[3]};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (i0 + e >= tokens) break;
                if (m.slots != nullptr) m.slots[i0 + e] = slot[e];
                if (m.positions != nullptr) m.positions[i0 + e] = position[e];
                if (m.sequences != nullptr) m.sequences[i0 + e] = sequence[e];
            }
        }
    }
    if (!last_of_all(a.p.state, &flag)) return;
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
        const int32_t b = b0 + k;
        if (k >= each || b >= batch) continue;
        if (len[k] >= 0 && count[k] > 0) a.t.lens[b] = len[k] + count[k];
        if (m.granted != nullptr) m.granted[b] = len[k] >= 0 ? count[k] : 0;
        if (m.starts != nullptr) m.starts[b] = (int32_t)start[b];
    }
    if (threadIdx.x == 0) {
        if (m.starts != nullptr) m.starts[batch] = (int32_t)total;
        if (!bad) *a.p.count = have - (int32_t)used;
    }
}

ccbStatus check(const ccbPagePool* p, const ccbPageTable* t, const int32_t* numbers, const int32_t* err)
{
    using ccb::aligned;
    if (p == nullptr || t == nullptr) return CCB_ERR_NULL_POINTER;
    if (p->numPages < 1 || p->numPages >= (1 << 30) || p->pageSize < 1 || p->pageSize > 32768 ||
        (p->pageSize & (p->pageSize - 1)) != 0 || t->batch < 0 || t->batch > CCB_PAGES_MAX_BATCH ||
        t->maxPages < 1 || (int64_t)t->maxPages * p->pageSize > (1 << 30) || t->stride < t->maxPages)
        return CCB_ERR_INVALID_VALUE;
    if (p->free == nullptr || p->count == nullptr || p->state == nullptr) return CCB_ERR_NULL_POINTER;
    if (t->batch > 0 && (t->pages == nullptr || t->lens == nullptr || numbers == nullptr)) return CCB_ERR_NULL_POINTER;
    if (!aligned(p->free, 4) || !aligned(p->count, 4) || !aligned(p->state, CCB_LINE_BYTES) || !aligned(t->pages, 4) ||
        !aligned(t->lens, 4) || !aligned(numbers, 4) || !aligned(err, 4))
        return CCB_ERR_INVALID_VALUE;
    return CCB_OK;
}

Pool pool_of(const ccbPagePool* p, const ccbPageTable* t, int32_t* err)
{
    Pool a;
    a.p = *p, a.t = *t, a.err = err;
    a.shift = __builtin_ctz((unsigned)p->pageSize);
    return a;
}

// Workgroups for so many tokens or pages, `each` and more for one.
int64_t groups_for(int64_t n, int64_t each, int64_t most)
{
    const int64_t g = (n + each - 1) / each;
    return g < 1 ? 1 : g < most ? g : most;
}

}  // namespace

extern "C" {

CCB_API ccbStatus ccb_pages_trim(const ccbPagePool* pool, const ccbPageTable* table,
                                 const int32_t* keep, int32_t* err, ccbStream stream)
{
    ccbStatus st = check(pool, table, keep, err);
    if (st != CCB_OK) return st;
    if (table->batch == 0) return CCB_OK;
    if ((st = ccb::device_ready()) != CCB_OK) return st;
    const Pool a = pool_of(pool, table, err);
    const int64_t pages = (int64_t)table->batch * table->maxPages;
    if (table->batch <= kShortBatch)
        return ccb::launch_status(kv8::enqueue(pages_k_trim<kShortBatch, 256>, groups_for(pages, 2048, kMostGroups), 256,
                                               (hipStream_t)stream, a, keep));
    return ccb::launch_status(kv8::enqueue(pages_k_trim<CCB_PAGES_MAX_BATCH, 1024>, groups_for(pages, 16384, kMostGroups),
                                           1024, (hipStream_t)stream, a, keep));
}

CCB_API ccbStatus ccb_pages_grow(const ccbPagePool* pool, const ccbPageTable* table,
                                 const int32_t* counts, const ccbSlotMaps* maps, int32_t* err,
                                 ccbStream stream)
{
    using ccb::aligned;
    ccbStatus st = check(pool, table, counts, err);
    if (st != CCB_OK) return st;
    if (maps == nullptr) return CCB_ERR_NULL_POINTER;
    if (maps->tokens < 0 || maps->tokens >= (1 << 30) || maps->reserved != 0 || !aligned(maps->slots, 16) ||
        !aligned(maps->positions, 16) || !aligned(maps->sequences, 16) || !aligned(maps->starts, 4) ||
        !aligned(maps->granted, 4))
        return CCB_ERR_INVALID_VALUE;
    if ((st = ccb::device_ready()) != CCB_OK) return st;
    const Pool a = pool_of(pool, table, err);
    if (table->batch <= kShortBatch)
        return ccb::launch_status(kv8::enqueue(pages_k_grow<kShortBatch, 512>, groups_for(maps->tokens, 2048, kMostGroups), 512,
                                               (hipStream_t)stream, a, counts, *maps));
    return ccb::launch_status(kv8::enqueue(pages_k_grow<CCB_PAGES_MAX_BATCH, 1024>,
                                           groups_for(maps->tokens, 4096, kMostGroups), 1024, (hipStream_t)stream, a, counts,
                                           *maps));
}

}  // extern "C"
