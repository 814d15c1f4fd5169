// ccb_kv8_cache.hip -- the kernels that fill, cut and read the 8-bit
// key/value cache: append, evict, read.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccb_kv8_internal.h"
#include "ccb_kv8_device.h"

namespace {

using namespace kv8;

constexpr int kThreads = 256;

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

// Picks the kernel instance for a cache's format and head size.
#define KV8_BY_DIM(dim, CALL) \
    ((dim) == 64    ? CALL(64) \
     : (dim) == 96  ? CALL(96) \
     : (dim) == 128 ? CALL(128) \
     : (dim) == 192 ? CALL(192) \
                    : CALL(256))

// ---------------------------------------------------------------------------
// append
//
// One team per touched page, head and side (K or V): the largest new value
// gives the block's scale, then the new values are rounded and, where the
// scale grew, the block's older codes are rounded again.  Blocks are
// independent, so there is nothing to join.  Bound by the bytes of the new
// values and codes (8 prompts of 8192 tokens: 402 MB in 75 to 87 us); one-token
// steps by latency (5 us).
// ---------------------------------------------------------------------------
template <int F, int T, int D>
__global__ __launch_bounds__(kThreads) void kv8_k_append(ccbKv8Cache c, ccbKv8Rows kNew,
                                                         ccbKv8Rows vNew, int32_t nNew,
                                                         const int32_t* counts, int32_t span,
                                                         uint32_t units, int32_t* err)
{
    __shared__ float scratch[4];
    const int32_t P = c.pageSize, shift = __builtin_ctz(P);
    const Team team(P, blockIdx.x);
    const uint32_t unit = team.unit < units ? team.unit : 0;
    bool works = team.unit < units;  // (the teams of a workgroup stay together)
    const bool isV = unit & 1;
    uint32_t rest = unit >> 1;
    const int32_t h = rest % (uint32_t)c.heads;
    rest /= (uint32_t)c.heads;
    const int32_t local = rest % (uint32_t)span;
    const int32_t b = rest / (uint32_t)span;

    const int32_t len = checked_len(c.lens[b], c.maxPages * P);
    const int32_t cnt = counts != nullptr ? counts[b] : nNew;
    if (works && (len < 0 || cnt < 0 || cnt > nNew || cnt > len)) {
        if (team.id == 0) report(err);
        works = false;
    }
    const int32_t start = works ? len - cnt : 0;
    const int32_t number = (start >> shift) + local;
    works = works && cnt > 0 && number * (int64_t)P < len;
    const int32_t lo = works && start > number * P ? start - number * P : 0;  // new slots lo .. hi - 1
    const int32_t hi = !works ? 0 : len - number * P < P ? len - number * P : P;
    if (!isV && c.weight != nullptr) {
        float* w = c.weight + ((int64_t)b * c.heads + h) * c.weightStride + (int64_t)number * P;
        for (int32_t i = lo + team.id; i < hi; i += team.size) w[i] = 0.0f;
    }
    const int32_t page = works ? checked_page(c.pageTable[b * c.tableStride + number], c.numPages) : 0;
    if (page < 0) {
        if (team.id == 0) report(err);
        works = false;
    }
    constexpr int V = D / 8;  // vectors of 8 values per token
    const ccbKv8Rows& rows = isV ? vNew : kNew;
    const uint16_t* src = (const uint16_t*)rows.data + b * rows.strideBatch + h * rows.strideHead +
                          (int64_t)(number * P + lo - start) * rows.strideToken;
    const int64_t block = (int64_t)(works ? page : 0) * c.heads + h;
    uint8_t* dst = (uint8_t*)(isV ? c.v : c.k) + block * P * D;
    float* scale = (isV ? c.vScale : c.kScale) + block;

    // the new values stay in registers between finding the scale and rounding
    constexpr int N = 128 * V / kThreads;  // vectors of a thread for the largest page
    const int32_t nVec = works ? (hi - lo) * V : 0;
    uint4 raw[N];
    float a = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int32_t i = k * team.size + team.id;
        raw[k] = make_uint4(0, 0, 0, 0);
        if (i < nVec) raw[k] = *(const uint4*)(src + (i / V) * rows.strideToken + (i % V) * 8);
    }
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) most = larger16(most, raw[k]);
    most = (most >> 16) > (most & 0xffffu) ? most >> 16 : most & 0xffffu;
    a = widen<T>(most);
    if (!(a < INFINITY)) {  // an infinity or NaN: the largest of the others
        a = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float x[8];
            widen8<T>(raw[k], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float m = fabsf(x[j]);
                a = (m > a && m < INFINITY) ? m : a;
            }
        }
    }
    const float s0 = works && lo > 0 ? *scale : 0.0f;
    a = team.largest(a, scratch);
    if (!works) return;
    const float s1 = block_scale<F>(a);
    const float s = s1 > s0 ? s1 : s0;
    const float inv = 1.0f / s;
    if (team.id == 0) *scale = s;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int32_t i = k * team.size + team.id;
        if (i < nVec) {
            float x[8];
            widen8<T>(raw[k], x);
            *(uint2*)(dst + (int64_t)lo * D + (int64_t)i * 8) = encode8<F>(x, inv, s);
        }
    }
    if (lo > 0 && s > s0) {  // older codes of a block whose scale grew
        for (int32_t i = team.id; i < lo * V; i += team.size) {
            uint2* p = (uint2*)(dst + (int64_t)i * 8);
            *p = encode8_again<F>(*p, s0, inv, s);
        }
    }
}

// ---------------------------------------------------------------------------
// read
//
// One team per page, head and side, so that page and scale are looked up
// once; a thread's 4 codes become one store of 16 (8) bytes beside its
// neighbours'.  Bound by the bytes written, which pass the caches by: 541 MB of
// floats in 105 us (6.4 TB/s with the codes read), 115 through them; 270 MB of
// 16-bit values in 60 us (6.8 TB/s).
// ---------------------------------------------------------------------------
template <int F, int T, int D>
__global__ __launch_bounds__(kThreads) void kv8_k_read(ccbKv8Cache c, ccbKv8Rows kOut,
                                                       ccbKv8Rows vOut, int32_t count,
                                                       const int32_t* first, int32_t span,
                                                       int32_t sides, uint32_t units, int32_t* err)
{
    constexpr int V = D / 4;
    const int32_t P = c.pageSize;
    const Team team(P, blockIdx.x);
    if (team.unit >= units) return;
    uint32_t rest = team.unit;
    const int32_t h = rest % (uint32_t)c.heads;
    rest /= (uint32_t)c.heads;
    const bool isV = sides == 2 || (sides == 3 && rest % 2 == 1);
    if (sides == 3) rest /= 2;
    const int32_t local = rest % (uint32_t)span;
    const int32_t b = rest / (uint32_t)span;
    int32_t len = checked_len(c.lens[b], c.maxPages * P);
    if (len < 0) {
        if (team.id == 0) report(err);
        len = 0;
    }
    const int64_t from = first != nullptr ? first[b] : 0;
    const int64_t start = (from & ~(int64_t)(P - 1)) + (int64_t)local * P;  // the page's first token
    const int32_t lo = start < from ? (int32_t)(from - start) : 0;          // slots lo .. hi - 1
    const int32_t hi = from + count - start < P ? (int32_t)(from + count - start) : P;
    if (lo >= hi) return;
    // slots below `held` have values
    int32_t held = start >= 0 && start < len ? (len - start < P ? (int32_t)(len - start) : P) : 0;
    int64_t block = 0;
    float s = 0.0f;
    if (held > lo) {
        const int32_t page = checked_page(c.pageTable[b * c.tableStride + (start >> __builtin_ctz(P))], c.numPages);
        if (page < 0) {
            if (team.id == 0) report(err);
            held = 0;
        } else {
            block = (int64_t)page * c.heads + h;
            s = (isV ? c.vScale : c.kScale)[block];
        }
    }
    const uint8_t* src = (const uint8_t*)(isV ? c.v : c.k) + block * P * D;
    const ccbKv8Rows& rows = isV ? vOut : kOut;
    const int64_t base = b * rows.strideBatch + h * rows.strideHead + (start - from) * rows.strideToken;
    for (int32_t i0 = lo * V + team.id; i0 < hi * V; i0 += 8 * team.size) {
        uint32_t w[8];  // eight loads in flight
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int32_t i = i0 + k * team.size;
            w[k] = 0;
            if (i < held * V && i < hi * V) w[k] = *(const uint32_t*)(src + i * 4);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int32_t i = i0 + k * team.size;
            if (i < hi * V) {
                float x[4];
                decode4<F>(w[k], x);  // code 0 is 0
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] *= s;
                const int64_t at = base + (i / V) * rows.strideToken + i % V * 4;
                if constexpr (T == CCB_KV8_FP32)
                    __builtin_nontemporal_store(f4{x[0], x[1], x[2], x[3]}, (f4*)((float*)rows.data + at));
                else
                    __builtin_nontemporal_store(u2{narrow<T>(x[0]) | (narrow<T>(x[1]) << 16),
                                                   narrow<T>(x[2]) | (narrow<T>(x[3]) << 16)},
                                                (u2*)((uint16_t*)rows.data + at));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// evict: the kept tokens into their new pages
//
// One team per new page, head and side: looks its tokens' places up once,
// gathers their codes into registers, finds the new scale, rounds the codes
// again and writes them.  Bound by instructions first: about 20 a code, 8 of
// them for rounding, fill the vector units for 2/3 of the time (16 x 1024 tokens of 8 heads, 66 MB in 26 us);
// of the waves' time 38% waits for their turn and 38% for memory, the chain
// token -> page -> codes.
// ---------------------------------------------------------------------------
struct MoveLds {
    int64_t place[128];  // where a token's codes start
    float scale[128];
    float reduce[4];
};

// One team's work: side isV of page `number` of a row, which is page `page` of
// the pool; the row's i-th kept token is token(i), `stay` stay.  Every thread
// of the workgroup calls this; a team that is not `valid` has nothing to do.
template <int F, int D, class Token>
__device__ __forceinline__ void move_page(const ccbKv8Cache& from, const ccbKv8Cache& to, int32_t budget,
                                          const Team& team, bool valid, int32_t row, int32_t number, bool isV,
                                          int32_t page, int32_t stay, int32_t* err, MoveLds& lds,
                                          Token&& token)
{
    constexpr int V = D / 16;              // vectors of 16 codes in a token
    constexpr int N = 128 * V / kThreads;  // of a thread for the largest page
    const int32_t P = from.pageSize, shift = __builtin_ctz(P);
    const int32_t b = row / (uint32_t)from.heads, h = row - b * from.heads;
    int64_t* place = lds.place + team.sub * P;
    float* tokenScale = lds.scale + team.sub * P;

    // (places past the kept tokens hold anything and are not used)
    const int32_t mine = number * P + team.id;
    const int32_t t = valid && team.id < P && mine < budget ? token(mine) : 0;
    page = checked_page(page, to.numPages);
    bool works = valid && number * P < stay;
    if (works && page < 0) {
        if (team.id == 0) report(err);
        works = false;
    }
    const int32_t n = !works ? 0 : stay - number * P < P ? stay - number * P : P;
    const uint8_t* codes = (const uint8_t*)(isV ? from.v : from.k);
    if (team.id < n) {
        const int32_t src = checked_page(from.pageTable[b * from.tableStride + (t >> shift)], from.numPages);
        if (src < 0) report(err);
        const int64_t block = (int64_t)(src < 0 ? 0 : src) * from.heads + h;
        place[team.id] = src < 0 ? -1 : (block * P + (t & (P - 1))) * D;
        tokenScale[team.id] = src < 0 ? 0.0f : (isV ? from.vScale : from.kScale)[block];
    }
    __syncthreads();
    uint4 raw[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int32_t i = k * team.size + team.id;
        raw[k] = make_uint4(0, 0, 0, 0);
        if (i < n * V) {
            const int64_t at = place[i / V];
            if (at >= 0) raw[k] = *(const uint4*)(codes + at + i % V * 16);
        }
    }
    float a = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int32_t i = k * team.size + team.id;
        if (i < n * V) {
            float x[16], m = 0.0f;
            decode4<F>(raw[k].x, x);
            decode4<F>(raw[k].y, x + 4);
            decode4<F>(raw[k].z, x + 8);
            decode4<F>(raw[k].w, x + 12);
#pragma unroll
            for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]));
            a = fmaxf(a, m * tokenScale[i / V]);
        }
    }
    a = team.largest(a, lds.reduce);
    if (!works) return;
    const float s = block_scale<F>(a);
    const float inv = 1.0f / s;
    const int64_t block = (int64_t)page * to.heads + h;
    if (team.id == 0) (isV ? to.vScale : to.kScale)[block] = s;
    uint4* dst = (uint4*)((uint8_t*)(isV ? to.v : to.k) + block * P * D);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int32_t i = k * team.size + team.id;
        if (i < n * V) {
            const float sOld = tokenScale[i / V];
            const uint2 x = encode8_again<F>(make_uint2(raw[k].x, raw[k].y), sOld, inv, s);
            const uint2 y = encode8_again<F>(make_uint2(raw[k].z, raw[k].w), sOld, inv, s);
            dst[i] = make_uint4(x.x, x.y, y.x, y.y);
        }
    }
}

template <int F, int D>
__global__ __launch_bounds__(kThreads) void kv8_k_move(ccbKv8Cache from, ccbKv8Cache to,
                                                       int32_t budget, uint32_t units,
                                                       const int32_t* index, int32_t* err)
{
    __shared__ MoveLds lds;
    const Team team(from.pageSize, blockIdx.x);
    const bool valid = team.unit < units;  // (the teams of a workgroup stay together)
    const uint32_t unit = valid ? team.unit >> 1 : 0;
    const uint32_t rows = (uint32_t)from.batch * (uint32_t)from.heads;
    const int32_t number = unit / rows, row = unit - number * rows;
    const int32_t* list = index + (int64_t)row * budget;
    const int32_t b = row / (uint32_t)from.heads;
    const int32_t page = to.pageTable[b * to.tableStride + number];
    int32_t len = checked_len(from.lens[b], from.maxPages * from.pageSize);
    if (len < 0) len = 0;  // the selection reports it
    move_page<F, D>(from, to, budget, team, valid, row, number, team.unit & 1, page, len < budget ? len : budget,
                    err, lds, [&](int32_t i) { return list[i]; });
}

// ---------------------------------------------------------------------------
// evict: which tokens stay
//
// The kept tokens are those whose key is above the k-th largest key, and the
// first few that equal it; the k-th largest is found 11, 11 and 10 bits at a
// time from the top with histograms in LDS (integer counts: the order of the
// atomics does not matter), and the search ends early where every key of the
// threshold's bin stays.  Each wave owns a run of tokens, so places among the
// kept ones need one scan over the waves' counts and then only votes within a
// wave.
//
// Rows of up to 16384 tokens are chosen from by one workgroup, which keeps
// them in registers (8 rows of 16000, with the move: 30 us, in segments 36; 512
// rows: 87 and 122).  A pass costs a CU about 0.2 us per 1024 tokens, so longer
// rows are cut into segments, one workgroup each, and the passes become
// kernels: each stage sums its row's histograms of the stage before, finds the
// bin, and counts the next bits of its segment.  Nothing waits inside a kernel.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kSelStep = 256;     // tokens of a wave's step, four to a lane
constexpr int kSelResident = 4;   // steps that stay in registers
constexpr int kSelShort = kSelWaves * kSelStep * kSelResident;
constexpr int kBins = 2048;

typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));

struct SelectArgs {
    ccbKv8Cache from, to;
    int32_t budget, recent, sinks;
    int32_t segments;  // of a row
    int32_t* index;    // [row][budget]
    int32_t* kept;
    int32_t* hist;     // [2][row][segment][kBins]
    int32_t* state;    // [2][row][kState]
    int2* counts;      // [row][segment]: tokens that stay for sure, and that equal the threshold
    int32_t* err;
};
constexpr int kState = 4;  // prefix, shift, need, whether the search is over

// Exclusive prefix sum of x over the workgroup.
__device__ __forceinline__ int32_t block_scan(int32_t x, int32_t* scratch)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int32_t v = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    if (lane == 63) scratch[wave] = v;
    __syncthreads();
    int32_t before = 0;
#pragma unroll
    for (int w = 0; w < kSelWaves; ++w) before += w < wave ? scratch[w] : 0;
    return before + v - x;
}

// Adds one to the bin of every lane that counts.  Lanes that share the first
// one's bin are added together: weights that are all alike would otherwise
// queue up 64 deep.
__device__ __forceinline__ void count_bin(int32_t* hist, uint32_t bin, bool counts)
{
    const uint64_t live = __ballot(counts);
    if (live == 0) return;
    const int leader = __builtin_ctzll(live);
    const uint32_t b0 = __builtin_amdgcn_readlane(bin, leader);
    const uint64_t same = __ballot(counts && bin == b0);
    if (counts && bin != b0) atomicAdd(&hist[bin], 1);
    if ((int)(threadIdx.x & 63) == leader) atomicAdd(&hist[b0], __popcll(same));
}

// What is known of a row's threshold.
struct Threshold {
    uint32_t prefix;  // its upper bits
    int32_t shift;    // below which they end
    int32_t need;     // how many of the tokens that equal it, so far, stay
    bool over;        // nothing is left to find
};

// The row's tokens and what is chosen among them.
struct Row {
    const float* w;
    int32_t len, low, high;  // chosen by weight: tokens low .. high - 1
    Threshold start;
};

__device__ __forceinline__ Row row_of(const SelectArgs& a, int64_t row)
{
    Row r;
    r.len = checked_len(a.from.lens[row / a.from.heads], a.from.maxPages * a.from.pageSize);
    if (r.len < 0) {
        if (threadIdx.x == 0) report(a.err);
        r.len = 0;
    }
    r.w = a.from.weight + row * a.from.weightStride;
    r.low = r.len > a.budget ? a.sinks : 0;
    r.high = r.len > a.budget ? r.len - a.recent : 0;
    const int32_t need = a.budget - a.sinks - a.recent;
    r.start = Threshold{0, 32, need, !(r.high > r.low && need > 0)};
    return r;
}

// Whether a token stays for sure, and whether it equals the threshold.
__device__ __forceinline__ void classify(const Row& r, const Threshold& th, int32_t t, float w, bool& sure,
                                         bool& equal)
{
    const bool middle = t >= r.low && t < r.high;
    const bool search = th.shift < 32;  // else none of the middle stays
    const uint32_t key = search ? weight_key(w) >> th.shift : 0u;
    sure = t < r.len && (!middle || (search && key > th.prefix));
    equal = middle && search && key == th.prefix;
}

// Four weights, those at and past `end` 0.
__device__ __forceinline__ f4u load4(const float* w, int32_t t, int32_t end)
{
    f4u v = {0, 0, 0, 0};
    if (t + 4 <= end) {
        v = *(const f4u*)(w + t);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (t + e < end) v[e] = w[t + e];
    }
    return v;
}

// Counts the bits [below, th.shift) of the tokens that share the threshold's
// upper bits; `each` goes over the workgroup's tokens.
template <class Each>
__device__ __forceinline__ void count_bits(const Row& r, const Threshold& th, int below, int32_t* hist,
                                           Each&& each)
{
    const uint32_t mask = (1u << (th.shift - below)) - 1;
    for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    each([&](int32_t t, const f4u& v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t key = weight_key(v[e]);
            count_bin(hist, (key >> below) & mask,
                      t + e >= r.low && t + e < r.high &&
                          (th.shift == 32 || (key >> (th.shift & 31)) == th.prefix));
        }
    });
    __syncthreads();
}

// The bin of the need-th largest, given this thread's two bins from the top.
__device__ __forceinline__ void find_bin(Threshold& th, int below, int32_t h0, int32_t h1, int32_t* scratch,
                                         int32_t* found)
{
    const int32_t before = block_scan(h0 + h1, scratch);
    if (before < th.need && th.need <= before + h0 + h1) {
        const bool second = th.need > before + h0;
        found[0] = kBins - 1 - 2 * (int32_t)threadIdx.x - (second ? 1 : 0);
        found[1] = before + (second ? h0 : 0);
        found[2] = second ? h1 : h0;
    }
    __syncthreads();
    th.prefix = (th.shift == 32 ? 0u : th.prefix << (th.shift - below)) | (uint32_t)found[0];
    th.need -= found[1];
    th.shift = below;
    th.over = below == 0 || th.need == found[2];
}

// This wave's tokens that stay for sure, and that equal the threshold.
template <class Each>
__device__ __forceinline__ int2 count_kept(const Row& r, const Threshold& th, Each&& each)
{
    int2 n = make_int2(0, 0);
    each([&](int32_t t, const f4u& v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bool s, q;
            classify(r, th, t + e, v[e], s, q);
            n.x += __popcll(__ballot(s)), n.y += __popcll(__ballot(q));
        }
    });
    return n;
}

// Writes the workgroup's kept tokens to `index` (the row's list) and to the
// results; `before` counts those ahead of them.
template <class Each>
__device__ __forceinline__ void write_kept(const SelectArgs& a, const Row& r, const Threshold& th, int64_t row,
                                           int32_t* index, int2 before, int2* scratch, Each&& each)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int2 n = count_kept(r, th, each);
    if (lane == 0) scratch[wave] = n;
    __syncthreads();
    for (int i = 0; i < wave; ++i) before.x += scratch[i].x, before.y += scratch[i].y;
    int32_t* kept = a.kept != nullptr ? a.kept + row * a.budget : nullptr;
    float* weight = a.to.weight != nullptr ? a.to.weight + row * a.to.weightStride : nullptr;
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    each([&](int32_t t, const f4u& v) {
        uint64_t sure[4], equal[4];
        int32_t s = before.x, q = before.y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bool isSure, isEqual;
            classify(r, th, t + e, v[e], isSure, isEqual);
            sure[e] = __ballot(isSure), equal[e] = __ballot(isEqual);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s += __popcll(sure[e] & below), q += __popcll(equal[e] & below);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool isSure = (sure[e] >> lane) & 1, isEqual = (equal[e] >> lane) & 1;
            if (isSure || (isEqual && q < th.need)) {
                const int32_t slot = s + (q < th.need ? q : th.need);
                index[slot] = t + e;
                if (kept != nullptr) kept[slot] = t + e;
                if (weight != nullptr) weight[slot] = v[e];
            }
            s += isSure, q += isEqual;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) before.x += __popcll(sure[e]), before.y += __popcll(equal[e]);
    });
}

// The end of a row: its length, and places that nothing was kept for.
__device__ __forceinline__ void finish_row(const SelectArgs& a, const Row& r, int64_t row)
{
    const int32_t stay = r.len < a.budget ? r.len : a.budget;
    if (threadIdx.x == 0 && row % a.from.heads == 0) a.to.lens[row / a.from.heads] = stay;
    for (int32_t i = stay + (int)threadIdx.x; i < a.budget; i += kSelThreads) {
        if (a.kept != nullptr) a.kept[row * a.budget + i] = -1;
        if (a.to.weight != nullptr) a.to.weight[row * a.to.weightStride + i] = 0.0f;
    }
}

// A row that one workgroup chooses from; `index` may lie in `hist`, which holds
// nothing any more when the list is written.
__device__ __forceinline__ void select_row(const SelectArgs& a, const Row& r, int64_t row, int32_t* index,
                                           int32_t* hist)
{
    __shared__ int32_t scratch[kSelWaves];
    __shared__ int2 places[kSelWaves];
    __shared__ int32_t found[3];
    // this wave's tokens: first + step * kSelStep + 4 * lane + e
    const int32_t steps = (r.len + kSelWaves * kSelStep - 1) / (kSelWaves * kSelStep);
    const int32_t first = (threadIdx.x >> 6) * steps * kSelStep + 4 * (threadIdx.x & 63);
    f4u held[kSelResident];
#pragma unroll
    for (int i = 0; i < kSelResident; ++i)
        if (i < steps) held[i] = load4(r.w, first + i * kSelStep, r.len);
    auto each = [&](auto&& f) {
#pragma unroll
        for (int i = 0; i < kSelResident; ++i)
            if (i < steps) f(first + i * kSelStep, held[i]);
    };
    Threshold th = r.start;
#pragma unroll 1
    for (int below = 21; !th.over; below = below == 21 ? 10 : 0) {
        count_bits(r, th, below, hist, each);
        const int32_t h0 = hist[kBins - 1 - 2 * threadIdx.x], h1 = hist[kBins - 2 - 2 * threadIdx.x];
        find_bin(th, below, h0, h1, scratch, found);
    }
    write_kept(a, r, th, row, index, make_int2(0, 0), places, each);
    finish_row(a, r, row);
}

__global__ __launch_bounds__(kSelThreads) void kv8_k_select_short(SelectArgs a)
{
    __shared__ int32_t hist[kBins];
    const int64_t row = blockIdx.x;
    select_row(a, row_of(a, row), row, a.index + row * a.budget, hist);
}

// The same, and the move of what was kept, where the workgroup's teams are as
// many as the row's new blocks (128 tokens, 256 in pages of 128): a launch less
// counts for more than other CUs' help.  204 rows that keep 28 tokens take 15
// us with the read after it instead of 18.7; with two rounds of blocks for a
// team, 12 rows of 138 tokens took 22.6 instead of 18.7.
template <int F, int D>
__global__ __launch_bounds__(kSelThreads) void kv8_k_select_move(SelectArgs a, int32_t nPages)
{
    __shared__ int32_t hist[kBins];
    __shared__ MoveLds lds[kSelThreads / kThreads];
    const int32_t row = blockIdx.x;
    const int32_t group = __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
    const Team team(a.from.pageSize, (uint32_t)group);
    const int32_t number = (int32_t)(team.unit >> 1);
    const bool valid = number < nPages;
    const int32_t page = a.to.pageTable[row / a.from.heads * a.to.tableStride + (valid ? number : 0)];
    const Row r = row_of(a, row);
    select_row(a, r, row, hist, hist);
    __syncthreads();  // the list is written
    move_page<F, D>(a.from, a.to, a.budget, team, valid, row, number, team.unit & 1, page,
                    r.len < a.budget ? r.len : a.budget, a.err, lds[group], [&](int32_t i) { return hist[i]; });
}

// One stage of a long row: 0, 1 and 2 count 11, 11 and 10 bits, 3 writes.
template <int S>
__global__ __launch_bounds__(kSelThreads) void kv8_k_select_long(SelectArgs a)
{
    __shared__ int32_t hist[kBins];
    __shared__ int32_t scratch[kSelWaves];
    __shared__ int2 places[kSelWaves];
    __shared__ int32_t found[3];
    const int64_t row = blockIdx.x / (uint32_t)a.segments;
    const int32_t seg = blockIdx.x % (uint32_t)a.segments;
    const int64_t rows = (int64_t)a.from.batch * a.from.heads;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // What the stage before left is asked for before the length says whether
    // there is a search at all (the workspace has the places in any case).
    int2 h = make_int2(0, 0), ahead = make_int2(0, 0);  // lower bin, higher bin; those of the segments before
    int4 st = make_int4(0, 0, 0, 0);
    if constexpr (S > 0) {
        const int32_t* in = a.hist + ((int64_t)((S + 1) & 1) * rows + row) * a.segments * kBins + kBins - 2 -
                            2 * (int32_t)threadIdx.x;
        if (S > 1) st = *(const int4*)(a.state + ((int64_t)((S + 1) & 1) * rows + row) * kState);
#pragma unroll 16
        for (int32_t i = 0; i < a.segments; ++i) {
            const int2 x = *(const int2*)(in + (int64_t)i * kBins);
            h.x += x.x, h.y += x.y;
            if (S == 3 && i < seg) ahead.x += x.x, ahead.y += x.y;
        }
    }
    const Row r = row_of(a, row);
    constexpr int32_t unit = kSelWaves * kSelStep;
    const int32_t size = (int32_t)(((r.len + (int64_t)a.segments * unit - 1) / ((int64_t)a.segments * unit)) * unit);
    const int64_t begin64 = (int64_t)seg * size;
    const int32_t begin = begin64 < r.len ? (int32_t)begin64 : r.len;
    const int32_t end = r.len - begin < size ? r.len : begin + size;
    const int32_t steps = (end - begin + unit - 1) / unit;
    const int32_t first = begin + wave * steps * kSelStep + 4 * lane;
    // the first two steps' weights come while the threshold is found
    f4u held[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (i < steps) held[i] = load4(r.w, first + i * kSelStep, end);
    auto each = [&](auto&& f) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (i < steps) f(first + i * kSelStep, held[i]);
        for (int32_t i = 2; i < steps; ++i) f(first + i * kSelStep, load4(r.w, first + i * kSelStep, end));
    };
    // tokens past the segment's end belong to the next one
    Row mine = r;
    mine.len = end;
    mine.high = r.high < end ? r.high : end;

    // the threshold, from the stage before
    Threshold th = r.start;
    if (S > 1 && !th.over) th.prefix = (uint32_t)st.x, th.shift = st.y, th.need = st.z, th.over = st.w != 0;
    const bool fresh = S > 0 && !th.over;
    if (fresh) find_bin(th, S == 1 ? 21 : S == 2 ? 10 : 0, h.y, h.x, scratch, found);
    if ((S == 1 || S == 2) && seg == 0 && threadIdx.x == 0) {
        *(int4*)(a.state + ((int64_t)(S & 1) * rows + row) * kState) =
            make_int4((int32_t)th.prefix, th.shift, th.need, th.over);
    }
    int2* counts = a.counts + row * a.segments;
    if constexpr (S == 2) {
        const int2 n = count_kept(mine, th, each);
        if (lane == 0) places[wave] = n;
        __syncthreads();
        if (threadIdx.x == 0) {
            int2 sum = make_int2(0, 0);
            for (int i = 0; i < kSelWaves; ++i) sum.x += places[i].x, sum.y += places[i].y;
            counts[seg] = sum;
        }
    }
    if constexpr (S < 3) {
        if (th.over) return;
        count_bits(mine, th, S == 0 ? 21 : S == 1 ? 10 : 0, hist, each);
        int32_t* out = a.hist + (((int64_t)(S & 1) * rows + row) * a.segments + seg) * kBins;
        for (int i = threadIdx.x; i < kBins; i += kSelThreads) out[i] = hist[i];
    } else {
        // kept in the segments before: what stage 2 was sure of, and by the last bits
        int2 before = make_int2(0, 0);
        if (fresh) {
            const int32_t low = kBins - 2 - 2 * (int32_t)threadIdx.x, bin = found[0];
            before.x = (low > bin ? ahead.x : 0) + (low + 1 > bin ? ahead.y : 0);
            before.y = low == bin ? ahead.x : low + 1 == bin ? ahead.y : 0;
        }
        for (int32_t i = threadIdx.x; i < seg; i += kSelThreads) {
            const int2 x = counts[i];
            before.x += x.x, before.y += fresh ? 0 : x.y;
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) {
            before.x += __shfl_xor(before.x, d, 64);
            before.y += __shfl_xor(before.y, d, 64);
        }
        if (lane == 0) places[wave] = before;
        __syncthreads();
        before = make_int2(0, 0);
        for (int i = 0; i < kSelWaves; ++i) before.x += places[i].x, before.y += places[i].y;
        __syncthreads();
        write_kept(a, mine, th, row, a.index + row * a.budget, before, places, each);
        if (seg == 0) finish_row(a, r, row);
    }
}

}  // namespace

namespace ccb {

// Blocks of the pages that n tokens can touch, starting anywhere in a page
// (one workgroup at most is rounded up: see team_groups); 0 for too many.
static int64_t touched_blocks(const ccbKv8Cache& c, int32_t n, int32_t sides)
{
    const int64_t pairs = (int64_t)c.batch * c.heads;
    const int64_t span = ((int64_t)n + c.pageSize - 2) / c.pageSize + 1;
    const int64_t blocks = pairs > INT32_MAX ? 0 : pairs * span * sides;
    return blocks <= INT32_MAX && kv8_launch_fits(team_groups(blocks, c.pageSize), kThreads) ? blocks : 0;
}

bool kv8_append_fits(const ccbKv8Cache& c, int32_t nNew) { return touched_blocks(c, nNew, 2) != 0; }

bool kv8_read_fits(const ccbKv8Cache& c, int32_t count, int32_t sides)
{
    return touched_blocks(c, count, sides) != 0;
}

hipError_t kv8_append(const ccbKv8Cache& c, const ccbKv8Rows& k, const ccbKv8Rows& v, int32_t nNew,
                      const int32_t* counts, int32_t* err, hipStream_t s)
{
    // pages that nNew tokens can touch, starting anywhere in a page
    const int32_t span = (nNew + c.pageSize - 2) / c.pageSize + 1;
    const int64_t blocks = touched_blocks(c, nNew, 2);
    const uint32_t units = (uint32_t)blocks;
    const int64_t groups = team_groups(blocks, c.pageSize);
#define KV8_APPEND(F, T, D) \
    enqueue(kv8_k_append<F, T, D>, groups, kThreads, s, c, k, v, nNew, counts, span, units, err)
#define KV8_APPEND_DIM(D) \
    (c.format == CCB_KV8_INT8 \
         ? (k.type == CCB_KV8_BF16 ? KV8_APPEND(kInt8, CCB_KV8_BF16, D) : KV8_APPEND(kInt8, CCB_KV8_FP16, D)) \
         : (k.type == CCB_KV8_BF16 ? KV8_APPEND(kE4m3, CCB_KV8_BF16, D) : KV8_APPEND(kE4m3, CCB_KV8_FP16, D)))
    return KV8_BY_DIM(c.headDim, KV8_APPEND_DIM);
}

hipError_t kv8_read(const ccbKv8Cache& c, const ccbKv8Rows* k, const ccbKv8Rows* v, int32_t count,
                    const int32_t* first, int32_t* err, hipStream_t s)
{
    const int32_t sides = (k != nullptr ? 1 : 0) | (v != nullptr ? 2 : 0);
    // pages that count tokens can touch, starting anywhere in a page
    const int32_t span = (int32_t)(((int64_t)count + c.pageSize - 2) / c.pageSize + 1);
    const int64_t blocks = touched_blocks(c, count, sides == 3 ? 2 : 1);
    const ccbKv8Rows kr = k != nullptr ? *k : *v, vr = v != nullptr ? *v : *k;
    const uint32_t units = (uint32_t)blocks;
    const int64_t groups = team_groups(blocks, c.pageSize);
#define KV8_READ(F, T, D) \
    enqueue(kv8_k_read<F, T, D>, groups, kThreads, s, c, kr, vr, count, first, span, sides, units, err)
#define KV8_READ_T(F, D) \
    (kr.type == CCB_KV8_BF16   ? KV8_READ(F, CCB_KV8_BF16, D) \
     : kr.type == CCB_KV8_FP16 ? KV8_READ(F, CCB_KV8_FP16, D) \
                               : KV8_READ(F, CCB_KV8_FP32, D))
#define KV8_READ_DIM(D) (c.format == CCB_KV8_INT8 ? KV8_READ_T(kInt8, D) : KV8_READ_T(kE4m3, D))
    return KV8_BY_DIM(c.headDim, KV8_READ_DIM);
}

// Segments of a row, 0 where one workgroup chooses by itself, and the
// workspace's parts; returns its bytes.  There is a sequence.
static size_t select_plan(SelectArgs& a, const ccbKv8Cache& from, int32_t budget, void* ws)
{
    const int64_t rows = (int64_t)from.batch * from.heads;
    const int64_t room = (int64_t)from.maxPages * from.pageSize;
    a.segments = 0;
    if (room > kSelShort) {
        // 8192 tokens and more for each, two workgroups on a CU at most
        const int64_t most = rows < 256 ? 512 / rows : 2;
        int64_t n = (room + 8191) / 8192;
        n = n < most ? n : most;
        a.segments = (int32_t)(n < 64 ? n : 64);
    }
    size_t bytes = 0;
    auto take = [&](int64_t n, size_t each) {
        char* here = (char*)ws + bytes;
        bytes += ((size_t)n * each + 127) / 128 * 128;
        return here;
    };
    a.index = (int32_t*)take(rows * budget, sizeof(int32_t));
    a.hist = (int32_t*)take(2 * rows * a.segments * kBins, sizeof(int32_t));
    a.state = (int32_t*)take(a.segments ? 2 * rows * kState : 0, sizeof(int32_t));
    a.counts = (int2*)take(rows * a.segments, sizeof(int2));
    return bytes;
}

size_t kv8_evict_bytes(const ccbKv8Cache& from, int32_t budget)
{
    if (from.batch == 0) return 0;
    SelectArgs a;
    return select_plan(a, from, budget, nullptr);
}

bool kv8_evict_fits(const ccbKv8Cache& from, int32_t budget)
{
    const int64_t rows = (int64_t)from.batch * from.heads;
    if (rows > INT32_MAX) return false;
    SelectArgs a;
    select_plan(a, from, budget, nullptr);
    const int64_t blocks = rows * ((budget + from.pageSize - 1) / from.pageSize) * 2;
    return kv8_launch_fits(rows * (a.segments > 0 ? a.segments : 1), kSelThreads) && blocks <= INT32_MAX &&
           kv8_launch_fits(team_groups(blocks, from.pageSize), kThreads);
}

hipError_t kv8_evict(const ccbKv8Cache& from, const ccbKv8Cache& to, int32_t budget, int32_t recent,
                     int32_t sinks, int32_t* kept, void* ws, int32_t* err, hipStream_t s)
{
    SelectArgs a;
    select_plan(a, from, budget, ws);
    a.from = from, a.to = to;
    a.budget = budget, a.recent = recent, a.sinks = sinks;
    a.kept = kept, a.err = err;
    const int32_t* index = a.index;
    const int32_t nPages = (budget + from.pageSize - 1) / from.pageSize;
    const int64_t rows = (int64_t)from.batch * from.heads;
    const int64_t blocks = rows * nPages * 2;
    const int32_t teams = kSelThreads / kThreads * (from.pageSize >= 64 ? 1 : 64 / from.pageSize);
    if (a.segments == 0 && 2 * nPages <= teams) {
#define KV8_SELECT_MOVE(F, D) enqueue(kv8_k_select_move<F, D>, rows, kSelThreads, s, a, nPages)
#define KV8_SELECT_MOVE_DIM(D) \
    (from.format == CCB_KV8_INT8 ? KV8_SELECT_MOVE(kInt8, D) : KV8_SELECT_MOVE(kE4m3, D))
        return KV8_BY_DIM(from.headDim, KV8_SELECT_MOVE_DIM);
    }
    hipError_t e = hipSuccess;
    if (a.segments == 0) {
        e = enqueue(kv8_k_select_short, rows, kSelThreads, s, a);
    } else {
        for (auto stage : {kv8_k_select_long<0>, kv8_k_select_long<1>, kv8_k_select_long<2>, kv8_k_select_long<3>})
            if (e == hipSuccess) e = enqueue(stage, rows * a.segments, kSelThreads, s, a);
    }
    if (e != hipSuccess) return e;
    const uint32_t units = (uint32_t)blocks;
    const int64_t groups = team_groups(blocks, from.pageSize);
#define KV8_MOVE(F, D) enqueue(kv8_k_move<F, D>, groups, kThreads, s, from, to, budget, units, index, err)
#define KV8_MOVE_DIM(D) (from.format == CCB_KV8_INT8 ? KV8_MOVE(kInt8, D) : KV8_MOVE(kE4m3, D))
    return KV8_BY_DIM(from.headDim, KV8_MOVE_DIM);
}

}  // namespace ccb
