// ccb_kv8_cache.hip -- the kernels that fill, cut and read the 8-bit
// key/value cache: append, evict, read.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccb_kv8_internal.h"
#include "ccb_kv8_device.h"

namespace {

using namespace kv8;

constexpr int kThreads = 256;

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
// One workgroup per touched page, head and side (K or V): the largest new
// value gives the block's scale, then the new values are rounded and, where
// the scale grew, the block's older codes are rounded again.  Blocks are
// independent, so there is nothing to join.  Bound by the bytes of the new
// values and codes; one-token steps by latency.
// ---------------------------------------------------------------------------
template <int F, int T, int D>
__global__ __launch_bounds__(kThreads) void kv8_k_append(ccbKv8Cache c, ccbKv8Rows kNew,
                                                         ccbKv8Rows vNew, int32_t nNew,
                                                         const int32_t* counts, int32_t span,
                                                         int32_t* err)
{
    __shared__ float scratch[4];
    const bool isV = blockIdx.x & 1;
    uint32_t rest = blockIdx.x >> 1;
    const int32_t h = rest % (uint32_t)c.heads;
    rest /= (uint32_t)c.heads;
    const int32_t local = rest % (uint32_t)span;
    const int32_t b = rest / (uint32_t)span;
    const int32_t P = c.pageSize;

    const int32_t len = checked_len(c.lens[b], c.maxPages * P);
    const int32_t cnt = counts != nullptr ? counts[b] : nNew;
    if (len < 0 || cnt < 0 || cnt > nNew || cnt > len) {
        if (threadIdx.x == 0) report(err);
        return;
    }
    const int32_t start = len - cnt;
    const int32_t number = start / P + local;
    if (cnt == 0 || number * P >= len) return;
    const int32_t lo = start > number * P ? start - number * P : 0;  // new slots lo .. hi - 1
    const int32_t hi = len - number * P < P ? len - number * P : P;
    if (!isV && c.weight != nullptr) {
        float* w = c.weight + ((int64_t)b * c.heads + h) * c.weightStride + (int64_t)number * P;
        for (int32_t i = lo + (int)threadIdx.x; i < hi; i += kThreads) w[i] = 0.0f;
    }
    const int32_t page = checked_page(c.pageTable[b * c.tableStride + number], c.numPages);
    if (page < 0) {
        if (threadIdx.x == 0) report(err);
        return;
    }
    constexpr int V = D / 8;  // vectors of 8 values per token
    const ccbKv8Rows& rows = isV ? vNew : kNew;
    const uint16_t* src = (const uint16_t*)rows.data + b * rows.strideBatch + h * rows.strideHead +
                          (int64_t)(number * P + lo - start) * rows.strideToken;
    const int64_t block = (int64_t)page * c.heads + h;
    uint8_t* dst = (uint8_t*)(isV ? c.v : c.k) + block * P * D;
    float* scale = (isV ? c.vScale : c.kScale) + block;

    // the new values stay in registers between finding the scale and rounding
    constexpr int N = 128 * V / kThreads;  // vectors of a thread for the largest page
    const int32_t nVec = (hi - lo) * V;
    uint4 raw[N];
    float a = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int32_t i = k * kThreads + (int32_t)threadIdx.x;
        raw[k] = make_uint4(0, 0, 0, 0);
        if (i < nVec) raw[k] = *(const uint4*)(src + (i / V) * rows.strideToken + (i % V) * 8);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (k * kThreads < nVec) {
            float x[8];
            widen8<T>(raw[k], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float m = fabsf(x[j]);
                a = (m > a && m < INFINITY) ? m : a;
            }
        }
    }
    const float s0 = lo > 0 ? *scale : 0.0f;
    a = block_max(a, scratch);
    const float s1 = block_scale<F>(a);
    const float s = s1 > s0 ? s1 : s0;
    const float inv = 1.0f / s;
    if (threadIdx.x == 0) *scale = s;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int32_t i = k * kThreads + (int32_t)threadIdx.x;
        if (i < nVec) {
            float x[8];
            widen8<T>(raw[k], x);
            *(uint2*)(dst + (int64_t)lo * D + (int64_t)i * 8) = encode8<F>(x, inv, s);
        }
    }
    if (lo > 0 && s > s0) {  // older codes of a block whose scale grew
        for (int32_t i = threadIdx.x; i < lo * V; i += kThreads) {
            uint2* p = (uint2*)(dst + (int64_t)i * 8);
            *p = encode8_again<F>(*p, s0, inv, s);
        }
    }
}

// ---------------------------------------------------------------------------
// read
//
// One workgroup per page, head and side, so that page and scale are looked up
// once; a thread's 4 codes become one store of 16 (8) bytes beside its
// neighbours'.  Bound by the bytes written.
// ---------------------------------------------------------------------------
template <int F, int T, int D>
__global__ __launch_bounds__(kThreads) void kv8_k_read(ccbKv8Cache c, ccbKv8Rows kOut,
                                                       ccbKv8Rows vOut, int32_t count,
                                                       const int32_t* first, int32_t span,
                                                       int32_t sides, int32_t* err)
{
    constexpr int V = D / 4;
    uint32_t rest = blockIdx.x;
    const int32_t h = rest % (uint32_t)c.heads;
    rest /= (uint32_t)c.heads;
    const bool isV = sides == 2 || (sides == 3 && rest % 2 == 1);
    if (sides == 3) rest /= 2;
    const int32_t local = rest % (uint32_t)span;
    const int32_t b = rest / (uint32_t)span;
    const int32_t P = c.pageSize;
    int32_t len = checked_len(c.lens[b], c.maxPages * P);
    if (len < 0) {
        if (threadIdx.x == 0) report(err);
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
        const int32_t page = checked_page(c.pageTable[b * c.tableStride + start / P], c.numPages);
        if (page < 0) {
            if (threadIdx.x == 0) report(err);
            held = 0;
        } else {
            block = (int64_t)page * c.heads + h;
            s = (isV ? c.vScale : c.kScale)[block];
        }
    }
    const uint8_t* src = (const uint8_t*)(isV ? c.v : c.k) + block * P * D;
    const ccbKv8Rows& rows = isV ? vOut : kOut;
    const int64_t base = b * rows.strideBatch + h * rows.strideHead + (start - from) * rows.strideToken;
    for (int32_t i0 = lo * V + (int32_t)threadIdx.x; i0 < hi * V; i0 += 8 * kThreads) {
        uint32_t w[8];  // eight loads in flight
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int32_t i = i0 + k * kThreads;
            w[k] = 0;
            if (i < held * V && i < hi * V) w[k] = *(const uint32_t*)(src + i * 4);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int32_t i = i0 + k * kThreads;
            if (i < hi * V) {
                float x[4];
                decode4<F>(w[k], x);  // code 0 is 0
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] *= s;
                const int64_t at = base + (i / V) * rows.strideToken + i % V * 4;
                if constexpr (T == CCB_KV8_FP32)
                    *(float4*)((float*)rows.data + at) = make_float4(x[0], x[1], x[2], x[3]);
                else
                    *(uint2*)((uint16_t*)rows.data + at) =
                        make_uint2(narrow<T>(x[0]) | (narrow<T>(x[1]) << 16),
                                   narrow<T>(x[2]) | (narrow<T>(x[3]) << 16));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// evict: which tokens stay
//
// One workgroup per sequence and head.  The kept tokens are those whose key
// is above the k-th largest key, and the first few that equal it; the k-th
// largest is found 11, 11 and 10 bits at a time from the top with a histogram
// in LDS (integer counts: the order of the atomics does not matter), and the
// search ends early where every key of the threshold's bin stays.
//
// Each wave owns a run of tokens, so places among the kept ones need one scan
// over the waves' counts and then only votes within the wave.  Rows of up to
// 16384 tokens stay in registers between the passes; longer ones are read
// again from L2 (four times in all).
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kSelStep = 256;     // tokens of a wave's step, four to a lane
constexpr int kSelResident = 4;   // steps that stay in registers
constexpr int kBins = 2048;

typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));

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

struct SelectOut {
    int32_t* index;
    int32_t* kept;
    float* weight;
};

template <bool R>
__device__ __forceinline__ void select_row(const float* w, int32_t len, int32_t low, int32_t high,
                                           int32_t need, const SelectOut& out, int32_t* hist,
                                           int32_t* scratch, int32_t* found)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // this wave's tokens: first + step * kSelStep + 4 * lane + e
    const int32_t steps = ((len + kSelWaves - 1) / kSelWaves + kSelStep - 1) / kSelStep;
    const int32_t first = wave * steps * kSelStep + 4 * lane;
    auto load = [&](int32_t step) {
        const int32_t t = first + step * kSelStep;
        f4u v = {0, 0, 0, 0};
        if (t + 4 <= len) {
            v = *(const f4u*)(w + t);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (t + e < len) v[e] = w[t + e];
        }
        return v;
    };
    f4u held[kSelResident];
    if (R) {
#pragma unroll
        for (int i = 0; i < kSelResident; ++i)
            if (i < steps) held[i] = load(i);
    }
    auto each = [&](auto&& f) {
        if (R) {
#pragma unroll
            for (int i = 0; i < kSelResident; ++i)
                if (i < steps) f(first + i * kSelStep, held[i]);
        } else {
            int32_t i = 0;
            for (; i + 4 <= steps; i += 4) {  // four loads in flight
                f4u v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = load(i + k);
#pragma unroll
                for (int k = 0; k < 4; ++k) f(first + (i + k) * kSelStep, v[k]);
            }
            for (; i < steps; ++i) f(first + i * kSelStep, load(i));
        }
    };

    uint32_t prefix = 0;  // the threshold's upper bits, found so far
    int shift = 32;       // below which they end
    const bool search = high > low && need > 0;
    for (int pass = 0; search && pass < 3; ++pass) {
        const int above = shift;
        shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = (1u << (above - shift)) - 1;
        for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        each([&](int32_t t, const f4u& v) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t key = weight_key(v[e]);
                count_bin(hist, (key >> shift) & mask,
                          t + e >= low && t + e < high && (pass == 0 || (key >> above) == prefix));
            }
        });
        __syncthreads();
        // the bin of the need-th largest: two bins to a thread, from the top
        const int32_t h0 = hist[kBins - 1 - 2 * threadIdx.x], h1 = hist[kBins - 2 - 2 * threadIdx.x];
        const int32_t before = block_scan(h0 + h1, scratch);
        if (before < need && need <= before + h0 + h1) {
            const bool second = need > before + h0;
            found[0] = kBins - 1 - 2 * (int32_t)threadIdx.x - (second ? 1 : 0);
            found[1] = before + (second ? h0 : 0);
            found[2] = second ? h1 : h0;
        }
        __syncthreads();
        prefix = (prefix << (above - shift)) | (uint32_t)found[0];
        need -= found[1];
        if (need == found[2]) break;  // (alike in every thread)
    }
    // need: how many of the tokens that equal the threshold, as far as it is known, stay
    auto votes = [&](int32_t t, const f4u& v, uint64_t* sure, uint64_t* equal) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool middle = t + e >= low && t + e < high;
            const uint32_t key = search ? weight_key(v[e]) >> shift : 0u;
            sure[e] = __ballot(t + e < len && (middle ? search && key > prefix : true));
            equal[e] = __ballot(middle && search && key == prefix);
        }
    };
    int32_t nSure = 0, nEqual = 0;
    each([&](int32_t t, const f4u& v) {
        uint64_t sure[4], equal[4];
        votes(t, v, sure, equal);
#pragma unroll
        for (int e = 0; e < 4; ++e) nSure += __popcll(sure[e]), nEqual += __popcll(equal[e]);
    });
    __syncthreads();
    if (lane == 0) hist[wave] = nSure, hist[kSelWaves + wave] = nEqual;
    __syncthreads();
    int32_t sureBefore = 0, equalBefore = 0;
    for (int i = 0; i < wave; ++i) sureBefore += hist[i], equalBefore += hist[kSelWaves + i];
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    each([&](int32_t t, const f4u& v) {
        uint64_t sure[4], equal[4];
        votes(t, v, sure, equal);
        int32_t s = sureBefore, q = equalBefore;
#pragma unroll
        for (int e = 0; e < 4; ++e) s += __popcll(sure[e] & below), q += __popcll(equal[e] & below);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool isSure = (sure[e] >> lane) & 1, isEqual = (equal[e] >> lane) & 1;
            if (isSure || (isEqual && q < need)) {
                const int32_t slot = s + (q < need ? q : need);
                out.index[slot] = t + e;
                if (out.kept != nullptr) out.kept[slot] = t + e;
                if (out.weight != nullptr) out.weight[slot] = v[e];
            }
            s += isSure, q += isEqual;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sureBefore += __popcll(sure[e]), equalBefore += __popcll(equal[e]);
    });
}

__global__ __launch_bounds__(kSelThreads) void kv8_k_select(ccbKv8Cache from, ccbKv8Cache to,
                                                            int32_t budget, int32_t recent,
                                                            int32_t sinks, int32_t* index,
                                                            int32_t* kept, int32_t* err)
{
    __shared__ int32_t hist[kBins];
    __shared__ int32_t scratch[kSelWaves];
    __shared__ int32_t found[3];
    const int32_t b = blockIdx.x / (uint32_t)from.heads;
    int32_t len = checked_len(from.lens[b], from.maxPages * from.pageSize);
    if (len < 0) {
        if (threadIdx.x == 0) report(err);
        len = 0;
    }
    const int64_t row = blockIdx.x;
    const float* w = from.weight + row * from.weightStride;
    SelectOut out;
    out.index = index + row * budget;
    out.kept = kept != nullptr ? kept + row * budget : nullptr;
    out.weight = to.weight != nullptr ? to.weight + row * to.weightStride : nullptr;
    const int32_t stay = len < budget ? len : budget;
    if (threadIdx.x == 0 && row % from.heads == 0) to.lens[b] = stay;
    // chosen by weight: `need` of the tokens between low and high
    const int32_t low = len > budget ? sinks : 0, high = len > budget ? len - recent : 0;
    const int32_t need = budget - sinks - recent;
    if (len <= kSelWaves * kSelResident * kSelStep)
        select_row<true>(w, len, low, high, need, out, hist, scratch, found);
    else
        select_row<false>(w, len, low, high, need, out, hist, scratch, found);
    for (int32_t i = stay + (int)threadIdx.x; i < budget; i += kSelThreads) {
        if (out.kept != nullptr) out.kept[i] = -1;
        if (out.weight != nullptr) out.weight[i] = 0.0f;
    }
}

// ---------------------------------------------------------------------------
// evict: the kept tokens into their new pages
//
// One workgroup per new page, head and side: looks its tokens' places up once,
// gathers their codes into registers, finds the new scale, rounds the codes
// again and writes them.  Bound by the gathered and written bytes.
// ---------------------------------------------------------------------------
template <int F, int D>
__global__ __launch_bounds__(kThreads) void kv8_k_move(ccbKv8Cache from, ccbKv8Cache to,
                                                       int32_t budget, int32_t nPages,
                                                       const int32_t* index, int32_t* err)
{
    constexpr int V = D / 16;              // vectors of 16 codes in a token
    constexpr int N = 128 * V / kThreads;  // of a thread for the largest page
    __shared__ float scratch[4];
    __shared__ int64_t place[128];    // where a token's codes start
    __shared__ float tokenScale[128];
    const bool isV = blockIdx.x & 1;
    uint32_t rest = blockIdx.x >> 1;
    const int32_t h = rest % (uint32_t)from.heads;
    rest /= (uint32_t)from.heads;
    const int32_t number = rest % (uint32_t)nPages;
    const int32_t b = rest / (uint32_t)nPages;
    const int32_t P = from.pageSize;

    int32_t len = checked_len(from.lens[b], from.maxPages * P);
    if (len < 0) len = 0;  // the selection reports it
    const int32_t stay = len < budget ? len : budget;
    if (number * P >= stay) return;
    const int32_t n = stay - number * P < P ? stay - number * P : P;
    const int32_t page = checked_page(to.pageTable[b * to.tableStride + number], to.numPages);
    if (page < 0) {
        if (threadIdx.x == 0) report(err);
        return;
    }
    const uint8_t* codes = (const uint8_t*)(isV ? from.v : from.k);
    if ((int32_t)threadIdx.x < n) {
        const int32_t t = index[((int64_t)b * from.heads + h) * budget + number * P + threadIdx.x];
        const int32_t src = checked_page(from.pageTable[b * from.tableStride + t / P], from.numPages);
        if (src < 0) report(err);
        const int64_t block = (int64_t)(src < 0 ? 0 : src) * from.heads + h;
        place[threadIdx.x] = src < 0 ? -1 : (block * P + t % P) * D;
        tokenScale[threadIdx.x] = src < 0 ? 0.0f : (isV ? from.vScale : from.kScale)[block];
    }
    __syncthreads();
    uint4 raw[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int32_t i = k * kThreads + (int32_t)threadIdx.x;
        raw[k] = make_uint4(0, 0, 0, 0);
        if (i < n * V) {
            const int64_t at = place[i / V];
            if (at >= 0) raw[k] = *(const uint4*)(codes + at + i % V * 16);
        }
    }
    float a = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int32_t i = k * kThreads + (int32_t)threadIdx.x;
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
    a = block_max(a, scratch);
    const float s = block_scale<F>(a);
    const float inv = 1.0f / s;
    const int64_t block = (int64_t)page * to.heads + h;
    if (threadIdx.x == 0) (isV ? to.vScale : to.kScale)[block] = s;
    uint4* dst = (uint4*)((uint8_t*)(isV ? to.v : to.k) + block * P * D);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int32_t i = k * kThreads + (int32_t)threadIdx.x;
        if (i < n * V) {
            const float sOld = tokenScale[i / V];
            const uint2 x = encode8_again<F>(make_uint2(raw[k].x, raw[k].y), sOld, inv, s);
            const uint2 y = encode8_again<F>(make_uint2(raw[k].z, raw[k].w), sOld, inv, s);
            dst[i] = make_uint4(x.x, x.y, y.x, y.y);
        }
    }
}

}  // namespace

namespace ccb {

hipError_t kv8_append(const ccbKv8Cache& c, const ccbKv8Rows& k, const ccbKv8Rows& v, int32_t nNew,
                      const int32_t* counts, int32_t* err, hipStream_t s)
{
    // pages that nNew tokens can touch, starting anywhere in a page
    const int32_t span = (nNew + c.pageSize - 2) / c.pageSize + 1;
    const int64_t blocks = (int64_t)c.batch * span * c.heads * 2;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
#define KV8_APPEND(F, T, D) \
    (kv8_k_append<F, T, D><<<dim3((unsigned)blocks), dim3(kThreads), 0, s>>>(c, k, v, nNew, counts, span, err), 0)
#define KV8_APPEND_DIM(D) \
    (c.format == CCB_KV8_INT8 \
         ? (k.type == CCB_KV8_BF16 ? KV8_APPEND(kInt8, CCB_KV8_BF16, D) : KV8_APPEND(kInt8, CCB_KV8_FP16, D)) \
         : (k.type == CCB_KV8_BF16 ? KV8_APPEND(kE4m3, CCB_KV8_BF16, D) : KV8_APPEND(kE4m3, CCB_KV8_FP16, D)))
    (void)KV8_BY_DIM(c.headDim, KV8_APPEND_DIM);
    return hipGetLastError();
}

hipError_t kv8_read(const ccbKv8Cache& c, const ccbKv8Rows* k, const ccbKv8Rows* v, int32_t count,
                    const int32_t* first, int32_t* err, hipStream_t s)
{
    const int32_t sides = (k != nullptr ? 1 : 0) | (v != nullptr ? 2 : 0);
    // pages that count tokens can touch, starting anywhere in a page
    const int32_t span = (int32_t)(((int64_t)count + c.pageSize - 2) / c.pageSize + 1);
    const int64_t blocks = (int64_t)c.batch * span * c.heads * (sides == 3 ? 2 : 1);
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    const ccbKv8Rows kr = k != nullptr ? *k : *v, vr = v != nullptr ? *v : *k;
#define KV8_READ(F, T, D) \
    (kv8_k_read<F, T, D><<<dim3((unsigned)blocks), dim3(kThreads), 0, s>>>(c, kr, vr, count, first, span, sides, err), 0)
#define KV8_READ_T(F, D) \
    (kr.type == CCB_KV8_BF16   ? KV8_READ(F, CCB_KV8_BF16, D) \
     : kr.type == CCB_KV8_FP16 ? KV8_READ(F, CCB_KV8_FP16, D) \
                               : KV8_READ(F, CCB_KV8_FP32, D))
#define KV8_READ_DIM(D) (c.format == CCB_KV8_INT8 ? KV8_READ_T(kInt8, D) : KV8_READ_T(kE4m3, D))
    (void)KV8_BY_DIM(c.headDim, KV8_READ_DIM);
    return hipGetLastError();
}

size_t kv8_evict_bytes(const ccbKv8Cache& from, int32_t budget)
{
    return (size_t)from.batch * from.heads * budget * sizeof(int32_t);
}

hipError_t kv8_evict(const ccbKv8Cache& from, const ccbKv8Cache& to, int32_t budget, int32_t recent,
                     int32_t sinks, int32_t* kept, void* ws, int32_t* err, int numCUs, hipStream_t s)
{
    (void)numCUs;
    int32_t* index = (int32_t*)ws;
    const int32_t nPages = (budget + from.pageSize - 1) / from.pageSize;
    const int64_t rows = (int64_t)from.batch * from.heads;
    const int64_t blocks = rows * nPages * 2;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    kv8_k_select<<<dim3((unsigned)rows), dim3(kSelThreads), 0, s>>>(from, to, budget, recent, sinks,
                                                                   index, kept, err);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
#define KV8_MOVE(F, D) \
    (kv8_k_move<F, D><<<dim3((unsigned)blocks), dim3(kThreads), 0, s>>>(from, to, budget, nPages, index, err), 0)
#define KV8_MOVE_DIM(D) (from.format == CCB_KV8_INT8 ? KV8_MOVE(kInt8, D) : KV8_MOVE(kE4m3, D))
    (void)KV8_BY_DIM(from.headDim, KV8_MOVE_DIM);
    return hipGetLastError();
}

}  // namespace ccb
