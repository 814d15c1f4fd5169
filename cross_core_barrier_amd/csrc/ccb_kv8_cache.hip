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

    float a = 0.0f;
    const int32_t nVec = (hi - lo) * V;
    for (int32_t i = threadIdx.x; i < nVec; i += kThreads) {
        float x[8];
        widen8<T>(*(const uint4*)(src + (i / V) * rows.strideToken + (i % V) * 8), x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float m = fabsf(x[j]);
            a = (m > a && m < INFINITY) ? m : a;
        }
    }
    const float s0 = lo > 0 ? *scale : 0.0f;
    a = block_max(a, scratch);
    const float s1 = block_scale<F>(a);
    const float s = s1 > s0 ? s1 : s0;
    const float inv = 1.0f / s;
    if (threadIdx.x == 0) *scale = s;
    for (int32_t i = threadIdx.x; i < nVec; i += kThreads) {
        float x[8];
        widen8<T>(*(const uint4*)(src + (i / V) * rows.strideToken + (i % V) * 8), x);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j / 4] |= (uint32_t)encode_value<F>(x[j], inv, s) << (8 * (j % 4));
        *(uint2*)(dst + (int64_t)lo * D + (int64_t)i * 8) = make_uint2(w[0], w[1]);
    }
    if (lo > 0 && s > s0) {  // older codes of a block whose scale grew
        for (int32_t i = threadIdx.x; i < lo * V; i += kThreads) {
            uint2* p = (uint2*)(dst + (int64_t)i * 8);
            const uint2 u = *p;
            float x[8];
            decode4<F>(u.x, x);
            decode4<F>(u.y, x + 4);
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j / 4] |= (uint32_t)encode_again<F>(x[j], s0, inv, s) << (8 * (j % 4));
            *p = make_uint2(w[0], w[1]);
        }
    }
}

// ---------------------------------------------------------------------------
// read
// ---------------------------------------------------------------------------
template <int F, int T, int D>
__global__ __launch_bounds__(kThreads) void kv8_k_read(ccbKv8Cache c, ccbKv8Rows kOut,
                                                       ccbKv8Rows vOut, int32_t count,
                                                       const int32_t* first, int32_t perGroup,
                                                       int32_t nGroups, int32_t sides, int32_t* err)
{
    constexpr int V = D / 8;
    uint32_t rest = blockIdx.x;
    const int32_t group = rest % (uint32_t)nGroups;
    rest /= (uint32_t)nGroups;
    const bool isV = sides == 2 || (sides == 3 && rest % 2 == 1);
    const int32_t b = sides == 3 ? rest / 2 : rest;
    const int32_t P = c.pageSize;
    int32_t len = checked_len(c.lens[b], c.maxPages * P);
    if (len < 0) {
        if (threadIdx.x == 0) report(err);
        len = 0;
    }
    const int64_t from = first != nullptr ? first[b] : 0;
    const ccbKv8Rows& rows = isV ? vOut : kOut;
    const int32_t i0 = group * perGroup;
    const int32_t n = count - i0 < perGroup ? count - i0 : perGroup;
    const int32_t perToken = c.heads * V;
    for (int32_t j = threadIdx.x; j < n * perToken; j += kThreads) {
        const int32_t i = i0 + j / perToken;
        const int32_t h = j % perToken / V;
        const int32_t d = j % V * 8;
        const int64_t t = from + i;
        float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (t >= 0 && t < len) {
            const int32_t page =
                checked_page(c.pageTable[b * c.tableStride + (int32_t)t / P], c.numPages);
            if (page < 0) {
                report(err);
            } else {
                const int64_t block = (int64_t)page * c.heads + h;
                const uint8_t* p =
                    (const uint8_t*)(isV ? c.v : c.k) + (block * P + (int32_t)t % P) * D + d;
                const float s = (isV ? c.vScale : c.kScale)[block];
                const uint2 u = *(const uint2*)p;
                decode4<F>(u.x, x);
                decode4<F>(u.y, x + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= s;
            }
        }
        const int64_t at = b * rows.strideBatch + i * rows.strideToken + h * rows.strideHead + d;
        if constexpr (T == CCB_KV8_FP32) {
            float4* o = (float4*)((float*)rows.data + at);
            o[0] = make_float4(x[0], x[1], x[2], x[3]);
            o[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = narrow<T>(x[2 * e]) | (narrow<T>(x[2 * e + 1]) << 16);
            *(uint4*)((uint16_t*)rows.data + at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ---------------------------------------------------------------------------
// evict: which tokens stay
//
// One workgroup per sequence and head.  The kept tokens are those whose key
// is above the k-th largest key, and the first few that equal it; the k-th
// largest is found 8 bits at a time from the top with a histogram in LDS
// (integer counts: the order of the atomics does not matter).
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;

// Exclusive prefix sum of x over the workgroup; *total gets the sum.
__device__ __forceinline__ int32_t block_scan(int32_t x, int32_t* scratch, int32_t* total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int32_t v = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    __syncthreads();
    if (lane == 63) scratch[wave] = v;
    __syncthreads();
    int32_t before = 0, all = 0;
    for (int w = 0; w < kSelThreads / 64; ++w) {
        const int32_t s = scratch[w];
        before += w < wave ? s : 0;
        all += s;
    }
    *total = all;
    return before + v - x;
}

__global__ __launch_bounds__(kSelThreads) void kv8_k_select(ccbKv8Cache from, ccbKv8Cache to,
                                                            int32_t budget, int32_t recent,
                                                            int32_t sinks, int32_t* index,
                                                            int32_t* kept, int32_t* err)
{
    __shared__ int32_t hist[256];
    __shared__ int32_t scratch[kSelThreads / 64];
    __shared__ int32_t found[2];
    const int32_t b = blockIdx.x / (uint32_t)from.heads;
    int32_t len = checked_len(from.lens[b], from.maxPages * from.pageSize);
    if (len < 0) {
        if (threadIdx.x == 0) report(err);
        len = 0;
    }
    const int64_t row = blockIdx.x;
    const float* w = from.weight + row * from.weightStride;
    float* wOut = to.weight != nullptr ? to.weight + row * to.weightStride : nullptr;
    int32_t* out = index + row * budget;
    int32_t* outKept = kept != nullptr ? kept + row * budget : nullptr;
    const int32_t stay = len < budget ? len : budget;
    if (threadIdx.x == 0 && row % from.heads == 0) to.lens[b] = stay;

    // the k-th largest key of the tokens between sinks and recent
    const int32_t low = len > budget ? sinks : 0, high = len > budget ? len - recent : 0;
    uint32_t prefix = 0;  // of the threshold key, found so far
    int32_t need = budget - sinks - recent;
    if (high > low && need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (threadIdx.x < 256) hist[threadIdx.x] = 0;
            __syncthreads();
            for (int32_t t = low + (int)threadIdx.x; t < high; t += kSelThreads) {
                const uint32_t key = weight_key(w[t]);
                if (shift == 24 || (key >> (shift + 8)) == prefix)
                    atomicAdd(&hist[(key >> shift) & 255], 1);
            }
            __syncthreads();
            // bin of the need-th largest: bins in descending order
            const int32_t mine = threadIdx.x < 256 ? hist[255 - threadIdx.x] : 0;
            int32_t total;
            const int32_t above = block_scan(mine, scratch, &total);
            if (threadIdx.x < 256 && above < need && need <= above + mine) {
                found[0] = 255 - threadIdx.x;
                found[1] = above;
            }
            __syncthreads();
            prefix = (prefix << 8) | (uint32_t)found[0];
            need -= found[1];
            __syncthreads();
        }
    }
    // need: how many of the tokens that equal the threshold stay
    int32_t equalBefore = 0, at = 0;
    for (int32_t t0 = 0; t0 < len; t0 += kSelThreads) {
        const int32_t t = t0 + (int)threadIdx.x;
        const float wt = t < len ? w[t] : 0.0f;
        bool keep = t < len && (t < low || t >= high);
        bool equal = false;
        if (t >= low && t < high && need > 0) {
            const uint32_t key = weight_key(wt);
            keep = key > prefix;
            equal = key == prefix;
        }
        int32_t nEqual, nKeep;
        const int32_t rank = equalBefore + block_scan(equal ? 1 : 0, scratch, &nEqual);
        keep = keep || (equal && rank < need);
        const int32_t slot = at + block_scan(keep ? 1 : 0, scratch, &nKeep);
        if (keep) {
            out[slot] = t;
            if (outKept != nullptr) outKept[slot] = t;
            if (wOut != nullptr) wOut[slot] = wt;
        }
        equalBefore += nEqual;
        at += nKeep;
    }
    for (int32_t i = stay + (int)threadIdx.x; i < budget; i += kSelThreads) {
        if (outKept != nullptr) outKept[i] = -1;
        if (wOut != nullptr) wOut[i] = 0.0f;
    }
}

// ---------------------------------------------------------------------------
// evict: the kept tokens into their new pages
//
// One workgroup per new page, head and side: gathers the page's tokens
// through LDS, finds the new scale, rounds the codes again and writes them.
// Bound by the gathered and written bytes.
// ---------------------------------------------------------------------------
template <int F, int D>
__global__ __launch_bounds__(kThreads) void kv8_k_move(ccbKv8Cache from, ccbKv8Cache to,
                                                       int32_t budget, int32_t nPages,
                                                       const int32_t* index, int32_t* err)
{
    constexpr int V = D / 8;
    extern __shared__ uint2 stage[];  // the page's codes, then its tokens' scales
    __shared__ float scratch[4];
    const bool isV = blockIdx.x & 1;
    uint32_t rest = blockIdx.x >> 1;
    const int32_t h = rest % (uint32_t)from.heads;
    rest /= (uint32_t)from.heads;
    const int32_t number = rest % (uint32_t)nPages;
    const int32_t b = rest / (uint32_t)nPages;
    const int32_t P = from.pageSize;
    float* tokenScale = (float*)(stage + P * V);

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
    const int32_t* idx = index + ((int64_t)b * from.heads + h) * budget + number * P;
    const uint8_t* codes = (const uint8_t*)(isV ? from.v : from.k);
    const float* scales = isV ? from.vScale : from.kScale;

    float a = 0.0f;
    for (int32_t i = threadIdx.x; i < n * V; i += kThreads) {
        const int32_t j = i / V;
        const int32_t t = idx[j];
        const int32_t src = checked_page(from.pageTable[b * from.tableStride + t / P], from.numPages);
        uint2 u = make_uint2(0, 0);
        float s = 0.0f;
        if (src < 0) {
            report(err);
        } else {
            const int64_t block = (int64_t)src * from.heads + h;
            u = *(const uint2*)(codes + (block * P + t % P) * D + i % V * 8);
            s = scales[block];
        }
        stage[i] = u;
        if (i % V == 0) tokenScale[j] = s;
        float x[8];
        decode4<F>(u.x, x);
        decode4<F>(u.y, x + 4);
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
        a = fmaxf(a, m * s);
    }
    a = block_max(a, scratch);
    const float s = block_scale<F>(a);
    const float inv = 1.0f / s;
    const int64_t block = (int64_t)page * to.heads + h;
    if (threadIdx.x == 0) (isV ? to.vScale : to.kScale)[block] = s;
    uint2* dst = (uint2*)((uint8_t*)(isV ? to.v : to.k) + block * P * D);
    for (int32_t i = threadIdx.x; i < n * V; i += kThreads) {
        const uint2 u = stage[i];
        const float sOld = tokenScale[i / V];
        float x[8];
        decode4<F>(u.x, x);
        decode4<F>(u.y, x + 4);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e / 4] |= (uint32_t)encode_again<F>(x[e], sOld, inv, s) << (8 * (e % 4));
        dst[i] = make_uint2(w[0], w[1]);
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
    // tokens per workgroup: about 4 vectors of 8 values per thread
    int32_t perGroup = 4 * kThreads * 8 / (c.heads * c.headDim);
    perGroup = perGroup < 1 ? 1 : perGroup;
    const int32_t nGroups = (count + perGroup - 1) / perGroup;
    const int64_t blocks = (int64_t)c.batch * nGroups * (sides == 3 ? 2 : 1);
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    const ccbKv8Rows kr = k != nullptr ? *k : *v, vr = v != nullptr ? *v : *k;
#define KV8_READ(F, T, D) \
    (kv8_k_read<F, T, D><<<dim3((unsigned)blocks), dim3(kThreads), 0, s>>>(c, kr, vr, count, first, perGroup, nGroups, sides, err), 0)
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
    const size_t lds = (size_t)from.pageSize * (from.headDim + sizeof(float));
#define KV8_MOVE(F, D) \
    (kv8_k_move<F, D><<<dim3((unsigned)blocks), dim3(kThreads), lds, s>>>(from, to, budget, nPages, index, err), 0)
#define KV8_MOVE_DIM(D) (from.format == CCB_KV8_INT8 ? KV8_MOVE(kInt8, D) : KV8_MOVE(kE4m3, D))
    (void)KV8_BY_DIM(from.headDim, KV8_MOVE_DIM);
    return hipGetLastError();
}

}  // namespace ccb
