// ccb_kv8_attend.hip -- attention of a decoding step over the 8-bit
// key/value cache.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccb_kv8_internal.h"
#include "ccb_kv8_device.h"

namespace {

using namespace kv8;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// A lane's share of a token's row: D / 64 values, lanes past the row hold 0.
template <int D>
struct Share {
    static constexpr int n = (D + 63) / 64;
};

// One workgroup per query row; its waves take every fourth token, keep a
// running maximum, sum and weighted values, and join at the end.
template <int F, int T, int D>
__global__ __launch_bounds__(kThreads) void kv8_k_attend_plain(ccb::Kv8AttendArgs a, float* lseOut)
{
    constexpr int N = Share<D>::n;
    __shared__ float sm[kWaves], sl[kWaves], sacc[kWaves][D];
    const ccbKv8Cache& c = a.c;
    uint32_t rest = blockIdx.x;
    const int32_t hq = rest % (uint32_t)a.headsQ;
    rest /= (uint32_t)a.headsQ;
    const int32_t i = rest % (uint32_t)a.nQuery;
    const int32_t b = rest / (uint32_t)a.nQuery;
    const int32_t h = hq / (a.headsQ / c.heads);
    const int32_t P = c.pageSize;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int32_t len = checked_len(c.lens[b], c.maxPages * P);
    if (len < 0) {
        if (threadIdx.x == 0) report(a.err);
        len = 0;
    }
    const int32_t end = len - a.nQuery + i + 1;
    const int32_t begin = a.window > 0 && end > a.window ? end - a.window : 0;
    const uint16_t* q = (const uint16_t*)a.q.data + b * a.q.strideBatch + i * a.q.strideToken +
                        hq * a.q.strideHead;
    float qv[N], acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        qv[e] = lane + 64 * e < D ? widen<T>(q[lane + 64 * e]) : 0.0f;
        acc[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int32_t t = begin + wave; t < end; t += kWaves) {
        const int32_t page = checked_page(c.pageTable[b * c.tableStride + t / P], c.numPages);
        if (page < 0) {
            if (lane == 0) report(a.err);
            continue;
        }
        const int64_t block = (int64_t)page * c.heads + h;
        const int64_t off = (block * P + t % P) * D;
        float s = 0.0f;
        float v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            float x[4] = {0, 0, 0, 0}, y[4] = {0, 0, 0, 0};
            if (lane + 64 * e < D) {
                decode4<F>(((const uint8_t*)c.k)[off + lane + 64 * e], x);
                decode4<F>(((const uint8_t*)c.v)[off + lane + 64 * e], y);
            }
            s += qv[e] * x[0];
            v[e] = y[0];
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d, 64);
        s *= c.kScale[block] * a.scale;
        const float mn = fmaxf(m, s);
        const float f = expf(m - mn), p = expf(s - mn);
        l = l * f + p;
        const float pv = p * c.vScale[block];
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = acc[e] * f + pv * v[e];
        m = mn;
    }
    if (lane == 0) sm[wave] = m, sl[wave] = l;
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (lane + 64 * e < D) sacc[wave][lane + 64 * e] = acc[e];
    __syncthreads();
    float mm = -INFINITY, ll = 0.0f;
    for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, sm[w]);
    for (int w = 0; w < kWaves; ++w) ll += sl[w] != 0.0f ? sl[w] * expf(sm[w] - mm) : 0.0f;
    uint16_t* out = (uint16_t*)a.out.data + b * a.out.strideBatch + i * a.out.strideToken +
                    hq * a.out.strideHead;
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float o = 0.0f;
        for (int w = 0; w < kWaves; ++w) o += sl[w] != 0.0f ? sacc[w][d] * expf(sm[w] - mm) : 0.0f;
        out[d] = (uint16_t)narrow<T>(ll != 0.0f ? o / ll : 0.0f);
    }
    if (threadIdx.x == 0) {
        const float lse = ll != 0.0f ? mm + logf(ll) : -INFINITY;
        lseOut[blockIdx.x] = lse;
        if (a.lse != nullptr) a.lse[blockIdx.x] = lse;
    }
}

// One thread per token and cache head adds the weights of every row.
template <int F, int T, int D>
__global__ __launch_bounds__(kThreads) void kv8_k_weights_plain(ccb::Kv8AttendArgs a, const float* lse,
                                                                int32_t perRow)
{
    const ccbKv8Cache& c = a.c;
    uint32_t rest = blockIdx.x;
    const int32_t t = (int32_t)(rest % (uint32_t)perRow) * kThreads + (int)threadIdx.x;
    rest /= (uint32_t)perRow;
    const int32_t h = rest % (uint32_t)c.heads;
    const int32_t b = rest / (uint32_t)c.heads;
    const int32_t P = c.pageSize, group = a.headsQ / c.heads;
    const int32_t len = checked_len(c.lens[b], c.maxPages * P);
    if (t >= len) return;
    const int32_t page = checked_page(c.pageTable[b * c.tableStride + t / P], c.numPages);
    if (page < 0) return;
    const int64_t block = (int64_t)page * c.heads + h;
    const uint8_t* k = (const uint8_t*)c.k + (block * P + t % P) * D;
    float sum = 0.0f;
    for (int32_t i = 0; i < a.nQuery; ++i) {
        const int32_t end = len - a.nQuery + i + 1;
        if (t >= end || (a.window > 0 && t < end - a.window)) continue;
        for (int32_t g = 0; g < group; ++g) {
            const int32_t hq = h * group + g;
            const uint16_t* q = (const uint16_t*)a.q.data + b * a.q.strideBatch +
                                i * a.q.strideToken + hq * a.q.strideHead;
            float s = 0.0f;
            for (int d = 0; d < D; d += 4) {
                float x[4];
                decode4<F>(*(const uint32_t*)(k + d), x);
                for (int e = 0; e < 4; ++e) s += widen<T>(q[d + e]) * x[e];
            }
            s *= c.kScale[block] * a.scale;
            sum += expf(s - lse[((int64_t)b * a.nQuery + i) * a.headsQ + hq]);
        }
    }
    c.weight[((int64_t)b * c.heads + h) * c.weightStride + t] += sum;
}

}  // namespace

namespace ccb {

size_t kv8_attend_bytes(const ccbKv8Cache& c, int32_t headsQ, int32_t nQuery, int32_t accumulate)
{
    (void)accumulate;
    return (size_t)c.batch * headsQ * nQuery * sizeof(float);
}

hipError_t kv8_attend(const Kv8AttendArgs& a, int numCUs, hipStream_t s)
{
    (void)numCUs;
    const ccbKv8Cache& c = a.c;
    float* lse = (float*)a.ws;
    const int64_t rows = (int64_t)c.batch * a.nQuery * a.headsQ;
    const int32_t perRow = (c.maxPages * c.pageSize + kThreads - 1) / kThreads;
    const int64_t blocks = (int64_t)c.batch * c.heads * perRow;
    if (rows > INT32_MAX || blocks > INT32_MAX) return hipErrorInvalidValue;
#define KV8_PLAIN(F, T, D) \
    kv8_k_attend_plain<F, T, D><<<dim3((unsigned)rows), dim3(kThreads), 0, s>>>(a, lse); \
    if (a.accumulate) \
        kv8_k_weights_plain<F, T, D><<<dim3((unsigned)blocks), dim3(kThreads), 0, s>>>(a, lse, perRow); \
    break;
#define KV8_PLAIN_DIM(F, T) \
    switch (c.headDim) { \
    case 64: KV8_PLAIN(F, T, 64) \
    case 96: KV8_PLAIN(F, T, 96) \
    case 128: KV8_PLAIN(F, T, 128) \
    case 192: KV8_PLAIN(F, T, 192) \
    default: KV8_PLAIN(F, T, 256) \
    }
    if (c.format == CCB_KV8_INT8) {
        if (a.q.type == CCB_KV8_BF16) {
            KV8_PLAIN_DIM(kInt8, CCB_KV8_BF16)
        } else {
            KV8_PLAIN_DIM(kInt8, CCB_KV8_FP16)
        }
    } else {
        if (a.q.type == CCB_KV8_BF16) {
            KV8_PLAIN_DIM(kE4m3, CCB_KV8_BF16)
        } else {
            KV8_PLAIN_DIM(kE4m3, CCB_KV8_FP16)
        }
    }
    return hipGetLastError();
}

}  // namespace ccb
