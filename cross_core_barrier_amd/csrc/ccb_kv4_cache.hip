// ccb_kv4_cache.hip -- append and read of the 4-bit key/value cache
// (include/ccb_kv4.h).  Both move memory: a thread takes 8 values of a key and
// the same of a value in append, 4 values in read.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccb_kv4_internal.h"
#include "ccb_kv8_device.h"

namespace {

using namespace kv8;

constexpr int kThreads = 256;

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

template <int T>
__device__ __forceinline__ constexpr uint32_t infinity16()
{
    return T == CCB_KV8_BF16 ? 0x7f80u : 0x7c00u;
}

// Eight 16-bit values as codes of the scale 2^e; the conversion rounds half to
// even and saturates, and no value is NaN.
template <int T>
__device__ __forceinline__ uint32_t encode8(const uint4& x, float scale)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t u = 0;
    if constexpr (T == CCB_KV8_BF16) {
        u = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(u, __builtin_bit_cast(bf2, w[0]), scale, 0);
        u = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(u, __builtin_bit_cast(bf2, w[1]), scale, 1);
        u = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(u, __builtin_bit_cast(bf2, w[2]), scale, 2);
        u = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(u, __builtin_bit_cast(bf2, w[3]), scale, 3);
    } else {
        u = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(u, __builtin_bit_cast(h2, w[0]), scale, 0);
        u = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(u, __builtin_bit_cast(h2, w[1]), scale, 1);
        u = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(u, __builtin_bit_cast(h2, w[2]), scale, 2);
        u = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(u, __builtin_bit_cast(h2, w[3]), scale, 3);
    }
    return u;
}

// The largest of a number over the four lanes that share a scale.
__device__ __forceinline__ uint32_t quad_max(uint32_t m)
{
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

// Eight values of 32 that four lanes hold: their codes, and the scale of all.
template <int T>
__device__ __forceinline__ uint32_t quantise(uint4 x, uint32_t& scale)
{
    uint32_t m = larger16(0, x);
    m = quad_max(max(m & 0xffffu, m >> 16));  // sizes order like whole numbers
    if (m >= infinity16<T>()) {  // an infinity or NaN, for the four lanes alike
        uint32_t* w = &x.x;
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int s = 0; s < 32; s += 16) {
                const uint32_t size = (w[i] >> s) & 0x7fffu;
                if (size < infinity16<T>()) m = max(m, size);
                if (size > infinity16<T>()) w[i] &= ~(0xffffu << s);
            }
        }
        m = quad_max(m);
    }
    // a = 1.f * 2^x is at most 7 * 2^(x - 2) where 1.f <= 1.75, else 7 * 2^(x - 1)
    const uint32_t a = bits(widen<T>(m));
    int32_t e = (int32_t)(a >> 23) - 127 - ((a & 0x7fffffu) > 0x600000u ? 1 : 2);
    e = e < -64 ? -64 : e > 125 ? 125 : e;
    scale = (uint32_t)(e + 127);
    return encode8<T>(x, of_bits(scale << 23));
}

// Four lanes share a scale, D / 8 a row; a workgroup takes as many rows of one
// head as it has threads for.
template <int T, int D>
__global__ __launch_bounds__(kThreads) void kv4_k_append(ccbKv4Cache c, ccbKv8Rows kNew, ccbKv8Rows vNew, int32_t n,
                                                         const int64_t* slots, int32_t* err)
{
    constexpr int C = D / 8, R = kThreads / C;
    const int32_t h = blockIdx.x % (uint32_t)c.heads;
    const int32_t r = (int32_t)threadIdx.x / C, at = (int32_t)threadIdx.x % C;
    const int64_t i = (int64_t)(blockIdx.x / (uint32_t)c.heads) * R + r;
    if (r >= R || i >= n) return;
    const int64_t slot = slots[i];
    const uint4 k = *(const uint4*)((const uint16_t*)kNew.data + i * kNew.strideToken + h * kNew.strideHead + at * 8);
    const uint4 v = *(const uint4*)((const uint16_t*)vNew.data + i * vNew.strideToken + h * vNew.strideHead + at * 8);
    const int shift = __builtin_ctz(c.pageSize);
    if (slot < 0 || slot >= (int64_t)c.numPages << shift) {
        if (slot != -1) report(err);
        return;
    }
    const int64_t row = (((slot >> shift) * c.heads + h) << shift) + (slot & (c.pageSize - 1));
    uint32_t ks, vs;
    const uint32_t ku = quantise<T>(k, ks), vu = quantise<T>(v, vs);
    *(uint32_t*)(c.k + row * (D / 2) + at * 4) = ku;
    *(uint32_t*)(c.v + row * (D / 2) + at * 4) = vu;
    if (at % 4 == 0) {
        c.kScale[row * (D / 32) + at / 4] = (uint8_t)ks;
        c.vScale[row * (D / 32) + at / 4] = (uint8_t)vs;
    }
}

constexpr int kReadEach = 8;  // loads of a thread in flight

// A workgroup takes the places of a sequence and head that its threads have
// room for, keys or values.
template <int T, int D>
__global__ __launch_bounds__(kThreads) void kv4_k_read(ccbKv4Cache c, ccbKv8Rows kOut, ccbKv8Rows vOut, int32_t count,
                                                       const int32_t* first, int32_t sides, uint32_t spans, int32_t* err)
{
    constexpr int V = D / 4;
    constexpr int R = kThreads * kReadEach / V;  // places
    uint32_t rest = blockIdx.x;
    const int32_t h = rest % (uint32_t)c.heads;
    rest /= (uint32_t)c.heads;
    const bool isV = sides == 2 || (sides == 3 && rest % 2 == 1);
    if (sides == 3) rest /= 2;
    const int32_t from = (int32_t)(rest % spans) * R, b = rest / spans;
    int32_t len = checked_len(c.lens[b], c.maxPages * c.pageSize);
    if (len < 0) {
        if (threadIdx.x == 0) report(err);
        len = 0;
    }
    const int shift = __builtin_ctz(c.pageSize);
    const int64_t start = first != nullptr ? first[b] : 0;
    const uint8_t* codes = isV ? c.v : c.k;
    const uint8_t* scales = isV ? c.vScale : c.kScale;
    const ccbKv8Rows& rows = isV ? vOut : kOut;
    int32_t page[kReadEach];
#pragma unroll
    for (int k = 0; k < kReadEach; ++k) {
        const int32_t i = from + (k * kThreads + (int)threadIdx.x) / V;
        const int64_t t = start + i;
        page[k] = -1;
        if (i < count && t >= 0 && t < len) {
            page[k] = checked_page(c.pageTable[b * c.tableStride + (t >> shift)], c.numPages);
            if (page[k] < 0) report(err);
        }
    }
    uint32_t w[kReadEach], s[kReadEach];
#pragma unroll
    for (int k = 0; k < kReadEach; ++k) {
        const int32_t u = k * kThreads + (int)threadIdx.x, at = u % V;
        const int64_t t = start + from + u / V;
        w[k] = 0, s[k] = 127;
        if (page[k] >= 0) {
            const int64_t row = (((int64_t)page[k] * c.heads + h) << shift) + (t & (c.pageSize - 1));
            w[k] = *(const uint16_t*)(codes + row * (D / 2) + at * 2);
            s[k] = scales[row * (D / 32) + at / 8];
        }
    }
#pragma unroll
    for (int k = 0; k < kReadEach; ++k) {
        const int32_t u = k * kThreads + (int)threadIdx.x, at = u % V, i = from + u / V;
        if (u / V >= R || i >= count) continue;
        // a scale of 0 is 2^-127, whose float has no exponent bits: in two steps
        const float f = of_bits((s[k] < 1 ? 1u : s[k]) << 23);
        const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 0);
        const f2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 1);
        f4 x = {a.x * f, a.y * f, e.x * f, e.y * f};
        if (s[k] < 1) x *= 0.5f;
        const int64_t o = b * rows.strideBatch + i * rows.strideToken + h * rows.strideHead + at * 4;
        if constexpr (T == CCB_KV8_FP32)
            __builtin_nontemporal_store(x, (f4*)((float*)rows.data + o));
        else
            __builtin_nontemporal_store(u2{narrow<T>(x.x) | (narrow<T>(x.y) << 16), narrow<T>(x.z) | (narrow<T>(x.w) << 16)},
                                        (u2*)((uint16_t*)rows.data + o));
    }
}

int64_t append_groups(const ccbKv4Cache& c, int32_t n)
{
    const int64_t rows = kThreads / (c.headDim / 8);
    return (n + rows - 1) / rows * c.heads;
}

int64_t read_spans(const ccbKv4Cache& c, int32_t count)
{
    const int64_t places = kThreads * kReadEach / (c.headDim / 4);
    return (count + places - 1) / places;
}

template <int T>
hipError_t append(const ccbKv4Cache& c, const ccbKv8Rows& k, const ccbKv8Rows& v, int32_t n, const int64_t* slots,
                  int32_t* err, hipStream_t s)
{
    const int64_t groups = append_groups(c, n);
    switch (c.headDim) {
    case 64: return enqueue(kv4_k_append<T, 64>, groups, kThreads, s, c, k, v, n, slots, err);
    case 96: return enqueue(kv4_k_append<T, 96>, groups, kThreads, s, c, k, v, n, slots, err);
    case 128: return enqueue(kv4_k_append<T, 128>, groups, kThreads, s, c, k, v, n, slots, err);
    case 192: return enqueue(kv4_k_append<T, 192>, groups, kThreads, s, c, k, v, n, slots, err);
    default: return enqueue(kv4_k_append<T, 256>, groups, kThreads, s, c, k, v, n, slots, err);
    }
}

template <int T>
hipError_t read(const ccbKv4Cache& c, const ccbKv8Rows& k, const ccbKv8Rows& v, int32_t count, const int32_t* first,
                int32_t sides, int32_t* err, hipStream_t s)
{
    const uint32_t spans = (uint32_t)read_spans(c, count);
    const int64_t groups = (int64_t)c.batch * c.heads * spans * (sides == 3 ? 2 : 1);
    switch (c.headDim) {
    case 64: return enqueue(kv4_k_read<T, 64>, groups, kThreads, s, c, k, v, count, first, sides, spans, err);
    case 96: return enqueue(kv4_k_read<T, 96>, groups, kThreads, s, c, k, v, count, first, sides, spans, err);
    case 128: return enqueue(kv4_k_read<T, 128>, groups, kThreads, s, c, k, v, count, first, sides, spans, err);
    case 192: return enqueue(kv4_k_read<T, 192>, groups, kThreads, s, c, k, v, count, first, sides, spans, err);
    default: return enqueue(kv4_k_read<T, 256>, groups, kThreads, s, c, k, v, count, first, sides, spans, err);
    }
}

}  // namespace

namespace ccb {

bool kv4_append_fits(const ccbKv4Cache& c, int32_t nNew) { return kv8_launch_fits(append_groups(c, nNew), kThreads); }

hipError_t kv4_append(const ccbKv4Cache& c, const ccbKv8Rows& k, const ccbKv8Rows& v, int32_t nNew,
                      const int64_t* slots, int32_t* err, hipStream_t s)
{
    return k.type == CCB_KV8_BF16 ? append<CCB_KV8_BF16>(c, k, v, nNew, slots, err, s)
                                  : append<CCB_KV8_FP16>(c, k, v, nNew, slots, err, s);
}

bool kv4_read_fits(const ccbKv4Cache& c, int32_t count)
{
    // (both sides, whichever are asked for)
    const int64_t pairs = (int64_t)c.batch * c.heads;
    return pairs <= INT32_MAX && kv8_launch_fits(pairs * 2 * read_spans(c, count), kThreads);
}

hipError_t kv4_read(const ccbKv4Cache& c, const ccbKv8Rows* k, const ccbKv8Rows* v, int32_t count,
                    const int32_t* first, int32_t* err, hipStream_t s)
{
    const int32_t sides = (k != nullptr ? 1 : 0) | (v != nullptr ? 2 : 0);
    const ccbKv8Rows &kr = k != nullptr ? *k : *v, &vr = v != nullptr ? *v : *k;
    switch (kr.type) {
    case CCB_KV8_BF16: return read<CCB_KV8_BF16>(c, kr, vr, count, first, sides, err, s);
    case CCB_KV8_FP16: return read<CCB_KV8_FP16>(c, kr, vr, count, first, sides, err, s);
    default: return read<CCB_KV8_FP32>(c, kr, vr, count, first, sides, err, s);
    }
}

}  // namespace ccb
