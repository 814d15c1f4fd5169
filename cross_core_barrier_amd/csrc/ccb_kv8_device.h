// ccb_kv8_device.h -- device helpers shared by the kernels of the 8-bit
// key/value cache.
#ifndef CCB_KV8_DEVICE_H
#define CCB_KV8_DEVICE_H

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include "ccb_kv8_internal.h"
#include "ccb_kv8_math.h"

namespace kv8 {

typedef float f2 __attribute__((ext_vector_type(2)));

// Report a bad page number, length or count (never cleared here).
__device__ __forceinline__ void report(int32_t* err)
{
    if (err != nullptr)
        __hip_atomic_store(err, (int32_t)CCB_ERR_INVALID_VALUE, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
}

// Four codes (one word, lowest byte first) as floats.
template <int F>
__device__ __forceinline__ void decode4(uint32_t w, float* x)
{
    if constexpr (F == kInt8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)((int32_t)(w << (24 - 8 * i)) >> 24);
    } else {
        const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
        const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    }
}

// A 16-bit value of the given type (low half of u) as a float.
template <int T>
__device__ __forceinline__ float widen(uint32_t u)
{
    if constexpr (T == CCB_KV8_BF16)
        return of_bits(u << 16);
    else
        return __half2float(__ushort_as_half((unsigned short)u));
}

// Eight 16-bit values as floats.
template <int T>
__device__ __forceinline__ void widen8(const uint4& u, float* x)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = widen<T>(w[i] & 0xffffu);
        x[2 * i + 1] = widen<T>(w[i] >> 16);
    }
}

// A float rounded once to 16 bits (half to even).
template <int T>
__device__ __forceinline__ uint32_t narrow(float x)
{
    if constexpr (T == CCB_KV8_BF16) {
        const __hip_bfloat16 h = __float2bfloat16(x);
        unsigned short u;
        __builtin_memcpy(&u, &h, 2);
        return u;
    } else {
        return __half_as_ushort(__float2half_rn(x));
    }
}

// Eight new values as codes of the block scale s; inv is 1 / s.
template <int F>
__device__ __forceinline__ uint2 encode8(const float* x, float inv, float s)
{
    if (!(s > 0.0f)) return make_uint2(0, 0);
    float t[8], odd = 0.0f;
    Near<F> near;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t[i] = x[i] * inv;
        odd = fmaf(x[i], 0.0f, odd);  // NaN if any value is NaN or infinite
    }
    uint2 u = make_uint2(encode4_near<F>(t, near), encode4_near<F>(t + 4, near));
    if (near.unsure(t) || odd != odd || s > 0x1p120f) {  // (there 1 / s loses bits)
        u = make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u.x |= (uint32_t)encode_value<F>(x[i], inv, s) << (8 * i);
            u.y |= (uint32_t)encode_value<F>(x[4 + i], inv, s) << (8 * i);
        }
    }
    return u;
}

// Eight codes (two words) of the scale sOld as codes of the scale s.
template <int F>
__device__ __forceinline__ uint2 encode8_again(const uint2& w, float sOld, float inv, float s)
{
    float v[8];
    decode4<F>(w.x, v);
    decode4<F>(w.y, v + 4);
    uint32_t u[2];
    encode8_again<F>(v, sOld, inv, s, u);
    return make_uint2(u[0], u[1]);
}

// The largest size among 16-bit values, two to a word, kept as bits: sizes
// order like whole numbers.
typedef unsigned short us2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t larger16(uint32_t m, const uint4& u)
{
    us2 x = __builtin_bit_cast(us2, m);
    x = __builtin_elementwise_max(x, __builtin_bit_cast(us2, u.x & 0x7fff7fffu));
    x = __builtin_elementwise_max(x, __builtin_bit_cast(us2, u.y & 0x7fff7fffu));
    x = __builtin_elementwise_max(x, __builtin_bit_cast(us2, u.z & 0x7fff7fffu));
    x = __builtin_elementwise_max(x, __builtin_bit_cast(us2, u.w & 0x7fff7fffu));
    return __builtin_bit_cast(uint32_t, x);
}

// The threads of a group of 256 (a workgroup, or a quarter of one) in teams, each for one block of a page: a
// wave for 16 tokens, two for 32, all four for 64 and 128.  With a workgroup
// for every block of 16 tokens, appending 65536 tokens took 135 us instead of
// 57, and moving 240,000 took 317 us instead of 225.
struct Team {
    int32_t size;   // threads
    int32_t id;     // of this thread in its team
    int32_t sub;    // the team's place in its group
    uint32_t unit;  // the team's number among all of group 0, 1, ..., alike in a wave

    __device__ __forceinline__ Team(int32_t pageSize, uint32_t group)
    {
        size = pageSize >= 64 ? 256 : pageSize * 4;
        id = (int32_t)threadIdx.x & (size - 1);
        sub = __builtin_amdgcn_readfirstlane(((int32_t)threadIdx.x & 255) / size);
        unit = group * (uint32_t)(256 / size) + (uint32_t)sub;
    }

    // The largest of a value over the team; x is not NaN.  Every thread of the
    // workgroup calls it, with its group's scratch.
    __device__ __forceinline__ float largest(float x, float* scratch) const
    {
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
        if (size == 64) return x;
        const int wave = (threadIdx.x >> 6) & 3;
        if ((threadIdx.x & 63) == 0) scratch[wave] = x;
        __syncthreads();
        x = fmaxf(scratch[wave], scratch[wave ^ 1]);
        return size == 128 ? x : fmaxf(x, fmaxf(scratch[wave ^ 2], scratch[wave ^ 3]));
    }
};

// Enqueues a kernel and returns that launch's own status: the runtime's last
// error may be of a call of the caller's that failed before.
template <class T>
struct Plain {
    using type = T;
};
template <class... P>
hipError_t enqueue(void (*kernel)(P...), int64_t groups, int threads, hipStream_t s, typename Plain<P>::type... p)
{
    void* args[] = {(void*)&p...};
    return hipLaunchKernel((const void*)kernel, dim3((unsigned)groups), dim3((unsigned)threads), args, 0, s);
}

inline unsigned team_groups(int64_t units, int32_t pageSize)
{
    const int32_t teams = pageSize >= 64 ? 1 : 64 / pageSize;
    return (unsigned)((units + teams - 1) / teams);
}

}  // namespace kv8

#endif  // CCB_KV8_DEVICE_H
