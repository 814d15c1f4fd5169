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

// The largest of a value over the workgroup (256 threads); x is not NaN.
__device__ __forceinline__ float block_max(float x, float* scratch)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
    const int wave = threadIdx.x >> 6;
    __syncthreads();  // scratch may still be read from an earlier use
    if ((threadIdx.x & 63) == 0) scratch[wave] = x;
    __syncthreads();
    return fmaxf(fmaxf(scratch[0], scratch[1]), fmaxf(scratch[2], scratch[3]));
}

}  // namespace kv8

#endif  // CCB_KV8_DEVICE_H
