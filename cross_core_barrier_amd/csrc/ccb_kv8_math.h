// ccb_kv8_math.h -- the arithmetic of the 8-bit key/value cache that has to
// come out the same everywhere: rounding to the code formats, block scales,
// and the lookups that keep every access in range.  Plain C++ that compiles
// for the host too, where the tests check it.
#ifndef CCB_KV8_MATH_H
#define CCB_KV8_MATH_H

#include <math.h>
#include <stdint.h>
#include <string.h>

#ifdef __HIPCC__
#define KV8_FN __host__ __device__ __forceinline__
#else
#define KV8_FN inline
#endif

namespace kv8 {

constexpr int kInt8 = 0, kE4m3 = 1;

KV8_FN uint32_t bits(float x)
{
    uint32_t u;
    memcpy(&u, &x, 4);
    return u;
}

KV8_FN float of_bits(uint32_t u)
{
    float x;
    memcpy(&x, &u, 4);
    return x;
}

template <int F>
KV8_FN constexpr float largest()
{
    return F == kInt8 ? 127.0f : 448.0f;
}

// The scale of a block whose largest value is a: at least 2^-64, so that the
// remainders in encode() below stay far above the smallest float.
template <int F>
KV8_FN float block_scale(float a)
{
    const float s = a / largest<F>();
    return a > 0.0f ? (s > 0x1p-64f ? s : 0x1p-64f) : 0.0f;
}

// The code nearest to (hi + lo) / s, ties to even, saturated; inv is 1 / s to
// a few units in the last place.  |lo| is at most half a unit of hi.
//
// The quotient is rounded once: u = |hi| * inv is only used to find the two
// codes around it, and the remainder against the border between them, |hi| -
// border * s, decides.  border has at most 8 bits and s 24, so close to a
// border the remainder is a small multiple of a quarter of s's unit and the
// fused multiply-add returns it exactly (its sign is right everywhere); lo then
// joins with one more rounding, which cannot change a sign either.  An error
// of u near a code picks the neighbouring pair, whose far border gives the
// same code.
template <int F>
KV8_FN uint8_t encode(float hi, float lo, float inv, float s)
{
    const uint32_t sign = bits(hi) >> 31;
    const float x = fabsf(hi);
    const float low = sign ? -lo : lo;
    const float t = x * inv;
    if (F == kInt8) {
        if (!(t < 127.0f)) return (uint8_t)(sign ? -127 : 127);
        const float n0 = floorf(t);
        const float d = fmaf(-(n0 + 0.5f), s, x) + low;
        int n = (int)n0;
        n += (d > 0.0f || (d == 0.0f && (n & 1))) ? 1 : 0;
        return (uint8_t)(sign ? -n : n);
    }
    if (!(t < 448.0f)) return (uint8_t)(0x7E | (sign << 7));
    // the binade of t (2^-6 and below: one step for all), step = 2^(e - 3)
    int e = (int)(bits(t) >> 23) - 127;
    e = e < -6 ? -6 : e;
    const float step = of_bits((uint32_t)(e - 3 + 127) << 23);
    const float n0 = floorf(t * of_bits((uint32_t)(3 - e + 127) << 23));
    const float d = fmaf(-(n0 + 0.5f) * step, s, x) + low;
    int n = (int)n0;
    n += (d > 0.0f || (d == 0.0f && (n & 1))) ? 1 : 0;
    // n = 16 carries into the next exponent by itself
    int code = ((e + 6) << 3) + n;
    code = code > 0x7E ? 0x7E : code;
    return (uint8_t)(code | (sign << 7));
}

// A new value's code: NaN is 0, an infinity saturates (encode() does that:
// its quotient is not below the largest).
template <int F>
KV8_FN uint8_t encode_value(float x, float inv, float s)
{
    return (x != x || !(s > 0.0f)) ? (uint8_t)0 : encode<F>(x, 0.0f, inv, s);
}

// A code's value (code times nothing) in the block scale sOld, as a code for
// the scale s.  v is the old code's value; v * sOld = hi + lo exactly.
template <int F>
KV8_FN uint8_t encode_again(float v, float sOld, float inv, float s)
{
    if (!(s > 0.0f)) return 0;
    const float hi = v * sOld;
    return encode<F>(hi, fmaf(v, sOld, -hi), inv, s);
}

// Whether quotients were too near a border between two codes to be sure.
// t, a product with 1 / s, is off by three roundings at most: 3 * 2^-24 of it.
// Unsure is, for int8, within 2^-15 of a border (t <= 127: 2^-15.4), and for
// e4m3 within 4 units of t's last place.  e4m3's step is the exponent's from
// 2^-6 on and stays 2^-9 below: smaller quotients are looked at again, raised
// by 2^-6 into the binade that has this step.
template <int F>
struct Near {
    float d = 0.0f;                      // int8: largest distance to a code
    uint32_t border = ~0u, small = ~0u;  // e4m3: place above a border's zone, size
    static constexpr uint32_t kZone = 4;
    KV8_FN void look(uint32_t u)
    {
        // the 20 bits below e4m3's three, 0 where a border's zone begins
        const uint32_t above = (u - (0x80000u - kZone)) << 12;
        border = above < border ? above : border;
    }
    KV8_FN bool unsure(const float* t)
    {
        if constexpr (F == kInt8) return d > 0.5f - 0x1p-15f;
        if (small < (0x3c800000u << 1) - 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (fabsf(t[i]) < 0x1p-6f) look(bits(fabsf(t[i]) + 0x1p-6f));
        }
        return border <= (2 * kZone) << 12;
    }
};

// Four quotients as the codes of one word (on the host: what the conversion
// instructions give).  None is further from 0 than the largest code by more
// than its error: s is at least the largest value / Q.
template <int F>
KV8_FN uint32_t encode4_near(const float* t, Near<F>& near)
{
    if constexpr (F == kInt8) {
        uint32_t n[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float r = __builtin_rintf(t[i]);
            near.d = fmaxf(near.d, fabsf(t[i] - r));
            n[i] = (uint32_t)(int32_t)r;
        }
#ifdef __HIP_DEVICE_COMPILE__
        const uint32_t a = __builtin_amdgcn_perm(n[1], n[0], 0x0c0c0400u);
        const uint32_t b = __builtin_amdgcn_perm(n[3], n[2], 0x04000c0cu);
        return a | b;
#else
        return (n[0] & 255) | (n[1] & 255) << 8 | (n[2] & 255) << 16 | n[3] << 24;
#endif
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = bits(t[i]);
            const uint32_t size = (u << 1) - 1;  // a 0 is not small
            near.look(u);
            near.small = size < near.small ? size : near.small;
        }
#ifdef __HIP_DEVICE_COMPILE__
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], w, true);
#else
        uint32_t w = 0;
        for (int i = 0; i < 4; ++i)
            w |= (uint32_t)(t[i] != t[i] ? 0x7F : encode<F>(t[i], 0.0f, 1.0f, 1.0f)) << (8 * i);
        return w;
#endif
    }
}

// Eight codes' values v of the block scale sOld as codes of the scale s, two
// words; inv is 1 / s.
template <int F>
KV8_FN void encode8_again(const float* v, float sOld, float inv, float s, uint32_t* w)
{
    w[0] = w[1] = 0;
    if (!(s > 0.0f)) return;
    float t[8];
    // Infinite only where every code is 0 (a code of 2^-9 would need an s above
    // sOld * 2^-18), and 0 has to stay 0.
    const float ratio = fminf(sOld * inv, 0x1.fffffep127f);
    Near<F> near;
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[i] * ratio;
    w[0] = encode4_near<F>(t, near);
    w[1] = encode4_near<F>(t + 4, near);
    if (near.unsure(t) || s > 0x1p120f) {
        w[0] = w[1] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i >> 2] |= (uint32_t)encode_again<F>(v[i], sOld, inv, s) << (8 * (i & 3));
    }
}

// lens[b] where it is possible, else -1.
KV8_FN int32_t checked_len(int32_t len, int32_t capacity)
{
    return (len < 0 || len > capacity) ? -1 : len;
}

// A page number where it is possible, else -1.
KV8_FN int32_t checked_page(int32_t page, int32_t numPages)
{
    return ((uint32_t)page < (uint32_t)numPages) ? page : -1;
}

// Order of weights as unsigned numbers: larger weight, larger key; every NaN
// is key 0, below -infinity; -0 and 0 are one key.
KV8_FN uint32_t weight_key(float w)
{
    if (w != w) return 0;
    const uint32_t u = bits(w == 0.0f ? 0.0f : w);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

}  // namespace kv8

#endif  // CCB_KV8_MATH_H
