// kvxfer_device.h -- device code that the kernels of append, rotation and attention share: vectors, plan records, and
// the conversions of 8- and 4-bit pool elements (not part of the public ABI).
#pragma once
#include <hip/hip_runtime.h>

#include "kvxfer_ops.h"

namespace kvx {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
#define KVX_GLOBAL __attribute__((address_space(1)))
#define KVX_LDS __attribute__((address_space(3)))
#define KVX_CONST __attribute__((address_space(4)))

// A plan record, the same for the whole workgroup and not written while kernels run: read
// through the constant space, by scalar loads into scalar registers.
template <class Rec>
__device__ __forceinline__ Rec plan_record(const Rec *at)
{
    constexpr int kWords = sizeof(Rec) / 4;
    union {
        Rec rec;
        uint32_t word[kWords];
    } u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) u.word[i] = ((const KVX_CONST uint32_t *)at)[i];
    return u.rec;
}

template <class T>
struct Vec {
    typedef T x2 __attribute__((ext_vector_type(2)));
    typedef T x4 __attribute__((ext_vector_type(4)));
    typedef T x8 __attribute__((ext_vector_type(8)));
};

// Four e4m3 values (one word) as T: every one is a value of both 16-bit types.
template <class T>
__device__ __forceinline__ typename Vec<T>::x4 from_e4m3(uint32_t w)
{
    typedef typename Vec<T>::x2 T2;
    T2 a, b;
    if constexpr (__is_same(T, __bf16)) {
        a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true);
    } else {
        a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, true);
    }
    return typename Vec<T>::x4{a[0], a[1], b[0], b[1]};
}

// Where the row bytes of eight consecutive values lie, and what they are read as: 16 bytes of 16-bit values, 8 of
// e4m3, 4 of mx4.  CACHE: what a pool's elements are.
enum Cache { kHalves, kE4m3, kMx4 };
inline Cache cache_of(int kv_type) { return kv_type == KV_TYPE_E4M3 ? kE4m3 : kv_type == KV_TYPE_MX4 ? kMx4 : kHalves; }

// A scale byte as the conversions take it: a 32-bit float of that exponent (0 is 2^-127 and 255 NaN for them too).
__device__ __forceinline__ float mx4_scale(uint32_t e) { return __builtin_bit_cast(float, e << 23); }

// Eight mx4 elements (one word) as T, times their group's scale: exact in bfloat16 and 32 bits, rounded in half.
template <class T>
__device__ __forceinline__ typename Vec<T>::x8 from_mx4(uint32_t w, float scale)
{
    typedef typename Vec<T>::x2 T2;
    T2 a, b, c, d;
    if constexpr (__is_same(T, __bf16)) {
        a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
        b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
        d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    } else if constexpr (__is_same(T, float)) {
        a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
        b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
        d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
    } else {
        a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0);
        b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2);
        d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3);
    }
    return typename Vec<T>::x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The scale byte of a group of 32 values, eight in each of four neighbouring lanes (a quad, all at work): the
// smallest e >= 1 with |x| <= 7 * 2^(e - 127), 255 where one is infinite or NaN.  As whole numbers the
// magnitudes order as their values do, NaN above infinity.
__device__ __forceinline__ uint32_t mx4_scale_of(const float (&x)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __builtin_bit_cast(uint32_t, x[i]) & 0x7fffffffu);
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xf, 0xf, true));  // the lane 1 away
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xf, 0xf, true));  // 2 away
    // 1.f * 2^k <= 7 * 2^s, with 7 = 1.75 * 2^2, for k = s + 2 where 1.f <= 1.75
    const int32_t k = (int32_t)(m >> 23);
    return k == 255 ? 255u : (uint32_t)max(k - ((m & 0x7fffffu) <= 0x600000u ? 2 : 1), 1);
}

// Eight values as mx4 elements, to nearest even, saturated; zeros in a group that is NaN.
__device__ __forceinline__ uint32_t to_mx4(const float (&x)[8], uint32_t e)
{
    const float scale = mx4_scale(e);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
    return e == 255 ? 0 : w;
}

}  // namespace kvx
