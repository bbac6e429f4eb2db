// 8-bit integer rows shared by the quantisation and product kernels.
//
// A row of elements x (one token, one output channel of a weight matrix, one
// hidden row) shares the scale s = amax / 127, amax its largest magnitude,
// rounded to fp32; its codes are the integers nearest to x / s, ties to the
// even one.  A row of zeros has s = 0 and codes 0; so has a row so small that
// s underflows.  A row that holds an infinity or a NaN has s = NaN and codes
// 0: every product with it is NaN.  Codes are row-major, one byte each.
#pragma once

#include "rmoe_mx.h"

namespace rmoe {

typedef unsigned u4 __attribute__((ext_vector_type(4)));
typedef unsigned u2 __attribute__((ext_vector_type(2)));

// What turns the elements of a row into codes.
struct I8Row {
    float scale;  // s, as it is stored
    float pre;    // a power of two that makes s normal: a code is the integer nearest to (x pre) / (s pre)
    float inv;    // 1 / (s pre), rounded; 0 where every code is 0
    float s;      // s pre
};
__device__ __forceinline__ I8Row i8_row(float amax) {
    I8Row r;
    r.scale = amax / 127.0f;
    if (!(amax < __builtin_inff())) r.scale = __builtin_nanf("");  // infinities, NaN
    r.pre = amax < 0x1p-100f ? 0x1p64f : 1.0f;
    r.s = r.scale * r.pre;
    r.inv = r.s > 0.0f ? 1.0f / r.s : 0.0f;
    return r;
}

// Codes of 8 elements, the exact nearest integers.  q = x inv is within 2^-23
// of x / s relatively (two roundings), 1.6e-5 absolutely, so rounding it gives
// the nearest integer n unless it lies that close to a border between two; a
// fused add of 1.5 2^23 rounds it (half a unit in the last place there is one
// half) and leaves n's low byte in the sum's.  Where |q - n| comes near one
// half (one element in 5000, one wave's 512 in 10), the remainder x - n s
// decides: the fused product is exact there (a multiple of the last place of s
// or of x below s) and is compared with s / 2.
constexpr float kI8Magic = 0x1.8p23f;
__device__ __forceinline__ unsigned i8_word(const float *t) {
    const unsigned a = __builtin_bit_cast(unsigned, t[0]), b = __builtin_bit_cast(unsigned, t[1]);
    const unsigned c = __builtin_bit_cast(unsigned, t[2]), d = __builtin_bit_cast(unsigned, t[3]);
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400), __builtin_amdgcn_perm(b, a, 0x0c0c0400),
                                 0x05040100);
}
__device__ __forceinline__ u2 i8_codes(const float (&x)[8], const I8Row &r) {
    float y[8], t[8], far = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = r.inv > 0.f ? x[i] * r.pre : 0.f;
        t[i] = __builtin_fmaf(y[i], r.inv, kI8Magic);
        const float n = t[i] - kI8Magic;
        far = fmaxf(far, __builtin_fabsf(__builtin_fmaf(y[i], r.inv, -n)));
    }
    // a scale below fp32's normal numbers is off by up to a half of itself: quotients up to 190
    if (far > 0.4999f || r.pre != 1.0f) {
        const float h = 0.5f * r.s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float n = t[i] - kI8Magic;
            const float e = __builtin_fmaf(-n, r.s, y[i]);
            const bool odd = __builtin_bit_cast(unsigned, t[i]) & 1u;
            if (e > h || (e == h && odd)) n += 1.0f;
            if (e < -h || (e == -h && odd)) n -= 1.0f;
            n = fminf(fmaxf(n, -127.0f), 127.0f);
            t[i] = n + kI8Magic;
        }
    }
    return u2{i8_word(t), i8_word(t + 4)};
}

}  // namespace rmoe
