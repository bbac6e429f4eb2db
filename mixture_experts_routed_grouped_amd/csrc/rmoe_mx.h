// MXFP4 format shared by the quantisation and product kernels.
//
// A block of 32 consecutive elements of a row shares one scale 2^(b - 127),
// held as the exponent byte b; an element is a 4-bit E2M1 code (sign, then
// the magnitudes 0 0.5 1 1.5 2 3 4 6), two per byte, the even element in the
// low nibble.  Codes are row-major, a row padded to whole chunks of 256
// elements (128 bytes: one LDS row of the product kernels, 8 blocks).  Scale
// bytes are stored chunk by chunk, [chunks][rows][8], so that the bytes of
// 32 rows of a chunk are 256 contiguous bytes: one DMA.  The 8 bytes of a
// (chunk, row) hold blocks 0 2 4 6 1 3 5 7: v_mfma_scale_f32_32x32x64 takes
// K = 64 per instruction, lanes 0-31 the first block of it and lanes 32-63
// the second, so one dword per lane holds its scales of a chunk's four
// instructions, picked by the instruction's byte select.
#pragma once

#include "rmoe_device.h"

namespace rmoe {

constexpr int kMxChunk = 256;     // elements per chunk
constexpr int kMxChunkBytes = 128;

// Byte of block j (0..7) of a chunk within its 8 scale bytes.
__device__ __forceinline__ int mx_pos(int j) { return ((j & 1) << 2) | (j >> 1); }

// Running maximum of magnitudes that keeps a NaN (v_maximum3_f32, two values
// per instruction).
__device__ __forceinline__ float mx_amax(float m, float a, float b) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b)), m);
}

// Swaps a's lanes 32-63 with b's lanes 0-31.
__device__ __forceinline__ void swap32(unsigned &a, unsigned &b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
// The maximum of lanes l and l ^ 32, in both.
__device__ __forceinline__ float mx_amax32(float m) {
    unsigned a = __builtin_bit_cast(unsigned, m), b = a;
    swap32(a, b);  // the lower half's in a, the upper's in b
    return mx_amax(0.f, __builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}

// Scale byte of a block by its largest magnitude: floor(log2(amax)) - 2 +
// 127, so that the largest element lands in [4, 8); at least 0 (amax <
// 2^-125, zero included).  Infinities and NaN give 255, the format's NaN.
__device__ __forceinline__ unsigned mx_scale_byte(float amax) {
    const int ex = (int)((__builtin_bit_cast(unsigned, amax) >> 23) & 255u);
    return ex == 255 ? 255u : ex > 2 ? (unsigned)(ex - 2) : 0u;
}

// E2M1 codes of 8 values over 2^(byte - 127), rounded to nearest even and
// clamped at 6 by the conversion instruction, which takes the scale's exponent
// field as it is (byte 0: 2^-127, subnormal values included).
__device__ __forceinline__ unsigned mx_pack8(const float *v, float scale) {
    unsigned r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], scale, 3);
    return r;
}
template <int N>
__device__ __forceinline__ void mx_codes(const float (&v)[N], unsigned byte, unsigned (&out)[N / 8]) {
    const float scale = __builtin_bit_cast(float, byte << 23);
#pragma unroll
    for (int i = 0; i < N / 8; ++i) out[i] = byte == 255u ? 0u : mx_pack8(v + 8 * i, scale);
}

}  // namespace rmoe
