// MXFP4 quantisation, its inverse, and the token pack that quantises on the
// way (format: rmoe_mx.h).  Bound by HBM: a row is read once and its codes
// (4.25 bits per element with the scales) are written once.  470 M elements
// (8 x 14336 x 4096), each direction by itself: bf16 200 us to quantise (6.0
// TB/s), 213 us back (5.6; 183 us right behind the quantisation, part of whose
// codes the last-level cache still holds); fp16 the same; fp32 425 us (5.0
// TB/s) and 500 us (4.3), its 32 bytes per lane in two halves.  The large
// layer's pack (16384 tokens of 7168 to 8 rows each) 202 us: 0.73 GB, 3.6
// TB/s, scale lines written 8 bytes at a time from several XCDs.  Small calls
// are bound by their launch.
//
// A half-wave takes one chunk of 256 elements of one row: 8 elements per
// lane (16-byte loads for fp16 and bf16, two for fp32), 4 lanes per block.
// The block's largest magnitude (a maximum that keeps NaN) is combined over
// the 4 lanes by DPP; the conversion instruction rounds two values per issue.  A lane stores 4 bytes
// of codes, a half-wave one 128-byte line.
#include "rmoe_internal.h"
#include "rmoe_mx.h"

namespace rmoe {
namespace {

typedef unsigned u4 __attribute__((ext_vector_type(4)));
typedef unsigned u2 __attribute__((ext_vector_type(2)));

// 8 elements at element offset 8 v of a row, as fp32
template <typename T>
struct Row8;
template <>
struct Row8<_Float16> {
    u4 a;
    __device__ __forceinline__ void load(const void *p, int64_t v) { a = __builtin_nontemporal_load((const u4 *)p + v); }
    __device__ __forceinline__ void get(float *f) const {
        const h8 h = __builtin_bit_cast(h8, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)h[i];
    }
    // the values of 8 codes under one scale; nan: NaN instead
    static __device__ __forceinline__ void put(void *p, int64_t v, unsigned q, float scale, bool nan) {
        u4 o;
        o[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, scale, 0));
        o[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, scale, 1));
        o[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, scale, 2));
        o[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, scale, 3));
        if (nan) o = u4{0x7e007e00u, 0x7e007e00u, 0x7e007e00u, 0x7e007e00u};
        __builtin_nontemporal_store(o, (u4 *)p + v);
    }
};
struct bf16_t {};
template <>
struct Row8<bf16_t> {
    u4 a;
    __device__ __forceinline__ void load(const void *p, int64_t v) { a = __builtin_nontemporal_load((const u4 *)p + v); }
    __device__ __forceinline__ void get(float *f) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __builtin_bit_cast(float, a[i] << 16);
            f[2 * i + 1] = __builtin_bit_cast(float, a[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void put(void *p, int64_t v, unsigned q, float scale, bool nan) {
        u4 o;
        o[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0));
        o[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1));
        o[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2));
        o[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3));
        if (nan) o = u4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
        __builtin_nontemporal_store(o, (u4 *)p + v);
    }
};
template <>
struct Row8<float> {
    u4 a, b;
    __device__ __forceinline__ void load(const void *p, int64_t v) {
        a = __builtin_nontemporal_load((const u4 *)p + 2 * v);
        b = __builtin_nontemporal_load((const u4 *)p + 2 * v + 1);
    }
    __device__ __forceinline__ void get(float *f) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // by value: a bit cast of a vector's element itself reads element 0
            const unsigned x = a[i], y = b[i];
            f[i] = __builtin_bit_cast(float, x);
            f[4 + i] = __builtin_bit_cast(float, y);
        }
    }
    static __device__ __forceinline__ void put(void *p, int64_t v, unsigned q, float scale, bool nan) {
        typedef float f2 __attribute__((ext_vector_type(2)));
        const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 1);
        const f2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 3);
        f4 x = {a.x, a.y, b.x, b.y}, y = {c.x, c.y, d.x, d.y};
        const float n = __builtin_nanf("");
        if (nan) x = y = f4{n, n, n, n};
        __builtin_nontemporal_store(x, (f4 *)p + 2 * v);
        __builtin_nontemporal_store(y, (f4 *)p + 2 * v + 1);
    }
};

// x from lane ^ 1 and lane ^ 2 (quad permutes)
template <int CTRL>
__device__ __forceinline__ float quad(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

struct Chunk {
    unsigned codes;   // 8 codes of this lane
    unsigned scales;  // lanes with (lane & 31) == 0 and 4: the chunk's low and high scale dword
};

// One chunk per half-wave: 8 values per lane (zeros past the row's end).
__device__ __forceinline__ Chunk quantize_chunk(float (&f)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) m = mx_amax(m, f[i], f[i + 1]);
    m = mx_amax(0.f, m, quad<0xB1>(m));
    m = mx_amax(0.f, m, quad<0x4E>(m));
    const unsigned byte = mx_scale_byte(m);
    Chunk c;
    unsigned codes[1];
    mx_codes<8>(f, byte, codes);
    c.codes = codes[0];
    // block g sits in lanes 4g .. 4g+3; its byte is byte g / 2 of dword g % 2
    const int g = (threadIdx.x & 31) >> 2;
    unsigned s = byte << (8 * (g >> 1));
    s |= (unsigned)__shfl_xor((int)s, 8);
    s |= (unsigned)__shfl_xor((int)s, 16);
    c.scales = s;
    return c;
}

// rows = every row of the batch, rpb = rows per matrix (scales are laid out
// per matrix).  U units (row, chunk) per half-wave, a stride of one grid pass
// apart, their loads issued before any is used.
template <typename T, int U>
__global__ __launch_bounds__(256) void quantize_kernel(const void *__restrict__ x, unsigned units, unsigned kc,
                                                       unsigned rpb, int64_t cols, unsigned char *__restrict__ codes,
                                                       unsigned char *__restrict__ scales) {
    const unsigned half = threadIdx.x >> 5, l = threadIdx.x & 31;
    const unsigned stride = gridDim.x * 8u;
    const int64_t vpr = cols / 8;  // 8-element vectors per row
    for (unsigned u0 = blockIdx.x * 8u + half; u0 < units; u0 += U * stride) {
        Row8<T> v[U];
        unsigned row[U], ch[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const unsigned u = u0 + i * stride;
            row[i] = u / kc;
            ch[i] = u - row[i] * kc;
            v[i] = Row8<T>{};
            if (u < units && (int64_t)ch[i] * 32 + l < vpr) v[i].load(x, row[i] * vpr + (int64_t)ch[i] * 32 + l);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const unsigned u = u0 + i * stride;
            float f[8];
            v[i].get(f);
            const Chunk c = quantize_chunk(f);
            if (u >= units) continue;
            *(unsigned *)(codes + ((int64_t)u * kMxChunkBytes + 4 * l)) = c.codes;
            if ((l & ~4u) == 0) {
                const unsigned b = row[i] / rpb, r = row[i] - b * rpb;
                *(unsigned *)(scales + (((int64_t)b * kc + ch[i]) * rpb + r) * 8 + l) = c.scales;
            }
        }
    }
}

template <typename T, int U>
__global__ __launch_bounds__(256) void dequantize_kernel(const unsigned char *__restrict__ codes,
                                                         const unsigned char *__restrict__ scales, unsigned units,
                                                         unsigned kc, unsigned rpb, int64_t cols, void *__restrict__ y) {
    const unsigned half = threadIdx.x >> 5, l = threadIdx.x & 31;
    const unsigned stride = gridDim.x * 8u;
    const int64_t vpr = cols / 8;
    for (unsigned u0 = blockIdx.x * 8u + half; u0 < units; u0 += U * stride) {
        unsigned q[U], sb[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const unsigned u = u0 + i * stride;
            q[i] = sb[i] = 0;
            if (u < units) {
                const unsigned row = u / kc, ch = u - row * kc, b = row / rpb, r = row - b * rpb;
                q[i] = __builtin_nontemporal_load((const unsigned *)(codes + ((int64_t)u * kMxChunkBytes + 4 * l)));
                sb[i] = scales[(((int64_t)b * kc + ch) * rpb + r) * 8 + mx_pos(l >> 2)];
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const unsigned u = u0 + i * stride;
            if (u >= units) continue;
            const unsigned row = u / kc, ch = u - row * kc;
            const int64_t v = (int64_t)ch * 32 + l;
            if (v >= vpr) continue;
            // value = E2M1 number times 2^(byte - 127), rounded once to the
            // output type by the conversion (two values each)
            Row8<T>::put(y, row * vpr + v, q[i], __builtin_bit_cast(float, sb[i] << 23), sb[i] == 255u);
        }
    }
}

// stacked codes and scales of pair p's padded row = MXFP4 of x[p / k]; the
// token's row is read and quantised once and its codes written k times.
// Pairs whose table entry is out of range move nothing.
__global__ __launch_bounds__(256) void pack_mx_kernel(const _Float16 *__restrict__ x, const float *__restrict__ topk_w,
                                                      const int32_t *__restrict__ prow,
                                                      const int32_t *__restrict__ cpos, unsigned units, unsigned kc,
                                                      int64_t T, int32_t k, int64_t cols, int64_t Tp,
                                                      unsigned char *__restrict__ codes,
                                                      unsigned char *__restrict__ scales,
                                                      float *__restrict__ w_compact) {
    const unsigned half = threadIdx.x >> 5, l = threadIdx.x & 31;
    const unsigned stride = gridDim.x * 8u;
    const int64_t vpr = cols / 8, pairs = T * k;
    for (unsigned ub = blockIdx.x * 8u; ub < units; ub += stride) {
        const unsigned u = ub + half;
        const unsigned t = u / kc, ch = u - t * kc;
        Row8<_Float16> v{};
        if (u < units && (int64_t)ch * 32 + l < vpr) v.load(x, t * vpr + (int64_t)ch * 32 + l);
        float f[8];
        v.get(f);
        const Chunk c = quantize_chunk(f);
        if (u >= units) continue;
        if (ch == 0) {  // the token's routed weights
            for (int j = l; j < k; j += 32) {
                const int64_t p = (int64_t)t * k + j, q = cpos[p];
                if (q >= 0 && q < pairs) w_compact[q] = topk_w[p];
            }
        }
        for (int j = 0; j < k; ++j) {
            const int64_t r = prow[(int64_t)t * k + j];
            if (r < 0 || r >= Tp) continue;
            *(unsigned *)(codes + (r * kc + ch) * kMxChunkBytes + 4 * l) = c.codes;
            if ((l & ~4u) == 0) *(unsigned *)(scales + ((int64_t)ch * Tp + r) * 8 + l) = c.scales;
        }
    }
}

// units per half-wave: 4 once every CU has several waves of work, else 1 so
// that a small call spreads over the chip.  470 M elements with 1, 4 and 8:
// bf16 210, 199, 207 us to quantise and 226, 213, 211 back (fp16 the same);
// fp32 382, 423, 419 and 543, 500, 582.  At most 2^20 workgroups, which stride
// beyond
constexpr int64_t kMxWideUnits = 256 * 8 * 16;
unsigned grid_units(int64_t units, int per) {
    const int64_t g = (units + 8 * per - 1) / (8 * per);
    return (unsigned)(g < 1 ? 1 : g > (1 << 20) ? 1 << 20 : g);
}

template <typename T>
hipError_t quantize_t(const void *x, int64_t batch, int64_t rows, int64_t cols, unsigned char *codes,
                      unsigned char *scales, hipStream_t s) {
    const int64_t kc = (cols + kMxChunk - 1) / kMxChunk, units = batch * rows * kc;
    if (units >= kMxWideUnits)
        hipLaunchKernelGGL((quantize_kernel<T, 4>), dim3(grid_units(units, 4)), dim3(256), 0, s, x, (unsigned)units,
                           (unsigned)kc, (unsigned)rows, cols, codes, scales);
    else
        hipLaunchKernelGGL((quantize_kernel<T, 1>), dim3(grid_units(units, 1)), dim3(256), 0, s, x, (unsigned)units,
                           (unsigned)kc, (unsigned)rows, cols, codes, scales);
    return hipGetLastError();
}

template <typename T>
hipError_t dequantize_t(const unsigned char *codes, const unsigned char *scales, int64_t batch, int64_t rows,
                        int64_t cols, void *y, hipStream_t s) {
    const int64_t kc = (cols + kMxChunk - 1) / kMxChunk, units = batch * rows * kc;
    if (units >= kMxWideUnits)
        hipLaunchKernelGGL((dequantize_kernel<T, 4>), dim3(grid_units(units, 4)), dim3(256), 0, s, codes, scales,
                           (unsigned)units, (unsigned)kc, (unsigned)rows, cols, y);
    else
        hipLaunchKernelGGL((dequantize_kernel<T, 1>), dim3(grid_units(units, 1)), dim3(256), 0, s, codes, scales,
                           (unsigned)units, (unsigned)kc, (unsigned)rows, cols, y);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(const void *x, MxType type, int64_t batch, int64_t rows, int64_t cols,
                           unsigned char *codes, unsigned char *scales, hipStream_t s) {
    switch (type) {
        case MxType::f16: return quantize_t<_Float16>(x, batch, rows, cols, codes, scales, s);
        case MxType::bf16: return quantize_t<bf16_t>(x, batch, rows, cols, codes, scales, s);
        default: return quantize_t<float>(x, batch, rows, cols, codes, scales, s);
    }
}

hipError_t launch_dequantize(const unsigned char *codes, const unsigned char *scales, MxType type, int64_t batch,
                             int64_t rows, int64_t cols, void *y, hipStream_t s) {
    switch (type) {
        case MxType::f16: return dequantize_t<_Float16>(codes, scales, batch, rows, cols, y, s);
        case MxType::bf16: return dequantize_t<bf16_t>(codes, scales, batch, rows, cols, y, s);
        default: return dequantize_t<float>(codes, scales, batch, rows, cols, y, s);
    }
}

hipError_t launch_pack_mx(const _Float16 *x, const float *topk_w, const int32_t *prow, const int32_t *cpos,
                          int64_t T, int32_t k, int64_t H, int64_t Tp, unsigned char *codes, unsigned char *scales,
                          float *w_compact, hipStream_t s) {
    const int64_t kc = (H + kMxChunk - 1) / kMxChunk, units = T * kc;
    int64_t g = (units + 7) / 8;
    if (g > 256 * 64) g = 256 * 64;  // the kernel strides beyond 64 workgroups per CU
    hipLaunchKernelGGL(pack_mx_kernel, dim3((unsigned)g), dim3(256), 0, s, x, topk_w, prow, cpos, (unsigned)units,
                       (unsigned)kc, T, k, H, Tp, codes, scales, w_compact);
    return hipGetLastError();
}

}  // namespace rmoe
