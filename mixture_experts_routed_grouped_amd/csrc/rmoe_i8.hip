// Quantisation to 8-bit integer rows (format: rmoe_i8.h), its inverse, the
// token pack that quantises on the way, and the quantisation of the hidden
// rows between the two products of the routed FFN.  Bound by HBM: a row is
// read once, held in registers while its largest magnitude is found, and its
// codes are written once.
//
// A row is taken by W waves (1, 4 or 16); a lane holds NV vectors of 8 elements
// (16 bytes of fp16 and bf16, 32 of fp32), all loaded before the first is
// used.  Rows longer than 64 W NV vectors are read twice, the second time
// from the caches.  One wave per row needs no barrier and is taken once there
// are several rows per CU; more waves shorten the one row that a small call
// waits for.  Rows of at most 64 vectors go without these loops: up to 32
// vectors several rows share a wave, from 33 on each has one.
//
// 8 x 14336 x 4096 bf16: 257 us there (5.5 TB/s), 229 back (6.2); 49152 hidden
// rows of 1408 fp32 60 us (5.8 TB/s); the pack of 8192 tokens of 2048 to 6 rows
// each 34 us.  Calls of some hundred rows take 3 to 7 us, a launch's latency
// and one trip to memory.
#include <type_traits>

#include "rmoe_i8.h"
#include "rmoe_internal.h"

namespace rmoe {
namespace {

// Element types: bytes, and how they are held in memory.
struct bf16_t {
    unsigned short bits;
};

// 8 elements at vector v of a row
template <typename T>
struct Vec8 {
    u4 a;
    __device__ __forceinline__ void load(const void *row, int64_t v) { a = ((const u4 *)row)[v]; }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        if constexpr (std::is_same<T, _Float16>::value) {
            const h8 h = __builtin_bit_cast(h8, a);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = (float)h[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __builtin_bit_cast(float, a[i] << 16);
                f[2 * i + 1] = __builtin_bit_cast(float, a[i] & 0xffff0000u);
            }
        }
    }
};
template <>
struct Vec8<float> {
    f4 a, b;
    __device__ __forceinline__ void load(const void *row, int64_t v) {
        a = ((const f4 *)row)[2 * v];
        b = ((const f4 *)row)[2 * v + 1];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    }
};
// The largest of a value over a wave, in every lane (NaN kept).
__device__ __forceinline__ float wave_amax(float m) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = mx_amax(0.f, m, __shfl_xor(m, d));
    return m;
}

// Quantises one row of vpr vectors with W waves: put(v, codes) for every
// vector v, and returns the row's scale (in every thread).  part: W floats of
// LDS, free on entry for W > 1 (a barrier lies between two rows).
template <typename T, int W, int NV, class Put>
__device__ __forceinline__ float quantize_row(const void *row, int64_t vpr, float *part, Put &&put) {
    const int tid = W == 1 ? threadIdx.x & 63 : threadIdx.x;
    constexpr int STEP = 64 * W;
    Vec8<T> x[NV];
    float m = 0.f;
    const bool once = vpr <= (int64_t)STEP * NV;
    for (int64_t v0 = 0; v0 < vpr; v0 += (int64_t)STEP * NV) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t v = v0 + tid + STEP * i;
            x[i] = Vec8<T>{};
            if (v < vpr) x[i].load(row, v);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[8];
            x[i].get(f);
#pragma unroll
            for (int j = 0; j < 8; j += 2) m = mx_amax(m, f[j], f[j + 1]);
        }
    }
    m = wave_amax(m);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) m = mx_amax(0.f, m, part[w]);
        __syncthreads();
    }
    const I8Row r = i8_row(m);
    for (int64_t v0 = 0; v0 < vpr; v0 += (int64_t)STEP * NV) {
        if (!once) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t v = v0 + tid + STEP * i;
                if (v < vpr) x[i].load(row, v);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t v = v0 + tid + STEP * i;
            float f[8];
            x[i].get(f);
            const u2 c = i8_codes(f, r);
            if (v < vpr) put(v, c);
        }
    }
    return r.scale;
}

template <typename T, int W, int NV>
__global__ __launch_bounds__(256) void quantize_kernel(const void *__restrict__ x, int64_t rows, int64_t vpr,
                                                       unsigned char *__restrict__ codes, float *__restrict__ scales) {
    __shared__ float part[4];
    constexpr int RPW = 4 / W;  // rows per workgroup
    for (int64_t r0 = (int64_t)blockIdx.x * RPW; r0 < rows; r0 += (int64_t)gridDim.x * RPW) {
        const int64_t row = r0 + (W == 1 ? threadIdx.x >> 6 : 0);
        if (W == 1 && row >= rows) continue;
        u2 *out = (u2 *)codes + row * vpr;
        const float s = quantize_row<T, W, NV>((const unsigned char *)x + row * vpr * 8 * (int64_t)sizeof(T), vpr, part,
                                               [&](int64_t v, u2 c) { out[v] = c; });
        if ((threadIdx.x & (64 * W - 1)) == 0) scales[row] = s;
    }
}

// Rows of up to 64 vectors: 1 << sh lanes each, the fewest that hold one.  Up
// to 32 vectors a wave takes several rows, where a wave for each spent its time
// on starting waves (54320 rows of 16 fp32 21.5 -> 2.6 us, 100000 of 64 fp16
// 39 -> 6); from 33 on a row still has its wave, and what it gains it gains by
// the straight body without quantize_row's loops (100000 of 512 46 -> 30).
template <typename T>
__global__ __launch_bounds__(256) void quantize_short_kernel(const void *__restrict__ x, int64_t rows, int vpr, int sh,
                                                             unsigned char *__restrict__ codes,
                                                             float *__restrict__ scales) {
    const int v = threadIdx.x & ((1 << sh) - 1), rpg = 256 >> sh;
    for (int64_t r0 = (int64_t)blockIdx.x * rpg; r0 < rows; r0 += (int64_t)gridDim.x * rpg) {
        const int64_t row = r0 + (threadIdx.x >> sh);
        const bool in = row < rows && v < vpr;
        Vec8<T> e{};
        if (in) e.load(x, row * vpr + v);
        float f[8], m = 0.f;
        e.get(f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) m = mx_amax(m, f[j], f[j + 1]);
        for (int d = 1; d < 1 << sh; d <<= 1) m = mx_amax(0.f, m, __shfl_xor(m, d));
        const I8Row r = i8_row(m);
        const u2 c = i8_codes(f, r);
        if (in) ((u2 *)codes)[row * vpr + v] = c;
        if (row < rows && v == 0) scales[row] = r.scale;
    }
}

// y[row, :] = codes times the row's scale, rounded once more to the type.
template <typename T>
__global__ __launch_bounds__(256) void dequantize_kernel(const unsigned char *__restrict__ codes,
                                                         const float *__restrict__ scales, int64_t n8, int64_t vpr,
                                                         void *__restrict__ y) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
        const u2 c = ((const u2 *)codes)[i];
        const float s = scales[i / vpr];
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (float)(int)(signed char)(c[j >> 2] >> (8 * (j & 3))) * s;
        if constexpr (std::is_same<T, float>::value) {
            ((f4 *)y)[2 * i] = f4{f[0], f[1], f[2], f[3]};
            ((f4 *)y)[2 * i + 1] = f4{f[4], f[5], f[6], f[7]};
        } else if constexpr (std::is_same<T, _Float16>::value) {
            h8 h;
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = (_Float16)f[j];
            ((h8 *)y)[i] = h;
        } else {
            typedef __bf16 b8 __attribute__((ext_vector_type(8)));
            b8 h;
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = (__bf16)f[j];
            ((b8 *)y)[i] = h;
        }
    }
}

// A token's row is read and quantised once, by W waves, and its codes and
// scale are written to its k padded rows.  Pairs whose table entry is out of
// range move nothing.  The first 64 entries are read beside the row.
template <int W, int NV>
__global__ __launch_bounds__(256) void pack_kernel(const _Float16 *__restrict__ x, const float *__restrict__ topk_w,
                                                   const int32_t *__restrict__ prow, const int32_t *__restrict__ cpos,
                                                   int64_t T, int32_t k, int64_t vpr, int64_t Tp,
                                                   unsigned char *__restrict__ codes, float *__restrict__ scales,
                                                   float *__restrict__ w_compact) {
    __shared__ float part[4];
    constexpr int TPG = 4 / W;  // tokens per workgroup
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t pairs = T * k;
    for (int64_t t0 = (int64_t)blockIdx.x * TPG; t0 < T; t0 += (int64_t)gridDim.x * TPG) {
        const int64_t t = t0 + (W == 1 ? wave : 0);
        if (W == 1 && t >= T) continue;
        const int first = lane < k ? prow[t * k + lane] : -1;
        const float s = quantize_row<_Float16, W, NV>(x + t * vpr * 8, vpr, part, [&](int64_t v, u2 c) {
            for (int j = 0; j < k; ++j) {
                const int64_t r = j < 64 ? __builtin_amdgcn_readlane(first, j) : prow[t * k + j];
                if (r >= 0 && r < Tp) ((u2 *)codes)[r * vpr + v] = c;
            }
        });
        for (int j = W == 1 ? lane : threadIdx.x; j < k; j += 64 * W) {
            const int64_t p = t * k + j, q = cpos[p], r = prow[p];
            if (q >= 0 && q < pairs) w_compact[q] = topk_w[p];
            if (r >= 0 && r < Tp) scales[r] = s;
        }
    }
}

// Hidden rows: the valid rows of every block, fp32 in, codes and scales out.
template <int W, int NV>
__global__ __launch_bounds__(W == 16 ? 1024 : 256) void hidden_kernel(
    const float *__restrict__ rows, const int32_t *__restrict__ gs, const int32_t *__restrict__ gpo,
    const int32_t *__restrict__ gidx, int32_t E, int64_t vpr, unsigned char *__restrict__ codes,
    float *__restrict__ scales) {
    __shared__ float part[W];
    const BlockInfo bi = block_info(gs, gpo, gidx, E, blockIdx.y);
    constexpr int RPW = W == 1 ? 4 : 1;
    for (int i0 = blockIdx.x * RPW; i0 < bi.rows; i0 += gridDim.x * RPW) {
        const int i = i0 + (W == 1 ? threadIdx.x >> 6 : 0);
        if (W == 1 && i >= bi.rows) continue;
        const int64_t row = (int64_t)blockIdx.y * kBlockM + i;
        u2 *out = (u2 *)codes + row * vpr;
        const float s = quantize_row<float, W, NV>(rows + row * vpr * 8, vpr, part, [&](int64_t v, u2 c) { out[v] = c; });
        if ((threadIdx.x & (64 * W - 1)) == 0) scales[row] = s;
    }
}

// Vectors per lane: the fewest that hold a row of vpr vectors in W waves,
// at most 8.
int vectors(int64_t vpr, int w) {
    const int64_t n = (vpr + 64 * w - 1) / (64 * w);
    return n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : 8;
}
// One wave per row once every CU has several rows and a row fits its
// registers; else four.
int waves(int64_t rows, int64_t vpr) { return vpr <= 64 * 4 && rows >= 4 * 256 ? 1 : vpr <= 64 ? 1 : 4; }

unsigned grid_of(int64_t n) { return (unsigned)(n < 1 ? 1 : n > (1 << 20) ? 1 << 20 : n); }

template <typename T>
hipError_t quantize_t(const void *x, int64_t rows, int64_t cols, unsigned char *codes, float *scales, hipStream_t s) {
    const int64_t vpr = cols / 8;
    if (vpr <= 64) {
        int sh = 0;
        while (1 << sh < vpr) ++sh;
        hipLaunchKernelGGL(quantize_short_kernel<T>, dim3(grid_of((rows + (256 >> sh) - 1) / (256 >> sh))), dim3(256), 0,
                           s, x, rows, (int)vpr, sh, codes, scales);
        return hipGetLastError();
    }
    const int w = waves(rows, vpr), nv = vectors(vpr, w);
    const dim3 grid(grid_of(w == 1 ? (rows + 3) / 4 : rows)), wg(256);
#define RMOE_Q(W, NV)                                                                                      \
    if (w == W && nv == NV) {                                                                              \
        hipLaunchKernelGGL((quantize_kernel<T, W, NV>), grid, wg, 0, s, x, rows, vpr, codes, scales);      \
        return hipGetLastError();                                                                          \
    }
    RMOE_Q(1, 2) RMOE_Q(1, 4) RMOE_Q(4, 1) RMOE_Q(4, 2) RMOE_Q(4, 4) RMOE_Q(4, 8)
#undef RMOE_Q
    return hipErrorInvalidValue;
}

template <typename T>
hipError_t dequantize_t(const unsigned char *codes, const float *scales, int64_t rows, int64_t cols, void *y,
                        hipStream_t s) {
    const int64_t n8 = rows * (cols / 8);
    hipLaunchKernelGGL(dequantize_kernel<T>, dim3(grid_of((n8 + 255) / 256)), dim3(256), 0, s, codes, scales, n8,
                       cols / 8, y);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_i8(const void *x, MxType type, int64_t rows, int64_t cols, unsigned char *codes,
                              float *scales, hipStream_t s) {
    switch (type) {
        case MxType::f16: return quantize_t<_Float16>(x, rows, cols, codes, scales, s);
        case MxType::bf16: return quantize_t<bf16_t>(x, rows, cols, codes, scales, s);
        default: return quantize_t<float>(x, rows, cols, codes, scales, s);
    }
}

hipError_t launch_dequantize_i8(const unsigned char *codes, const float *scales, MxType type, int64_t rows,
                                int64_t cols, void *y, hipStream_t s) {
    switch (type) {
        case MxType::f16: return dequantize_t<_Float16>(codes, scales, rows, cols, y, s);
        case MxType::bf16: return dequantize_t<bf16_t>(codes, scales, rows, cols, y, s);
        default: return dequantize_t<float>(codes, scales, rows, cols, y, s);
    }
}

hipError_t launch_pack_i8(const _Float16 *x, const float *topk_w, const int32_t *prow, const int32_t *cpos, int64_t T,
                          int32_t k, int64_t H, int64_t Tp, unsigned char *codes, float *scales, float *w_compact,
                          hipStream_t s) {
    const int64_t vpr = H / 8;
    const int w = waves(T, vpr), nv = vectors(vpr, w);
    const dim3 grid(grid_of(w == 1 ? (T + 3) / 4 : T)), wg(256);
#define RMOE_P(W, NV)                                                                                            \
    if (w == W && nv == NV) {                                                                                    \
        hipLaunchKernelGGL((pack_kernel<W, NV>), grid, wg, 0, s, x, topk_w, prow, cpos, T, k, vpr, Tp, codes,    \
                           scales, w_compact);                                                                   \
        return hipGetLastError();                                                                                \
    }
    RMOE_P(1, 1) RMOE_P(1, 2) RMOE_P(1, 4) RMOE_P(4, 1) RMOE_P(4, 2) RMOE_P(4, 4) RMOE_P(4, 8)
#undef RMOE_P
    return hipErrorInvalidValue;
}

hipError_t launch_quantize_hidden_i8(const I8Args &a, int64_t pairs, hipStream_t s) {
    const int64_t vpr = a.N / 8;
    // few long rows: 16 waves each, as one row's latency is the launch's (128 rows of 14336: 8.5 -> 5.6 us)
    const int w = pairs <= 1024 && vpr > 256 ? 16 : waves(pairs, vpr), nv = vectors(vpr, w);
    const dim3 grid(32, (unsigned)a.M), wg(w == 16 ? 1024 : 256);
#define RMOE_H(W, NV)                                                                                          \
    if (w == W && nv == NV) {                                                                                  \
        hipLaunchKernelGGL((hidden_kernel<W, NV>), grid, wg, 0, s, a.rows, a.gs, a.gpo, a.gidx, a.E, vpr,      \
                           a.yc, a.ys);                                                                        \
        return hipGetLastError();                                                                              \
    }
    RMOE_H(16, 1) RMOE_H(16, 2) RMOE_H(16, 4) RMOE_H(16, 8)
    RMOE_H(1, 1) RMOE_H(1, 2) RMOE_H(1, 4) RMOE_H(4, 1) RMOE_H(4, 2) RMOE_H(4, 4) RMOE_H(4, 8)
#undef RMOE_H
    return hipErrorInvalidValue;
}

}  // namespace rmoe
