// Backward pass of the router: with p the probabilities of a token, g its
// routed weights' gradients, c the experts' counts, n the tokens that count,
// and a and b the gradients of the balance and the z loss,
//
//     dp[e] = sum_{j: id[j] = e} g[j] + a E c[e] / (k n^2)
//     dl[e] = p[e] (dp[e] - sum_i p[i] dp[i]) + 2 b lse p[e] / n
//     dx    = dl . W             (a sum over the experts)
//     dW[e] = sum_t dl[t, e] x[t]
//
// Three steps: dl, 64 tokens per workgroup; dx; dW.  The products run on fp16
// MFMA, so dl, which is fp32, becomes two fp16 operands, the value rounded
// and what that rounding left (22 bits): once scaled by a power of two per
// token (for dx), once by one per expert and 64 tokens (for dW), so that the
// largest value of either lies in [2^13, 2^14) and small gradients stay far
// from fp16's subnormal numbers.  Both are stored in the order in which a wave
// reads its MFMA operands: 1 KB per operand, 16 bytes per lane.
//
// Bound by memory: x is read once for dW, dx written once (and added to what
// came through the experts, read once).
#include <atomic>

#include "rmoe_internal.h"
#include "rmoe_kmajor.h"

namespace rmoe {
namespace {

constexpr int BT = 64;      // tokens per block
constexpr int HS = 256;     // columns of H per workgroup of the products: 64 per wave
constexpr int FRAG = 1024;  // bytes of one MFMA operand of a wave
constexpr int GT = 4;       // expert tiles (of 32) per workgroup of dW

// The scratch: what the first step leaves for the others.
struct Scratch {
    int64_t nb;             // blocks of 64 tokens
    int et;                 // expert tiles of 32
    int slices, groups;     // of dW: column slices, groups of expert tiles
    int splits;             // parts of the token range in dW
    unsigned char *dlx;     // [nb][2 halves of 32 tokens][et * 2 steps of 16 experts][hi, lo] operands
    unsigned char *dlw;     // [nb][et][4 steps of 16 tokens][hi, lo] operands
    float *sx;              // [nb * 64] inverse scale of a token
    float *sw;              // [nb][32 et] inverse scale of an expert in a block
    uint64_t *live;         // [nb] bit t: token 64 b + t counts
    unsigned char *zeros;   // 128 bytes
    float *parts;           // [splits][E][H]
    int64_t bytes;
};
Scratch scratch_of(unsigned char *base, int64_t T, int64_t H, int32_t E) {
    Scratch s;
    s.nb = (T + BT - 1) / BT;
    s.et = (E + 31) / 32;
    s.slices = (int)((H + HS - 1) / HS);
    s.groups = (s.et + GT - 1) / GT;
    // one workgroup per CU, and at least 4 blocks of tokens for each
    const int64_t units = (int64_t)s.slices * s.groups;
    int64_t n = units >= 256 ? 1 : 256 / units;
    if (n > s.nb / 4) n = s.nb / 4;
    s.splits = (int)(n < 1 ? 1 : n);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        unsigned char *p = base + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    const int64_t half = s.nb * s.et * 4 * 2 * FRAG;
    s.dlx = take(half);
    s.dlw = take(half);
    s.sx = (float *)take(s.nb * BT * 4);
    s.sw = (float *)take(s.nb * s.et * 32 * 4);
    s.live = (uint64_t *)take(s.nb * 8);
    s.zeros = take(128);
    s.parts = (float *)take(s.splits > 1 ? s.splits * E * H * 4 : 0);
    s.bytes = at;
    return s;
}

// A power of two that brings a largest magnitude into [2^13, 2^14), and its
// inverse; at most 2^126.
struct Scale {
    float up, down;
};
__device__ __forceinline__ Scale scale_of(float amax) {
    const int ex = (int)((__builtin_bit_cast(unsigned, amax) >> 23) & 255u);
    const int se = min(267 - ex, 253);
    return Scale{__builtin_bit_cast(float, (unsigned)se << 23), __builtin_bit_cast(float, (unsigned)(254 - se) << 23)};
}
// Two operands of 8 values each, hi at p and lo FRAG behind it.
__device__ __forceinline__ void store_split(unsigned char *p, const float (&v)[8], float up) {
    h8 hi, lo;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float s = v[i] * up;
        hi[i] = (_Float16)s;
        lo[i] = (_Float16)(s - (float)hi[i]);
    }
    *(h8 *)p = hi;
    *(h8 *)(p + FRAG) = lo;
}

// ---- dl: one workgroup per block of 64 tokens, 4 lanes per token.
__global__ __launch_bounds__(256) void dlogits_kernel(RouterBackArgs a, Scratch s) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int EP = 32 * s.et, ld = EP + 4;  // row stride: 16 tokens x 4 lanes on 64 banks
    float *L = reinterpret_cast<float *>(smem);  // [64][ld]
    __shared__ float up_x[BT], up_w[256];
    const int tid = threadIdx.x, tok = tid >> 2, sub = tid & 3;
    const int64_t b = blockIdx.x, t = b * BT + tok;
    const bool live = t < a.T && (a.mask == nullptr || a.mask[t] != 0);
    const float n = (float)a.counts[a.E];
    const float ca = a.dlosses && n > 0.f ? a.dlosses[0] * (float)a.E / ((float)a.k * n * n) : 0.f;
    const float cz = a.dlosses && n > 0.f ? a.dlosses[1] * 2.0f / n : 0.f;
    float *row = L + tok * ld;
    const float *p = a.probs + t * a.E;

    auto gradient = [&](int j) {  // of routed weight j of this token
        const int64_t i = t * a.k + j, q = a.cpos ? a.cpos[i] : i;
        return q >= 0 && q < a.T * a.k ? a.drw[q] : 0.f;
    };
    float dot = 0.f;
    if (live) {
        for (int e = sub; e < a.E; e += 4) dot += p[e] * (ca * (float)a.counts[e]);
        for (int j = sub; j < a.k; j += 4) {
            const int id = a.ids[t * a.k + j];
            if (id >= 0 && id < a.E) dot += p[id] * gradient(j);
        }
    }
    dot += __shfl_xor(dot, 1);
    dot += __shfl_xor(dot, 2);
    const float z = live ? cz * a.lse[t] - dot : 0.f;
    for (int e = sub; e < EP; e += 4) row[e] = live && e < a.E ? p[e] * (ca * (float)a.counts[e] + z) : 0.f;
    __syncthreads();
    if (live && sub == 0)
        for (int j = 0; j < a.k; ++j) {
            const int id = a.ids[t * a.k + j];
            if (id >= 0 && id < a.E) row[id] += p[id] * gradient(j);
        }
    __syncthreads();
    // scales: of a token, over its 4 lanes; of an expert
    float m = 0.f;
    for (int e = sub; e < EP; e += 4) m = __builtin_elementwise_maximum(m, __builtin_fabsf(row[e]));
    m = __builtin_elementwise_maximum(m, __shfl_xor(m, 1));
    m = __builtin_elementwise_maximum(m, __shfl_xor(m, 2));
    if (sub == 0) {
        const Scale c = scale_of(m);
        up_x[tok] = c.up;
        s.sx[t] = c.down;
    }
    if (tid < EP) {
        float w = 0.f;
#pragma unroll 8
        for (int i = 0; i < BT; ++i) w = __builtin_elementwise_maximum(w, __builtin_fabsf(L[i * ld + tid]));
        const Scale c = scale_of(w);
        up_w[tid] = c.up;
        s.sw[b * EP + tid] = c.down;
    }
    const uint64_t bits = __ballot(live);  // 16 tokens per wave, 4 equal bits each
    __shared__ uint16_t on[4];
    if ((tid & 63) == 0) {
        unsigned w = 0;
        for (int i = 0; i < 16; ++i) w |= (unsigned)(bits >> (4 * i) & 1) << i;
        on[tid >> 6] = (uint16_t)w;
    }
    if (b == 0 && tid < 8) ((h8 *)s.zeros)[tid] = h8{0, 0, 0, 0, 0, 0, 0, 0};
    __syncthreads();
    if (tid == 0)
        s.live[b] = (uint64_t)on[0] | (uint64_t)on[1] << 16 | (uint64_t)on[2] << 32 | (uint64_t)on[3] << 48;
    // operands of dx: lane = token % 32 + 32 (octet of experts % 2)
    for (int i = tid; i < BT * EP / 8; i += 256) {
        const int tk = i & 63, o = i >> 6;  // token, octet of experts
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = L[tk * ld + 8 * o + j];
        unsigned char *f = s.dlx + (((b * 2 + (tk >> 5)) * (2 * s.et) + (o >> 1)) * 2) * FRAG;
        store_split(f + ((tk & 31) + 32 * (o & 1)) * 16, v, up_x[tk]);
    }
    // operands of dW: lane = expert % 32 + 32 (octet of tokens % 2)
    for (int i = tid; i < EP * 8; i += 256) {
        const int o = i / EP, e = i - o * EP;  // octet of tokens, expert
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = L[(8 * o + j) * ld + e];
        unsigned char *f = s.dlw + (((b * s.et + (e >> 5)) * 4 + (o >> 1)) * 2) * FRAG;
        store_split(f + ((e & 31) + 32 * (o & 1)) * 16, v, up_w[e]);
    }
}

// ---- dx: a workgroup takes 256 columns; its 4 waves hold the gate matrix's
// 64 columns each as MFMA operands in registers and run over tiles of 32
// tokens, whose operands come from the caches.
template <int ET>
__global__ __launch_bounds__(256) void dx_kernel(RouterBackArgs a, Scratch s, int chunks) {
    constexpr int KS = 2 * ET;  // steps of 16 experts
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int lr = lane & 31, lh = lane >> 5;
    // an XCD's workgroups take neighbouring chunks of tokens, whose operands its L2 holds
    const int total = s.slices * chunks, per = (total + 7) / 8;
    const int at = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || at >= total) return;
    const int chunk = at / s.slices, slice = at - chunk * s.slices;
    const int64_t c0 = (int64_t)slice * HS + 64 * wave;  // this wave's columns
    const int64_t cl = c0 < a.H ? c0 : a.H - 64;         // idle waves read valid ones
    const unsigned lds = (unsigned)(uintptr_t)smem + wave * ET * 4 * FRAG;
    const int r8 = lane >> 3;
#pragma unroll
    for (int g = 0; g < 4 * ET; ++g) {
        const int e = 8 * g + r8, c = (lane & 7) ^ swz_k(r8);
        const void *src = e < a.E ? (const void *)(a.w + e * a.H + cl + 8 * c) : (const void *)(s.zeros + 16 * c);
        dma16(src, lds + g * FRAG);
    }
    wait_vm<0>();
    bar();
    h8 w[2][KS];
    const unsigned char *slot = smem + wave * ET * 4 * FRAG;
#pragma unroll
    for (int ht = 0; ht < 2; ++ht)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            w[ht][k].lo = tr_read(slot + 2048 * k + tr_off(lane, ht, 0));
            w[ht][k].hi = tr_read(slot + 2048 * k + tr_off(lane, ht, 1));
        }
    __syncthreads();  // the slots become staging pieces: 32 tokens x 64 columns of fp32 per wave
    unsigned char *st = smem + wave * 8192;
    const int64_t tiles = (a.T + 31) / 32, lo = tiles * chunk / chunks, hi = tiles * (chunk + 1) / chunks;
    const int c8 = lane & 7;
    for (int64_t i = lo; i < hi; ++i) {
        const unsigned char *f = s.dlx + i * KS * 2 * FRAG + lane * 16;
        h8 add[4];
        if (a.add && c0 < a.H) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t t = 32 * i + 8 * j + r8;
                if (t < a.T) add[j] = *(const h8 *)(a.add + t * a.H + c0 + 8 * c8);
            }
        }
        f16x acc[2];
#pragma unroll
        for (int ht = 0; ht < 2; ++ht)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[ht][r] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const h8 dh = *(const h8 *)(f + (2 * k) * FRAG), dl = *(const h8 *)(f + (2 * k + 1) * FRAG);
#pragma unroll
            for (int ht = 0; ht < 2; ++ht) {
                acc[ht] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w[ht][k], dh, acc[ht], 0, 0, 0);
                acc[ht] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w[ht][k], dl, acc[ht], 0, 0, 0);
            }
        }
        // register 4q + r of tile ht: column 32 ht + 8q + 4lh + r of token lr
        const float down = s.sx[32 * i + lr];
#pragma unroll
        for (int ht = 0; ht < 2; ++ht)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(f4 *)(st + lr * 256 + (((8 * ht + 2 * q + lh) ^ (lr & 15)) << 4)) =
                    f4{acc[ht][4 * q] * down, acc[ht][4 * q + 1] * down, acc[ht][4 * q + 2] * down, acc[ht][4 * q + 3] * down};
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        asm volatile("" ::: "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 8 * j + r8;
            const f4 v0 = *(const f4 *)(st + r * 256 + (((2 * c8) ^ (r & 15)) << 4));
            const f4 v1 = *(const f4 *)(st + r * 256 + (((2 * c8 + 1) ^ (r & 15)) << 4));
            const int64_t t = 32 * i + r;
            if (t < a.T && c0 < a.H) {
                h8 y;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    float v = q < 4 ? v0[q & 3] : v1[q & 3];
                    if (a.add) v += (float)add[j][q];
                    y[q] = (_Float16)v;
                }
                *(h8 *)(a.dx + t * a.H + c0 + 8 * c8) = y;
            }
        }
        asm volatile("" ::: "memory");
    }
}

// ---- dW: a workgroup takes 256 columns of H, up to 4 expert tiles and a
// part of the blocks of tokens; x travels as a k-major slot, the operands of
// dl as they are.  A block's sums are scaled back and added up in fp32.
template <int ET>
__global__ __launch_bounds__(256) void dw_kernel(RouterBackArgs a, Scratch s, int tile0) {
    constexpr int XB = BT * HS * 2, DB = ET * 8 * FRAG, SLOT = XB + DB;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int lr = lane & 31, lh = lane >> 5, r8 = lane >> 3;
    const int total = s.slices * s.splits, per = (total + 7) / 8;
    const int at = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || at >= total) return;
    const int split = at / s.slices, slice = at - split * s.slices;
    const int64_t c0 = (int64_t)slice * HS + 64 * wave, cl = c0 < a.H ? c0 : a.H - 64;
    const int64_t b0 = s.nb * split / s.splits, b1 = s.nb * (split + 1) / s.splits;
    const unsigned lds = (unsigned)(uintptr_t)smem;
    const int c = (lane & 7) ^ swz_k(r8);
    // x: this wave's column group, 8 instructions of 8 tokens; dl: 2 ET of its 8 ET operands
    auto fill = [&](int64_t b, int slot) {
        const uint64_t on = s.live[b];
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            const int t = 8 * g + r8;
            const void *src = on >> t & 1 ? (const void *)(a.x + (b * BT + t) * a.H + cl + 8 * c) : (const void *)(s.zeros + 16 * c);
            dma16(src, lds + slot * SLOT + wave * 8 * FRAG + g * FRAG);
        }
        const unsigned char *d = s.dlw + (b * s.et + tile0) * 8 * FRAG + lane * 16;
#pragma unroll
        for (int g = 0; g < 2 * ET; ++g) {
            const int o = wave * 2 * ET + g;
            dma16(d + o * FRAG, lds + slot * SLOT + XB + o * FRAG);
        }
    };
    f16x sum[ET][2];
#pragma unroll
    for (int et = 0; et < ET; ++et)
#pragma unroll
        for (int ht = 0; ht < 2; ++ht)
#pragma unroll
            for (int r = 0; r < 16; ++r) sum[et][ht][r] = 0.f;
    unsigned off[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) off[i >> 1][i & 1] = tr_off(lane, i >> 1, i & 1);
    if (b0 < b1) fill(b0, 0);
    for (int64_t b = b0; b < b1; ++b) {
        const int slot = (int)(b - b0) & 1;
        float down[ET];
#pragma unroll
        for (int et = 0; et < ET; ++et) down[et] = s.sw[b * 32 * s.et + 32 * (tile0 + et) + lr];
        wait_vm<0>();
        __syncthreads();  // block b is there; everyone is done with the other slot
        if (b + 1 < b1) fill(b + 1, slot ^ 1);
        const unsigned char *xs = smem + slot * SLOT + wave * 8 * FRAG, *ds = smem + slot * SLOT + XB + lane * 16;
        h8 xa[2][4];
#pragma unroll
        for (int ht = 0; ht < 2; ++ht)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                xa[ht][k].lo = tr_read(xs + 2048 * k + off[ht][0]);
                xa[ht][k].hi = tr_read(xs + 2048 * k + off[ht][1]);
            }
#pragma unroll
        for (int et = 0; et < ET; ++et) {
            f16x acc[2];
#pragma unroll
            for (int ht = 0; ht < 2; ++ht)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[ht][r] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const h8 dh = *(const h8 *)(ds + ((et * 4 + k) * 2) * FRAG), dl = *(const h8 *)(ds + ((et * 4 + k) * 2 + 1) * FRAG);
#pragma unroll
                for (int ht = 0; ht < 2; ++ht) {
                    acc[ht] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xa[ht][k], dh, acc[ht], 0, 0, 0);
                    acc[ht] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xa[ht][k], dl, acc[ht], 0, 0, 0);
                }
            }
#pragma unroll
            for (int ht = 0; ht < 2; ++ht)
#pragma unroll
                for (int r = 0; r < 16; ++r) sum[et][ht][r] = __builtin_fmaf(acc[ht][r], down[et], sum[et][ht][r]);
        }
    }
    if (c0 >= a.H) return;
    float *y = s.splits > 1 ? s.parts + (int64_t)split * a.E * a.H : a.dw;
#pragma unroll
    for (int et = 0; et < ET; ++et) {
        const int e = 32 * (tile0 + et) + lr;
        if (e >= a.E) continue;
#pragma unroll
        for (int ht = 0; ht < 2; ++ht)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(f4 *)(y + e * a.H + c0 + 32 * ht + 8 * q + 4 * lh) =
                    f4{sum[et][ht][4 * q], sum[et][ht][4 * q + 1], sum[et][ht][4 * q + 2], sum[et][ht][4 * q + 3]};
    }
}

// The parts' sum, in order.
__global__ __launch_bounds__(256) void dw_sum_kernel(const f4 *__restrict__ parts, int splits, int64_t n, f4 *__restrict__ y) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        f4 v = parts[i];
        for (int p = 1; p < splits; ++p) v += parts[p * n + i];
        y[i] = v;
    }
}

template <int ET>
hipError_t launch_dx(const RouterBackArgs &a, const Scratch &s, hipStream_t st) {
    constexpr int LDS = ET * 16 * FRAG > 32768 ? ET * 16 * FRAG : 32768;
    static std::atomic<uint64_t> lds_set{0};
    hipError_t e = lds_opt_in_once((const void *)dx_kernel<ET>, LDS, lds_set);
    if (e != hipSuccess) return e;
    const int64_t tiles = (a.T + 31) / 32;
    int64_t chunks = s.slices >= 512 ? 1 : (512 + s.slices - 1) / s.slices;
    if (chunks > tiles) chunks = tiles;
    const int64_t total = (s.slices * chunks + 7) / 8 * 8;
    hipLaunchKernelGGL(dx_kernel<ET>, dim3((unsigned)total), dim3(256), LDS, st, a, s, (int)chunks);
    return hipGetLastError();
}

template <int ET>
hipError_t launch_dw(const RouterBackArgs &a, const Scratch &s, int tile0, hipStream_t st) {
    constexpr int LDS = 2 * (BT * HS * 2 + ET * 8 * FRAG);
    static_assert(LDS <= 160 * 1024, "LDS");
    static std::atomic<uint64_t> lds_set{0};
    hipError_t e = lds_opt_in_once((const void *)dw_kernel<ET>, LDS, lds_set);
    if (e != hipSuccess) return e;
    const int total = (s.slices * s.splits + 7) / 8 * 8;
    hipLaunchKernelGGL(dw_kernel<ET>, dim3((unsigned)total), dim3(256), LDS, st, a, s, tile0);
    return hipGetLastError();
}

}  // namespace

int64_t router_backward_scratch(int64_t T, int64_t H, int32_t E) { return scratch_of(nullptr, T, H, E).bytes; }

hipError_t launch_router_backward(const RouterBackArgs &a, hipStream_t st) {
    const Scratch s = scratch_of(a.scratch, a.T, a.H, a.E);
    if (s.nb > 0) {
        const int lds = BT * (32 * s.et + 4) * 4;
        static std::atomic<uint64_t> lds_set{0};
        hipError_t e = lds_opt_in_once((const void *)dlogits_kernel, BT * (256 + 4) * 4, lds_set);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(dlogits_kernel, dim3((unsigned)s.nb), dim3(256), lds, st, a, s);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
#define RMOE_X(N) case N: e = launch_dx<N>(a, s, st); break;
        switch (s.et) {
            RMOE_X(1) RMOE_X(2) RMOE_X(3) RMOE_X(4) RMOE_X(5) RMOE_X(6) RMOE_X(7) RMOE_X(8)
            default: return hipErrorInvalidValue;
        }
#undef RMOE_X
        if (e != hipSuccess) return e;
    }
    for (int t = 0; t < s.et; t += GT) {
        hipError_t e = hipSuccess;
        switch (s.et - t) {
            case 1: e = launch_dw<1>(a, s, t, st); break;
            case 2: e = launch_dw<2>(a, s, t, st); break;
            case 3: e = launch_dw<3>(a, s, t, st); break;
            default: e = launch_dw<4>(a, s, t, st); break;
        }
        if (e != hipSuccess) return e;
    }
    if (s.splits > 1) {
        const int64_t n = a.E * a.H / 4;
        int64_t g = (n + 255) / 256;
        if (g > 256 * 16) g = 256 * 16;
        hipLaunchKernelGGL(dw_sum_kernel, dim3((unsigned)g), dim3(256), 0, st, (const f4 *)s.parts, s.splits, n, (f4 *)a.dw);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace rmoe
