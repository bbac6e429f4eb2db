// Backward pass of the router: with p the probabilities of a token, g its
// routed weights' gradients, c the experts' counts, n the tokens that count,
// and a and b the gradients of the balance and the z loss,
//
//     dp[e] = sum_{j: id[j] = e} g[j] + a E c[e] / (k n^2)
//     dl[e] = p[e] (dp[e] - sum_i p[i] dp[i]) + 2 b lse p[e] / n
//     dx    = dl . W             (a sum over the experts)
//     dW[e] = sum_t dl[t, e] x[t]
//
// Steps: dl, 64 tokens per workgroup; dx and dW, in one launch up to 128
// experts; the parts of dW added up.  The products run on fp16
// MFMA, so dl, which is fp32, becomes two fp16 operands, the value rounded
// and what that rounding left (22 bits): once scaled by a power of two per
// token (for dx), once by one per expert and 64 tokens (for dW), so that the
// largest value of either lies in [2^13, 2^14) and small gradients stay far
// from fp16's subnormal numbers.  Both are stored in the order in which a wave
// reads its MFMA operands: 1 KB per operand, 16 bytes per lane.
//
// Bound by memory: x is read once for dW, dx written once (and added to what
// came through the experts, read once).  16384 tokens of 7168, 128 experts, an
// eighth left out: 200 us, 188 of them dx and dW (752 MB by the counters: 4.0
// TB/s, the matrix cores busy 28%), dl 15, the sum of the parts 9.  8191 tokens of 2048, 64
// experts: 35 us (9 + 21 + 5), three launches of which each waits for its first
// loads; 9 tokens of 256: 13 us, most of it the host's.
#include <atomic>
#include <type_traits>

#include "rmoe_internal.h"
#include "rmoe_kloop.h"
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

// ---- dl: one workgroup per block of 64 tokens.  Thread (token, lane, part):
// a token's experts are cut into 4 parts of EP / 4, each taken by 4 lanes.
__global__ __launch_bounds__(1024) void dlogits_kernel(RouterBackArgs a, Scratch s) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int EP = 32 * s.et, ld = EP + 4;  // row stride: 16 tokens x 4 lanes on 64 banks
    float *L = reinterpret_cast<float *>(smem);            // [64][ld] dl
    float *pg = L + BT * ld;                               // [64 k] a routed weight's gradient
    int *pid = reinterpret_cast<int *>(pg + BT * a.k);     // [64 k] its expert, -1: none
    __shared__ float red[4][BT], big[4][BT], up_x[BT], up_w[256];
    __shared__ uint16_t on[4];
    const int tid = threadIdx.x, sub = tid & 3, tok = (tid >> 2) & 63, part = tid >> 8;
    const int64_t b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, t0 = b * BT, t = t0 + tok;  // grid_rows
    if (b >= s.nb) return;
    const bool live = t < a.T && (a.mask == nullptr || a.mask[t] != 0);
    const float n = (float)a.counts[a.E];
    const float ca = a.dlosses && n > 0.f ? a.dlosses[0] * (float)a.E / ((float)a.k * n * n) : 0.f;
    const float cz = a.dlosses && n > 0.f ? a.dlosses[1] * 2.0f / n : 0.f;
    float *row = L + tok * ld;
    const float *p = a.probs + t * a.E;
    const int e0 = part * (EP / 4) + sub, ne = EP / 16;  // this thread's experts: e0 + 4 i, i < ne
    float pv[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) pv[i] = i < ne && live && e0 + 4 * i < a.E ? p[e0 + 4 * i] : 0.f;

    // the block's pairs are one contiguous piece
    const int64_t np = (a.T - t0 < BT ? a.T - t0 : BT) * a.k;
    for (int i = tid; i < np; i += 1024) {
        const int tk = i / a.k, id = a.ids[t0 * a.k + i];
        const bool use = id >= 0 && id < a.E && (a.mask == nullptr || a.mask[t0 + tk] != 0);
        const int64_t q = a.cpos ? (int64_t)a.cpos[t0 * a.k + i] : t0 * a.k + i;
        pg[i] = use && q >= 0 && q < a.T * a.k ? a.drw[q] : 0.f;
        pid[i] = use ? id : -1;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < ne) row[e0 + 4 * i] = e0 + 4 * i < a.E ? ca * (float)a.counts[e0 + 4 * i] : 0.f;
    if (tid < 256) {  // 16 tokens per wave, 4 equal bits each
        const uint64_t bits = __ballot(live);
        if ((tid & 63) == 0) {
            unsigned w = 0;
            for (int i = 0; i < 16; ++i) w |= (unsigned)(bits >> (4 * i) & 1) << i;
            on[tid >> 6] = (uint16_t)w;
        }
    }
    __syncthreads();
    if (tid == 0)
        s.live[b] = (uint64_t)on[0] | (uint64_t)on[1] << 16 | (uint64_t)on[2] << 32 | (uint64_t)on[3] << 48;
    if (b == 0 && tid < 8) ((h8 *)s.zeros)[tid] = h8{0, 0, 0, 0, 0, 0, 0, 0};
    if (live && tid < 256 && sub == 0)
        for (int j = 0; j < a.k; ++j) {
            const int id = pid[tok * a.k + j];
            if (id >= 0) row[id] += pg[tok * a.k + j];
        }
    __syncthreads();
    // dl from dp - sum p dp: what is large in both cancels before the rest is
    // added (exactly where one expert has all the probability)
    float dv[16], dot = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        dv[i] = i < ne ? row[e0 + 4 * i] : 0.f;
        dot += pv[i] * dv[i];
    }
    dot += __shfl_xor(dot, 1);
    dot += __shfl_xor(dot, 2);
    if (sub == 0) red[part][tok] = dot;
    __syncthreads();
    dot = (red[0][tok] + red[1][tok]) + (red[2][tok] + red[3][tok]);
    const float z = live ? cz * a.lse[t] : 0.f;
    // and the scales: of a token, over its lanes and parts; of an expert
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < ne) {
            const float dl = live && e0 + 4 * i < a.E ? pv[i] * ((dv[i] - dot) + z) : 0.f;
            row[e0 + 4 * i] = dl;
            m = __builtin_elementwise_maximum(m, __builtin_fabsf(dl));
        }
    m = __builtin_elementwise_maximum(m, __shfl_xor(m, 1));
    m = __builtin_elementwise_maximum(m, __shfl_xor(m, 2));
    if (sub == 0) big[part][tok] = m;
    __syncthreads();
    if (tid < EP) {
        float w = 0.f;
#pragma unroll 16
        for (int i = 0; i < BT; ++i) w = __builtin_elementwise_maximum(w, __builtin_fabsf(L[i * ld + tid]));
        const Scale c = scale_of(w);
        up_w[tid] = c.up;
        s.sw[b * EP + tid] = c.down;
    } else if (tid >= 1024 - BT) {
        const int tk = tid - (1024 - BT);
        m = big[0][tk];
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __builtin_elementwise_maximum(m, big[i][tk]);
        const Scale c = scale_of(m);
        up_x[tk] = c.up;
        s.sx[t0 + tk] = c.down;
    }
    __syncthreads();
    // operands of dx: lane = token % 32 + 32 (octet of experts % 2)
    for (int i = tid; i < BT * EP / 8; i += 1024) {
        const int tk = i & 63, o = i >> 6;  // token, octet of experts
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = L[tk * ld + 8 * o + j];
        unsigned char *f = s.dlx + (((b * 2 + (tk >> 5)) * (2 * s.et) + (o >> 1)) * 2) * FRAG;
        store_split(f + ((tk & 31) + 32 * (o & 1)) * 16, v, up_x[tk]);
    }
    // operands of dW: lane = expert % 32 + 32 (octet of tokens % 2)
    for (int i = tid; i < EP * 8; i += 1024) {
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
// tokens.  A tile's operands travel through a ring in LDS that all four read;
// the rows to be added go to a piece of each wave's own, where the sum
// replaces them (fp16, its one rounding) before it leaves as whole lines.
// Everything that is read in the loop comes by DMA, one tile ahead: the waits
// count memory instructions and leave the stores of the tile before in flight.
template <int ET>
struct DxCfg {
    static constexpr int KS = 2 * ET;                // steps of 16 experts
    static constexpr int OPS = KS * 2 * FRAG;        // operands of a tile of tokens
    static constexpr int PIECE = 32 * 128;           // 32 tokens x 64 columns of fp16
    static constexpr int WAVE = PIECE + 256;         // and the tokens' scales, twice
    static constexpr int SLOT = OPS + 4 * WAVE, D = 2;
    static constexpr int W = ET * 16 * FRAG;         // the gate matrix's 256 columns, before the loop
    static constexpr int LDS = W > D * SLOT ? W : D * SLOT;
};
// A value that is the same in every lane, in a scalar register (under two
// nested branches the compiler kept LDS addresses in vector registers, which
// the DMA's M0 cannot take).
__device__ __forceinline__ unsigned scalar(unsigned x) { return __builtin_amdgcn_readfirstlane(x); }
// 256-byte DMA: lane i stores the dword at g to LDS byte lds + 4 i (s_nop: as
// in dma16)
__device__ __forceinline__ void dma4(const void *g, unsigned lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(g) : "memory", "m0");
}
template <int ET, bool ADD>
__device__ __forceinline__ void dx_body(const RouterBackArgs &a, const Scratch &s, int chunks, int block,
                                        unsigned char *smem) {
    using C = DxCfg<ET>;
    constexpr int KS = C::KS;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int lr = lane & 31, lh = lane >> 5;
    // an XCD's workgroups take neighbouring chunks of tokens, whose operands its L2 holds
    const int total = s.slices * chunks, per = (total + 7) / 8;
    const int at = (block & 7) * per + (block >> 3);
    if ((block >> 3) >= per || at >= total) return;
    const int chunk = at / s.slices, slice = at - chunk * s.slices;
    const int64_t c0 = (int64_t)slice * HS + 64 * wave;  // this wave's columns
    const bool mine = c0 < a.H;
    const int64_t cl = mine ? c0 : a.H - 64;             // idle waves read valid ones
    const unsigned lds0 = (unsigned)(uintptr_t)smem;
    const int r8 = lane >> 3, c8 = lane & 7;
#pragma unroll
    for (int g = 0; g < 4 * ET; ++g) {
        const int e = 8 * g + r8, c = c8 ^ swz_k(r8);
        const void *src = e < a.E ? (const void *)(a.w + e * a.H + cl + 8 * c) : (const void *)(s.zeros + 16 * c);
        dma16(src, lds0 + (wave * ET * 4 + g) * FRAG);
    }
    wait_vm<0>();
    __syncthreads();
    h8 w[2][KS];
    const unsigned char *slot = smem + wave * ET * 4 * FRAG;
#pragma unroll
    for (int ht = 0; ht < 2; ++ht)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            w[ht][k].lo = tr_read(slot + 2048 * k + tr_off(lane, ht, 0));
            w[ht][k].hi = tr_read(slot + 2048 * k + tr_off(lane, ht, 1));
        }
    __syncthreads();  // the gate matrix is in registers: its LDS becomes the ring
    const int64_t tiles = (a.T + 31) / 32, lo = tiles * chunk / chunks, hi = tiles * (chunk + 1) / chunks;
    // a tile's 4 ET operands, ET per wave; its scales; its rows to be added,
    // whose 16-byte chunks are XOR-swizzled by row pair (lds_swz)
    const unsigned char *ops = uniform(s.dlx + wave * ET * FRAG);
    const _Float16 *addbase = uniform(a.add + cl);
    unsigned aoff[2];  // lane offset of rows 8 j ..: their swizzle repeats with j's parity
#pragma unroll
    for (int j = 0; j < 2; ++j) aoff[j] = (unsigned)((8 * j + r8) * a.H * 2) + 16 * (c8 ^ lds_swz(8 * j + r8));
    const unsigned row16 = (unsigned)(32 * a.H);
    auto fill = [&](int64_t i) {
        const unsigned d = lds0 + (unsigned)(i & 1) * C::SLOT, mypiece = d + C::OPS + wave * C::WAVE;
#pragma unroll
        for (int g = 0; g < ET; ++g) dma16_sb(ops + i * C::OPS + g * FRAG, 16 * lane, d + (wave * ET + g) * FRAG);
        dma4(s.sx + 32 * i + lr, mypiece + C::PIECE);
        if constexpr (ADD) {
            const _Float16 *rows = addbase + 32 * i * a.H;
            const int left = a.T - 32 * i < 32 ? (int)(a.T - 32 * i) : 32;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                unsigned o = aoff[j & 1] + (j >> 1) * row16;
                // behind the last token: its row again
                if (left < 32 && 8 * j + r8 >= left) o = (unsigned)((left - 1) * a.H * 2) + 16 * c8;
                dma16_sb(rows, o, mypiece + 1024 * j);
            }
        }
    };
    _Float16 *out = a.dx + c0;
    const unsigned yoff = (unsigned)(r8 * a.H * 2) + 16 * c8, row8 = (unsigned)(16 * a.H);
    if (lo < hi) fill(lo);
    for (int64_t i = lo; i < hi; ++i) {
        // all but the stores of the tile before, which is a whole one
        if (i > lo && mine)
            wait_vm<4>();
        else
            wait_vm<0>();
        bar();  // tile i is there; everyone is done with the other slot
        if (i + 1 < hi) fill(i + 1);
        const unsigned char *f = smem + (i & 1) * C::SLOT + lane * 16;
        unsigned char *st = smem + (i & 1) * C::SLOT + C::OPS + wave * C::WAVE;
        f16x acc[2];
#pragma unroll
        for (int ht = 0; ht < 2; ++ht)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[ht][r] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const h8 dh = *(const h8 *)(f + (2 * k) * FRAG), dl = *(const h8 *)(f + (2 * k + 1) * FRAG);
#pragma unroll
            for (int ht = 0; ht < 2; ++ht) acc[ht] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w[ht][k], dh, acc[ht], 0, 0, 0);
#pragma unroll
            for (int ht = 0; ht < 2; ++ht) acc[ht] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w[ht][k], dl, acc[ht], 0, 0, 0);
        }
        // register 4q + r of tile ht: column 32 ht + 8q + 4lh + r of token lr
        const float down = *(const float *)(st + C::PIECE + 4 * lr);
        unsigned char *row = st + lr * 128 + 8 * lh;
#pragma unroll
        for (int ht = 0; ht < 2; ++ht)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                h4 *at4 = (h4 *)(row + (((4 * ht + q) ^ lds_swz(lr)) << 4));
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = acc[ht][4 * q + r] * down;
                if constexpr (ADD) {
                    const h4 add = *at4;
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] += (float)add[r];
                }
                *at4 = to_h4(v[0], v[1], v[2], v[3]);
            }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's rows are written
        asm volatile("" ::: "memory");
        h8 y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *(const h8 *)(st + (8 * j + r8) * 128 + ((c8 ^ lds_swz(8 * j + r8)) << 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t t = 32 * i + 8 * j + r8;
            if (t < a.T && mine) *(h8 *)((unsigned char *)(out + 32 * i * a.H) + yoff + j * row8) = y[j];
        }
        asm volatile("" ::: "memory");
    }
}

// ---- dW: a workgroup takes 256 columns of H, up to 4 expert tiles and a
// part of the blocks of tokens, which it runs through in steps of 32 tokens: x
// as a k-major slot, the operands of dl as they are, and the experts' scales,
// all by DMA D - 1 steps ahead.  NW = 8 waves, 4 groups of 64 columns x 2
// halves of the expert tiles: two per SIMD, one's scaling and addresses beside
// the other's MFMAs; or 4, each with every tile.  A block's sums are scaled
// back and added up in fp32 after its second step.
template <int ET, int NW, int D_>
struct DwCfg {
    static constexpr int XB = 32 * HS * 2, DB = ET * 4 * FRAG, SB = NW * 256;  // bytes of a step: tokens, operands, scales
    static constexpr int SLOT = XB + DB + SB, D = D_;
    static constexpr int TPW = NW == 8 ? (ET + 1) / 2 : ET;  // expert tiles per wave
    static constexpr int XPW = 16 / NW;                      // instructions of x per wave
    static constexpr int OPW = (4 * ET + NW - 1) / NW;       // operands moved per wave
    static constexpr int DMAS = XPW + OPW + 1;               // per wave and step
    static constexpr int LDS = D * SLOT;
};
template <int ET, int NW, int D>
__device__ __forceinline__ void dw_body(const RouterBackArgs &a, const Scratch &s, int tile0, int block,
                                        unsigned char *smem) {
    using C = DwCfg<ET, NW, D>;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int lr = lane & 31, lh = lane >> 5, r8 = lane >> 3;
    const int cg = wave & 3, t0 = (wave >> 2) * C::TPW;  // this wave's columns, its first tile
    const int total = s.slices * s.splits, per = (total + 7) / 8;
    const int at = (block & 7) * per + (block >> 3);
    if ((block >> 3) >= per || at >= total) return;
    const int split = at / s.slices, slice = at - split * s.slices;
    const int64_t b0 = s.nb * split / s.splits, n = 2 * (s.nb * (split + 1) / s.splits - b0);  // first block, steps
    const unsigned lds = (unsigned)(uintptr_t)smem;
    // the kernel before wrote it: scalar loads (the waits below count the
    // vector memory instructions)
    typedef const __attribute__((address_space(4))) uint64_t *Words;
    const Words live = (Words)(uintptr_t)s.live;
    // x: this wave moves 8 XPW tokens of one column group
    const int64_t cx = (int64_t)slice * HS + 64 * (wave * C::XPW >> 2);
    const _Float16 *xbase = uniform(a.x + (cx < a.H ? cx : a.H - 64));  // idle columns read valid ones
    const int tx = 8 * (wave * C::XPW & 3) + r8;
    const unsigned xstep = (unsigned)(16 * a.H), xoff = (unsigned)(tx * a.H * 2) + 16 * ((lane & 7) ^ swz_k(r8));
    // step i; past the last one the last again, so that every wait counts the
    // same.  The mask of the next step is requested here and used there.
    uint64_t mask = n > 0 ? live[b0] : 0;
    auto fill = [&](int64_t i) {
        const unsigned d = lds + (unsigned)(i % C::D) * C::SLOT;
        const int64_t j = i < n ? i : n - 1, b = b0 + (j >> 1);
        const int half = (int)(j & 1);
        const unsigned on = (unsigned)(mask >> (32 * half));
        mask = live[b0 + ((i + 1 < n ? i + 1 : n - 1) >> 1)];
        const _Float16 *src = xbase + (b * BT + 32 * half) * a.H;
        if (on == ~0u) {
#pragma unroll
            for (int g = 0; g < C::XPW; ++g) dma16_sb(src, xoff + g * xstep, scalar(d + (wave * C::XPW + g) * FRAG));
        } else {
#pragma unroll
            for (int g = 0; g < C::XPW; ++g) {
                const unsigned char *row = (const unsigned char *)src + xoff + g * xstep;
                dma16(on >> (tx + 8 * g) & 1 ? row : s.zeros + 16 * (lane & 7), scalar(d + (wave * C::XPW + g) * FRAG));
            }
        }
        // the step's operands: tile o / 4, of its 8 the half's 4 (some moved twice)
        const unsigned char *f = s.dlw + (b * s.et + tile0) * 8 * FRAG + half * 4 * FRAG;
#pragma unroll
        for (int g = 0; g < C::OPW; ++g) {
            const int o = (wave * C::OPW + g) % (4 * ET);
            dma16_sb(uniform(f + ((o >> 2) * 8 + (o & 3)) * FRAG), 16 * lane, scalar(d + C::XB + o * FRAG));
        }
        dma4(s.sw + b * 32 * s.et + 32 * (tile0 + (wave < ET ? wave : 0)) + lr, scalar(d + C::XB + C::DB + wave * 256));
    };
    f16x sum[C::TPW][2], acc[C::TPW][2];
#pragma unroll
    for (int et = 0; et < C::TPW; ++et)
#pragma unroll
        for (int ht = 0; ht < 2; ++ht)
#pragma unroll
            for (int r = 0; r < 16; ++r) sum[et][ht][r] = 0.f;
    unsigned off[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) off[i >> 1][i & 1] = tr_off(lane, i >> 1, i & 1);
    auto step = [&](int64_t i, auto second) __attribute__((always_inline)) {
        wait_vm<(D - 2) * C::DMAS>();        // all but the steps after this one
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's reads of the step before
        bar();                               // step i is there; everyone is done with the slot of the one before
        fill(i + D - 1);
        const unsigned char *slot = smem + (i % C::D) * C::SLOT, *xs = slot + cg * 4 * FRAG;
        const unsigned char *ds = slot + C::XB + t0 * 4 * FRAG + lane * 16;
        h8 xa[2][2];
#pragma unroll
        for (int ht = 0; ht < 2; ++ht)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                xa[ht][k].lo = tr_read(xs + 2048 * k + off[ht][0]);
                xa[ht][k].hi = tr_read(xs + 2048 * k + off[ht][1]);
            }
#pragma unroll
        for (int et = 0; et < C::TPW; ++et) {
            if (NW == 8 && ET % 2 && t0 + et >= ET) continue;  // an odd count's idle tile
            if constexpr (!second) {
#pragma unroll
                for (int ht = 0; ht < 2; ++ht)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[et][ht][r] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const h8 dh = *(const h8 *)(ds + (et * 4 + k * 2) * FRAG), dl = *(const h8 *)(ds + (et * 4 + k * 2 + 1) * FRAG);
#pragma unroll
                for (int ht = 0; ht < 2; ++ht) acc[et][ht] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xa[ht][k], dh, acc[et][ht], 0, 0, 0);
#pragma unroll
                for (int ht = 0; ht < 2; ++ht) acc[et][ht] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xa[ht][k], dl, acc[et][ht], 0, 0, 0);
            }
            if constexpr (second) {
                const float down = *(const float *)(slot + C::XB + C::DB + (t0 + et) * 256 + 4 * lr);
#pragma unroll
                for (int ht = 0; ht < 2; ++ht)
#pragma unroll
                    for (int r = 0; r < 16; ++r) sum[et][ht][r] = __builtin_fmaf(acc[et][ht][r], down, sum[et][ht][r]);
            }
        }
    };
    if (n > 0) {
#pragma unroll
        for (int i = 0; i < D - 1; ++i) fill(i);
        for (int64_t i = 0; i < n; i += 2) {
            step(i, std::integral_constant<bool, false>{});
            step(i + 1, std::integral_constant<bool, true>{});
        }
        wait_vm<0>();  // no DMA is left in flight
    }
    const int64_t c0 = (int64_t)slice * HS + 64 * cg;
    if (c0 >= a.H) return;
    float *y = s.splits > 1 ? s.parts + (int64_t)split * a.E * a.H : a.dw;
#pragma unroll
    for (int et = 0; et < C::TPW; ++et) {
        const int e = 32 * (tile0 + t0 + et) + lr;
        if (e >= a.E || t0 + et >= ET) continue;
#pragma unroll
        for (int ht = 0; ht < 2; ++ht)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(f4 *)(y + e * a.H + c0 + 32 * ht + 8 * q + 4 * lh) =
                    f4{sum[et][ht][4 * q], sum[et][ht][4 * q + 1], sum[et][ht][4 * q + 2], sum[et][ht][4 * q + 3]};
    }
}

template <int ET>
__global__ __launch_bounds__(512) void dw_kernel(RouterBackArgs a, Scratch s, int tile0) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    dw_body<ET, 8, 4>(a, s, tile0, blockIdx.x, smem);
}
template <int ET, bool ADD>
__global__ __launch_bounds__(256) void dx_kernel(RouterBackArgs a, Scratch s, int chunks) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    dx_body<ET, ADD>(a, s, chunks, blockIdx.x, smem);
}
// Both in one launch, up to 4 expert tiles: workgroups 0 .. dws - 1 (a
// multiple of 8) dW's, the others dx's.  Up to 3 expert tiles two workgroups
// fit a CU, all are there at once, and dW waits for its loads where dx stores.
// With 4 (186 vector and 128 accumulation registers: one wave per SIMD) a CU
// holds one: dW's go first and dx's follow as CUs fall free, which saves a
// launch and the drain between the two, no more.  Against a launch each: 16384
// tokens of 7168, 128 experts 217 -> 202 us for the whole pass, 4096 tokens of
// the same 83 -> 73, 8191 tokens of 2048, 64 experts 39 -> 36, 9 tokens of 256
// 16 -> 12.
template <int ET, bool ADD>
__global__ __launch_bounds__(256) void grads_kernel(RouterBackArgs a, Scratch s, int chunks, int dws) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    if ((int)blockIdx.x < dws)
        dw_body<ET, 4, 2>(a, s, 0, blockIdx.x, smem);
    else
        dx_body<ET, ADD>(a, s, chunks, blockIdx.x - dws, smem);
}

// The parts' sum, in order.
__global__ __launch_bounds__(64) void dw_sum_kernel(const f4 *__restrict__ parts, int splits, int64_t n, f4 *__restrict__ y) {
    for (int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 64) {
        f4 v = parts[i];
#pragma unroll 8
        for (int p = 1; p < splits; ++p) v += parts[p * n + i];
        y[i] = v;
    }
}

// dx: parts of the tiles of tokens, for wgs workgroups in all
int64_t dx_chunks(const RouterBackArgs &a, const Scratch &s, int64_t wgs) {
    const int64_t tiles = (a.T + 31) / 32, n = wgs / s.slices;
    return n > tiles ? tiles : n < 1 ? 1 : n;
}

template <int ET, bool ADD>
hipError_t launch_dx(const RouterBackArgs &a, const Scratch &s, hipStream_t st) {
    constexpr int LDS = DxCfg<ET>::LDS;
    static_assert(LDS <= 160 * 1024, "LDS");
    static std::atomic<uint64_t> lds_set{0};
    hipError_t e = lds_opt_in_once((const void *)dx_kernel<ET, ADD>, LDS, lds_set);
    if (e != hipSuccess) return e;
    const int64_t chunks = dx_chunks(a, s, 512 + s.slices - 1), total = (s.slices * chunks + 7) / 8 * 8;
    hipLaunchKernelGGL((dx_kernel<ET, ADD>), dim3((unsigned)total), dim3(256), LDS, st, a, s, (int)chunks);
    return hipGetLastError();
}

template <int ET>
hipError_t launch_dw(const RouterBackArgs &a, const Scratch &s, int tile0, hipStream_t st) {
    constexpr int LDS = DwCfg<ET, 8, 4>::LDS;
    static_assert(LDS <= 160 * 1024, "LDS");
    static std::atomic<uint64_t> lds_set{0};
    hipError_t e = lds_opt_in_once((const void *)dw_kernel<ET>, LDS, lds_set);
    if (e != hipSuccess) return e;
    const int total = (s.slices * s.splits + 7) / 8 * 8;
    hipLaunchKernelGGL(dw_kernel<ET>, dim3((unsigned)total), dim3(512), LDS, st, a, s, tile0);
    return hipGetLastError();
}

template <int ET, bool ADD>
hipError_t launch_grads(const RouterBackArgs &a, const Scratch &s, hipStream_t st) {
    constexpr int LDS = DwCfg<ET, 4, 2>::LDS > DxCfg<ET>::LDS ? DwCfg<ET, 4, 2>::LDS : DxCfg<ET>::LDS;
    static_assert(LDS <= 80 * 1024, "LDS of two workgroups per CU");
    static std::atomic<uint64_t> lds_set{0};
    hipError_t e = lds_opt_in_once((const void *)grads_kernel<ET, ADD>, LDS, lds_set);
    if (e != hipSuccess) return e;
    // 512 workgroups in all: two per CU (with 4 expert tiles one after the other)
    const int64_t dws = (s.slices * s.splits + 7) / 8 * 8, chunks = dx_chunks(a, s, 512 - dws), dxs = (s.slices * chunks + 7) / 8 * 8;
    hipLaunchKernelGGL((grads_kernel<ET, ADD>), dim3((unsigned)(dws + dxs)), dim3(256), LDS, st, a, s, (int)chunks, (int)dws);
    return hipGetLastError();
}

hipError_t launch_sum(const RouterBackArgs &a, const Scratch &s, hipStream_t st) {
    if (s.splits <= 1) return hipSuccess;
    const int64_t n = a.E * a.H / 4;
    int64_t g = (n + 63) / 64;
    if (g > 256 * 32) g = 256 * 32;  // strides beyond
    hipLaunchKernelGGL(dw_sum_kernel, dim3((unsigned)g), dim3(64), 0, st, (const f4 *)s.parts, s.splits, n, (f4 *)a.dw);
    return hipGetLastError();
}

}  // namespace

int64_t router_backward_scratch(int64_t T, int64_t H, int32_t E) { return scratch_of(nullptr, T, H, E).bytes; }

hipError_t launch_router_backward(const RouterBackArgs &a, hipStream_t st) {
    const Scratch s = scratch_of(a.scratch, a.T, a.H, a.E);
    if (s.nb > 0) {
        const int lds = BT * (32 * s.et + 4 + 2 * a.k) * 4;
        static std::atomic<uint64_t> lds_set{0};
        hipError_t e = lds_opt_in_once((const void *)dlogits_kernel, BT * (256 + 4 + 2 * 32) * 4, lds_set);
        if (e != hipSuccess) return e;
        const GridRows grid = grid_rows(s.nb);
        hipLaunchKernelGGL(dlogits_kernel, dim3(grid.x, grid.y), dim3(1024), lds, st, a, s);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (s.et <= GT) {
#define RMOE_G(N) case N: e = a.add ? launch_grads<N, true>(a, s, st) : launch_grads<N, false>(a, s, st); break;
            switch (s.et) {
                RMOE_G(1) RMOE_G(2) RMOE_G(3)
                default: e = a.add ? launch_grads<GT, true>(a, s, st) : launch_grads<GT, false>(a, s, st);
            }
#undef RMOE_G
            return e != hipSuccess ? e : launch_sum(a, s, st);
        }
#define RMOE_X(N) case N: e = a.add ? launch_dx<N, true>(a, s, st) : launch_dx<N, false>(a, s, st); break;
        switch (s.et) {
            RMOE_X(5) RMOE_X(6) RMOE_X(7) RMOE_X(8)
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
    return launch_sum(a, s, st);
}

}  // namespace rmoe
