// Tiled grouped GEMM on MXFP4 tokens and weights, for blocks with many rows.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 on E2M1 operands takes 16 bytes per lane
// and operand, as v_mfma_f32_32x32x16_f16 does, and the same time: a K step
// of 128 bytes per row holds 256 elements instead of 64, so the 256 x 256
// tile, its DMAs and its LDS traffic are those of the fp16 tiled kernels at
// four times the products.  Each step adds 8 scale bytes per row: 2 KB per
// slot, one 1 KB DMA per wave, and one dword per lane and operand tile that
// serves the step's four sub-steps.  The two extra scale slots per operand
// leave LDS for two operand slots each (136 KB).
//
// The gate/up epilogue quantises the hidden rows on the way out: a lane
// holds 16 of a block's 32 features of one token, its partner lane + 32 the
// others, so the block's maximum is 15 register maxima and one shuffle, and
// the hidden rows cost 4.25 bits per element of memory traffic.
#include <atomic>

#include "rmoe_internal.h"
#include "rmoe_kloop.h"
#include "rmoe_mx.h"
#include "rmoe_sched.h"

namespace rmoe {
namespace {

constexpr int SLOT = 256 * kMxChunkBytes;  // 32 KB: a K step of 256 rows
constexpr int NS = 2;                      // slots per operand
constexpr int SSLOT = 256 * 8;             // scale bytes of a step
constexpr int W_OFF = 0, T_OFF = NS * SLOT, WS_OFF = 2 * NS * SLOT, TS_OFF = WS_OFF + NS * SSLOT;
constexpr int LDS_BYTES = TS_OFF + NS * SSLOT;
static_assert(LDS_BYTES <= 160 * 1024, "LDS");
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u4 __attribute__((ext_vector_type(4)));

struct MxOps {
    typedef i32x4 Frag;
    static constexpr int AR = 1, BR = 1;
    static constexpr int DMAS = 17, LATE = 0, PARTS = 2, PRE = 2;

    unsigned char *smem;
    unsigned dwave;        // LDS address of this wave's 64 rows of a slot
    const unsigned char *tbase, *wbase, *sbase;  // uniform: token rows, weight rows, this wave's scale rows
    int64_t sstep;         // bytes between a step's scales and the next step's
    unsigned sdst;         // LDS address of this wave's scale half
    unsigned soff;         // 16 * lane
    unsigned tkoff[8], woff[8];
    int nk;
    int lr, lh, arow, trow0;  // arow: first A row of this wave's tile 0; tile t at arow + 32 (t & 1) + astep (t / 2)
    int astep;
    unsigned sa[4], sb[4], sna[4], snb[4];

    __device__ __forceinline__ void dma(int d, int j) {
        const int kt = min(j + NS, nk - 1), slot = (j + NS) % NS;
        if (d == 0)
            dma16_sb(sbase + (int64_t)kt * sstep, soff, sdst + slot * SSLOT);
        else if (d <= 8)
            dma16_sb(tbase + (int64_t)kt * kMxChunkBytes, tkoff[d - 1], dwave + T_OFF + slot * SLOT + 1024 * (d - 1));
        else
            dma16_sb(wbase + (int64_t)kt * kMxChunkBytes, woff[d - 9], dwave + W_OFF + slot * SLOT + 1024 * (d - 9));
    }
    __device__ __forceinline__ int row_a(int t) const { return arow + 32 * (t & 1) + astep * (t >> 1); }
    __device__ __forceinline__ void read(int k, int s, int i, Frag *a, Frag *b) {
        const int ch = 2 * s + lh;
        if (i < 4)
            a[i] = *(const Frag *)(smem + W_OFF + (k % NS) * SLOT + lds_off(row_a(i) + lr, ch));
        else
            b[i - 4] = *(const Frag *)(smem + T_OFF + (k % NS) * SLOT + lds_off(trow0 + 32 * (i - 4) + lr, ch));
    }
    __device__ __forceinline__ void step(int k) {
        const unsigned char *ws = smem + WS_OFF + (k % NS) * SSLOT, *ts = smem + TS_OFF + (k % NS) * SSLOT;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            sna[t] = *(const unsigned *)(ws + (row_a(t) + lr) * 8 + 4 * lh);
            snb[t] = *(const unsigned *)(ts + (trow0 + 32 * t + lr) * 8 + 4 * lh);
        }
    }
    __device__ __forceinline__ void next() {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            sa[t] = sna[t];
            sb[t] = snb[t];
        }
    }
    template <int S>
    __device__ __forceinline__ void mma(const Frag &x, const Frag &y, f16x &c, int t, int u) {
        const i32x8 xa = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
        const i32x8 ya = __builtin_shufflevector(y, y, 0, 1, 2, 3, -1, -1, -1, -1);
        c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xa, ya, c, 4, 4, S, (int)sa[t], S, (int)sb[u]);
    }
    __device__ __forceinline__ void publish(int) {}
};

// One work item: blocks bx (rows0 valid rows) and bx+1 (rows1; has1: of the
// same expert) against weight slice nt.
template <bool DUAL>
__device__ __forceinline__ void run_item(const MxArgs &a, unsigned char *smem, const TileItem &it) {
    const int rows0 = a.gidx[it.bx] == it.e ? it.rows0 : 0;
    const int rows1 = (it.rows1 > 0 && a.gidx[it.bx + 1] == it.e) ? it.rows1 : 0;
    if (rows0 == 0 && rows1 == 0) return;
    const bool has1 = rows1 > 0;
    const int64_t N = a.N, rb = (int64_t)a.kc * kMxChunkBytes;
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // opaque per item: addresses are not hoisted out of the item loop
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, lr = lane & 31, lh = lane >> 5;
    const int ww = wave & 1, wt = wave >> 1;  // weight half, token half (= block bx + wt)
    const int64_t n0 = (int64_t)it.nt * (DUAL ? 128 : 256);

    MxOps p;
    p.smem = smem;
    p.nk = a.kc;
    p.lr = lr;
    p.lh = lh;
    p.trow0 = 128 * wt;
    p.arow = DUAL ? 64 * ww : 128 * ww;  // gate/up: tiles 0, 1 gate rows, 2, 3 the same up rows
    p.astep = DUAL ? 128 : 64;
    // weight rows 64 w .. of the slot: gate rows for waves 0, 1, up rows for 2, 3
    const unsigned char *wmat = DUAL && wave >= 2 ? a.w1 : a.w0;
    int64_t wrow0 = n0 + (DUAL ? (64 * wave) & 127 : 64 * wave);
    wrow0 = wrow0 < N ? wrow0 : N - 64;  // a narrow last slice: idle rows read valid rows
    p.wbase = wmat + ((int64_t)it.e * N + wrow0) * rb;
    p.tbase = a.x + (int64_t)it.bx * kBlockM * rb;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int r = 64 * wave + 8 * j + (lane >> 3);
        const int c = (lane & 7) ^ lds_swz(r);
        p.woff[j] = (unsigned)((8 * j + (lane >> 3)) * rb + 16 * c);
        int tr = r;
        if (r >= kBlockM && !has1) tr -= kBlockM;  // absent second block: stay in bounds
        p.tkoff[j] = (unsigned)(tr * rb + 16 * c);
    }
    const unsigned lds0 = (unsigned)(uintptr_t)smem;
    p.dwave = lds0 + 64 * wave * kMxChunkBytes;
    // scales: waves 0, 1 move the weight rows' (128 rows each), waves 2, 3
    // the two blocks' token rows'
    if (wave < 2) {
        int64_t r0 = DUAL ? n0 : n0 + 128 * wave;
        r0 = r0 < N ? r0 : N - 128;
        p.sbase = (DUAL && wave == 1 ? a.w1s : a.w0s) + ((int64_t)it.e * a.kc * N + r0) * 8;
        p.sstep = N * 8;
        p.sdst = lds0 + WS_OFF + 1024 * wave;
    } else {
        p.sbase = a.xs + ((int64_t)it.bx + (wave == 3 && has1 ? 1 : 0)) * kBlockM * 8;
        p.sstep = a.Tp * 8;
        p.sdst = lds0 + TS_OFF + 1024 * (wave - 2);
    }
    p.soff = 16 * lane;

    const int myrows = wt ? rows1 : rows0;
    const bool wlive = DUAL || n0 + 128 * ww < N;
    const int ntt = wlive ? (myrows + 31) / 32 : 0;
    f16x acc[4][4];
    zero_acc(acc);
    kloop_tiles(p, a.kc, ntt, acc);
    if (ntt == 0) return;
    const int64_t row0 = (int64_t)(it.bx + wt) * kBlockM;

    if constexpr (DUAL) {
        // hidden block t (32 features) of token lr of tile u: register 4q + r
        // holds feature 8q + 4lh + r.  Lanes 0-31 assemble and store block 0,
        // lanes 32-63 block 1.
        const int64_t orb = (int64_t)((N + kMxChunk - 1) / kMxChunk) * kMxChunkBytes;
        const int64_t blk = (n0 + 64 * ww) / 32;  // first of the wave's two blocks
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (u >= ntt) continue;
            unsigned c01[2], c23[2], byte[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float v[16];
                unsigned m = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    v[i] = silu(acc[t][u][i]) * acc[t + 2][u][i];
                    m = max(m, __builtin_bit_cast(unsigned, v[i]) & 0x7fffffffu);
                }
                m = max(m, (unsigned)__shfl_xor((int)m, 32));
                byte[t] = mx_scale_byte(m);
                const float up = mx_up(byte[t]), sc = mx_scale(byte[t]);
                c01[t] = mx_codes4(v[0], v[1], v[2], v[3], up, sc) | (mx_codes4(v[4], v[5], v[6], v[7], up, sc) << 16);
                c23[t] = mx_codes4(v[8], v[9], v[10], v[11], up, sc) |
                         (mx_codes4(v[12], v[13], v[14], v[15], up, sc) << 16);
                if (byte[t] == 255u) c01[t] = c23[t] = 0;
            }
            // send the other lane half its block, keep the own one
            const unsigned s01 = lh ? c01[0] : c01[1], s23 = lh ? c23[0] : c23[1];
            const unsigned r01 = (unsigned)__shfl_xor((int)s01, 32), r23 = (unsigned)__shfl_xor((int)s23, 32);
            const unsigned m01 = lh ? c01[1] : c01[0], m23 = lh ? c23[1] : c23[0];
            const unsigned l01 = lh ? r01 : m01, h01 = lh ? m01 : r01, l23 = lh ? r23 : m23, h23 = lh ? m23 : r23;
            u4 o;
            o[0] = (l01 & 0xffffu) | (h01 << 16);
            o[1] = (l01 >> 16) | (h01 & 0xffff0000u);
            o[2] = (l23 & 0xffffu) | (h23 << 16);
            o[3] = (l23 >> 16) | (h23 & 0xffff0000u);
            const int row = 32 * u + lr;
            if (row < myrows) {
                const int64_t b = blk + lh;
                *(u4 *)(a.yc + (row0 + row) * orb + 16 * b) = o;
                a.ys[((b >> 3) * a.Tp + row0 + row) * 8 + mx_pos((int)(b & 7))] = (unsigned char)(lh ? byte[1] : byte[0]);
                // the last slice zero-fills the rest of an odd last chunk
                // (this wave: 32 of its 64 bytes and 2 of its 4 scales)
                if (n0 + 128 == N && (N & 255)) {
                    *(u4 *)(a.yc + (row0 + row) * orb + 16 * (b + 4)) = u4{0, 0, 0, 0};
                    a.ys[((b >> 3) * a.Tp + row0 + row) * 8 + mx_pos((int)((b + 4) & 7))] = 0;
                }
            }
        }
    } else {
        // out rows, staged through LDS for whole-line stores: a wave stages
        // into its own 8 KB pieces of the operand slots (its DMAs have all
        // landed, and no wave reads the ring after the last barrier): 128
        // rows of 128 features, 16-byte chunks XOR-swizzled by row, 32 rows
        // per piece
        auto stage_row = [&](int row) { return smem + (row / 32) * SLOT + wave * 8192 + (row % 32) * 256; };
        float wtok[4] = {0.f, 0.f, 0.f, 0.f};
        const float *rwe = a.rw + a.go[it.e] + it.off + kBlockM * wt;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (u < ntt && 32 * u + lr < myrows) wtok[u] = rwe[32 * u + lr];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (u >= ntt) continue;
            const int row = 32 * u + lr;
            unsigned char *srow = stage_row(row);
            const float w = wtok[u];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f16x &o = acc[t][u];
                    const int c = (4 * t + q) ^ (row & 15);
                    *(h4 *)(srow + (c << 4) + 8 * lh) =
                        to_h4(o[4 * q + 0] * w, o[4 * q + 1] * w, o[4 * q + 2] * w, o[4 * q + 3] * w);
                }
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's staging writes are done
        _Float16 *ybase = a.y + row0 * N + n0 + 128 * ww;
        const int c = lane & 15;
#pragma unroll 4
        for (int r0 = 0; r0 < 32 * ntt; r0 += 4) {
            const int row = r0 + (lane >> 4);
            if (row < myrows) *(h8 *)(ybase + (int64_t)row * N + 8 * c) = *(const h8 *)(stage_row(row) + ((c ^ (row & 15)) << 4));
        }
    }
}

// Persistent, one workgroup per CU, items in the order of rmoe_sched.h.
template <bool DUAL>
__global__ __launch_bounds__(256) void mx_tile_kernel(MxArgs a, int NT) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const TileSeq seq = tile_seq(a.gs, a.E, NT, blockIdx.x % kXcd, kXcd);
    const int nl = gridDim.x / kXcd;
    TileCursor cur;
    for (int i = blockIdx.x / kXcd; i < seq.n; i += nl) run_item<DUAL>(a, smem, tile_item(a.gs, a.gpo, seq, i, cur));
}

template <bool DUAL>
hipError_t launch(const MxArgs &a, int NT, hipStream_t s) {
    unsigned grid = 0;
    hipError_t e = persistent_grid(grid);
    if (e != hipSuccess) return e;
    static std::atomic<uint64_t> lds_set{0};
    e = lds_opt_in_once((const void *)mx_tile_kernel<DUAL>, LDS_BYTES, lds_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(mx_tile_kernel<DUAL>, dim3(grid), dim3(256), LDS_BYTES, s, a, NT);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_tile_gate_up(const MxArgs &a, hipStream_t s) { return launch<true>(a, (int)(a.N / 128), s); }
hipError_t launch_mx_tile_down(const MxArgs &a, hipStream_t s) { return launch<false>(a, (int)((a.N + 255) / 256), s); }

}  // namespace rmoe
