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
// others, so the block's maximum is eight three-value maxima, a swap of the
// halves and one more, and the hidden rows cost 4.25 bits per element of
// memory traffic.
#include <atomic>

#include "rmoe_kloop.h"
#include "rmoe_mx.h"

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

// NEXT: the epilogue uses no LDS, so the second step's first DMAs may be
// issued ahead of it too.
template <bool NEXT>
struct MxOps {
    typedef i32x4 Frag;
    static constexpr int AR = 1, BR = 1;
    static constexpr int DMAS = 17, LATE = 0, PARTS = 2, PRE = 2, FILL = NEXT;

    unsigned char *smem;
    unsigned dwave;        // LDS address of this wave's 64 rows of a slot
    const unsigned char *tbase, *wbase, *sbase;  // uniform: token rows, weight rows, this wave's scale rows
    int64_t sstep;         // bytes between a step's scales and the next step's
    unsigned sdst;         // LDS address of this wave's scale half
    unsigned soff;         // 16 * lane
    unsigned row16;        // bytes of 16 rows
    unsigned off[2];       // lane offsets of instructions 0 and 1 of a slot; j: 16 rows past j - 2
    unsigned to[2], wo[2];
    int nk;
    int lane, lr, lh, arow, trow0;  // arow: first A row of this wave's tile 0; tile t at arow + 32 (t & 1) + astep (t / 2)
    int astep;
    unsigned sa[4], sb[4], sna[4], snb[4];

    __device__ __forceinline__ void begin() {
        const int l = fresh(lane);
        lr = l & 31;
        lh = l >> 5;
    }
    __device__ __forceinline__ void dma(int d, int j) {
        const int kt = min(j + NS, nk - 1), slot = (j + NS) % NS;
        if (d == 0) {
            dma16_sb(sbase + (int64_t)kt * sstep, soff, sdst + slot * SSLOT);
        } else if (d <= 8) {
            const unsigned o = row_off(to, d - 1);
            dma16_sb(tbase + (int64_t)kt * kMxChunkBytes, o, dwave + T_OFF + slot * SLOT + 1024 * (d - 1));
        } else {
            const unsigned o = row_off(wo, d - 9);
            dma16_sb(wbase + (int64_t)kt * kMxChunkBytes, o, dwave + W_OFF + slot * SLOT + 1024 * (d - 9));
        }
    }
    // lane offset of instruction j of a slot, whose instructions go out in order
    __device__ __forceinline__ unsigned row_off(unsigned (&o)[2], int j) {
        o[j & 1] = j < 2 ? (unsigned)fresh((int)off[j]) : o[j & 1] + row16;
        return o[j & 1];
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

// What a lane and a wave hold for the whole launch, and the item's bases.
template <bool DUAL>
struct Tile {
    const MxArgs &a;
    unsigned char *smem;
    int wave, lane, ww, wt;  // ww: weight half, wt: token half (= block bx + wt)
    int64_t N, rb;
    MxOps<DUAL> p;

    __device__ __forceinline__ Tile(const MxArgs &args, unsigned char *s) : a(args), smem(s) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        lane = threadIdx.x & 63;
        ww = wave & 1;
        wt = wave >> 1;
        N = a.N;
        rb = (int64_t)a.kc * kMxChunkBytes;
        p.smem = smem;
        p.nk = a.kc;
        p.lane = lane;
        p.trow0 = 128 * wt;
        p.arow = DUAL ? 64 * ww : 128 * ww;  // gate/up: tiles 0, 1 gate rows, 2, 3 the same up rows
        p.astep = DUAL ? 128 : 64;
        // instruction j moves rows 64 w + 8 j + lane / 8 of a slot, physical
        // chunk lane % 8; the rows' swizzle repeats with j's parity
        p.row16 = (unsigned)(16 * rb);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 8 * j + (lane >> 3);
            p.off[j] = (unsigned)(r * rb + 16 * ((lane & 7) ^ lds_swz(r)));
        }
        const unsigned lds0 = (unsigned)(uintptr_t)smem;
        p.dwave = lds0 + 64 * wave * kMxChunkBytes;
        p.sdst = lds0 + (wave < 2 ? WS_OFF : TS_OFF) + 1024 * (wave & 1);
        p.sstep = 8 * (wave < 2 ? N : a.Tp);
        p.soff = 16 * lane;
    }
    __device__ __forceinline__ void set(const TileItem &it) {
        const int64_t n0 = (int64_t)it.nt * (DUAL ? 128 : 256);
        // weight rows 64 w .. of the slot: gate rows for waves 0, 1, up rows for 2, 3
        int64_t wrow0 = n0 + (DUAL ? (64 * wave) & 127 : 64 * wave);
        wrow0 = wrow0 < N ? wrow0 : N - 64;  // a narrow last slice: idle rows read valid rows
        p.wbase = uniform((DUAL && wave >= 2 ? a.w1 : a.w0) + ((int64_t)it.e * N + wrow0) * rb);
        // an absent second block: its half reads the first block's rows
        const bool two = it.rows1 > 0;
        p.tbase = uniform(a.x + ((int64_t)it.bx * kBlockM + (two ? 64 * wave : (64 * wave) & 127)) * rb);
        // scales: waves 0, 1 move the weight rows' (128 rows each), waves 2,
        // 3 the two blocks' token rows'
        if (wave < 2) {
            int64_t r0 = DUAL ? n0 : n0 + 128 * wave;
            r0 = r0 < N ? r0 : N - 128;
            p.sbase = uniform((DUAL && wave == 1 ? a.w1s : a.w0s) + ((int64_t)it.e * a.kc * N + r0) * 8);
        } else {
            p.sbase = uniform(a.xs + ((int64_t)it.bx + (wave == 3 && two ? 1 : 0)) * kBlockM * 8);
        }
    }
    // valid rows and live token tiles of this wave
    __device__ __forceinline__ int rows(const TileItem &it) const { return wt ? it.rows1 : it.rows0; }
    __device__ __forceinline__ int tiles(const TileItem &it) const {
        return DUAL || (int64_t)it.nt * 256 + 128 * ww < N ? (rows(it) + 31) / 32 : 0;
    }

    // gate/up: hidden block t (32 features) of token lr of tile u: register
    // 4q + r holds feature 8q + 4lh + r.  Lanes 0-31 assemble and store block
    // 0, lanes 32-63 block 1.
    template <int NTT>
    __device__ __forceinline__ void hidden(const TileItem &it, f16x (&acc)[4][4]) const {
        const int ln = fresh(lane), lr = ln & 31, lh = ln >> 5;
        const int64_t n0 = (int64_t)it.nt * 128, row0 = (int64_t)(it.bx + wt) * kBlockM;
        const int64_t orb = (int64_t)((N + kMxChunk - 1) / kMxChunk) * kMxChunkBytes;
        const int64_t b = (n0 + 64 * ww) / 32 + lh;  // block that this lane stores
        const int myrows = rows(it);
#pragma unroll
        for (int u = 0; u < NTT; ++u) {
            unsigned cd[2][2], byte[2];  // quads 0, 1 and 2, 3 of each block: 16 bits each
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float v[16], m = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = silu(acc[t][u][i]) * acc[t + 2][u][i];
#pragma unroll
                for (int i = 0; i < 16; i += 2) m = mx_amax(m, v[i], v[i + 1]);
                byte[t] = mx_scale_byte(mx_amax32(m));
                mx_codes<16>(v, byte[t], cd[t]);
            }
            // lower lanes take block 0, upper ones block 1: after the swaps
            // cd[0] holds the lower lanes' half of it, cd[1] the upper ones'
            swap32(cd[0][0], cd[1][0]);
            swap32(cd[0][1], cd[1][1]);
            u4 o;
            o[0] = (cd[0][0] & 0xffffu) | (cd[1][0] << 16);
            o[1] = (cd[0][0] >> 16) | (cd[1][0] & 0xffff0000u);
            o[2] = (cd[0][1] & 0xffffu) | (cd[1][1] << 16);
            o[3] = (cd[0][1] >> 16) | (cd[1][1] & 0xffff0000u);
            const int row = 32 * u + lr;
            if (row < myrows) {
                unsigned char *ys = a.ys + ((b >> 3) * a.Tp + row0 + row) * 8;
                *(u4 *)(a.yc + (row0 + row) * orb + 16 * b) = o;
                ys[mx_pos((int)(b & 7))] = (unsigned char)(lh ? byte[1] : byte[0]);
                // the last slice zero-fills the rest of an odd last chunk
                // (this lane: 16 of its 64 bytes and one of its 4 scales)
                if (n0 + 128 == N && (N & 255)) {
                    *(u4 *)(a.yc + (row0 + row) * orb + 16 * (b + 4)) = u4{0, 0, 0, 0};
                    ys[mx_pos((int)((b + 4) & 7))] = 0;
                }
            }
        }
    }

    // down: out rows, 64 at a time staged through LDS for whole-line stores.
    // A wave stages into its own 8 KB pieces of the operands' slots 1, which
    // only its own DMAs fill (all landed, and no wave reads the ring after
    // the last barrier; the next item's first step goes to slots 0): 128
    // columns per row, 16-byte chunks XOR-swizzled by row.
    template <int NTT>
    __device__ __forceinline__ void out(const TileItem &it, f16x (&acc)[4][4]) const {
        const int ln = fresh(lane), lr = ln & 31, lh = ln >> 5;
        const int64_t row0 = (int64_t)(it.bx + wt) * kBlockM;
        const int myrows = rows(it);
        unsigned char *piece[2] = {smem + W_OFF + SLOT + wave * 8192, smem + T_OFF + SLOT + wave * 8192};
        const float *rwe = a.rw + table(a.go)[it.e] + it.off + kBlockM * wt;
        _Float16 *ybase = a.y + row0 * N + (int64_t)it.nt * 256 + 128 * ww;
        const int c = ln & 15;
#pragma unroll
        for (int u0 = 0; u0 < NTT; u0 += 2) {
            __builtin_amdgcn_sched_barrier(0);  // no accumulator is copied out early: registers
            float w[2] = {0.f, 0.f};
#pragma unroll
            for (int u = u0; u < u0 + 2 && u < NTT; ++u)
                if (32 * u + lr < myrows) w[u - u0] = rwe[32 * u + lr];
#pragma unroll
            for (int u = u0; u < u0 + 2 && u < NTT; ++u)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f16x &o = acc[t][u];
                        *(h4 *)(piece[u - u0] + lr * 256 + (((4 * t + q) ^ (lr & 15)) << 4) + 8 * lh) = to_h4(
                            o[4 * q + 0] * w[u - u0], o[4 * q + 1] * w[u - u0], o[4 * q + 2] * w[u - u0],
                            o[4 * q + 3] * w[u - u0]);
                    }
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's staging writes are done
#pragma unroll
            for (int u = u0; u < u0 + 2 && u < NTT; ++u) {
                h8 v[8];  // read together: one LDS round trip, not eight
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = 4 * j + (ln >> 4);
                    v[j] = *(const h8 *)(piece[u - u0] + r * 256 + ((c ^ (r & 15)) << 4));
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int row = 32 * u + 4 * j + (ln >> 4);
                    if (row < myrows) *(h8 *)(ybase + (int64_t)row * N + 8 * c) = v[j];
                }
            }
        }
    }

    template <int NTT, class F>
    __device__ __forceinline__ bool finish(const TileItem &it, f16x (&acc)[4][4], F &&fill) const {
        fill();
        if constexpr (DUAL)
            hidden<NTT>(it, acc);
        else
            out<NTT>(it, acc);
        return !DUAL && NTT == 4 && rows(it) == kBlockM;  // a whole block of out rows: 32 stores
    }
};

template <bool DUAL>
__global__ __launch_bounds__(256) void mx_tile_kernel(MxArgs a, int NT) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    Tile<DUAL> tile(a, smem);
    run_items(tile, a.gs, a.gpo, a.gidx, a.E, NT);
}

template <bool DUAL>
hipError_t launch(const MxArgs &a, int NT, hipStream_t s) {
    unsigned grid = 0;
    hipError_t e = cu_grid(grid);
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
