// Tiled grouped GEMM on 8-bit integer tokens and weights, for blocks with
// many rows.
//
// v_mfma_i32_32x32x32_i8 takes 16 bytes per lane and operand, as
// v_mfma_f32_32x32x16_f16 does, and the same time: a K step of 128 bytes per
// row holds 128 elements instead of 64, so the 256 x 256 tile, its DMAs and
// its LDS traffic are those of the fp16 tiled kernels at twice the products.
// The sums are exact 32-bit integers (K is limited so that they fit); the
// token's and the channel's scale enter in the epilogue.
//
// A hidden row's scale needs the whole row, whose slices are spread over
// workgroups: the gate/up epilogue writes the rows in fp32 and a second
// launch turns them into codes.
//
// Bound by the matrix cores and their power limit, then by the epilogue, which
// one wave per SIMD cannot overlap with them.  16384 tokens, 8 of 128 experts,
// 7168 x 2048: gate/up 3360 us, down 2190 (2.3 and 1.75 POP/s; a large library
// product 2.1).  8192 tokens, 6 of 64 experts, 2048 x 1408 (11 K steps in
// down): 380 and 220 us (counters: 822 MB read and 287 written, 422 and 217; the
// matrix cores busy 41 and 33% of the time).  The kernels fill all 512 registers
// and spill a few outside the K loop's body (gate/up 5 per lane, down 27; the
// fp16 tiles 1, the MXFP4 ones 4).  Measured and not kept: two slots for the weights as
// well (slower), a next group of 32 tokens computed while the last one's rows
// are stored (no gain), non-temporal stores (no gain).
#include <atomic>

#include "rmoe_i8.h"
#include "rmoe_kloop.h"

namespace rmoe {
namespace {

constexpr int BK = 128;             // K per step
constexpr int SLOT = 256 * BK;      // 32 KB: a K step of 256 rows
constexpr int NAS = 3, NBS = 2;     // A (weight) and B (token) slots: A runs two steps ahead, B one
constexpr int B_OFF = NAS * SLOT;
constexpr int LDS_BYTES = (NAS + NBS) * SLOT;
static_assert(LDS_BYTES <= 160 * 1024, "LDS");
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct I8Ops {
    typedef i32x4 Frag;
    static constexpr int AR = 1, BR = 1;
    static constexpr int DMAS = 16, LATE = 8, PARTS = 4, PRE = 3, FILL = 0;

    unsigned char *smem;
    unsigned dwave;                      // LDS address of this wave's 64 rows of a slot
    const unsigned char *tbase, *wbase;  // uniform: token rows, weight rows
    unsigned row16;                      // bytes of 16 rows
    unsigned off[2];                     // lane offsets of instructions 0 and 1 of a slot; j: 16 rows past j - 2
    unsigned to[2], wo[2];
    int nk;
    int lane, lr, lh, arow, trow0;  // arow: first A row of this wave's tile 0; tile t at arow + 32 (t & 1) + astep (t / 2)
    int astep;

    __device__ __forceinline__ void begin() {
        const int l = fresh(lane);
        lr = l & 31;
        lh = l >> 5;
    }
    __device__ __forceinline__ void dma(int d, int j) {
        if (d < 8) {
            const unsigned o = row_off(to, d);
            dma16_sb(tbase + (int64_t)min(j + NBS, nk - 1) * BK, o, dwave + B_OFF + ((j + NBS) % NBS) * SLOT + 1024 * d);
        } else {
            const unsigned o = row_off(wo, d - 8);
            dma16_sb(wbase + (int64_t)min(j + NAS, nk - 1) * BK, o, dwave + ((j + NAS) % NAS) * SLOT + 1024 * (d - 8));
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
            a[i] = *(const Frag *)(smem + (k % NAS) * SLOT + lds_off(row_a(i) + lr, ch));
        else
            b[i - 4] = *(const Frag *)(smem + B_OFF + (k % NBS) * SLOT + lds_off(trow0 + 32 * (i - 4) + lr, ch));
    }
    __device__ __forceinline__ void step(int) {}
    __device__ __forceinline__ void next() {}
    // the accumulators are integers held in the K loop's fp32 registers
    template <int S>
    __device__ __forceinline__ void mma(const Frag &x, const Frag &y, f16x &c, int, int) {
        c = __builtin_bit_cast(f16x, __builtin_amdgcn_mfma_i32_32x32x32_i8(x, y, __builtin_bit_cast(i32x16, c), 0, 0, 0));
    }
    __device__ __forceinline__ void publish(int) {}
};

// (by value: the cast of a vector's element takes its first one)
__device__ __forceinline__ int bits_of(float c) { return __builtin_bit_cast(int, c); }
__device__ __forceinline__ float sum_of(float c) { return (float)bits_of(c); }

// The down product whole, or a part of its K per item: out rows' sums, which
// another launch adds up (exact integers: the same results).
enum Stage { GATE_UP, DOWN, DOWN_PART };

// What a lane and a wave hold for the whole launch, and the item's bases.
template <int STAGE>
struct Tile {
    static constexpr bool DUAL = STAGE == GATE_UP, PART = STAGE == DOWN_PART;
    const I8Args &a;
    unsigned char *smem;
    int wave, lane, ww, wt;  // ww: weight half, wt: token half (= block bx + wt)
    int64_t N, K;
    int cols;  // parts: column tiles, an item's slice being part * cols + column tile
    I8Ops p;
    // The scales of the item whose products run: of the wave's 128 weight rows
    // (gate/up: 64 gate, 64 up rows) and of its 128 tokens (down: times the
    // routed weight), two of each per lane.  Requested with the item's first
    // step, under the epilogue before it: a request at the epilogue's start
    // would hold up the next item's first step by its own round trip.
    float fs[2], ts[2];

    __device__ __forceinline__ Tile(const I8Args &args, unsigned char *s) : a(args), smem(s) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        lane = threadIdx.x & 63;
        ww = wave & 1;
        wt = wave >> 1;
        N = a.N;
        K = a.K;
        cols = PART ? (int)((N + 255) / 256) : 0;
        p.smem = smem;
        p.nk = (int)(K / BK);
        p.lane = lane;
        p.trow0 = 128 * wt;
        p.arow = DUAL ? 64 * ww : 128 * ww;  // gate/up: tiles 0, 1 gate rows, 2, 3 the same up rows
        p.astep = DUAL ? 128 : 64;
        // instruction j moves rows 64 w + 8 j + lane / 8 of a slot, physical
        // chunk lane % 8; the rows' swizzle repeats with j's parity
        p.row16 = (unsigned)(16 * K);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 8 * j + (lane >> 3);
            p.off[j] = (unsigned)(r * K + 16 * ((lane & 7) ^ lds_swz(r)));
        }
        p.dwave = (unsigned)(uintptr_t)smem + 64 * wave * BK;
    }
    __device__ __forceinline__ int part(const TileItem &it) const { return PART ? it.nt / cols : 0; }
    __device__ __forceinline__ int64_t first(const TileItem &it) const {  // its first column
        return (int64_t)(PART ? it.nt % cols : it.nt) * (DUAL ? 128 : 256);
    }
    __device__ __forceinline__ void set(const TileItem &it) {
        const int64_t n0 = first(it);
        // weight rows 64 w .. of the slot: gate rows for waves 0, 1, up rows for 2, 3
        int64_t wrow0 = n0 + (DUAL ? (64 * wave) & 127 : 64 * wave);
        wrow0 = wrow0 < N ? wrow0 : N - 64;  // a narrow last slice: idle rows read valid rows
        p.wbase = uniform((DUAL && wave >= 2 ? a.w1 : a.w0) + ((int64_t)it.e * N + wrow0) * K);
        // an absent second block: its half reads the first block's rows
        p.tbase = uniform(a.x + ((int64_t)it.bx * kBlockM + (it.rows1 > 0 ? 64 * wave : (64 * wave) & 127)) * K);
        if constexpr (PART) {
            const int nk = (int)(K / BK), k0 = nk * part(it) / a.splits;
            p.nk = nk * (part(it) + 1) / a.splits - k0;
            p.wbase += k0 * BK;
            p.tbase += k0 * BK;
            return;
        }
        // an idle wave (a narrow last slice, an absent second block) reads valid ones
        const int64_t c0 = n0 + (DUAL ? 64 : 128) * ww, f = (int64_t)it.e * N + (c0 < N ? c0 : N - 128) + lane;
        const int64_t row = ((int64_t)it.bx + (rows(it) > 0 ? wt : 0)) * kBlockM + lane;
        fs[0] = a.w0s[f];
        fs[1] = DUAL ? a.w1s[f] : a.w0s[f + 64];
        ts[0] = a.xs[row];
        ts[1] = a.xs[row + 64];
        if constexpr (!DUAL) {
            const float *rwe = a.rw + table(a.go)[it.e] + it.off + kBlockM * wt;
            const int n = rows(it);
            ts[0] *= lane < n ? rwe[lane] : 0.f;
            ts[1] *= lane + 64 < n ? rwe[lane + 64] : 0.f;
        }
    }
    // valid rows and live token tiles of this wave
    __device__ __forceinline__ int rows(const TileItem &it) const { return wt ? it.rows1 : it.rows0; }
    __device__ __forceinline__ int tiles(const TileItem &it) const {
        return DUAL || first(it) + 128 * ww < N ? (rows(it) + 31) / 32 : 0;
    }
    // Two pieces of 8 KB of this wave's LDS: in A's slot 2 and B's slot 1,
    // which only its own DMAs fill (all landed after the K loop; no wave reads
    // the ring after the last barrier, and the next item's first step goes to
    // the other slots).  Rows are staged in the first; the second takes the
    // scales, 128 of weight rows and 128 of tokens.  A wave's LDS accesses
    // happen in their order, so rows may follow rows without waiting.
    __device__ __forceinline__ unsigned char *piece(int i) const {
        return smem + (i ? B_OFF + SLOT : 2 * SLOT) + wave * 8192;
    }
    __device__ __forceinline__ void keep_scales() const {
        float *sc = (float *)piece(1);
        sc[lane] = fs[0];
        sc[64 + lane] = fs[1];
        sc[128 + lane] = ts[0];
        sc[192 + lane] = ts[1];
    }

    // gate/up: hidden rows in fp32, 32 tokens of 64 features at a time (256
    // bytes per row, 16-byte chunks XOR-swizzled by row), whole lines out.
    // Register 4q + r of tile t holds feature 32 t + 8q + 4lh + r.
    template <int NTT, class F>
    __device__ __forceinline__ void hidden(const TileItem &it, f16x (&acc)[4][4], F &&fill) {
        const int ln = fresh(lane), lr = ln & 31, lh = ln >> 5, c = ln & 15;
        const int64_t n0 = (int64_t)it.nt * 128 + 64 * ww, row0 = (int64_t)(it.bx + wt) * kBlockM;
        const int myrows = rows(it);
        keep_scales();
        fill();
        const float *sc = (const float *)piece(1);
        unsigned char *st = piece(0);
        float *ybase = a.rows + row0 * N + n0 + 4 * c;
#pragma unroll
        for (int u = 0; u < NTT; ++u) {
            __builtin_amdgcn_sched_barrier(0);  // no accumulator is copied out early: registers
            const float xs = sc[128 + 32 * u + lr];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f4 gs = *(const f4 *)(sc + 32 * t + 8 * q + 4 * lh), us = *(const f4 *)(sc + 64 + 32 * t + 8 * q + 4 * lh);
                    f4 h;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float g = sum_of(acc[t][u][4 * q + r]) * (xs * gs[r]);
                        const float v = sum_of(acc[t + 2][u][4 * q + r]) * (xs * us[r]);
                        h[r] = silu(g) * v;
                    }
                    *(f4 *)(st + lr * 256 + (((8 * t + 2 * q + lh) ^ (lr & 15)) << 4)) = h;
                }
            f4 v[8];  // read together: one LDS round trip, not eight
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = 4 * j + (ln >> 4);
                v[j] = *(const f4 *)(st + r * 256 + ((c ^ (r & 15)) << 4));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int row = 32 * u + 4 * j + (ln >> 4);
                if (row < myrows) *(f4 *)(ybase + (int64_t)row * N) = v[j];
            }
        }
    }

    // down: out rows, 32 tokens of 128 columns at a time, staged as above.
    template <int NTT, class F>
    __device__ __forceinline__ void out(const TileItem &it, f16x (&acc)[4][4], F &&fill) {
        const int ln = fresh(lane), lr = ln & 31, lh = ln >> 5, c = ln & 15;
        const int64_t row0 = (int64_t)(it.bx + wt) * kBlockM, n0 = first(it) + 128 * ww;
        const int myrows = rows(it);
        keep_scales();
        fill();
        const float *sc = (const float *)piece(1);
        unsigned char *st = piece(0);
        _Float16 *ybase = a.y + row0 * N + n0 + 8 * c;
#pragma unroll
        for (int u = 0; u < NTT; ++u) {
            __builtin_amdgcn_sched_barrier(0);  // no accumulator is copied out early: registers
            const float w = sc[128 + 32 * u + lr];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f16x &o = acc[t][u];
                    const f4 d = *(const f4 *)(sc + 32 * t + 8 * q + 4 * lh);
                    *(h4 *)(st + lr * 256 + (((4 * t + q) ^ (lr & 15)) << 4) + 8 * lh) =
                        to_h4(sum_of(o[4 * q + 0]) * (w * d[0]), sum_of(o[4 * q + 1]) * (w * d[1]),
                              sum_of(o[4 * q + 2]) * (w * d[2]), sum_of(o[4 * q + 3]) * (w * d[3]));
                }
            h8 v[8];  // read together: one LDS round trip, not eight
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = 4 * j + (ln >> 4);
                v[j] = *(const h8 *)(st + r * 256 + ((c ^ (r & 15)) << 4));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int row = 32 * u + 4 * j + (ln >> 4);
                if (row < myrows) *(h8 *)(ybase + (int64_t)row * N) = v[j];
            }
        }
    }

    // a part's sums, 32 tokens of 64 columns at a time, staged as hidden rows
    template <int NTT, class F>
    __device__ __forceinline__ void sums(const TileItem &it, f16x (&acc)[4][4], F &&fill) {
        const int ln = fresh(lane), lr = ln & 31, lh = ln >> 5, c = ln & 15;
        const int64_t row0 = (int64_t)(it.bx + wt) * kBlockM, n0 = first(it) + 128 * ww;
        const int myrows = rows(it);
        int32_t *ybase = a.part + ((int64_t)part(it) * a.Tp + row0) * N + n0 + 4 * c;
        fill();
        unsigned char *st = piece(0);
#pragma unroll
        for (int u = 0; u < NTT; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                __builtin_amdgcn_sched_barrier(0);  // no accumulator is copied out early: registers
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        i32x4 v;
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = bits_of(acc[2 * h + t][u][4 * q + r]);
                        *(i32x4 *)(st + lr * 256 + (((8 * t + 2 * q + lh) ^ (lr & 15)) << 4)) = v;
                    }
                i32x4 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = 4 * j + (ln >> 4);
                    v[j] = *(const i32x4 *)(st + r * 256 + ((c ^ (r & 15)) << 4));
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int row = 32 * u + 4 * j + (ln >> 4);
                    if (row < myrows) *(i32x4 *)(ybase + (int64_t)row * N + 64 * h) = v[j];
                }
            }
    }

    template <int NTT, class F>
    __device__ __forceinline__ bool finish(const TileItem &it, f16x (&acc)[4][4], F &&fill) {
        if constexpr (DUAL)
            hidden<NTT>(it, acc, fill);
        else if constexpr (PART)
            sums<NTT>(it, acc, fill);
        else
            out<NTT>(it, acc, fill);
        return NTT == 4 && rows(it) == kBlockM;  // a whole block of rows: 32 stores and more
    }
};

template <int STAGE>
__global__ __launch_bounds__(256) void i8_tile_kernel(I8Args a, int NT) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    Tile<STAGE> tile(a, smem);
    run_items(tile, a.gs, a.gpo, a.gidx, a.E, NT);
}

// out from the parts' sums: 4 columns per thread, every gridDim.z'th row of
// block y.
__global__ __launch_bounds__(256) void i8_join_kernel(I8Args a) {
    const BlockInfo bi = block_info(a.gs, a.gpo, a.gidx, a.E, blockIdx.y);
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (bi.rows == 0 || c >= a.N) return;
    const f4 d = *(const f4 *)(a.w0s + (int64_t)bi.e * a.N + c);
    const float *rw = a.rw + a.go[bi.e] + bi.token_offset;
    for (int i = blockIdx.z; i < bi.rows; i += gridDim.z) {
        const int64_t row = (int64_t)blockIdx.y * kBlockM + i;
        const int32_t *p = a.part + row * a.N + c;
        i32x4 v = *(const i32x4 *)p;
#pragma unroll 4
        for (int s = 1; s < a.splits; ++s) v += *(const i32x4 *)(p + s * a.Tp * a.N);
        const float w = a.xs[row] * rw[i];
        *(h4 *)(a.y + row * a.N + c) = to_h4((float)v[0] * (w * d[0]), (float)v[1] * (w * d[1]),
                                             (float)v[2] * (w * d[2]), (float)v[3] * (w * d[3]));
    }
}

template <int STAGE>
hipError_t launch(const I8Args &a, int NT, hipStream_t s) {
    unsigned grid = 0;
    hipError_t e = cu_grid(grid);
    if (e != hipSuccess) return e;
    static std::atomic<uint64_t> lds_set{0};
    e = lds_opt_in_once((const void *)i8_tile_kernel<STAGE>, LDS_BYTES, lds_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(i8_tile_kernel<STAGE>, dim3(grid), dim3(256), LDS_BYTES, s, a, NT);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_tile_gate_up(const I8Args &a, hipStream_t s) { return launch<GATE_UP>(a, (int)(a.N / 128), s); }

// Few experts and rows make few tiles of out, each a long sum, at 1 us or more
// per step of 128 elements on its own CU.  K is cut into n parts where those
// find free CUs, have 8 steps each and fit the room for their sums, and gain
// more than the sums cost: a launch and the way out and back (8 us and 8 TB/s,
// mostly in the caches).  One expert, 4096 x 14336, 256 rows: forward 176 ->
// 112 us (n = 3); 1024 rows: 248 -> 213; one of 1024 x 4096, 1024 rows: 75 ->
// 65 (n = 4); 4 of those, 2048 rows each, which stay whole: 48 us for the down
// product, 55 in two parts.
hipError_t launch_i8_tile_down(const I8Args &args, int64_t pairs, hipStream_t s) {
    I8Args a = args;
    unsigned cus = 0;
    hipError_t e = cu_grid(cus);
    if (e != hipSuccess) return e;
    const int cols = (int)((a.N + 255) / 256);
    const int64_t live = pairs < a.E ? pairs : a.E, full = (pairs + 255) / 256;  // items per column: at least
    const int64_t items = (live > full ? live : full) * cols;
    int n = 1;
    double gain = 0.0;
    for (int64_t i = 2; a.part != nullptr && i * items <= cus && i * a.N <= a.K && i * 8 * BK <= a.K; ++i) {
        const double g = (double)(a.K / BK) * (1.0 - 1.0 / (double)i) - 8.0 - 1e-6 * (double)(i * pairs * a.N);
        if (g > gain) {
            gain = g;
            n = (int)i;
        }
    }
    if (n < 2) return launch<DOWN>(a, cols, s);
    a.splits = n;
    e = launch<DOWN_PART>(a, cols * n, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(i8_join_kernel, dim3((unsigned)((a.N + 1023) / 1024), (unsigned)a.M, 32), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace rmoe
