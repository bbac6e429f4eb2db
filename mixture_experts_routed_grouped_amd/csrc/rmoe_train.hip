// Backward pass of the routed expert FFN.  For a row r of expert e with
// routed weight w, token row x, kept pre-activations g, u and output gradient
// dy (all rows of the padded layout):
//
//     b  = dy . Wd[e]              (a sum over H)
//     dw = sum_i b silu(g) u       dh = w b
//     dg = dh u silu'(g)           du = dh silu(g)       hw = w silu(g) u
//     dx = dg . Wg[e] + du . Wu[e] (a sum over I, twice)
//     dWg[e] = sum_r dg^T x        dWu[e] = sum_r du^T x  dWd[e] = sum_r dy^T hw
//
// with silu'(g) = s + g s (1 - s), s = 1 / (1 + e^-g).  Everything between
// the fp16 inputs and outputs is fp32; dg, du and hw are rounded to fp16
// once, as operands of the products that follow (a split into two fp16
// operands would double those products).  That rounding and the results' own
// put dx and the weight gradients 2.9e-4 of their norm from 64 bits on normal
// inputs; the results' rounding alone, 2.1e-4.
//
// All three products run on the 256 x 256 tiles of rmoe_kloop.h with fp16
// MFMA (v_mfma_f32_32x32x16_f16), bound by the matrix cores and by operand
// delivery as the forward's tiles are (median dispatches on several cards; 64
// experts of 2048 x 1408, 49152 skewed rows: hidden stage 490-505 us, 0.56-0.58
// PFLOP/s, 36-42% of an item the epilogue's 690 MB; dx 561-577 us, 0.98-1.01;
// weight gradients 1072-1119 us, 0.76-0.79; 8 experts of 4096 x 14336, 8192
// rows: 0.92-0.96, 0.97-1.00 and 0.98 PFLOP/s at 1.5-1.7 GHz).  Their sums run
// along the row index of a row-major matrix (Wd over H, Wg and Wu over I; for
// the weight gradients both operands, over the tokens), so those operands lie
// k-major: an LDS slot holds 64 k rows of 256 columns, and ds_read_b64_tr_b16
// turns it into MFMA operands: a group of 16 lanes reads 4 k rows of 16 columns
// and each lane receives its column's 4 values.  DMA instructions move 8 k rows
// x 128 bytes, the pattern the L2 serves best.
//
// k-major slot: [4 column groups of 64][8 k groups of 8] blocks of 1 KB =
// 8 rows x 128 bytes; 16-byte chunk c of row r sits at c ^ swz_k(r), which
// spreads the 4 rows x 64 bytes that 32 lanes read over all 64 banks.
#include <atomic>

#include "rmoe_kloop.h"

namespace rmoe {
namespace {

constexpr int BK = 64;               // K per step
constexpr int SLOT = 256 * BK * 2;   // 32 KB
constexpr int NAS = 3, NBS = 2;      // A (weight) and B (token) slots: A runs two steps ahead, B one
constexpr int B_OFF = NAS * SLOT;
constexpr int LDS_BYTES = (NAS + NBS) * SLOT;
static_assert(LDS_BYTES <= 160 * 1024, "LDS");
typedef short s4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int swz_k(int r) { return ((r >> 1) & 1) * 4 | ((r >> 2) & 1) * 2; }

// Lane offset in a k-major slot of read half h of a 32-column tile of parity
// tp: rows 4h .. 4h+3 of k group lane / 32 (sub-step s: + 2048 s; column
// group nb: + 8192 nb).
__device__ __forceinline__ unsigned tr_off(int lane, int tp, int h) {
    const int i = lane & 15, n16 = (lane >> 4) & 1, lh = lane >> 5;
    const int r = 4 * h + (i >> 2), c = 4 * tp + 2 * n16 + ((i & 3) >> 1);
    return lh * 1024 + r * 128 + ((c ^ swz_k(r)) << 4) + (i & 1) * 8;
}
__device__ __forceinline__ h4 tr_read(const unsigned char *p) {
    return __builtin_bit_cast(
        h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4 *)p));
}

// Lane offsets of a slot's instructions, which go out in order: a row-major
// slot's rows 8 j .. 8 j + 7 (the swizzle repeats with j's parity), a k-major
// slot's k rows 8 j ...  One vector add per instruction (from a fresh first
// one, so that the sums are not kept per instruction: 16 registers through
// the epilogue, which spill); as scalar base additions they delayed the MFMAs
// (5% of the row products' time).
struct RowSteps {
    unsigned first[2], step, cur[2];  // bytes: of 16 rows
    __device__ __forceinline__ void init(int lane, int64_t K) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 8 * j + (lane >> 3);
            first[j] = (unsigned)((r * K + 8 * ((lane & 7) ^ lds_swz(r))) * 2);
        }
        step = (unsigned)(32 * K);
    }
    __device__ __forceinline__ unsigned at(int j) {
        cur[j & 1] = j < 2 ? (unsigned)fresh((int)first[j]) : cur[j & 1] + step;
        return cur[j & 1];
    }
};
struct ColSteps {
    unsigned first, step, cur;  // bytes: of 8 k rows
    __device__ __forceinline__ void init(int lane, int64_t N) {
        const int r = lane >> 3;
        first = (unsigned)((r * N + 8 * ((lane & 7) ^ swz_k(r))) * 2);
        step = (unsigned)(16 * N);
    }
    __device__ __forceinline__ unsigned at(int j) {
        cur = j == 0 ? (unsigned)fresh((int)first) : cur + step;
        return cur;
    }
};

struct OpsBase {
    typedef h8 Frag;
    static constexpr int DMAS = 16, LATE = 8, PARTS = 4, PRE = 3, FILL = 0;
    __device__ __forceinline__ void step(int) {}
    __device__ __forceinline__ void next() {}
    template <int S>
    __device__ __forceinline__ void mma(const Frag &x, const Frag &y, f16x &c, int, int) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, y, c, 0, 0, 0);
    }
};

// A: weight rows k-major [K, N]; B: token rows row-major [rows, K].  The sum
// may run over two pairs of matrices of K = 64 n1 each, one after the other.
struct RowOps : OpsBase {
    static constexpr int AR = 2, BR = 1;
    unsigned char *smem;
    unsigned dwave;
    const _Float16 *w[2], *t[2];  // uniform bases of the two pairs
    ColSteps ws;
    RowSteps ts;
    int64_t N;                    // elements per weight row
    int nk, n1;
    unsigned la[2][2];            // tr_off of tile parity, half
    int nb0;                      // first column group of this wave's A half
    int trow0, lane, lr, lh;

    __device__ __forceinline__ void begin() {
        const int l = fresh(lane);
        lr = l & 31;
        lh = l >> 5;
#pragma unroll
        for (int i = 0; i < 4; ++i) la[i >> 1][i & 1] = tr_off(l, i >> 1, i & 1);
    }
    __device__ __forceinline__ void dma(int d, int j) {
        if (d < 8) {
            const int k = min(j + NBS, nk - 1), two = k >= n1;
            const unsigned o = ts.at(d);
            dma16_sb((two ? t[1] : t[0]) + (int64_t)(two ? k - n1 : k) * BK, o,
                     dwave + B_OFF + ((j + NBS) % NBS) * SLOT + 1024 * d);
        } else {
            const int k = min(j + NAS, nk - 1), two = k >= n1;
            const unsigned o = ws.at(d - 8);
            dma16_sb((two ? w[1] : w[0]) + (int64_t)(two ? k - n1 : k) * BK * N, o,
                     dwave + ((j + NAS) % NAS) * SLOT + 1024 * (d - 8));
        }
    }
    __device__ __forceinline__ void read(int k, int s, int i, Frag *a, Frag *b) {
        if (i < 8) {
            const int tt = i >> 1, h = i & 1;
            const h4 v = tr_read(smem + (k % NAS) * SLOT + (nb0 + (tt >> 1)) * 8192 + 2048 * s + la[tt & 1][h]);
            if (h) a[tt].hi = v; else a[tt].lo = v;
        } else {
            b[i - 8] = *(const h8 *)(smem + B_OFF + (k % NBS) * SLOT + lds_off(trow0 + 32 * (i - 8) + lr, 2 * s + lh));
        }
    }
    __device__ __forceinline__ void publish(int) {}
};

// A (gate and up weight rows) and B (token rows) row-major, K = H.
struct DualOps : OpsBase {
    static constexpr int AR = 1, BR = 1;
    unsigned char *smem;
    unsigned dwave;
    const _Float16 *w, *t;        // uniform bases: this wave's 64 weight rows, its 64 token rows
    int64_t row8;                 // elements of 8 rows
    unsigned off[2];              // lane offset of instruction j from its rows 8 j: j even, odd
    const _Float16 *wcur, *tcur;  // first row of the instruction issued last (a group's go out in order)
    int nk, lane, lr, lh, arow, trow0;

    __device__ __forceinline__ void begin() {
        const int l = fresh(lane);
        lr = l & 31;
        lh = l >> 5;
    }
    __device__ __forceinline__ void dma(int d, int j) {
        if (d < 8) {
            tcur = d == 0 ? t + (int64_t)min(j + NBS, nk - 1) * BK : tcur + row8;
            dma16_sb(tcur, off[d & 1], dwave + B_OFF + ((j + NBS) % NBS) * SLOT + 1024 * d);
        } else {
            wcur = d == 8 ? w + (int64_t)min(j + NAS, nk - 1) * BK : wcur + row8;
            dma16_sb(wcur, off[d & 1], dwave + ((j + NAS) % NAS) * SLOT + 1024 * (d - 8));
        }
    }
    __device__ __forceinline__ void read(int k, int s, int i, Frag *a, Frag *b) {
        const int ch = 2 * s + lh;
        if (i < 4)  // tiles 0, 1 gate rows, 2, 3 the same up rows
            a[i] = *(const h8 *)(smem + (k % NAS) * SLOT + lds_off(arow + 32 * (i & 1) + 128 * (i >> 1) + lr, ch));
        else
            b[i - 4] = *(const h8 *)(smem + B_OFF + (k % NBS) * SLOT + lds_off(trow0 + 32 * (i - 4) + lr, ch));
    }
    __device__ __forceinline__ void publish(int) {}
};

// A and B k-major: the sum runs over token rows.
struct ColOps : OpsBase {
    static constexpr int AR = 2, BR = 2;
    unsigned char *smem;
    unsigned dwave;
    const _Float16 *a, *b;
    ColSteps as, bs;
    int64_t NA, NB;               // elements per row
    const _Float16 *acur, *bcur;  // first row of the instruction issued last (a group's go out in order)
    int nk, tail;                 // rows of the last step, 0: a whole one
    unsigned la[2][2];
    int lane, na0, nb0;           // first column groups of this wave's halves

    __device__ __forceinline__ void begin() {
        const int l = fresh(lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) la[i >> 1][i & 1] = tr_off(l, i >> 1, i & 1);
    }

    __device__ __forceinline__ void dma(int d, int j) {
        if (d < 8) {
            bcur = d == 0 ? b + (int64_t)min(j + NBS, nk - 1) * BK * NB : bcur + 8 * NB;
            dma16_sb(bcur, bs.first, dwave + B_OFF + ((j + NBS) % NBS) * SLOT + 1024 * d);
        } else {
            acur = d == 8 ? a + (int64_t)min(j + NAS, nk - 1) * BK * NA : acur + 8 * NA;
            dma16_sb(acur, as.first, dwave + ((j + NAS) % NAS) * SLOT + 1024 * (d - 8));
        }
    }
    __device__ __forceinline__ void read(int k, int s, int i, Frag *fa, Frag *fb) {
        const int tt = (i & 7) >> 1, h = i & 1;
        const unsigned char *slot = i < 8 ? smem + (k % NAS) * SLOT : smem + B_OFF + (k % NBS) * SLOT;
        const h4 v = tr_read(slot + ((i < 8 ? na0 : nb0) + (tt >> 1)) * 8192 + 2048 * s + la[tt & 1][h]);
        Frag *f = i < 8 ? fa : fb;
        if (h) f[tt].hi = v; else f[tt].lo = v;
    }
    // the rows past the group's last one hold padding (anything): zero them
    // in both operands before anyone reads the last step
    __device__ __forceinline__ void publish(int k) {
        if (k != nk - 1 || tail == 0) return;
        unsigned char *sa = smem + (k % NAS) * SLOT, *sb = smem + B_OFF + (k % NBS) * SLOT;
        const int i = threadIdx.x & 31;  // column group i / 8, chunk i % 8
        const h8 z = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int r = tail + (threadIdx.x >> 5); r < BK; r += 8) {
            const int o = (i >> 3) * 8192 + (r >> 3) * 1024 + (r & 7) * 128 + (i & 7) * 16;
            *(h8 *)(sa + o) = z;
            *(h8 *)(sb + o) = z;
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        bar();
    }
};

// Pieces of this wave's LDS for staging: 8 KB each in A's slot 2 and B's slot
// 1, which only its own DMAs fill (all landed after the K loop; no wave reads
// the ring after the last barrier, and the next item's first step goes to
// the other slots).
__device__ __forceinline__ unsigned char *piece(unsigned char *smem, int wave, int i) {
    return smem + (i ? B_OFF + SLOT : 2 * SLOT) + wave * 8192;
}

// The wave's block as fp16 rows of 128 columns: B index (token or output
// row) = row, A index = column.  Staged 64 rows at a time (256 bytes per row,
// 16-byte chunks XOR-swizzled), then stored as whole lines.
template <int NTT, bool NT>
__device__ __forceinline__ void store_block(const f16x (&acc)[4][4], unsigned char *smem, int wave, int lane, int rows,
                                            _Float16 *y, int64_t N) {
    const int lr = lane & 31, lh = lane >> 5, c = lane & 15;
#pragma unroll
    for (int u0 = 0; u0 < NTT; u0 += 2) {
#pragma unroll
        for (int u = u0; u < u0 + 2 && u < NTT; ++u)
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f16x &o = acc[t][u];
                    *(h4 *)(piece(smem, wave, u - u0) + lr * 256 + (((4 * t + q) ^ (lr & 15)) << 4) + 8 * lh) =
                        to_h4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's staging writes are done
#pragma unroll
        for (int u = u0; u < u0 + 2 && u < NTT; ++u) {
            h8 v[8];  // read together: one LDS round trip, not eight
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = 4 * j + (lane >> 4);
                v[j] = *(const h8 *)(piece(smem, wave, u - u0) + r * 256 + ((c ^ (r & 15)) << 4));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int row = 32 * u + 4 * j + (lane >> 4);
                if (row >= rows) continue;
                h8 *dst = (h8 *)(y + (int64_t)row * N + 8 * c);
                if constexpr (NT)
                    __builtin_nontemporal_store(v[j], dst);
                else
                    *dst = v[j];
            }
        }
    }
}

// Kept values beyond fp16's range (infinities) as its largest numbers: the
// forward used them in fp32, where silu and its derivative were finite.  NaN
// stays.
__device__ __forceinline__ h8 finite(h8 x) {
    const _Float16 m = (_Float16)65504.f;
    const h8 hi = {m, m, m, m, m, m, m, m}, lo = -hi;
    return __builtin_elementwise_minimum(__builtin_elementwise_maximum(x, lo), hi);
}

// Sum over the 16 lanes of a row (DPP rotations: every lane gets it).
template <int CTRL>
__device__ __forceinline__ float rot(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum16(float x) {
    x += rot<0x128>(x);  // row_ror:8
    x += rot<0x124>(x);
    x += rot<0x122>(x);
    x += rot<0x121>(x);
    return x;
}

// HID: the hidden stage (b = dy . Wd and everything that follows from it
// element by element); otherwise dx.  Holds what a lane and a wave keep for
// the whole launch, and the item's bases.
template <bool HID>
struct Rows {
    const TrainArgs &a;
    unsigned char *smem;
    int wave, lane, ww, wt;          // ww: column half, wt: token half
    int64_t K, N;                    // of one pair of matrices
    RowOps p;

    __device__ __forceinline__ Rows(const TrainArgs &args, unsigned char *s) : a(args), smem(s) {
        K = HID ? a.H : a.I;
        N = HID ? a.I : a.H;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        lane = threadIdx.x & 63;
        ww = wave & 1;
        wt = wave >> 1;
        p.smem = smem;
        p.dwave = (unsigned)(uintptr_t)smem + 8192 * wave;
        p.n1 = (int)(K / BK);
        p.nk = HID ? p.n1 : 2 * p.n1;
        p.N = N;
        p.ws.init(lane, N);
        p.ts.init(lane, K);
        p.nb0 = 2 * ww;
        p.trow0 = 128 * wt;
        p.lane = lane;
    }
    __device__ __forceinline__ void set(const TileItem &it) {
        int64_t col = (int64_t)it.nt * 256 + 64 * wave;
        col = col < N ? col : N - 64;  // a narrow last slice: idle columns read valid ones
        // an absent second block: its half reads the first block's rows
        const int row = it.rows1 > 0 ? 64 * wave : (64 * wave) & 127;
        const int64_t wofs = (int64_t)it.e * K * N + col, tofs = ((int64_t)it.bx * kBlockM + row) * K;
        p.w[0] = uniform((HID ? a.wd : a.wg) + wofs);
        p.t[0] = uniform((HID ? a.dy : a.dg) + tofs);
        p.w[1] = HID ? p.w[0] : uniform(a.wu + wofs);
        p.t[1] = HID ? p.t[0] : uniform(a.du + tofs);
    }
    __device__ __forceinline__ int rows(const TileItem &it) const { return wt ? it.rows1 : it.rows0; }
    __device__ __forceinline__ int tiles(const TileItem &it) const {
        return (int64_t)it.nt * 256 + 128 * ww < N ? (rows(it) + 31) / 32 : 0;
    }

    // Epilogue; fill() issues the next item's first step.  Returns whether at
    // least kNewer memory instructions followed it for sure.
    template <int NTT, class F>
    __device__ __forceinline__ bool finish(const TileItem &it, f16x (&acc)[4][4], F &&fill) const {
        const int lane = fresh(this->lane), lr = lane & 31, lh = lane >> 5;
        const int64_t row0 = (int64_t)(it.bx + wt) * kBlockM, col0 = (int64_t)it.nt * 256 + 128 * ww;
        const int nrows = rows(it);
        if constexpr (!HID) {
            fill();
            store_block<NTT, false>(acc, smem, wave, lane, nrows, a.dx + row0 * N + col0, N);
        } else {
            // 32 tokens at a time: b staged in fp32 (512 bytes per row over two
            // pieces: columns 0-63 and 64-127), read back 8 columns per lane,
            // 16 lanes and 4 rows per pass, next to 16-byte loads of g and u;
            // a pass requests its rows of the next 32 tokens once it is done
            // with its own
            const int64_t c0 = table(a.go)[it.e] + it.off + kBlockM * wt;  // compact index of the block's first row
            const int r4 = lane >> 4, cl = lane & 15;
            const int64_t np = N / 128;
            h8 g[8], p8[8];
            float w[8];
            auto request = [&](int u, int i) __attribute__((always_inline)) {
                const int row = 32 * u + 4 * i + r4;
                if (row < nrows) {
                    const int64_t o = (row0 + row) * N + col0 + 8 * cl;
                    g[i] = *(const h8 *)(a.g + o);
                    p8[i] = *(const h8 *)(a.u + o);
                    w[i] = a.rw[c0 + row];
                }
            };
            if constexpr (NTT > 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) request(0, i);
            }
#pragma unroll
            for (int u = 0; u < NTT; ++u) {
                // the last requests have landed before the next item's DMAs
                // go out: a later wait for one would wait for the DMAs too
                if (u + 1 == NTT) {
                    wait_vm<0>();
                    fill();
                }
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f16x &o = acc[t][u];
                        const int c = (8 * (t & 1) + 2 * q + lh) ^ (lr & 15);
                        *(f4 *)(piece(smem, wave, t >> 1) + lr * 256 + (c << 4)) =
                            f4{o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]};
                    }
                __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int sr = 4 * i + r4, row = 32 * u + sr;
                    const unsigned char *src = (cl >> 3 ? piece(smem, wave, 1) : piece(smem, wave, 0)) + sr * 256;
                    const int c = 2 * (cl & 7);
                    const f4 b0 = *(const f4 *)(src + ((c ^ (sr & 15)) << 4));
                    const f4 b1 = *(const f4 *)(src + (((c + 1) ^ (sr & 15)) << 4));
                    const h8 gc = finite(g[i]), uc = finite(p8[i]);
                    float dw = 0.f;
                    h8 dg, du, hw;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float b = j < 4 ? b0[j & 3] : b1[j & 3];
                        const float gf = (float)gc[j], uf = (float)uc[j], wf = w[i];
                        const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-gf * 1.4426950408889634f));
                        const float sl = gf * s, h = sl * uf, dh = wf * b;
                        dw += b * h;
                        dg[j] = (_Float16)(dh * uf * (s + sl * (1.0f - s)));
                        du[j] = (_Float16)(dh * sl);
                        hw[j] = (_Float16)(wf * h);
                    }
                    dw = sum16(dw);
                    if (row < nrows) {
                        const int64_t o = (row0 + row) * N + col0 + 8 * cl;
                        *(h8 *)(a.dg + o) = dg;
                        *(h8 *)(a.du + o) = du;
                        *(h8 *)(a.hw + o) = hw;
                        if (cl == 0) a.part[(c0 + row) * np + col0 / 128] = dw;
                    }
                    if (u + 1 < NTT) request(u + 1, i);
                }
            }
            if constexpr (NTT == 0) fill();
        }
        return NTT == 4 && nrows == kBlockM;  // 32 stores, or the last tile's 24 and more
    }
};

// drw[c] = the sum of c's partial sums, one per 128 columns: 16 lanes per c
// take every 16th in ascending order, then the lanes are added.
__device__ __forceinline__ void sum_drw(const TrainArgs &a) {
    const int64_t n = min((int64_t)a.go[a.E], a.pairs);
    const int np = (int)(a.I / 128), l = threadIdx.x & 15;
    for (int64_t c0 = (int64_t)blockIdx.x * 16; c0 < n; c0 += (int64_t)gridDim.x * 16) {
        const int64_t c = c0 + (threadIdx.x >> 4);
        float s = 0.f;
        if (c < n)
            for (int j = l; j < np; j += 16) s += a.part[c * np + j];
        s = sum16(s);
        if (c < n && l == 0) a.drw[c] = s;
    }
}

template <bool HID>
__global__ __launch_bounds__(256) void rows_kernel(TrainArgs a, int NT) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    Rows<HID> r(a, smem);
    run_items(r, a.gs, a.gpo, a.gidx, a.E, NT);
}

// The training forward's gate/up stage: 128 features per item, their gate
// rows in the first half of the A slot and the same up rows in the second, so
// that a lane holds gate and up of the same (token, feature).
struct Forward {
    const TrainArgs &a;
    unsigned char *smem;
    int wave, lane, ww, wt;  // ww: feature half, wt: token half
    DualOps p;

    __device__ __forceinline__ Forward(const TrainArgs &args, unsigned char *s) : a(args), smem(s) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        lane = threadIdx.x & 63;
        ww = wave & 1;
        wt = wave >> 1;
        p.smem = smem;
        p.dwave = (unsigned)(uintptr_t)smem + 8192 * wave;
        p.nk = (int)(a.H / BK);
        p.row8 = 8 * a.H;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            p.off[j] = (unsigned)(((lane >> 3) * a.H + 8 * ((lane & 7) ^ lds_swz(8 * j + (lane >> 3)))) * 2);
        p.arow = 64 * ww;
        p.trow0 = 128 * wt;
        p.lane = lane;
    }
    __device__ __forceinline__ void set(const TileItem &it) {
        const int64_t f0 = (int64_t)it.nt * 128 + ((64 * wave) & 127);
        const int row = it.rows1 > 0 ? 64 * wave : (64 * wave) & 127;  // as in Rows::set
        p.w = uniform((wave < 2 ? a.wg : a.wu) + ((int64_t)it.e * a.I + f0) * a.H);
        p.t = uniform(a.x + ((int64_t)it.bx * kBlockM + row) * a.H);
    }
    __device__ __forceinline__ int rows(const TileItem &it) const { return wt ? it.rows1 : it.rows0; }
    __device__ __forceinline__ int tiles(const TileItem &it) const { return (rows(it) + 31) / 32; }

    // gate, up and hidden rows, one after the other through the staging
    // pieces: 128 rows of 64 features, 64 rows per piece
    template <int NTT, class F>
    __device__ __forceinline__ bool finish(const TileItem &it, f16x (&acc)[4][4], F &&fill) const {
        fill();
        const int ln = fresh(lane), lr = ln & 31, lh = ln >> 5, c = ln & 7;
        const int nrows = rows(it);
        const int64_t o = ((int64_t)(it.bx + wt) * kBlockM) * a.I + (int64_t)it.nt * 128 + 64 * ww + 8 * c;
#pragma unroll
        for (int m = 0; m < 3; ++m) {
#pragma unroll
            for (int u = 0; u < NTT; ++u)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f16x &g = acc[t][u], &p2 = acc[t + 2][u];
                        float v[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            v[r] = m == 0 ? g[4 * q + r] : m == 1 ? p2[4 * q + r] : silu(g[4 * q + r]) * p2[4 * q + r];
                        *(h4 *)(piece(smem, wave, u >> 1) + (32 * (u & 1) + lr) * 128 + (((4 * t + q) ^ (lr & 7)) << 4) +
                                8 * lh) = to_h4(v[0], v[1], v[2], v[3]);
                    }
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's staging writes are done
            _Float16 *y = (m == 0 ? a.yg : m == 1 ? a.yu : a.yh) + o;
#pragma unroll
            for (int u = 0; u < NTT; ++u) {
                h8 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 8 * j + (ln >> 3);
                    v[j] = *(const h8 *)(piece(smem, wave, u >> 1) + (32 * (u & 1) + r) * 128 + ((c ^ (r & 7)) << 4));
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = 32 * u + 8 * j + (ln >> 3);
                    if (row < nrows) *(h8 *)(y + (int64_t)row * a.I) = v[j];
                }
            }
        }
        return NTT == 4 && nrows == kBlockM;  // 48 stores
    }
};

__global__ __launch_bounds__(256) void forward_kernel(TrainArgs a, int NT) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    Forward f(a, smem);
    run_items(f, a.gs, a.gpo, a.gidx, a.E, NT);
}

__global__ __launch_bounds__(256) void drw_kernel(TrainArgs a) { sum_drw(a); }

// Weight gradients: every 256 x 256 tile of the three matrices of every
// expert, its sum over the expert's rows; an expert without rows gets zeros.
// Persistent, one workgroup per CU; the tiles' order and who takes them:
// rmoe_sched.h.
struct Cols {
    const TrainArgs &a;
    unsigned char *smem;
    int wave, lane, ww, wt;  // ww: A half, wt: B half
    int nh, ni;              // tiles along H and I
    ColOps p;

    struct Tile {
        int e, m, n;           // expert, matrix, rows
        int64_t a0, b0, row0;  // first A column (contiguous in the output), first B column (its row), first row
    };

    __device__ __forceinline__ Cols(const TrainArgs &args, unsigned char *s) : a(args), smem(s) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        lane = threadIdx.x & 63;
        ww = wave & 1;
        wt = wave >> 1;
        nh = (int)((a.H + 255) / 256);
        ni = (int)((a.I + 255) / 256);
        p.smem = smem;
        p.dwave = (unsigned)(uintptr_t)smem + 8192 * wave;
        p.lane = lane;
        p.na0 = 2 * ww;
        p.nb0 = 2 * wt;
    }
    // matrix m: 0 dWg, 1 dWu (A = x, B = dg or du), 2 dWd (A = hw, B = dy)
    __device__ __forceinline__ int64_t cols_a(int m) const { return m < 2 ? a.H : a.I; }
    __device__ __forceinline__ int64_t cols_b(int m) const { return m < 2 ? a.I : a.H; }

    // Tile `item`; false where a group's tables break the contract (nothing
    // is read out of bounds, its gradients are left out).
    __device__ __forceinline__ bool at(int item, Tile &t) const {
        const GradTile g = grad_tile(item, nh, ni);
        t.e = g.e;
        t.m = g.m;
        t.a0 = (int64_t)g.a * 256;
        t.b0 = (int64_t)g.b * 256;
        t.n = table(a.gs)[t.e];
        t.row0 = table(a.gpo)[t.e];
        return t.n >= 0 && t.row0 >= 0 && t.row0 + ((int64_t)t.n + BK - 1) / BK * BK <= a.Tp;
    }
    __device__ __forceinline__ void set(const Tile &t) {
        const int64_t NA = cols_a(t.m), NB = cols_b(t.m);
        p.nk = (t.n + BK - 1) / BK;
        p.tail = t.n % BK;
        p.NA = NA;
        p.NB = NB;
        p.as.init(lane, NA);
        p.bs.init(lane, NB);
        int64_t ca = t.a0 + 64 * wave, cb = t.b0 + 64 * wave;
        ca = ca < NA ? ca : NA - 64;  // narrow last tiles: idle columns read valid ones
        cb = cb < NB ? cb : NB - 64;
        const _Float16 *g = t.m == 0 ? a.dg : t.m == 1 ? a.du : a.dy;
        p.a = uniform((t.m < 2 ? a.x : a.hw) + t.row0 * NA + ca);
        p.b = uniform(g + t.row0 * NB + cb);
    }
    __device__ __forceinline__ bool live(const Tile &t) const {
        return t.a0 + 128 * ww < cols_a(t.m) && t.b0 + 128 * wt < cols_b(t.m);
    }
    __device__ __forceinline__ _Float16 *out(const Tile &t) const {
        const int64_t NA = cols_a(t.m);
        return (t.m == 0 ? a.dwg : t.m == 1 ? a.dwu : a.dwd) + (int64_t)t.e * a.H * a.I + (t.b0 + 128 * wt) * NA +
               t.a0 + 128 * ww;
    }
    __device__ __forceinline__ void zeros(const Tile &t) const {
        if (!live(t)) return;
        const h8 z = {0, 0, 0, 0, 0, 0, 0, 0};
        _Float16 *y = out(t) + 8 * (lane & 15);
        for (int r = lane >> 4; r < 128; r += 4) __builtin_nontemporal_store(z, (h8 *)(y + r * cols_a(t.m)));
    }
};

// The tiles of one workgroup (GradWalk).
__device__ __forceinline__ void run_cols(const TrainArgs &a, unsigned char *smem, int total, int busy, int lead) {
    Cols c(a, smem);
    GradWalk walk(total, busy, lead, (int)blockIdx.x, (int)gridDim.x);
    // the next tile whose expert holds rows; the zeros of the others on the way
    auto advance = [&](Cols::Tile &t) __attribute__((always_inline)) {
        for (;;) {
            const int item = walk.next();
            if (item < 0) return false;
            if (!c.at(item, t)) continue;
            if (t.n > 0) return true;
            c.zeros(t);
        }
    };
    Cols::Tile t;
    if (!advance(t)) return;
    c.set(t);
    kfill(c.p);
    bool newer = false, more = true;
    while (more) {
        auto finish = [&](auto &acc, auto n) __attribute__((always_inline)) {
            const Cols::Tile now = t;
            more = advance(t);
            if (more) {
                c.set(t);
                kfill(c.p);
            }
            constexpr int NTT = decltype(n)::value;
            store_block<NTT, true>(acc, smem, c.wave, fresh(c.lane), kBlockM, c.out(now), c.cols_a(now.m));
            newer = NTT == 4;  // 32 stores
        };
        if (c.live(t))
            krun<4>(c.p, newer, finish);
        else
            krun<0>(c.p, newer, finish);
    }
}

__global__ __launch_bounds__(256) void cols_kernel(TrainArgs a, int total) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    run_cols(a, smem, total, 0, 0);
}

// The rest of a whole backward pass in one launch: drw, dx, and the weight
// gradients, which need nothing from dx.  dx has few, long items (8 experts
// of 4096 x 14336, 8192 rows: 592 of 448 K steps for 256 workgroups, 2.3
// rounds, 23% of its launch idle): the workgroups that have one item fewer
// than the others of their XCD start on the weight gradients meanwhile, as
// many tiles as an item's K steps are certainly worth: tiles of the expert
// with the most rows (by the average, the start ran late on 64 uneven experts,
// 2% of their pass).  6 steps stand for what surrounds a K loop.
// Against the two launches: 9 tokens of 256 x 128 27.6 -> 20.6 us, the 8192 rows
// above 5935 -> 5825 (6030 with the free workgroups waiting), 64 experts equal.
__global__ __launch_bounds__(256) void grads_kernel(TrainArgs a, int NT, int total) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    sum_drw(a);
    const int nl = gridDim.x / kXcd, items = tile_seq(table(a.gs), a.E, NT, blockIdx.x % kXcd, kXcd).n;  // of this XCD
    {
        Rows<false> r(a, smem);
        run_items(r, a.gs, a.gpo, a.gidx, a.E, NT);
    }
    __syncthreads();
    int most = 0;
    for (int e = 0; e < a.E; ++e) most = max(most, (int)table(a.gs)[e]);
    const int busy = items % nl;
    run_cols(a, smem, total, busy, busy ? ((int)(2 * a.I / BK) + 6) / (most / BK + 6) : 0);
}

template <bool HID>
hipError_t launch_rows(const TrainArgs &a, hipStream_t s) {
    unsigned grid = 0;
    hipError_t e = cu_grid(grid);
    if (e != hipSuccess) return e;
    static std::atomic<uint64_t> lds_set{0};
    e = lds_opt_in_once((const void *)rows_kernel<HID>, LDS_BYTES, lds_set);
    if (e != hipSuccess) return e;
    const int64_t N = HID ? a.I : a.H;
    hipLaunchKernelGGL(rows_kernel<HID>, dim3(grid), dim3(256), LDS_BYTES, s, a, (int)((N + 255) / 256));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gate_up_train(const TrainArgs &a, hipStream_t s) {
    unsigned grid = 0;
    hipError_t e = cu_grid(grid);
    if (e != hipSuccess) return e;
    static std::atomic<uint64_t> lds_set{0};
    e = lds_opt_in_once((const void *)forward_kernel, LDS_BYTES, lds_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(forward_kernel, dim3(grid), dim3(256), LDS_BYTES, s, a, (int)(a.I / 128));
    return hipGetLastError();
}

hipError_t launch_hidden_grad(const TrainArgs &a, hipStream_t s) { return launch_rows<true>(a, s); }

hipError_t launch_drw(const TrainArgs &a, hipStream_t s) {
    int64_t g = (a.pairs + 15) / 16;
    if (g > 256 * 16) g = 256 * 16;  // strides beyond
    if (g == 0) return hipSuccess;
    hipLaunchKernelGGL(drw_kernel, dim3((unsigned)g), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_gate_up_backward(const TrainArgs &a, hipStream_t s) { return launch_rows<false>(a, s); }

int64_t weight_grad_tiles(int64_t H, int64_t I, int32_t E) {
    return 3 * (int64_t)E * ((H + 255) / 256) * ((I + 255) / 256);
}

hipError_t launch_weight_grad(const TrainArgs &a, hipStream_t s) {
    static std::atomic<uint64_t> lds_set{0};
    hipError_t e = lds_opt_in_once((const void *)cols_kernel, LDS_BYTES, lds_set);
    if (e != hipSuccess) return e;
    unsigned grid = 0;
    e = cu_grid(grid);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(cols_kernel, dim3(grid), dim3(256), LDS_BYTES, s, a,
                       (int)weight_grad_tiles(a.H, a.I, a.E));
    return hipGetLastError();
}

hipError_t launch_grads(const TrainArgs &a, hipStream_t s) {
    static std::atomic<uint64_t> lds_set{0};
    hipError_t e = lds_opt_in_once((const void *)grads_kernel, LDS_BYTES, lds_set);
    if (e != hipSuccess) return e;
    unsigned grid = 0;
    e = cu_grid(grid);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(grads_kernel, dim3(grid), dim3(256), LDS_BYTES, s, a, (int)((a.H + 255) / 256),
                       (int)weight_grad_tiles(a.H, a.I, a.E));
    return hipGetLastError();
}

}  // namespace rmoe
