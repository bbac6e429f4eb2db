// Weight-streaming grouped GEMM on 8-bit integer tokens and weights, for
// blocks with few rows (decode-shaped batches): bound by reading the routed
// experts' weights, one byte each, from HBM once.
//
// As the MXFP4 streaming family, a workgroup takes one 128-row block x 2
// tiles of 32 weight rows (gate and up of 32 features, or 64 features of the
// down product), its KS waves split K into contiguous ranges and run without
// barriers, and operands travel by DMA into per-wave rings: 32 weight rows x
// 128 bytes per tile and chunk, and the pass's token rows.  The partial sums
// are integers, so their order does not matter; scales enter at the end.
//
// 64 tokens, 2 of 8 experts, 4096 x 14336: gate/up 160 us for 940 MB of
// weights, down 76 us for 470 (5.9 and 6.2 TB/s; a contiguous read-only sweep
// reaches 7.07).  One wave per workgroup with two ring slots where that gives
// enough workgroups: the more independent sweeps, the fuller the channels.
#include <atomic>

#include "rmoe_i8.h"
#include "rmoe_internal.h"

namespace rmoe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int BK = 128;          // K per chunk
constexpr int TILE_B = 32 * BK;  // 32 rows of a chunk

template <bool DUAL, int KS, int TT>
struct Cfg {
    static constexpr int FT = DUAL ? 1 : 2;  // feature tiles per workgroup
    static constexpr int NM = 2;             // weight tiles: gate and up, or two of down
    static constexpr int D = 2;              // ring slots per wave
    static constexpr int SLOT = (NM + TT) * TILE_B;
    static constexpr int RING = KS * D * SLOT;
    static constexpr int RED = KS > 1 ? KS * NM * TT * 16 * 64 * 4 : 0;
    static constexpr int LDS_BYTES = RING > RED ? RING : RED;
    static_assert(LDS_BYTES <= 160 * 1024, "LDS");
};

// One pass: token rows p0 .. p0 + 32 TT - 1 of block bx (the first 8 TD of
// them are moved: LDS rows past them keep stale values, which only reach
// output columns that are not stored) against features n0 ...
template <bool DUAL, int KS, int TT, int TD>
__device__ __forceinline__ void stream_pass(const I8Args &a, const BlockInfo &bi, int bx, int p0, int n0,
                                            unsigned char *smem, int wave, int lane) {
    using C = Cfg<DUAL, KS, TT>;
    constexpr int NM = C::NM, D = C::D;
    constexpr int DMA_PER_CHUNK = 4 * NM + TD;
    static_assert((D - 1) * DMA_PER_CHUNK < 64, "vmcnt range");
    const int64_t N = a.N, K = a.K;
    const int lr = lane & 31, lh = lane >> 5;
    const int kc = (int)(K / BK);
    const int c_begin = (int)((int64_t)kc * wave / KS);
    const int n = (int)((int64_t)kc * (wave + 1) / KS) - c_begin;

    const unsigned char *wsrc[NM][4], *tsrc[TD];
    const int64_t row0 = (int64_t)bx * kBlockM + p0;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        const unsigned char *w = DUAL && m ? a.w1 : a.w0;
        const int64_t nf = n0 + (DUAL ? 0 : 32 * m);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 8 * j + (lane >> 3);
            const int c = (lane & 7) ^ lds_swz(r);
            wsrc[m][j] = w + ((int64_t)bi.e * N + nf + r) * K + (int64_t)c_begin * BK + 16 * c;
        }
    }
#pragma unroll
    for (int j = 0; j < TD; ++j) {
        const int r = 8 * j + (lane >> 3);
        const int c = (lane & 7) ^ lds_swz(r);
        tsrc[j] = a.x + (row0 + r) * K + (int64_t)c_begin * BK + 16 * c;
    }

    const unsigned wbase = (unsigned)(uintptr_t)smem + wave * D * C::SLOT;
    const unsigned char *wring = smem + wave * D * C::SLOT;
    // Rows a multiple of 4 KB apart share their memory channels: workgroups
    // that sweep K in step would all read through a few of them at a time, so
    // neighbours start at different chunks (the sums are exact in any order).
    // 8 experts of 14336 rows of K = 4096, 16 tokens each: 105 -> 83 us; 8192
    // rows of 8192: 120 -> 83; at other K (1024 to 14336) within 4% either way,
    // so those sweep as they are.
    const int first = n > 0 && K % 4096 == 0 ? (int)((blockIdx.x * 5u) % (unsigned)n) : 0;
    auto dma_chunk = [&](int i, int slot) {
        i = i + first < n ? i + first : i + first - n;
        const unsigned sb = wbase + slot * C::SLOT;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) dma16_nt(wsrc[m][j] + (int64_t)i * BK, sb + m * TILE_B + 1024 * j);
#pragma unroll
        for (int j = 0; j < TD; ++j) dma16(tsrc[j] + (int64_t)i * BK, sb + NM * TILE_B + 1024 * j);
    };

    i32x16 acc[NM][TT];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][t][i] = 0;

    if (n > 0) {
#pragma unroll
        for (int j = 0; j < D - 1; ++j) dma_chunk(min(j, n - 1), j);
        for (int i = 0; i < n; ++i) {
            // refill the slot of chunk i-1, whose reads are done (clamped:
            // repeats land in slots no later chunk reads), then wait for
            // chunk i, the oldest in flight
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
            dma_chunk(min(i + D - 1, n - 1), (i + D - 1) % D);
            wait_vm<(D - 1) * DMA_PER_CHUNK>();
            const unsigned char *slot = wring + (i % D) * C::SLOT;
            i32x4 af[NM][4], bf[TT][4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
#pragma unroll
                for (int m = 0; m < NM; ++m) af[m][s] = *(const i32x4 *)(slot + m * TILE_B + lds_off(lr, 2 * s + lh));
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    bf[t][s] = *(const i32x4 *)(slot + NM * TILE_B + lds_off(32 * t + lr, 2 * s + lh));
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int m = 0; m < NM; ++m)
                        acc[m][t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(af[m][s], bf[t][s], acc[m][t], 0, 0, 0);
        }
    }
    wait_vm<0>();  // no DMA may land in the ring once it holds partial sums
    __syncthreads();

    int *red = reinterpret_cast<int *>(smem);  // [KS][NM][TT][16][64]
    if constexpr (KS > 1) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) red[(((wave * NM + m) * TT + t) * 16 + r) * 64 + lane] = acc[m][t][r];
        __syncthreads();
    }
    auto sum = [&](int m, int t, int r) {
        if constexpr (KS == 1) return (float)acc[m][t][r];
        int s = red[((m * TT + t) * 16 + r) * 64 + lane];
#pragma unroll
        for (int w = 1; w < KS; ++w) s += red[(((w * NM + m) * TT + t) * 16 + r) * 64 + lane];
        return (float)s;
    };
    // quad q (4 features) of feature tile m and token tile t belongs to wave
    // q % KS; register 4q + r holds feature 8q + 4lh + r
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int tok = p0 + 32 * t + lr;
        if (tok >= bi.rows) continue;
        const int64_t row = (int64_t)bx * kBlockM + tok;
        const float xs = a.xs[row];
        if constexpr (DUAL) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (q % KS != wave) continue;
                const int64_t f = n0 + 8 * q + 4 * lh;
                const f4 gs = *(const f4 *)(a.w0s + (int64_t)bi.e * N + f), us = *(const f4 *)(a.w1s + (int64_t)bi.e * N + f);
                f4 h;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    h[r] = silu(sum(0, t, 4 * q + r) * (xs * gs[r])) * (sum(1, t, 4 * q + r) * (xs * us[r]));
                *(f4 *)(a.rows + row * N + f) = h;
            }
        } else {
            const float w = xs * a.rw[a.go[bi.e] + bi.token_offset + tok];
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q % KS != wave) continue;
                    const int64_t f = n0 + 32 * m + 8 * q + 4 * lh;
                    const f4 d = *(const f4 *)(a.w0s + (int64_t)bi.e * N + f);
                    *(h4 *)(a.y + row * N + f) =
                        to_h4(sum(m, t, 4 * q) * (w * d[0]), sum(m, t, 4 * q + 1) * (w * d[1]),
                              sum(m, t, 4 * q + 2) * (w * d[2]), sum(m, t, 4 * q + 3) * (w * d[3]));
                }
        }
    }
    __syncthreads();  // the next pass refills the ring that holds red[]
}

// grid: (N / (32 FT), num_blocks_m), 64 KS threads.  A block of up to 64 rows
// reads its expert's weights once, a larger one once per 64 rows.
template <bool DUAL, int KS>
__global__ __launch_bounds__(64 * KS) void i8_stream_kernel(I8Args a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int bx = blockIdx.y;
    const BlockInfo bi = block_info(a.gs, a.gpo, a.gidx, a.E, bx);
    if (bi.rows == 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int n0 = blockIdx.x * 32 * Cfg<DUAL, KS, 1>::FT;
    for (int p0 = 0; p0 < bi.rows; p0 += 64) {
        const int td = (bi.rows - p0 + 7) / 8;  // token rows of the pass, in 8s
        if (td <= 1) stream_pass<DUAL, KS, 1, 1>(a, bi, bx, p0, n0, smem, wave, lane);
        else if (td == 2) stream_pass<DUAL, KS, 1, 2>(a, bi, bx, p0, n0, smem, wave, lane);
        else if (td <= 4) stream_pass<DUAL, KS, 1, 4>(a, bi, bx, p0, n0, smem, wave, lane);
        else if (td <= 6) stream_pass<DUAL, KS, 2, 6>(a, bi, bx, p0, n0, smem, wave, lane);
        else stream_pass<DUAL, KS, 2, 8>(a, bi, bx, p0, n0, smem, wave, lane);
    }
}

template <bool DUAL, int KS>
hipError_t launch_ks(const I8Args &a, hipStream_t s) {
    using C = Cfg<DUAL, KS, 2>;  // the largest pass's LDS
    static std::atomic<uint64_t> lds_set{0};
    hipError_t e = lds_opt_in_once((const void *)i8_stream_kernel<DUAL, KS>, C::LDS_BYTES, lds_set);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(a.N / (32 * C::FT)), (unsigned)a.M);
    hipLaunchKernelGGL((i8_stream_kernel<DUAL, KS>), grid, dim3(64 * KS), C::LDS_BYTES, s, a);
    return hipGetLastError();
}

constexpr int64_t kWg1 = 512;  // from here on one wave each
// Waves per workgroup, by the workgroups that will hold rows (at most one
// block per pair or, with few rows, per expert).
template <bool DUAL>
hipError_t launch(const I8Args &a, int64_t pairs, hipStream_t s) {
    const int64_t wgs = a.N / (32 * Cfg<DUAL, 1, 2>::FT) * (pairs < a.E ? pairs : a.E);
    if (wgs >= kWg1) return launch_ks<DUAL, 1>(a, s);
    if (wgs >= kWg1 / 2) return launch_ks<DUAL, 2>(a, s);
    return launch_ks<DUAL, 4>(a, s);
}

}  // namespace

hipError_t launch_i8_stream_gate_up(const I8Args &a, int64_t pairs, hipStream_t s) { return launch<true>(a, pairs, s); }
hipError_t launch_i8_stream_down(const I8Args &a, int64_t pairs, hipStream_t s) { return launch<false>(a, pairs, s); }

}  // namespace rmoe
