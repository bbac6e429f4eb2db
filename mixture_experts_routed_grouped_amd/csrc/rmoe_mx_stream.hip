// Weight-streaming grouped GEMM on MXFP4 tokens and weights, for blocks with
// few rows (decode-shaped batches): bound by reading the routed experts'
// weights, 4.25 bits each, from HBM once.
//
// As the fp16 streaming family, a workgroup takes one 128-row block x FT
// tiles of 32 output features, its KS waves split K into contiguous ranges
// and run without barriers, and everything travels by DMA into per-wave
// rings: 32 weight rows x 128 bytes (256 elements) per tile and chunk, the
// pass's token rows, and 256 bytes of scales per 32 rows (one dword per lane:
// global_load_lds_dword).  A row is a quarter as long as in fp16 (16 chunks at
// K = 4096), so a workgroup's start and end weigh more; what hides them is
// small workgroups, many per CU.  One wave per workgroup (KS = 1: no reduction
// either) with two ring slots, 34 KB of LDS for passes of up to 64 tokens,
// measured best on a decode batch (64 tokens, 8 experts, 4096 x 14336): its
// two stages take 124 us, 6.0 TB/s of weights; two waves 128, four 160, three
// ring slots 127.  KS = 2 and 4 serve calls with few workgroups, where one
// wave's K loop would be the whole time.
#include <atomic>
#include <type_traits>

#include "rmoe_internal.h"
#include "rmoe_mx.h"

namespace rmoe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u4 __attribute__((ext_vector_type(4)));

constexpr int TILE_B = 32 * 128;     // 32 rows of a chunk
constexpr int SCALE_B = 32 * 8;      // their scales
constexpr int TILE_ALL = TILE_B + SCALE_B;

// 256-byte DMA: lane i stores the dword at g to LDS byte lds + 4 i (s_nop: as
// in dma16)
__device__ __forceinline__ void dma4(const void *g, unsigned lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(g) : "memory", "m0");
}

template <bool DUAL, int KS, int TT>
struct Cfg {
    static constexpr int FT = DUAL ? 1 : 2;            // feature tiles per workgroup
    static constexpr int NM = 2;                       // weight tiles: gate and up, or two of down
    static constexpr int D = 2;                        // ring slots per wave
    static constexpr int SLOT = (NM + TT) * TILE_ALL;  // tiles, then their scales
    static constexpr int RING = KS * D * SLOT;
    static constexpr int RED = KS > 1 ? KS * NM * TT * 16 * 64 * 4 : 0;
    static constexpr int LDS_BYTES = RING > RED ? RING : RED;
    static_assert(LDS_BYTES <= 160 * 1024, "LDS");
};

// One pass: token rows p0 .. p0 + 32 TT - 1 of block bx (the first 8 TD of
// them are moved: LDS rows past them keep stale values, which only reach
// output columns that are not stored) against features n0 ...
template <bool DUAL, int KS, int TT, int TD>
__device__ __forceinline__ void stream_pass(const MxArgs &a, const BlockInfo &bi, int bx, int p0, int n0,
                                            unsigned char *smem, int wave, int lane) {
    using C = Cfg<DUAL, KS, TT>;
    constexpr int NM = C::NM, D = C::D;
    constexpr int DMA_PER_CHUNK = 4 * NM + TD + NM + TT;
    static_assert((D - 1) * DMA_PER_CHUNK < 64, "vmcnt range");
    const int64_t N = a.N, rb = (int64_t)a.kc * kMxChunkBytes;
    const int lr = lane & 31, lh = lane >> 5;
    const int c_begin = (a.kc * wave) / KS;
    const int n = (a.kc * (wave + 1)) / KS - c_begin;

    const unsigned char *wsrc[NM][4], *tsrc[TD], *wscl[NM], *tscl[TT];
    const int64_t row0 = (int64_t)bx * kBlockM + p0;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        const unsigned char *w = DUAL && m ? a.w1 : a.w0;
        const unsigned char *ws = DUAL && m ? a.w1s : a.w0s;
        const int64_t nf = n0 + (DUAL ? 0 : 32 * m);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 8 * j + (lane >> 3);
            const int c = (lane & 7) ^ lds_swz(r);
            wsrc[m][j] = w + ((int64_t)bi.e * N + nf + r) * rb + (int64_t)c_begin * kMxChunkBytes + 16 * c;
        }
        wscl[m] = ws + (((int64_t)bi.e * a.kc + c_begin) * N + nf) * 8 + 4 * lane;
    }
#pragma unroll
    for (int j = 0; j < TD; ++j) {
        const int r = 8 * j + (lane >> 3);
        const int c = (lane & 7) ^ lds_swz(r);
        tsrc[j] = a.x + (row0 + r) * rb + (int64_t)c_begin * kMxChunkBytes + 16 * c;
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) tscl[t] = a.xs + ((int64_t)c_begin * a.Tp + row0 + 32 * t) * 8 + 4 * lane;

    const unsigned wbase = (unsigned)(uintptr_t)smem + wave * D * C::SLOT;
    const unsigned char *wring = smem + wave * D * C::SLOT;
    auto dma_chunk = [&](int i, int slot) {
        const unsigned sb = wbase + slot * C::SLOT;
        const unsigned ss = sb + (NM + TT) * TILE_B;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
#pragma unroll
            for (int j = 0; j < 4; ++j) dma16_nt(wsrc[m][j] + (int64_t)i * kMxChunkBytes, sb + m * TILE_B + 1024 * j);
            dma4(wscl[m] + (int64_t)i * N * 8, ss + m * SCALE_B);
        }
#pragma unroll
        for (int j = 0; j < TD; ++j) dma16(tsrc[j] + (int64_t)i * kMxChunkBytes, sb + NM * TILE_B + 1024 * j);
#pragma unroll
        for (int t = 0; t < TT; ++t) dma4(tscl[t] + (int64_t)i * a.Tp * 8, ss + (NM + t) * SCALE_B);
    };

    f16x acc[NM][TT];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][t][i] = 0.f;

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
            const unsigned char *ss = slot + (NM + TT) * TILE_B;
            i32x4 af[NM][4], bf[TT][4];
            unsigned sa[NM], sb[TT];
#pragma unroll
            for (int m = 0; m < NM; ++m) sa[m] = *(const unsigned *)(ss + m * SCALE_B + 8 * lr + 4 * lh);
#pragma unroll
            for (int t = 0; t < TT; ++t) sb[t] = *(const unsigned *)(ss + (NM + t) * SCALE_B + 8 * lr + 4 * lh);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
#pragma unroll
                for (int m = 0; m < NM; ++m) af[m][s] = *(const i32x4 *)(slot + m * TILE_B + lds_off(lr, 2 * s + lh));
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    bf[t][s] = *(const i32x4 *)(slot + NM * TILE_B + lds_off(32 * t + lr, 2 * s + lh));
            }
            auto sub = [&](auto sc) {
                constexpr int S = decltype(sc)::value;
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        const i32x8 x = __builtin_shufflevector(af[m][S], af[m][S], 0, 1, 2, 3, -1, -1, -1, -1);
                        const i32x8 y = __builtin_shufflevector(bf[t][S], bf[t][S], 0, 1, 2, 3, -1, -1, -1, -1);
                        acc[m][t] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc[m][t], 4, 4, S, (int)sa[m],
                                                                                    S, (int)sb[t]);
                    }
            };
            sub(std::integral_constant<int, 0>{});
            sub(std::integral_constant<int, 1>{});
            sub(std::integral_constant<int, 2>{});
            sub(std::integral_constant<int, 3>{});
        }
    }
    wait_vm<0>();  // no DMA may land in the ring once it holds partial sums
    __syncthreads();

    // ---- fixed-order reduction of the KS partial sums
    float *red = reinterpret_cast<float *>(smem);  // [KS][NM][TT][16][64]
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
        if constexpr (KS == 1) return acc[m][t][r];
        float s = red[((m * TT + t) * 16 + r) * 64 + lane];
#pragma unroll
        for (int w = 1; w < KS; ++w) s += red[(((w * NM + m) * TT + t) * 16 + r) * 64 + lane];
        return s;
    };
    if constexpr (DUAL) {
        // token tile t belongs to wave t % KS, whose lane pair (lr, lr + 32)
        // holds one token's 32 features: one block of the hidden row.
        // Register 4q + r holds feature 8q + 4lh + r.
        const int64_t orb = (int64_t)((N + kMxChunk - 1) / kMxChunk) * kMxChunkBytes;
        const int b = n0 / 32;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            if (t % KS != wave) continue;
            float v[16], m = 0.f;
#pragma unroll
            for (int r = 0; r < 16; ++r) v[r] = silu(sum(0, t, r)) * sum(1, t, r);
#pragma unroll
            for (int r = 0; r < 16; r += 2) m = mx_amax(m, v[r], v[r + 1]);
            const unsigned byte = mx_scale_byte(mx_amax32(m));
            unsigned lo[2];  // quads 0, 1 and 2, 3: 16 bits each
            mx_codes<16>(v, byte, lo);
            unsigned hi[2] = {lo[0], lo[1]};  // the upper lanes' half
            swap32(lo[0], hi[0]);
            swap32(lo[1], hi[1]);
            const int tok = p0 + 32 * t + lr;
            if (lh == 0 && tok < bi.rows) {
                u4 o;
                o[0] = (lo[0] & 0xffffu) | (hi[0] << 16);
                o[1] = (lo[0] >> 16) | (hi[0] & 0xffff0000u);
                o[2] = (lo[1] & 0xffffu) | (hi[1] << 16);
                o[3] = (lo[1] >> 16) | (hi[1] & 0xffff0000u);
                const int64_t row = (int64_t)bx * kBlockM + tok;
                *(u4 *)(a.yc + row * orb + 16 * b) = o;
                unsigned char *ys = a.ys + ((int64_t)(b >> 3) * a.Tp + row) * 8;
                ys[mx_pos(b & 7)] = (unsigned char)byte;
                if (n0 + 32 == N && (N & 255)) {  // zero-fill the rest of an odd last chunk
#pragma unroll
                    for (int j = 1; j <= 4; ++j) {
                        *(u4 *)(a.yc + row * orb + 16 * (b + j)) = u4{0, 0, 0, 0};
                        ys[mx_pos((b + j) & 7)] = 0;
                    }
                }
            }
        }
    } else {
        // output quad q (4 features) of feature tile m and token tile t
        // belongs to wave q % KS
        const float *rwe = a.rw + a.go[bi.e] + bi.token_offset;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int tok = p0 + 32 * t + lr;
            if (tok >= bi.rows) continue;
            const float w = rwe[tok];
            const int64_t row = (int64_t)bx * kBlockM + tok;
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q % KS != wave) continue;
                    *(h4 *)(a.y + row * N + n0 + 32 * m + 8 * q + 4 * lh) =
                        to_h4(sum(m, t, 4 * q) * w, sum(m, t, 4 * q + 1) * w, sum(m, t, 4 * q + 2) * w,
                              sum(m, t, 4 * q + 3) * w);
                }
        }
    }
    __syncthreads();  // the next pass refills the ring that holds red[]
}

// grid: (N / (32 FT), num_blocks_m), 64 KS threads.  A block of up to 64 rows
// reads its expert's weights once, a larger one once per 64 rows.
template <bool DUAL, int KS>
__global__ __launch_bounds__(64 * KS) void mx_stream_kernel(MxArgs a) {
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
hipError_t launch_ks(const MxArgs &a, hipStream_t s) {
    using C = Cfg<DUAL, KS, 2>;  // the largest pass's LDS
    static std::atomic<uint64_t> lds_set{0};
    hipError_t e = lds_opt_in_once((const void *)mx_stream_kernel<DUAL, KS>, C::LDS_BYTES, lds_set);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(a.N / (32 * C::FT)), (unsigned)a.M);
    hipLaunchKernelGGL((mx_stream_kernel<DUAL, KS>), grid, dim3(64 * KS), C::LDS_BYTES, s, a);
    return hipGetLastError();
}

constexpr int64_t kWg1 = 512;  // from here on one wave each
// Waves per workgroup, by the workgroups that will hold rows (at most one
// block per pair or, with few rows, per expert).  Measured borders of 256,
// 512 and 1024 (one MI355X, both stages, one token): 1 expert (4096, 14336)
// 28, 27, 32 us; 2 of 8 experts 40, 38, 39; 6 of 64 (2048, 1408) 15.5, 16.3,
// 18.5; 64 tokens over 8 experts 124, 124, 126.
template <bool DUAL>
hipError_t launch(const MxArgs &a, int64_t pairs, hipStream_t s) {
    const int64_t wgs = a.N / (32 * Cfg<DUAL, 1, 2>::FT) * (pairs < a.E ? pairs : a.E);
    if (wgs >= kWg1) return launch_ks<DUAL, 1>(a, s);
    if (wgs >= kWg1 / 2) return launch_ks<DUAL, 2>(a, s);
    return launch_ks<DUAL, 4>(a, s);
}

}  // namespace

hipError_t launch_mx_stream_gate_up(const MxArgs &a, int64_t pairs, hipStream_t s) { return launch<true>(a, pairs, s); }
hipError_t launch_mx_stream_down(const MxArgs &a, int64_t pairs, hipStream_t s) { return launch<false>(a, pairs, s); }

}  // namespace rmoe
