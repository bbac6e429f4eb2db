// Router: logits = x W^T, softmax over the experts, top-k ids and scores
// ("MetaX-TileLang工具链", section 2.4: the reference router is a linear gate,
// a softmax, a top-k; no renormalisation of the k scores is stated, so the
// scores are the softmax probabilities).
//
// One workgroup = TOK tokens (64 or 32) x every expert (E padded to a
// multiple of 32, at most 256), 4 computing waves and one that only requests
// tokens.  Tokens and gate rows travel HBM/L2 -> LDS by DMA in K-chunks of 64
// (8 rows x 128 bytes per instruction) through two rings of 4 stages (one
// barrier per chunk): the fifth wave's requests of x never wait behind the
// others' gate rows, which arrive sooner.  v_mfma_f32_32x32x16_f16 with gate
// rows as A and a 32-token tile as B, fp32 logits.  TOK = 64: the 4 waves are
// 2 token halves x 2 interleaved sets of 32-expert tiles; TOK = 32: one token
// tile, 4 interleaved sets of expert tiles -- or, with fewer than four
// expert tiles (E <= 64), the waves also split each chunk's four K-steps
// (E <= 32: one K-step per wave; E <= 64: two), so that every wave has work
// and a chunk costs one or two dependent MFMAs instead of four (64 tokens,
// E = 8, H = 4096: two workgroups of 64 chunks); their partial logits are
// added in a fixed order.  TOK = 32 gives twice the workgroups, i.e. more
// memory streams per CU, for batches that would not fill the chip.
// The logits go through LDS, rows four banks apart; 4 lanes per token then
// hold its scores in registers and take the row maximum, the exponential sum
// and k rounds of arg-max (equal scores: lower expert index first), combining
// with lane shuffles.  The gate matrix ([E, H], ~1.8 MB at E = 128, H = 7168)
// stays in L2; x is read once (counters: 265 MB for 235 and the gate rows; the
// matrix cores busy 15% of the time), and HBM bounds large batches: 16384
// tokens, H = 7168, E = 128 take 73 us with x from HBM (3.2 TB/s), 4096 of them
// 45.  Small ones are bound by the latency of their H / 64 chunks: 64 tokens,
// H = 4096, E = 8 take 11 us.  (Figures of the form a -> b in this file are
// those of the step that they explain, on its own box.)
// Measured and not kept: an 8-stage token ring with 3 stages of gate rows, so
// fewer workgroups per CU (4096 tokens, H = 4096, E = 8: 15.7 against 12.2 us;
// E = 64 up to 48 against 35; nothing gained elsewhere).
#include "rmoe_device.h"
#include "rmoe_internal.h"

namespace rmoe {
namespace {

constexpr int RT_CK = 64;   // K per chunk
constexpr int RT_XST = 4;   // LDS ring stages of the tokens: DMA runs 3 chunks ahead
constexpr int RT_WST = 4;   // and of the gate rows

template <int EP, int TOK>
struct RouterCfg {
    static constexpr int TROWS = TOK;             // LDS token rows
    static constexpr int XSTAGE = TROWS * 128, WSTAGE = EP * 128;  // bytes of a chunk: tokens, gate rows
    static constexpr int W_OFF = RT_XST * XSTAGE;
    static constexpr int NIX = TROWS / 8;         // DMA instructions per chunk: tokens, by the fifth wave,
    static constexpr int NIW = EP / 32;           // gate rows, by each of the others
    static constexpr int NT = EP / 32;            // 32-expert tiles
    static constexpr int EW = TOK == 64 ? 2 : 4;  // waves sharing the expert tiles
    static constexpr int TPW = (NT + EW - 1) / EW;  // tiles per wave
    // waves per expert tile that split a chunk's 4 K-steps (TOK = 32 only)
    static constexpr int KSW = TOK == 32 && NT == 1 ? 4 : TOK == 32 && NT == 2 ? 2 : 1;
    // Two sets of operands: a chunk's MFMAs run while the next one's operands
    // come from LDS (64 tokens, H = 7168, E = 128: 33 -> 28 us; 8192 of 4096,
    // E = 96: 22 -> 19).  With 64 tokens the registers cost more than that
    // (16384 of 7168, E = 128: 68 -> 73 us; 20000 of 2048, E = 256: 71 -> 339,
    // spilled), and where the waves split the K-steps nothing changes.
    static constexpr bool TWO = TOK == 32 && KSW == 1;
    static constexpr int LD = EP + 4;             // words per row of logits
    static constexpr int LDS_BYTES = W_OFF + RT_WST * WSTAGE;  // >= the TROWS x LD fp32 logits
    static_assert(TOK == 64 || TOK == 32, "tokens per workgroup: whole 32-token tiles");
    static_assert(LDS_BYTES >= KSW * TROWS * LD * 4 && LDS_BYTES >= 64 * LD * 4, "partial logits fit in the rings");
    static_assert(LDS_BYTES <= 160 * 1024, "LDS");
    static_assert((RT_XST - 2) * NIX < 64 && (RT_WST - 2) * NIW < 64, "vmcnt range");
};

__device__ __forceinline__ bool better(float s, int e, float s2, int e2) {
    return s > s2 || (s == s2 && e < e2);
}

// The losses and the count of tokens from the sums over all tokens.
__device__ __forceinline__ void router_losses(double sum_pc, double z, int n, const RouterTrainArgs &a) {
    a.counts[a.E] = n;
    a.losses[0] = n > 0 ? (float)(sum_pc * a.E / ((double)a.k * n * n)) : 0.f;
    a.losses[1] = n > 0 ? (float)(z / n) : 0.f;
}

// ---- softmax and top-k of the logits L: 4 consecutive lanes per token, lane
// `sub` owns experts sub, sub + 4, ..., NE scores in registers.  NE is EP / 4,
// but 2 for at most 8 experts, whose lanes would spend the time on scores that
// do not exist (8 experts, inputs from HBM: 300000 tokens of H = 64 25.2 ->
// 22.7 us, 300000 of 256 42.5 -> 40.6, 131072 of 1024 52.1 -> 50.7; 64 of
// 4096 10.0 -> 9.5).
template <int EP, int TOK, int NE, bool TRAIN>
__device__ __forceinline__ void router_scores(float *L, unsigned block, int64_t t0, int64_t T, int32_t E, int32_t k,
                                              int32_t *__restrict__ ids, float *__restrict__ vals,
                                              const RouterTrainArgs &tr) {
    using C = RouterCfg<EP, TOK>;
    constexpr int LD = C::LD;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int tok = tid >> 2, sub = tid & 3;
    float *row = L + tok * LD;
    float v[NE], m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        v[i] = sub + 4 * i < E ? row[sub + 4 * i] : -__builtin_inff();
        m = fmaxf(m, v[i]);
    }
    m = fmaxf(m, __shfl_xor(m, 1));
    m = fmaxf(m, __shfl_xor(m, 2));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        v[i] = __builtin_amdgcn_exp2f((v[i] - m) * 1.4426950408889634f);
        sum += v[i];
    }
    sum += __shfl_xor(sum, 1);
    sum += __shfl_xor(sum, 2);
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < NE; ++i) v[i] *= inv;
    const bool live = tok < TOK && t0 + tok < T;
    // behind the logits: the workgroup's pairs per expert, and of each token
    // lse^2 and whether it counts
    static_assert(!TRAIN || C::LDS_BYTES >= (C::TROWS * LD + EP + 2 * TOK) * 4, "LDS behind the logits");
    int32_t *cnt = reinterpret_cast<int32_t *>(L + C::TROWS * LD);
    float *zs = reinterpret_cast<float *>(cnt + EP), *on = zs + TOK;
    bool counts = live;
    if constexpr (TRAIN) {
        counts = live && (tr.mask == nullptr || tr.mask[t0 + tok] != 0);
        __syncthreads();  // idle threads (tok >= TOK) have read their rows there
        for (int e = tid; e < EP; e += 256) cnt[e] = 0;
        if (tok < TOK) {
#pragma unroll
            for (int i = 0; i < NE; ++i) row[sub + 4 * i] = counts ? v[i] : 0.f;
            if (sub == 0) {
                const float lse = counts ? m + __builtin_amdgcn_logf(sum) * 0.6931471805599453f : 0.f;
                zs[tok] = lse * lse;
                on[tok] = counts ? 1.f : 0.f;
                if (live) tr.lse[t0 + tok] = lse;
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) v[i] = sub + 4 * i < E ? v[i] : -2.f;
    for (int j = 0; j < k; ++j) {
        float bs = -1.f;
        int be = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (v[i] > bs) {  // in ascending order: the first of equal scores stays
                bs = v[i];
                be = sub + 4 * i;
            }
#pragma unroll
        for (int d = 1; d <= 2; d <<= 1) {
            const float os = __shfl_xor(bs, d);
            const int oe = __shfl_xor(be, d);
            if (better(os, oe, bs, be)) {
                bs = os;
                be = oe;
            }
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] = be == sub + 4 * i ? -2.f : v[i];  // taken
        if (live && sub == 0) {
            if constexpr (TRAIN) {
                ids[(t0 + tok) * k + j] = counts ? be : -1;
                vals[(t0 + tok) * k + j] = counts ? bs : 0.f;
                // a row of NaN picks no expert (be past E)
                if (counts && be < E) atomicAdd(&cnt[be], 1);
            } else {
                ids[(t0 + tok) * k + j] = be;
                vals[(t0 + tok) * k + j] = bs;
            }
        }
    }
    if constexpr (TRAIN) {
        __syncthreads();
        const int nt = T - t0 < TOK ? (int)(T - t0) : TOK;
        for (int t = wave; t < nt; t += 4)
            for (int e = lane; e < E; e += 64) tr.probs[(t0 + t) * E + e] = L[t * LD + e];
        // sums over the workgroup's tokens, in a fixed order
        float sum_p = 0.f, z = 0.f, n = 0.f;
        if (tid < E) {
#pragma unroll 8
            for (int t = 0; t < nt; ++t) sum_p += L[t * LD + tid];
        }
        if (wave == 3) {  // zs and on hold TOK entries, zeros past the last token
            z = lane < TOK ? zs[lane] : 0.f;
            n = lane < TOK ? on[lane] : 0.f;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                z += __shfl_xor(z, d);
                n += __shfl_xor(n, d);
            }
        }
        if (T > TOK) {
            if (tid < E) tr.parts[(int64_t)block * E + tid] = RouterPart{sum_p, cnt[tid]};
            if (tid == 192) tr.tokens[block] = RouterPart{z, (int)n};
            if (block == 0 && tid == 0) tr.losses[0] = 0.f;  // the next kernel counts there
        } else {  // the batch's only workgroup gives the losses itself
            double term = tid < E ? (double)sum_p * cnt[tid] : 0.0;
            if (tid < E) tr.counts[tid] = cnt[tid];
            for (int d = 1; d < 64; d <<= 1) term += __shfl_xor(term, d);
            __syncthreads();  // the rows are done with
            double *part = reinterpret_cast<double *>(L);
            if (lane == 0) part[wave] = term;
            if (tid == 192) {
                part[4] = z;
                part[5] = n;
            }
            __syncthreads();
            if (tid == 0)
                router_losses((part[0] + part[1]) + (part[2] + part[3]), part[4], (int)part[5], tr);
        }
    }
}

// TRAIN: the training forward, which also keeps the probabilities and each
// token's logsumexp, leaves out masked tokens and sums what the losses need
// over the workgroup's tokens.
template <int EP, int TOK, bool TRAIN>
__device__ __forceinline__ void router_body(const _Float16 *__restrict__ x, const _Float16 *__restrict__ w, int64_t T,
                                            int64_t H, int32_t E, int32_t k, int32_t lag_, int32_t *__restrict__ ids,
                                            float *__restrict__ vals, const RouterTrainArgs &tr) {
    using C = RouterCfg<EP, TOK>;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const unsigned block = blockIdx.y * gridDim.x + blockIdx.x;  // grid_rows
    const int64_t t0 = (int64_t)block * TOK;
    if (t0 >= T) return;
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, lr = lane & 31, lh = lane >> 5;
    // token tile of this wave, and its first expert tile (then every EW-th)
    // (with KSW > 1: expert tile wave % NT, K-steps s with s % KSW == ks)
    const int ks = C::KSW > 1 ? wave / C::NT : 0;
    const int th = TOK == 64 ? (wave & 1) : 0;
    const int eh = TOK == 64 ? (wave >> 1) : C::KSW > 1 ? wave % C::NT : wave;

    // every workgroup reads the same gate rows: each starts its K sweep at a
    // different chunk, so that concurrent workgroups do not ask the L2 for
    // the same lines at the same moment (a token's sum order stays fixed).
    // With a lag the two halves of 64 tokens are sums of two workgroups of 32:
    // the second half joins the sweep lag chunks after the first, where its
    // own workgroup would have started, and goes on as long after the first's
    // end (the same sums, the gate rows read once for both).
    const int nk = (int)(H / RT_CK);
    const int lag = TOK == 64 ? lag_ : 0, sweep = nk + lag;
    const int kofs = (int)((block * (TOK == 64 && lag ? 14u : 7u)) % (unsigned)nk);
    auto chunk = [&](int kc) -> int64_t {  // element offset; clamped at the end: repeats land in stages no later chunk reads
        kc = (kc < sweep ? kc : sweep - 1) + kofs;
        kc = kc < nk ? kc : kc - nk;
        return (int64_t)(kc < nk ? kc : kc - nk) * RT_CK;
    };
    const unsigned lds0 = (unsigned)(uintptr_t)smem;
    // DMA instruction j moves rows 8j .. 8j+7 of a chunk (tokens clamped to
    // the last one, gate rows to the last expert: padding rows feed outputs
    // nobody reads)
    if (wave == 4) {
        const _Float16 *src[C::NIX];
#pragma unroll
        for (int i = 0; i < C::NIX; ++i) {
            const int r = 8 * i + (lane >> 3);
            src[i] = x + (t0 + r < T ? t0 + r : T - 1) * H + 8 * ((lane & 7) ^ lds_swz(r));
        }
        auto dma = [&](int kc) {
#pragma unroll
            for (int i = 0; i < C::NIX; ++i)
                dma16(src[i] + chunk(kc), lds0 + (kc % RT_XST) * C::XSTAGE + i * 1024);
        };
#pragma unroll
        for (int p = 0; p < RT_XST - 1; ++p) dma(p);
        for (int kc = 0; kc < sweep; ++kc) {
            wait_vm<(RT_XST - 2) * C::NIX>();  // chunk kc landed
            bar();
            dma(kc + RT_XST - 1);
        }
        wait_vm<0>();
        bar();
        return;
    }
    const _Float16 *src[C::NIW];
#pragma unroll
    for (int i = 0; i < C::NIW; ++i) {
        const int e = 8 * (wave * C::NIW + i) + (lane >> 3);
        src[i] = w + (int64_t)(e < E ? e : E - 1) * H + 8 * ((lane & 7) ^ lds_swz(e));
    }
    auto dma = [&](int kc) {
#pragma unroll
        for (int i = 0; i < C::NIW; ++i)
            dma16(src[i] + chunk(kc), lds0 + C::W_OFF + (kc % RT_WST) * C::WSTAGE + (wave * C::NIW + i) * 1024);
    };

    constexpr bool whole = C::KSW > 1 || C::NT % C::EW == 0;  // every wave has TPW expert tiles
    f16x acc[C::TPW];
#pragma unroll
    for (int t = 0; t < C::TPW; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[t][i] = 0.f;

#pragma unroll
    for (int p = 0; p < RT_WST - 1; ++p) dma(p);
    constexpr int NS = 4 / C::KSW;  // K-steps of this wave: s = KSW i + ks
    struct Ops {
        h8 b[NS], a[C::TPW][NS];
    } ops[C::TWO ? 2 : 1];
    auto mul = [&](const Ops &o) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int t = 0; t < C::TPW; ++t)
                acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(o.a[t][i], o.b[i], acc[t], 0, 0, 0);
    };
    // requests the operands of chunk kc and multiplies those of `ready`
    auto step = [&](int kc, Ops &o, const Ops &ready) {
        wait_vm<(RT_WST - 2) * C::NIW>();    // chunk kc landed (own DMAs) ...
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's reads of chunk kc-1
        bar();  // ... and everyone's; and every wave is done with chunk kc-1's stages
        if (lag && (th ? kc < lag : kc >= nk)) {  // the other half's part of the sweep
            dma(kc + RT_WST - 1);
            return;
        }
        // the wave's operands of the chunk, all requested before the first MFMA
        const unsigned char *bx = smem + (kc % RT_XST) * C::XSTAGE;
        const unsigned char *bw = smem + C::W_OFF + (kc % RT_WST) * C::WSTAGE;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int ch = 2 * (C::KSW * i + ks) + lh;
            o.b[i] = *(const h8 *)(bx + lds_off(32 * th + lr, ch));
#pragma unroll
            for (int t = 0; t < C::TPW; ++t) {
                // an idle last tile reads the tile before it
                const int et = whole || eh + C::EW * t < C::NT ? eh + C::EW * t : C::NT - 1;
                o.a[t][i] = *(const h8 *)(bw + lds_off(32 * et + lr, ch));
            }
        }
        if constexpr (C::TWO) __builtin_amdgcn_sched_barrier(0);
        dma(kc + RT_WST - 1);
        mul(ready);
    };
    if constexpr (C::TWO) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {  // before the first chunk: adds zeros
            ops[1].b[i] = h8{};
#pragma unroll
            for (int t = 0; t < C::TPW; ++t) ops[1].a[t][i] = h8{};
        }
        int kc = 0;
        for (; kc + 1 < sweep; kc += 2) {
            step(kc, ops[0], ops[1]);
            step(kc + 1, ops[1], ops[0]);
        }
        if (kc < sweep) step(kc, ops[0], ops[1]);
        mul(kc < sweep ? ops[0] : ops[1]);
    } else {
        for (int kc = 0; kc < sweep; ++kc) step(kc, ops[0], ops[0]);
    }
    wait_vm<0>();
    bar();

    // ---- logits -> LDS [TROWS tokens][EP experts] fp32 (partial logits of
    //      K-split ks at L + ks * TROWS * LD, then added in order of ks).
    //      32x32 accumulator layout: register 4q + r holds expert row
    //      8q + 4lh + r, token lr.  Rows are 4 words apart modulo the banks:
    //      the 16 tokens x 4 lanes that read together touch all 64 (at a
    //      stride of EP they shared 4 of them).
    float *L = reinterpret_cast<float *>(smem);
    constexpr int LD = C::LD;
#pragma unroll
    for (int t = 0; t < C::TPW; ++t) {
        const int et = eh + C::EW * t;
        if (whole || et < C::NT) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(f4 *)(L + ks * C::TROWS * LD + (32 * th + lr) * LD + 32 * et + 8 * q + 4 * lh) =
                    f4{acc[t][4 * q], acc[t][4 * q + 1], acc[t][4 * q + 2], acc[t][4 * q + 3]};
        }
    }
    __syncthreads();
    if constexpr (C::KSW > 1) {
        for (int i = tid; i < C::TROWS * LD; i += 256) {
            float v = L[i];
#pragma unroll
            for (int j = 1; j < C::KSW; ++j) v += L[j * C::TROWS * LD + i];
            L[i] = v;
        }
        __syncthreads();
    }

    if constexpr (EP == 32) {
        if (E <= 8) {
            router_scores<EP, TOK, 2, TRAIN>(L, block, t0, T, E, k, ids, vals, tr);
            return;
        }
    }
    router_scores<EP, TOK, EP / 4, TRAIN>(L, block, t0, T, E, k, ids, vals, tr);
}

template <int EP, int TOK>
__global__ __launch_bounds__(320) void router_kernel(const _Float16 *__restrict__ x,
                                                     const _Float16 *__restrict__ w, int64_t T,
                                                     int64_t H, int32_t E, int32_t k, int32_t lag,
                                                     int32_t *__restrict__ ids,
                                                     float *__restrict__ vals) {
    router_body<EP, TOK, false>(x, w, T, H, E, k, lag, ids, vals, RouterTrainArgs{});
}

template <int EP, int TOK>
__global__ __launch_bounds__(320) void router_train_kernel(RouterTrainArgs a) {
    router_body<EP, TOK, true>(a.x, a.w, a.T, a.H, a.E, a.k, a.lag, a.ids, a.vals, a);
}

// Sums of the workgroups' parts and the losses.  A workgroup takes 32 experts
// (512 parts of 128 experts read by one workgroup cost 11 us, by four 5), 32
// slices of the parts each, then the slices in order; it leaves its experts'
// share of the balance loss where its first part was (which no other one
// reads), and the last to finish adds the shares in order.  The count of
// finished workgroups is kept in losses[0], zeroed by the kernel before.
__global__ __launch_bounds__(1024) void router_losses_kernel(RouterTrainArgs a, int parts) {
    __shared__ double ps[1024], zsum[16];
    __shared__ int32_t cs[1024], nsum[16];
    __shared__ bool last;
    const int tid = threadIdx.x, sl = tid >> 5, e = blockIdx.x * 32 + (tid & 31);
    if (parts == 0) {
        if (sl == 0 && e < a.E) a.counts[e] = 0;
        if (e == 0 && sl == 0) {
            a.counts[a.E] = 0;
            a.losses[0] = a.losses[1] = 0.f;
        }
        return;
    }
    double p = 0.0, z = 0.0;
    int32_t c = 0, n = 0;
    if (e < a.E)
#pragma unroll 16
        for (int b = sl; b < parts; b += 32) {
            const RouterPart r = a.parts[(int64_t)b * a.E + e];
            p += r.sum;
            c += r.count;
        }
    for (int b = tid; b < parts; b += 1024) {
        const RouterPart r = a.tokens[b];
        z += r.sum;
        n += r.count;
    }
    for (int d = 1; d < 64; d <<= 1) {
        z += __shfl_xor(z, d);
        n += __shfl_xor(n, d);
    }
    ps[tid] = p;
    cs[tid] = c;
    if ((tid & 63) == 0) {
        zsum[tid >> 6] = z;
        nsum[tid >> 6] = n;
    }
    __syncthreads();
    double *share = reinterpret_cast<double *>(a.parts + blockIdx.x * 32);
    if (tid < 32) {
        for (int i = 1; i < 32; ++i) {
            p += ps[32 * i + tid];
            c += cs[32 * i + tid];
        }
        if (e < a.E) a.counts[e] = c;
        double term = p * c;
        for (int d = 1; d < 32; d <<= 1) term += __shfl_xor(term, d, 32);
        if (tid == 0) {
            __hip_atomic_store(share, term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(reinterpret_cast<int32_t *>(a.losses), 1, __ATOMIC_ACQ_REL,
                                          __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last || tid != 0) return;
    z = 0.0;
    n = 0;
    for (int i = 0; i < 16; ++i) {
        z += zsum[i];
        n += nsum[i];
    }
    double s = 0.0;
    for (unsigned i = 0; i < gridDim.x; ++i)
        s += __hip_atomic_load(reinterpret_cast<double *>(a.parts + i * 32), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    router_losses(s, z, n, a);
}

template <int EP, int TOK>
hipError_t launch_ep(const _Float16 *x, const _Float16 *w, int64_t T, int64_t H, int32_t E,
                     int32_t k, int32_t lag, int32_t *ids, float *vals, hipStream_t s) {
    using C = RouterCfg<EP, TOK>;
    static std::atomic<uint64_t> lds_set{0};
    hipError_t e = lds_opt_in_once((const void *)router_kernel<EP, TOK>, C::LDS_BYTES, lds_set);
    if (e != hipSuccess) return e;
    const GridRows grid = grid_rows((T + TOK - 1) / TOK);
    hipLaunchKernelGGL((router_kernel<EP, TOK>), dim3(grid.x, grid.y), dim3(320), C::LDS_BYTES, s, x, w, T, H,
                       E, k, lag, ids, vals);
    return hipGetLastError();
}

template <int EP, int TOK>
hipError_t launch_train_ep(const RouterTrainArgs &a, hipStream_t s) {
    using C = RouterCfg<EP, TOK>;
    static std::atomic<uint64_t> lds_set{0};
    hipError_t e = lds_opt_in_once((const void *)router_train_kernel<EP, TOK>, C::LDS_BYTES, lds_set);
    if (e != hipSuccess) return e;
    const GridRows grid = grid_rows((a.T + TOK - 1) / TOK);
    hipLaunchKernelGGL((router_train_kernel<EP, TOK>), dim3(grid.x, grid.y), dim3(320), C::LDS_BYTES, s, a);
    return hipGetLastError();
}

// Compute units of the current device (cached per device).
hipError_t cu_count(int &n) {
    static std::atomic<int> cached[64];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    n = dev < 64 ? cached[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        e = hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev);
        if (e != hipSuccess) return e;
        if (n < 1) n = 1;
        if (dev < 64) cached[dev].store(n, std::memory_order_relaxed);
    }
    return hipSuccess;
}

// Tokens per workgroup: 64 once that still gives two workgroups per CU; from
// one per CU on, 64 as two lagging halves (16384 tokens, H = 7168, E = 128,
// training forward: 94 -> 79 us) where workgroups of 32 do not split a chunk's K-steps, whose
// sums are another order.
hipError_t tokens_per_workgroup(int64_t T, int64_t H, int32_t E, int &tok, int32_t &lag) {
    int cus = 0;
    const hipError_t e = cu_count(cus);
    if (e != hipSuccess) return e;
    const bool halves = E > 64 && T >= (int64_t)64 * cus && T < (int64_t)64 * 2 * cus;
    tok = halves || T >= (int64_t)64 * 2 * cus ? 64 : 32;
    lag = halves ? (int32_t)(7 % (H / RT_CK)) : 0;
    return hipSuccess;
}

}  // namespace

int64_t router_train_parts(int64_t T) { return (T + 31) / 32; }

hipError_t launch_router_train(const RouterTrainArgs &args, hipStream_t s) {
    RouterTrainArgs a = args;
    int tok = 0;
    hipError_t e = tokens_per_workgroup(a.T, a.H, a.E, tok, a.lag);
    if (e != hipSuccess) return e;
    if (a.T > 0) {
#define RMOE_R(N) \
    case N: e = tok == 64 ? launch_train_ep<32 * N, 64>(a, s) : launch_train_ep<32 * N, 32>(a, s); break;
        switch ((a.E + 31) / 32) {
            RMOE_R(1) RMOE_R(2) RMOE_R(3) RMOE_R(4) RMOE_R(5) RMOE_R(6) RMOE_R(7) RMOE_R(8)
            default: return hipErrorInvalidValue;
        }
#undef RMOE_R
        if (e != hipSuccess) return e;
    }
    if (a.T > 0 && a.T <= tok) return hipSuccess;
    hipLaunchKernelGGL(router_losses_kernel, dim3((unsigned)((a.E + 31) / 32)), dim3(1024), 0, s, a,
                       (int)((a.T + tok - 1) / tok));
    return hipGetLastError();
}

hipError_t launch_router(const _Float16 *x, const _Float16 *w, int64_t T, int64_t H, int32_t E,
                         int32_t k, int32_t *ids, float *vals, hipStream_t s) {
    if (T == 0 || k == 0) return hipSuccess;
    int tok = 0;
    int32_t lag = 0;
    hipError_t e = tokens_per_workgroup(T, H, E, tok, lag);
    if (e != hipSuccess) return e;
#define RMOE_R(N)                                                                        \
    case N:                                                                              \
        return tok == 64 ? launch_ep<32 * N, 64>(x, w, T, H, E, k, lag, ids, vals, s)    \
                         : launch_ep<32 * N, 32>(x, w, T, H, E, k, 0, ids, vals, s);
    switch ((E + 31) / 32) {
        RMOE_R(1) RMOE_R(2) RMOE_R(3) RMOE_R(4) RMOE_R(5) RMOE_R(6) RMOE_R(7) RMOE_R(8)
        default: return hipErrorInvalidValue;
    }
#undef RMOE_R
}

}  // namespace rmoe
