// K loop of the 256 x 256 tiled kernels on MXFP4 operands and with k-major
// operands: four waves, 2 (A half) x 2 (B half), each holding a 128 x 128
// fp32 block as 4 x 4 tiles of 32 x 32; operands travel global -> LDS by DMA
// through a ring of slots and reach the matrix instructions through LDS
// reads of one sub-step (a quarter of a K step) ahead.
//
// The pipeline is rotated by one sub-step: the wait and barrier that publish
// step k+1 sit before the last sub-step of step k, whose MFMAs cover the
// first LDS reads of step k+1.  Group g(j) is the DMAs that refill the slots
// of step j once every wave is done with them; its parts are spread over the
// sub-steps that follow that barrier, between the MFMAs, so that the memory
// instructions leave the in-order wave while the matrix core is busy.
//
// P, the operands, provides
//   Frag                     one 16-byte MFMA operand
//   AR, BR                   LDS reads per A / B operand tile of a sub-step
//   DMAS, LATE, PARTS        DMAs of a group per wave; how many of the last
//                            of them fill the step after the next (0 or the
//                            A slot's); sub-steps over which a group is spread
//   PRE                      steps that the ring holds: 2, or 3 for A
//   dma(d, j)                DMA d of group g(j): steps are clamped to the
//                            last one (the repeats land in slots that no
//                            later step reads)
//   read(k, s, i, a, b)      LDS read i of sub-step s of step k
//   step(k), next()          a step's further operands (scales): read ahead
//                            with its first sub-step, and taken over
//   mma<S>(a, b, acc, t, u)  the matrix instruction of sub-step S
//   publish(k)               after the barrier that publishes step k
#pragma once

#include <type_traits>

#include "rmoe_device.h"

namespace rmoe {

constexpr int kSub = 4;  // sub-steps per K step

template <int NTT, class P>
__device__ __forceinline__ void kloop(P &p, int nk, f16x (&acc)[4][4]) {
    constexpr int NMF = 4 * NTT;                            // MFMAs per sub-step
    constexpr int NRD = NTT > 0 ? 4 * P::AR + NTT * P::BR : 0;  // operand reads per sub-step
    constexpr int DPS = (P::DMAS + P::PARTS - 1) / P::PARTS;
    typename P::Frag a[2][4], b[2][4];
    // MFMAs of sub-step S (buffer S & 1), interleaved with the reads of
    // sub-step sr of step kr and part `part` of group g(gj)
    auto substep = [&](auto sc, bool rd, int kr, int sr, int gj, int part) {
        constexpr int S = decltype(sc)::value;
        const int nrd = rd ? NRD : 0;
        const int d0 = DPS * part;
        const int ndma = part < P::PARTS ? (P::DMAS - d0 < DPS ? P::DMAS - d0 : DPS) : 0;
        const int nmem = nrd + ndma;
        const int nslot = NMF > nmem ? NMF : nmem;
        const int m = nrd < ndma ? nrd : ndma;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < nslot; ++i) {
            if (i < NMF) p.template mma<S>(a[S & 1][i % 4], b[S & 1][i / 4], acc[i % 4][i / 4], i % 4, i / 4);
            int r = -1, d = -1;  // memory slot i: reads on even slots, DMAs between
            if (i < 2 * m) {
                if (i & 1) d = i / 2; else r = i / 2;
            } else if (i - m < nrd && nrd > ndma) {
                r = i - m;
            } else if (i - m < ndma && ndma > nrd) {
                d = i - m;
            }
            if (r >= 0) p.read(kr, sr, r, a[sr & 1], b[sr & 1]);
            if (d >= 0) p.dma(d0 + d, gj);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr std::integral_constant<int, 0> s0{};
    constexpr std::integral_constant<int, 1> s1{};
    constexpr std::integral_constant<int, 2> s2{};
    constexpr std::integral_constant<int, 3> s3{};
    // prologue: step 0 whole (with a ring of 3 also A of step 1), the first
    // part of the group that follows
    if constexpr (P::PRE == 3) {
#pragma unroll
        for (int d = P::DMAS - P::LATE; d < P::DMAS; ++d) p.dma(d, -3);
    }
#pragma unroll
    for (int d = 0; d < P::DMAS; ++d) p.dma(d, -2);
#pragma unroll
    for (int d = 0; d < DPS; ++d) p.dma(d, -1);
    wait_vm<P::LATE + DPS>();
    bar();
    p.publish(0);
    if constexpr (NTT > 0) {
        p.step(0);
#pragma unroll
        for (int i = 0; i < NRD; ++i) p.read(0, 0, i, a[0], b[0]);
        p.next();
    }
    for (int k = 0; k < nk; ++k) {
        if (k > 0) {  // end of step k-1
            if constexpr (NTT > 0) p.step(k);
            substep(s3, true, k, 0, k - 1, 0);
            if constexpr (NTT > 0) p.next();
        }
        substep(s0, true, k, 1, k - 1, 1);
        substep(s1, true, k, 2, k - 1, 2);
        substep(s2, true, k, 3, k - 1, 3);
        // publish step k+1 and retire this wave's reads of step k, whose
        // slots the next group refills
        wait_vm<P::LATE>();
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        bar();
        p.publish(k + 1);
    }
    substep(s3, false, 0, 0, 0, P::PARTS);  // end of step nk-1
    wait_vm<0>();
}

// kloop for the wave's live token tiles (a uniform count)
template <class P>
__device__ __forceinline__ void kloop_tiles(P &p, int nk, int ntt, f16x (&acc)[4][4]) {
    switch (ntt) {
        case 4: kloop<4>(p, nk, acc); break;
        case 3: kloop<3>(p, nk, acc); break;
        case 2: kloop<2>(p, nk, acc); break;
        case 1: kloop<1>(p, nk, acc); break;
        default: kloop<0>(p, nk, acc); break;
    }
}

__device__ __forceinline__ void zero_acc(f16x (&acc)[4][4]) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[t][u][i] = 0.f;
}

}  // namespace rmoe
