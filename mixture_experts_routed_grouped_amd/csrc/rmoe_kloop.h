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
// A persistent workgroup overlaps its items: kfill issues the first step's
// DMAs of the next item before the epilogue of the current one, whose vector
// work then covers their round trip (a first step took 5-8 k cycles of a 46 k
// cycle item when it was fetched at the item's start).
//
// P, the operands, provides
//   Frag                     one 16-byte MFMA operand
//   AR, BR                   LDS reads per A / B operand tile of a sub-step
//   DMAS, LATE, PARTS        DMAs of a group per wave; how many of the last
//                            of them fill the step after the next (0 or the
//                            A slot's); sub-steps over which a group is spread
//   PRE                      steps that the ring holds: 2, or 3 for A
//   FILL                     parts of group g(-1) that kfill issues too (0, 1)
//   nk                       K steps
//   begin()                  before an item's K loop: its lane indexes, fresh
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
#include "rmoe_internal.h"
#include "rmoe_sched.h"

namespace rmoe {

// A pointer known to be the same in every lane, in scalar registers.
template <class T>
__device__ __forceinline__ const T *uniform(const T *p) {
    const uint64_t u = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u), hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
    return (const T *)(((uint64_t)hi << 32) | lo);
}

// A table that no kernel of the launch writes, in the constant address space:
// a uniform index reads it with a scalar load, also after stores (which the
// compiler must otherwise assume may have changed it: such vector loads cost
// 1-2 k cycles each in a persistent kernel's step to its next item).
typedef const __attribute__((address_space(4))) int32_t *Table;
__device__ __forceinline__ Table table(const int32_t *p) { return (Table)(uintptr_t)p; }
typedef ItemWalk<Table> Walk;

// x, as if it were a new value: keeps the compiler from computing what
// depends on it ahead of a loop, where it would stay live (and spill).
__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

template <class P>
constexpr int kPart = (P::DMAS + P::PARTS - 1) / P::PARTS;  // DMAs of a group's part

// The DMAs of the first step.  The workgroup must be past the last barrier of
// the K loop before (the slots are then free; the epilogue may still use this
// wave's pieces of the slots that are not filled here: with PRE 2 all but
// slot 0 of both operands, with PRE 3 all but A's 0 and 1 and B's 0).
template <class P>
__device__ __forceinline__ void kfill(P &p) {
    if constexpr (P::PRE == 3) {
#pragma unroll
        for (int d = P::DMAS - P::LATE; d < P::DMAS; ++d) p.dma(d, -3);
    }
#pragma unroll
    for (int d = 0; d < P::DMAS; ++d) p.dma(d, -2);
    if constexpr (P::FILL > 0) {
#pragma unroll
        for (int d = 0; d < kPart<P>; ++d) p.dma(d, -1);
    }
}

// newer: memory instructions that this wave has certainly issued since kfill
// (0 or kNewer): the wait for the first step leaves that many in flight.
constexpr int kNewer = 24;

template <int NTT, class P>
__device__ __forceinline__ void kloop(P &p, bool newer, f16x (&acc)[4][4]) {
    constexpr int NMF = 4 * NTT;                            // MFMAs per sub-step
    constexpr int NRD = NTT > 0 ? 4 * P::AR + NTT * P::BR : 0;  // operand reads per sub-step
    constexpr int DPS = kPart<P>;
    const int nk = p.nk;
    typename P::Frag a[2][4], b[2][4];
    // MFMAs of sub-step S (buffer S & 1), interleaved with the reads of
    // sub-step sr of step kr and part `part` of group g(gj)
    auto substep = [&](auto sc, bool rd, int kr, int sr, int gj, int part) __attribute__((always_inline)) {
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
    if constexpr (P::FILL == 0) {
#pragma unroll
        for (int d = 0; d < DPS; ++d) p.dma(d, -1);
    }
    static_assert(P::LATE + DPS + kNewer < 64, "vmcnt range");
    if (newer)
        wait_vm<P::LATE + DPS + kNewer>();
    else
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

__device__ __forceinline__ void zero_acc(f16x (&acc)[4][4]) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[t][u][i] = 0.f;
}

// The K loop for the wave's live token tiles (a uniform count), then
// done(accumulators, count as a constant): one copy of the epilogue per
// count, so that the accumulators stay in the registers of their loop (one
// copy after all loops cost 336 register moves per item).
template <int NTT, class P, class F>
__device__ __forceinline__ void krun(P &p, bool newer, F &&done) {
    p.begin();
    f16x acc[4][4];
    zero_acc(acc);
    kloop<NTT>(p, newer, acc);
    done(acc, std::integral_constant<int, NTT>{});
}
template <class P, class F>
__device__ __forceinline__ void ktiles(P &p, int ntt, bool newer, F &&done) {
    switch (ntt) {
        case 4: krun<4>(p, newer, done); break;
        case 3: krun<3>(p, newer, done); break;
        case 2: krun<2>(p, newer, done); break;
        case 1: krun<1>(p, newer, done); break;
        default: krun<0>(p, newer, done); break;
    }
}

// Runs a persistent workgroup (one per CU).  T, the tile, provides p (its
// operands), set(item) (their bases), tiles(item) (this wave's live token
// tiles) and finish<NTT>(item, acc, fill): the epilogue, which calls fill()
// once, where the next item's first step may go out, and returns whether at
// least kNewer memory instructions of this wave certainly followed it.
template <class T>
__device__ __forceinline__ void run_items(T &tile, const int32_t *group_sizes, const int32_t *padded_offsets,
                                          const int32_t *block_experts, int E, int NT) {
    Walk walk(table(group_sizes), table(padded_offsets), table(block_experts), E, NT, (int)blockIdx.x, (int)gridDim.x);
    TileItem it;
    if (!walk.next(it)) return;
    tile.set(it);
    kfill(tile.p);
    bool newer = false, more = true;
    while (more) {
        ktiles(tile.p, tile.tiles(it), newer, [&](auto &acc, auto n) __attribute__((always_inline)) {
            const TileItem now = it;
            newer = tile.template finish<decltype(n)::value>(now, acc, [&]() __attribute__((always_inline)) {
                more = walk.next(it);
                if (more) {
                    tile.set(it);
                    kfill(tile.p);
                }
            });
        });
    }
}

}  // namespace rmoe
