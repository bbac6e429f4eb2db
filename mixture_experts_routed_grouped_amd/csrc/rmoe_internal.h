// Internal interface between the C-ABI host code (rmoe_api.cpp) and the
// gfx950 kernel launchers (*.hip).  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "rmoe_sched.h"

namespace rmoe {

// Opt a kernel into `bytes` of dynamic LDS, once per device: the attribute
// stays set for the process, so later launches skip the runtime call.
// `done` is the kernel's own per-device flag word (bit d: device d).
inline hipError_t lds_opt_in_once(const void *fn, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return hipSuccess;
    e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess && bit) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// Workgroup slots of the persistent kernel on the current device: its CU
// count rounded down to a multiple of 8 (cached per device).
inline hipError_t cu_grid(unsigned &grid) {
    static std::atomic<int> cached[64];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    int n = dev < 64 ? cached[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        e = hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev);
        if (e != hipSuccess) return e;
        n = n / kXcd * kXcd;
        if (n < kXcd) n = kXcd;
        if (dev < 64) cached[dev].store(n, std::memory_order_relaxed);
    }
    grid = (unsigned)n;
    return hipSuccess;
}

// One stage of the routed expert FFN as the kernels see it: a grouped GEMM
// Y[r, n] = epilogue( sum_k X[r, k] * W[e(r), n, k] ) over the valid rows r
// of every 128-row block.  For the gate/up stage W0 = gate_w, W1 = up_w and
// the epilogue is fp16(silu(g) * u); for the down stage W0 = down_w and the
// epilogue is fp16(acc * routed_weight[compact row]).
struct StageArgs {
    const _Float16 *x;      // [Tp, K]
    const _Float16 *w0;     // [E, N, K]
    const _Float16 *w1;     // [E, N, K] (gate/up only)
    const float *rw;        // [pairs] compact order (down only)
    const int32_t *gs;      // group_sizes [E]
    const int32_t *go;      // group_offsets [E+1] (down only)
    const int32_t *gpo;     // group_padded_offsets [E+1]
    const int32_t *gidx;    // group_idx_for_bx [M]
    _Float16 *y;            // [Tp, N]
    int64_t K, N;
    int32_t E, M;
    int64_t pairs;
};

// Kernel-family launchers; return hipSuccess or the launch error.
hipError_t launch_stream_gate_up(const StageArgs &a, hipStream_t s);
hipError_t launch_stream_down(const StageArgs &a, hipStream_t s);
hipError_t launch_tile_gate_up(const StageArgs &a, hipStream_t s);
hipError_t launch_tile_down(const StageArgs &a, hipStream_t s);
// Both tiled stages in one persistent launch (gu.y = dn.x = the hidden
// workspace); sync as described for rmoe_forward_fused_f16; a down tile
// waits at most wait_us for its pair's hidden rows.  local: each XCD runs
// whole entries and the hidden rows stay in its L2 (the kernel's LOCAL
// mode); otherwise entries are spread over all XCDs with write-through
// hand-over.
hipError_t launch_fused(const StageArgs &gu, const StageArgs &dn, int32_t *sync, int64_t wait_us,
                        bool local, hipStream_t s);

hipError_t launch_pack(const _Float16 *x, const float *topk_w, const int32_t *prow,
                       const int32_t *cpos, int64_t pairs, int32_t top_k, int64_t H, int64_t Tp,
                       _Float16 *stacked, float *w_compact, hipStream_t s);
hipError_t launch_combine(const _Float16 *out, const int32_t *prow, int64_t T, int32_t top_k,
                          int64_t H, int64_t Tp, _Float16 *y, hipStream_t s);

// Router: top-k ids and softmax scores of x W^T (E <= 256).
hipError_t launch_router(const _Float16 *x, const _Float16 *w, int64_t T, int64_t H, int32_t E,
                         int32_t k, int32_t *ids, float *vals, hipStream_t s);

// A workgroup's sum and count.
struct alignas(8) RouterPart {
    float sum;
    int32_t count;
};

// The training router: what the forward keeps, and the losses.
struct RouterTrainArgs {
    const _Float16 *x, *w;  // [T, H], [E, H]
    const uint8_t *mask;    // [T], 0: the token is left out; null: none is
    int64_t T, H;
    int32_t E, k;
    int32_t *ids;           // [T, k]
    float *vals;            // [T, k]
    float *probs, *lse;     // [T, E], [T]
    int32_t *counts;        // [E + 1]: pairs per expert, tokens that count
    float *losses;          // [2]: balance, z
    RouterPart *parts;      // [parts, E] probabilities, pairs
    RouterPart *tokens;     // [parts] lse^2, tokens
    int32_t lag;            // set by the launcher
};
int64_t router_train_parts(int64_t T);  // at most
hipError_t launch_router_train(const RouterTrainArgs &a, hipStream_t s);

// Its backward pass (rmoe_router_train.hip).
struct RouterBackArgs {
    const _Float16 *x, *w;  // [T, H], [E, H]
    const uint8_t *mask;
    const int32_t *ids;     // [T, k]
    const float *probs, *lse;
    const int32_t *counts;  // [E + 1]
    const float *drw;       // [pairs]: in pair order, or in compact order with cpos
    const int32_t *cpos;    // [T, k] or null
    const float *dlosses;   // [2] or null
    const _Float16 *add;    // [T, H] or null
    _Float16 *dx;           // [T, H]
    float *dw;              // [E, H]
    unsigned char *scratch;
    int64_t T, H;
    int32_t E, k;
};
int64_t router_backward_scratch(int64_t T, int64_t H, int32_t E);
hipError_t launch_router_backward(const RouterBackArgs &a, hipStream_t s);

// Device-side check of the contract tables: writes the number of violated
// rules to *violations (one workgroup, no memset needed).
hipError_t launch_validate(const int32_t *gs, const int32_t *go, const int32_t *gpo,
                           const int32_t *gidx, int32_t E, int32_t M, int64_t pairs,
                           int32_t *violations, hipStream_t s);

// ---- MXFP4 (rmoe_mx.h)

enum class MxType { f16, bf16, f32 };

// x [batch, rows, cols] -> codes [batch, rows, 128 ceil(cols / 256)], scales
// [batch, ceil(cols / 256), rows, 8]; and back.
hipError_t launch_quantize(const void *x, MxType type, int64_t batch, int64_t rows, int64_t cols,
                           unsigned char *codes, unsigned char *scales, hipStream_t s);
hipError_t launch_dequantize(const unsigned char *codes, const unsigned char *scales, MxType type, int64_t batch,
                             int64_t rows, int64_t cols, void *y, hipStream_t s);
hipError_t launch_pack_mx(const _Float16 *x, const float *topk_w, const int32_t *prow, const int32_t *cpos,
                          int64_t T, int32_t k, int64_t H, int64_t Tp, unsigned char *codes, unsigned char *scales,
                          float *w_compact, hipStream_t s);

// One stage of the routed FFN on MXFP4 operands, as StageArgs.
struct MxArgs {
    const unsigned char *x, *xs;               // token codes [Tp, 128 kc], scales [kc, Tp, 8]
    const unsigned char *w0, *w0s, *w1, *w1s;  // weight codes [E, N, 128 kc], scales [E, kc, N, 8]; w1 gate/up only
    const float *rw;                           // [pairs] compact order (down only)
    const int32_t *gs, *go, *gpo, *gidx;
    unsigned char *yc, *ys;                    // gate/up: hidden codes [Tp, 128 ceil(N / 256)], scales
    _Float16 *y;                               // down: out [Tp, N]
    int64_t N, Tp;
    int32_t kc;                                // chunks of 256 along K
    int32_t E, M;
};
hipError_t launch_mx_tile_gate_up(const MxArgs &a, hipStream_t s);
hipError_t launch_mx_tile_down(const MxArgs &a, hipStream_t s);
hipError_t launch_mx_stream_gate_up(const MxArgs &a, int64_t pairs, hipStream_t s);
hipError_t launch_mx_stream_down(const MxArgs &a, int64_t pairs, hipStream_t s);

// ---- 8-bit integers (rmoe_i8.h)

hipError_t launch_quantize_i8(const void *x, MxType type, int64_t rows, int64_t cols, unsigned char *codes,
                              float *scales, hipStream_t s);
hipError_t launch_dequantize_i8(const unsigned char *codes, const float *scales, MxType type, int64_t rows,
                                int64_t cols, void *y, hipStream_t s);
hipError_t launch_pack_i8(const _Float16 *x, const float *topk_w, const int32_t *prow, const int32_t *cpos, int64_t T,
                          int32_t k, int64_t H, int64_t Tp, unsigned char *codes, float *scales, float *w_compact,
                          hipStream_t s);

// One stage of the routed FFN on 8-bit rows, as StageArgs.
struct I8Args {
    const unsigned char *x;                    // token codes [Tp, K]
    const float *xs;                           // their scales [Tp]
    const unsigned char *w0, *w1;              // weight codes [E, N, K]; w1 gate/up only
    const float *w0s, *w1s;                    // their scales [E, N]
    const float *rw;                           // [pairs] compact order (down only)
    const int32_t *gs, *go, *gpo, *gidx;
    float *rows;                               // gate/up: hidden rows [Tp, N] in fp32
    unsigned char *yc;                         // gate/up: their codes [Tp, N]
    float *ys;                                 // and scales [Tp]
    _Float16 *y;                               // down: out [Tp, N]
    int32_t *part;                             // down, tiled: room for K / N parts of sums [Tp, N], or null
    int64_t K, N, Tp;
    int32_t E, M, splits;                      // splits: parts of K (set by the launch)
};
// The products of the gate/up stage write rows, the quantisation yc and ys.
hipError_t launch_i8_tile_gate_up(const I8Args &a, hipStream_t s);
hipError_t launch_i8_tile_down(const I8Args &a, int64_t pairs, hipStream_t s);
hipError_t launch_i8_stream_gate_up(const I8Args &a, int64_t pairs, hipStream_t s);
hipError_t launch_i8_stream_down(const I8Args &a, int64_t pairs, hipStream_t s);
hipError_t launch_quantize_hidden_i8(const I8Args &a, int64_t pairs, hipStream_t s);

// ---- training (rmoe_train.hip)

struct TrainArgs {
    const _Float16 *x, *dy;             // [Tp, H] token rows, output gradient
    const _Float16 *wg, *wu, *wd;       // [E, I, H], [E, I, H], [E, H, I]
    const float *rw;                    // [pairs] compact order
    const _Float16 *g, *u;              // [Tp, I] kept pre-activations
    const int32_t *gs, *go, *gpo, *gidx;
    _Float16 *yg, *yu, *yh;             // [Tp, I] the training forward's gate, up and hidden rows
    _Float16 *dg, *du, *hw;             // [Tp, I] (dg, du may be g, u themselves)
    float *part, *drw;                  // [pairs, I / 128] partial sums; [pairs]
    _Float16 *dx;                       // [Tp, H]
    _Float16 *dwg, *dwu, *dwd;
    int64_t H, I, Tp, pairs;
    int32_t E, M;
};
hipError_t launch_gate_up_train(const TrainArgs &a, hipStream_t s);     // yg, yu, yh
hipError_t launch_hidden_grad(const TrainArgs &a, hipStream_t s);       // dg, du, hw, part
hipError_t launch_drw(const TrainArgs &a, hipStream_t s);               // drw from part
hipError_t launch_gate_up_backward(const TrainArgs &a, hipStream_t s);  // dx
hipError_t launch_weight_grad(const TrainArgs &a, hipStream_t s);       // dwg, dwu, dwd
hipError_t launch_grads(const TrainArgs &a, hipStream_t s);             // the last three in one launch
int64_t weight_grad_tiles(int64_t H, int64_t I, int32_t E);

// Words of the static scratch the allocation-free contract build uses
// (1 MiB per GPU): contract_chunks(pairs) * (E + 1) must not exceed it.
constexpr int64_t kNoAllocScratchWords = (int64_t)1 << 18;
// Device address of that scratch on the current device (looked up once per
// device, cached).
hipError_t noalloc_scratch(int32_t **ptr);

// Device-side contract build.  ws holds contract_chunks(pairs) * (E + 1)
// int32 of scratch.
int64_t contract_chunks(int64_t pairs);
hipError_t launch_contract(const int32_t *ids, int64_t pairs, int32_t E, int32_t M, int32_t *gs,
                           int32_t *go, int32_t *gpo, int32_t *gidx, int32_t *order, int32_t *prow,
                           int32_t *cpos, int32_t *bad, int32_t *ws, hipStream_t s);

}  // namespace rmoe
