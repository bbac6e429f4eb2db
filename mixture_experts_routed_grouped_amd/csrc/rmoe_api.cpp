// C-ABI entry points of the routed fused-MoE library: host-side dispatch
// contract, its validator, argument checking and kernel dispatch.  Nothing
// here allocates device memory, synchronises, or reads device tables.
#include "../../include/routed_moe.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <vector>

#include "rmoe_internal.h"

namespace {

constexpr int64_t B = RMOE_BLOCK_M;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
constexpr int32_t kMaxDeviceExperts = 8192;  // the device contract keeps per-expert tables in LDS
// default bound on how long a fused down tile waits for its pair's hidden
// rows (the longest real wait is one gate/up stage: milliseconds)
constexpr int64_t kFusedWaitUs = 2000000;

// ceil(a / b) without forming a + b - 1, which wraps around next to INT64_MAX
int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b > 0); }

// Shape checks shared by the forward and the two stage entry points.
int check_dims(int64_t hidden, int64_t intermediate, int32_t num_experts,
               int64_t total_padded_tokens, int32_t num_blocks_m) {
    if (hidden <= 0 || intermediate <= 0 || num_experts < 1 || num_blocks_m < 0 ||
        total_padded_tokens < 0)
        return RMOE_ERR_INVALID_ARGUMENT;
    if (hidden % 128 != 0 || intermediate % 128 != 0) return RMOE_ERR_UNSUPPORTED_SHAPE;
    if ((int64_t)num_blocks_m * B > total_padded_tokens) return RMOE_ERR_INVALID_ARGUMENT;
    if (num_blocks_m > 65535) return RMOE_ERR_UNSUPPORTED_SHAPE;  // grid y limit
    if (hidden > (int64_t)1 << 20 || intermediate > (int64_t)1 << 20)
        return RMOE_ERR_UNSUPPORTED_SHAPE;
    return RMOE_OK;
}

// Kernel family: the weight-streaming family when experts hold few rows on
// average (then a weight byte serves a handful of tokens and the stage is
// HBM-bound), the LDS-tiled family otherwise.  A streaming block takes the
// narrowest pass of 32, 64 or 96 tokens that holds its rows (96 then 32 for
// 97-128 rows), so blocks of up to 96 rows read their weights once; a group
// of g rows reads its expert's weights about g/64 times beyond that.
//
// Average threshold by expert count, from forward times of both families
// (one MI355X, uniform and Zipf routing, 16-112 rows per expert):
//   E <= 4: 96 rows -- the tiled family has very few work items (E=4,
//     H=4096: 64 down-stage items for 256 CUs); E=4 (4096, 14336) streams
//     14-42% faster at 48-96, tiles 13-14% faster at 112;
//   E <= 8: 56 -- at 56, E=8 (4096, 14336) streams 15% faster (uniform) and
//     1-4% (Zipf 1.2), (6144, 16384) 1-4%; at 64 the Zipf batch tiles 9%
//     faster;
//   E < 32: 32 -- E=16 (4096, 14336) tiles up to 5% faster at 40-48
//     uniform, 7% from 40 under Zipf;
//   E >= 32: 36 -- E=64 (2048, 1408) streams 2-4% faster at 36 and tiles
//     2% faster at 42; E=128 (7168, 2048) tiles 4-6% faster at 40 (E=32
//     (4096, 2048) streams faster up to 64 rows, 18% at 40).
// When the caller knows the largest group (max_group_rows >= 0, from host
// tables):
//   * with fewer than 32 experts streaming also needs every group to fit
//     one 128-row block: the few experts' extra weight reads then weigh on
//     the whole batch (E=16 Zipf 1.2, 40 rows per expert, largest group 197:
//     tiling 7% faster).  With 32 or more experts the extra reads of the
//     large groups are a small share (E=128 Zipf 1.2 at 8-32 rows, largest
//     group 120-485: streaming 2-18% faster; E=64 Zipf 1.1 at 24-36,
//     largest 219-330: 4-9%);
//   * batches of at most 32 experts whose every group fits one pass stream
//     whatever their average while the largest group is at most 64 rows,
//     and up to 96 rows at an average of at most 80 (E <= 8) or 48 rows:
//     each weight byte is then read once, while the tiled family has too
//     few work items (E=8 (4096, 14336) at 64-80 rows, largest 75-94:
//     streaming 5-15% faster, (2048, 5632) 41-52%, (6144, 16384) between
//     2% faster and 8% slower; E=32 (4096, 2048) at 40-48, largest 57-72:
//     14-18% faster; E=16 (4096, 14336) at 40-48, largest 51-62: within 5%
//     either way).
constexpr int64_t kStreamMaxGroupRows = B;
constexpr int32_t kManyExperts = 32;
int64_t stream_max_avg_rows(int32_t num_experts) {
    return num_experts <= 4 ? 96 : num_experts <= 8 ? 56 : num_experts < kManyExperts ? 32 : 36;
}
int pick_variant(int32_t variant, int64_t pairs, int32_t num_experts, int64_t max_group_rows = -1) {
    if (variant == RMOE_VARIANT_STREAM || variant == RMOE_VARIANT_TILE) return variant;
    const int32_t E = num_experts;
    const bool few = pairs <= stream_max_avg_rows(E) * (int64_t)E;
    const bool fits = max_group_rows < 0 || max_group_rows <= kStreamMaxGroupRows || E >= kManyExperts;
    const bool one_pass =
        max_group_rows >= 0 && E <= kManyExperts &&
        (max_group_rows <= 64 || (max_group_rows <= 96 && pairs <= (E <= 8 ? 80 : 48) * (int64_t)E));
    return (few && fits) || one_pass ? RMOE_VARIANT_STREAM : RMOE_VARIANT_TILE;
}
int to_status(hipError_t e) { return e == hipSuccess ? RMOE_OK : RMOE_ERR_LAUNCH; }

// Hand-over of the single launch.  AUTO hands hidden rows across XCDs: the
// XCD-local hand-over is correct on every shape but measured slower on all
// workloads (large 14.0 against 10.9 ms, fine 1.28-1.36 against 0.92 ms):
// a write-back L2 still writes every hidden row out, and running each
// entry's slices on one XCD raises the operand traffic beyond L2 by ~20%.
int pick_handover(int32_t handover) {
    return handover == RMOE_FUSED_LOCAL ? RMOE_FUSED_LOCAL : RMOE_FUSED_GLOBAL;
}
int gate_up_impl(const void *x, const void *gate_w, const void *up_w, const int32_t *gs,
                 const int32_t *gpo, const int32_t *gidx, void *workspace, int64_t hidden,
                 int64_t intermediate, int32_t E, int64_t Tp, int32_t M, int64_t pairs,
                 int32_t variant, void *stream) {
    rmoe::StageArgs a{};
    a.x = static_cast<const _Float16 *>(x);
    a.w0 = static_cast<const _Float16 *>(gate_w);
    a.w1 = static_cast<const _Float16 *>(up_w);
    a.gs = gs;
    a.gpo = gpo;
    a.gidx = gidx;
    a.y = static_cast<_Float16 *>(workspace);
    a.K = hidden;
    a.N = intermediate;
    a.E = E;
    a.M = M;
    a.pairs = pairs;
    (void)Tp;
    if (M == 0) return RMOE_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (pick_variant(variant, pairs, E) == RMOE_VARIANT_STREAM)
        return to_status(rmoe::launch_stream_gate_up(a, s));
    return to_status(rmoe::launch_tile_gate_up(a, s));
}

int down_impl(const void *workspace, const void *down_w, const float *rw, const int32_t *gs,
              const int32_t *go, const int32_t *gpo, const int32_t *gidx, void *out,
              int64_t hidden, int64_t intermediate, int32_t E, int64_t Tp, int32_t M,
              int64_t pairs, int32_t variant, void *stream) {
    rmoe::StageArgs a{};
    a.x = static_cast<const _Float16 *>(workspace);
    a.w0 = static_cast<const _Float16 *>(down_w);
    a.rw = rw;
    a.gs = gs;
    a.go = go;
    a.gpo = gpo;
    a.gidx = gidx;
    a.y = static_cast<_Float16 *>(out);
    a.K = intermediate;
    a.N = hidden;
    a.E = E;
    a.M = M;
    a.pairs = pairs;
    (void)Tp;
    if (M == 0) return RMOE_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (pick_variant(variant, pairs, E) == RMOE_VARIANT_STREAM)
        return to_status(rmoe::launch_stream_down(a, s));
    return to_status(rmoe::launch_tile_down(a, s));
}

bool bad_variant(int32_t v) {
    return v != RMOE_VARIANT_AUTO && v != RMOE_VARIANT_STREAM && v != RMOE_VARIANT_TILE;
}

}  // namespace

extern "C" {

const char *rmoe_status_str(int status) {
    switch (status) {
        case RMOE_OK: return "ok";
        case RMOE_ERR_INVALID_ARGUMENT: return "invalid argument";
        case RMOE_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
        case RMOE_ERR_MISALIGNED: return "misaligned pointer";
        case RMOE_ERR_LAUNCH: return "kernel launch failed";
        case RMOE_ERR_CONTRACT: return "tables violate the dispatch contract";
        case RMOE_ERR_CAPACITY: return "output table too small";
        case RMOE_ERR_SCRATCH: return "batch exceeds the library's static scratch";
        default: return "unknown status";
    }
}

const char *rmoe_version(void) { return "routed_moe 0.1 gfx950"; }

int rmoe_build_contract(const int32_t *topk_ids, int64_t num_tokens, int32_t top_k,
                        int32_t num_experts, int32_t *group_sizes, int32_t *group_offsets,
                        int32_t *group_padded_offsets, int32_t *group_idx_for_bx,
                        int64_t capacity_blocks, int32_t *num_blocks_m, int32_t *order,
                        int32_t *padded_row_of_pair, int32_t *compact_pos_of_pair) {
    if (num_tokens < 0 || top_k < 0 || num_experts < 1 || !group_sizes || !group_offsets ||
        !group_padded_offsets || !num_blocks_m || (num_tokens > 0 && top_k > 0 && !topk_ids))
        return RMOE_ERR_INVALID_ARGUMENT;
    const int64_t pairs = num_tokens * top_k;
    if (pairs > INT32_MAX / 2) return RMOE_ERR_INVALID_ARGUMENT;
    const int32_t E = num_experts;
    // every padded row index (up to 128*M) must fit the int32 tables
    const int64_t M = ceil_div(pairs, B) + E;
    if (M * B > INT32_MAX) return RMOE_ERR_INVALID_ARGUMENT;
    if (capacity_blocks < M || (M > 0 && !group_idx_for_bx)) return RMOE_ERR_CAPACITY;
    // counts (and id range check before anything is written)
    std::vector<int64_t> cnt(E, 0);
    for (int64_t p = 0; p < pairs; ++p) {
        const int32_t e = topk_ids[p];
        if (e < 0 || e >= E) return RMOE_ERR_INVALID_ARGUMENT;
        cnt[e]++;
    }
    // compact and padded offsets (E+1 entries each)
    group_offsets[0] = 0;
    group_padded_offsets[0] = 0;
    for (int32_t e = 0; e < E; ++e) {
        group_sizes[e] = (int32_t)cnt[e];
        group_offsets[e + 1] = group_offsets[e] + (int32_t)cnt[e];
        group_padded_offsets[e + 1] = group_padded_offsets[e] + (int32_t)(ceil_div(cnt[e] + 1, B) * B);
    }
    *num_blocks_m = (int32_t)M;
    // block -> last expert whose padded start is <= bx*128 (starts strictly increase)
    int32_t e = 0;
    for (int64_t bx = 0; bx < M; ++bx) {
        while (e + 1 < E && (int64_t)group_padded_offsets[e + 1] <= bx * B) ++e;
        group_idx_for_bx[bx] = e;
    }
    // stable counting sort of the pairs by expert
    std::vector<int32_t> next(group_offsets, group_offsets + E);
    for (int64_t p = 0; p < pairs; ++p) {
        const int32_t ex = topk_ids[p];
        const int32_t c = next[ex]++;
        const int32_t rank = c - group_offsets[ex];
        if (order) order[c] = (int32_t)p;
        if (padded_row_of_pair) padded_row_of_pair[p] = group_padded_offsets[ex] + rank;
        if (compact_pos_of_pair) compact_pos_of_pair[p] = c;
    }
    return RMOE_OK;
}

int rmoe_validate_contract(const int32_t *gs, const int32_t *go, const int32_t *gpo,
                           const int32_t *gidx, int32_t E, int32_t M, int64_t Tp, int64_t pairs) {
    if (!gs || !go || !gpo || E < 1 || M < 0 || (M > 0 && !gidx)) return RMOE_ERR_INVALID_ARGUMENT;
    if (go[0] != 0 || gpo[0] != 0) return RMOE_ERR_CONTRACT;
    for (int32_t e = 0; e < E; ++e) {
        if (gs[e] < 0) return RMOE_ERR_CONTRACT;
        if ((int64_t)go[e + 1] - go[e] != gs[e]) return RMOE_ERR_CONTRACT;
        if ((int64_t)gpo[e + 1] - gpo[e] != ((int64_t)gs[e] / B + 1) * B) return RMOE_ERR_CONTRACT;
    }
    if ((int64_t)go[E] != pairs) return RMOE_ERR_CONTRACT;
    if ((int64_t)M != ceil_div(pairs, B) + E) return RMOE_ERR_CONTRACT;
    if ((int64_t)gpo[E] > (int64_t)M * B || (int64_t)M * B > Tp) return RMOE_ERR_CONTRACT;
    int32_t e = 0;
    for (int64_t bx = 0; bx < M; ++bx) {
        while (e + 1 < E && (int64_t)gpo[e + 1] <= bx * B) ++e;
        if (gidx[bx] != e) return RMOE_ERR_CONTRACT;
    }
    return RMOE_OK;
}

size_t rmoe_workspace_bytes(int64_t total_padded_tokens, int64_t intermediate) {
    if (total_padded_tokens <= 0 || intermediate <= 0) return 0;
    return (size_t)total_padded_tokens * (size_t)intermediate * 2u;
}

int rmoe_contract_sizes(int64_t num_pairs, int32_t num_experts, int32_t *num_blocks_m,
                        int64_t *total_padded_tokens) {
    if (num_pairs < 0 || num_experts < 1 || num_pairs > INT32_MAX / 2)
        return RMOE_ERR_INVALID_ARGUMENT;
    const int64_t M = ceil_div(num_pairs, B) + num_experts;
    if (M * B > INT32_MAX) return RMOE_ERR_INVALID_ARGUMENT;
    if (num_blocks_m) *num_blocks_m = (int32_t)M;
    if (total_padded_tokens) *total_padded_tokens = M * B;
    return RMOE_OK;
}

int rmoe_pick_variant(int32_t variant, int64_t num_pairs, int32_t num_experts,
                      int64_t max_group_rows) {
    if (bad_variant(variant) || num_pairs < 0 || num_experts < 1 || max_group_rows > num_pairs)
        return RMOE_ERR_INVALID_ARGUMENT;
    return pick_variant(variant, num_pairs, num_experts, max_group_rows);
}

int rmoe_validate_contract_device(const int32_t *gs, const int32_t *go, const int32_t *gpo,
                                  const int32_t *gidx, int32_t num_experts, int32_t num_blocks_m,
                                  int64_t total_padded_tokens, int64_t total_valid_tokens,
                                  int32_t *violations, void *stream) {
    if (!gs || !go || !gpo || !violations || num_experts < 1 || num_blocks_m < 0 ||
        total_valid_tokens < 0 || (num_blocks_m > 0 && !gidx))
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned4(gs) || !aligned4(go) || !aligned4(gpo) || !aligned4(gidx) || !aligned4(violations))
        return RMOE_ERR_MISALIGNED;
    // the size rules need no table: they are checked here, synchronously
    if (total_valid_tokens > INT32_MAX / 2 ||
        (int64_t)num_blocks_m != ceil_div(total_valid_tokens, B) + num_experts ||
        (int64_t)num_blocks_m * B > total_padded_tokens)
        return RMOE_ERR_CONTRACT;
    return to_status(rmoe::launch_validate(gs, go, gpo, gidx, num_experts, num_blocks_m,
                                           total_valid_tokens, violations,
                                           static_cast<hipStream_t>(stream)));
}

int rmoe_gate_up_f16(const void *x, const void *gate_w, const void *up_w, const int32_t *gs,
                     const int32_t *gpo, const int32_t *gidx, void *workspace, int64_t hidden,
                     int64_t intermediate, int32_t num_experts, int64_t total_padded_tokens,
                     int64_t total_valid_tokens, int32_t num_blocks_m, int32_t variant,
                     void *stream) {
    int st = check_dims(hidden, intermediate, num_experts, total_padded_tokens, num_blocks_m);
    if (st != RMOE_OK) return st;
    if (bad_variant(variant) || total_valid_tokens < 0) return RMOE_ERR_INVALID_ARGUMENT;
    if (!x || !gate_w || !up_w || !gs || !gpo || !workspace || (num_blocks_m > 0 && !gidx))
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(gate_w) || !aligned16(up_w) || !aligned16(workspace) ||
        !aligned4(gs) || !aligned4(gpo) || !aligned4(gidx))
        return RMOE_ERR_MISALIGNED;
    // the same family choice as rmoe_down_f16 and the forward for this batch
    return gate_up_impl(x, gate_w, up_w, gs, gpo, gidx, workspace, hidden, intermediate,
                        num_experts, total_padded_tokens, num_blocks_m, total_valid_tokens,
                        variant, stream);
}

int rmoe_down_f16(const void *workspace, const void *down_w, const float *rw, const int32_t *gs,
                  const int32_t *go, const int32_t *gpo, const int32_t *gidx, void *out,
                  int64_t hidden, int64_t intermediate, int32_t num_experts,
                  int64_t total_padded_tokens, int64_t total_valid_tokens, int32_t num_blocks_m,
                  int32_t variant, void *stream) {
    int st = check_dims(hidden, intermediate, num_experts, total_padded_tokens, num_blocks_m);
    if (st != RMOE_OK) return st;
    if (bad_variant(variant) || total_valid_tokens < 0) return RMOE_ERR_INVALID_ARGUMENT;
    if (!workspace || !down_w || !gs || !go || !gpo || !out || (num_blocks_m > 0 && !gidx) ||
        (total_valid_tokens > 0 && !rw))
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(workspace) || !aligned16(down_w) || !aligned16(out) || !aligned4(rw) ||
        !aligned4(gs) || !aligned4(go) || !aligned4(gpo) || !aligned4(gidx))
        return RMOE_ERR_MISALIGNED;
    return down_impl(workspace, down_w, rw, gs, go, gpo, gidx, out, hidden, intermediate,
                     num_experts, total_padded_tokens, num_blocks_m, total_valid_tokens, variant,
                     stream);
}

int rmoe_forward_f16_variant(const void *x, const void *gate_w, const void *up_w,
                             const void *down_w, const float *rw, const int32_t *gs,
                             const int32_t *go, const int32_t *gpo, const int32_t *gidx,
                             void *workspace, void *out, int64_t hidden, int64_t intermediate,
                             int32_t num_experts, int64_t total_padded_tokens,
                             int64_t total_valid_tokens, int32_t num_blocks_m, int32_t variant,
                             void *stream) {
    int st = check_dims(hidden, intermediate, num_experts, total_padded_tokens, num_blocks_m);
    if (st != RMOE_OK) return st;
    if (bad_variant(variant) || total_valid_tokens < 0) return RMOE_ERR_INVALID_ARGUMENT;
    if (!x || !gate_w || !up_w || !down_w || !gs || !go || !gpo || !workspace || !out ||
        (num_blocks_m > 0 && !gidx) || (total_valid_tokens > 0 && !rw))
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(gate_w) || !aligned16(up_w) || !aligned16(down_w) ||
        !aligned16(workspace) || !aligned16(out) || !aligned4(rw) || !aligned4(gs) ||
        !aligned4(go) || !aligned4(gpo) || !aligned4(gidx))
        return RMOE_ERR_MISALIGNED;
    const int v = pick_variant(variant, total_valid_tokens, num_experts);
    st = gate_up_impl(x, gate_w, up_w, gs, gpo, gidx, workspace, hidden, intermediate,
                      num_experts, total_padded_tokens, num_blocks_m, total_valid_tokens, v,
                      stream);
    if (st != RMOE_OK) return st;
    return down_impl(workspace, down_w, rw, gs, go, gpo, gidx, out, hidden, intermediate,
                     num_experts, total_padded_tokens, num_blocks_m, total_valid_tokens, v,
                     stream);
}

int rmoe_forward_f16(const void *x, const void *gate_w, const void *up_w, const void *down_w,
                     const float *rw, const int32_t *gs, const int32_t *go, const int32_t *gpo,
                     const int32_t *gidx, void *workspace, void *out, int64_t hidden,
                     int64_t intermediate, int32_t num_experts, int64_t total_padded_tokens,
                     int64_t total_valid_tokens, int32_t num_blocks_m, void *stream) {
    return rmoe_forward_f16_variant(x, gate_w, up_w, down_w, rw, gs, go, gpo, gidx, workspace,
                                    out, hidden, intermediate, num_experts, total_padded_tokens,
                                    total_valid_tokens, num_blocks_m, RMOE_VARIANT_AUTO, stream);
}

size_t rmoe_fused_sync_words(int32_t num_blocks_m) {
    return num_blocks_m < 0 ? 0 : (size_t)RMOE_FUSED_SYNC_HEAD + (size_t)num_blocks_m;
}

int rmoe_forward_fused_f16(const void *x, const void *gate_w, const void *up_w,
                           const void *down_w, const float *rw, const int32_t *gs,
                           const int32_t *go, const int32_t *gpo, const int32_t *gidx,
                           void *workspace, void *out, int32_t *sync, int64_t hidden,
                           int64_t intermediate, int32_t num_experts, int64_t total_padded_tokens,
                           int64_t total_valid_tokens, int32_t num_blocks_m, int32_t max_wait_us,
                           int32_t handover, void *stream) {
    int st = check_dims(hidden, intermediate, num_experts, total_padded_tokens, num_blocks_m);
    if (st != RMOE_OK) return st;
    if (total_valid_tokens < 0 || handover < RMOE_FUSED_AUTO || handover > RMOE_FUSED_GLOBAL)
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!x || !gate_w || !up_w || !down_w || !gs || !go || !gpo || !workspace || !out || !sync ||
        (num_blocks_m > 0 && !gidx) || (total_valid_tokens > 0 && !rw))
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(gate_w) || !aligned16(up_w) || !aligned16(down_w) ||
        !aligned16(workspace) || !aligned16(out) || !aligned4(rw) || !aligned4(gs) ||
        !aligned4(go) || !aligned4(gpo) || !aligned4(gidx) || !aligned4(sync))
        return RMOE_ERR_MISALIGNED;
    if (num_blocks_m == 0) return RMOE_OK;
    rmoe::StageArgs gu{}, dn{};
    gu.x = static_cast<const _Float16 *>(x);
    gu.w0 = static_cast<const _Float16 *>(gate_w);
    gu.w1 = static_cast<const _Float16 *>(up_w);
    gu.y = static_cast<_Float16 *>(workspace);
    gu.K = hidden;
    gu.N = intermediate;
    dn.x = static_cast<const _Float16 *>(workspace);
    dn.w0 = static_cast<const _Float16 *>(down_w);
    dn.rw = rw;
    dn.y = static_cast<_Float16 *>(out);
    dn.K = intermediate;
    dn.N = hidden;
    for (rmoe::StageArgs *a : {&gu, &dn}) {
        a->gs = gs;
        a->go = go;
        a->gpo = gpo;
        a->gidx = gidx;
        a->E = num_experts;
        a->M = num_blocks_m;
        a->pairs = total_valid_tokens;
    }
    const int64_t wait_us = max_wait_us > 0 ? max_wait_us : kFusedWaitUs;
    const bool local = pick_handover(handover) == RMOE_FUSED_LOCAL;
    return to_status(
        rmoe::launch_fused(gu, dn, sync, wait_us, local, static_cast<hipStream_t>(stream)));
}

int rmoe_pack_f16(const void *x, const float *topk_weights, const int32_t *prow,
                  const int32_t *cpos, int64_t num_tokens, int32_t top_k, int64_t hidden,
                  void *stacked, float *w_compact, int64_t total_padded_tokens, void *stream) {
    if (num_tokens < 0 || top_k < 0 || hidden <= 0 || total_padded_tokens < 0)
        return RMOE_ERR_INVALID_ARGUMENT;
    if (hidden % 8 != 0 || hidden / 8 > ((int64_t)1 << 30)) return RMOE_ERR_UNSUPPORTED_SHAPE;
    const int64_t pairs = num_tokens * top_k;
    if (pairs == 0) return RMOE_OK;
    if (!x || !topk_weights || !prow || !cpos || !stacked || !w_compact)
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(stacked) || !aligned4(topk_weights) || !aligned4(prow) ||
        !aligned4(cpos) || !aligned4(w_compact))
        return RMOE_ERR_MISALIGNED;
    return to_status(rmoe::launch_pack(static_cast<const _Float16 *>(x), topk_weights, prow, cpos,
                                       pairs, top_k, hidden, total_padded_tokens,
                                       static_cast<_Float16 *>(stacked), w_compact,
                                       static_cast<hipStream_t>(stream)));
}

int rmoe_combine_f16(const void *out, const int32_t *prow, int64_t num_tokens, int32_t top_k,
                     int64_t hidden, void *y, int64_t total_padded_tokens, void *stream) {
    if (num_tokens < 0 || top_k < 0 || hidden <= 0 || total_padded_tokens < 0)
        return RMOE_ERR_INVALID_ARGUMENT;
    if (hidden % 8 != 0 || hidden / 8 > ((int64_t)1 << 30)) return RMOE_ERR_UNSUPPORTED_SHAPE;
    if (num_tokens == 0) return RMOE_OK;
    if (!y || (top_k > 0 && (!out || !prow))) return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(y) || !aligned16(out) || !aligned4(prow)) return RMOE_ERR_MISALIGNED;
    return to_status(rmoe::launch_combine(static_cast<const _Float16 *>(out), prow, num_tokens,
                                          top_k, hidden, total_padded_tokens,
                                          static_cast<_Float16 *>(y), static_cast<hipStream_t>(stream)));
}

// ---- device-side contract ------------------------------------------------

size_t rmoe_contract_workspace_bytes(int64_t num_pairs, int32_t num_experts) {
    if (num_pairs < 0 || num_experts < 1 || num_experts > kMaxDeviceExperts) return 0;
    const int64_t nch = rmoe::contract_chunks(num_pairs);
    const size_t n = (size_t)(nch * ((int64_t)num_experts + 1));
    return n > 0 ? n * sizeof(int32_t) : 4;
}

}  // extern "C"

namespace {

// Argument checks of the device contract build (both entry points), before
// any HIP call; on success *M holds the block count.  The scratch is
// checked by the caller.
int check_contract_device(const int32_t *topk_ids, int64_t num_tokens, int32_t top_k,
                          int32_t num_experts, const int32_t *group_sizes,
                          const int32_t *group_offsets, const int32_t *group_padded_offsets,
                          const int32_t *group_idx_for_bx, int64_t capacity_blocks,
                          const int32_t *num_blocks_m, const int32_t *order,
                          const int32_t *padded_row_of_pair, const int32_t *compact_pos_of_pair,
                          const int32_t *bad_ids, int64_t *M) {
    if (num_tokens < 0 || top_k < 0 || num_experts < 1 || !num_blocks_m) return RMOE_ERR_INVALID_ARGUMENT;
    if (num_experts > kMaxDeviceExperts) return RMOE_ERR_UNSUPPORTED_SHAPE;
    const int64_t pairs = num_tokens * top_k;
    if (pairs > INT32_MAX / 2) return RMOE_ERR_INVALID_ARGUMENT;
    *M = ceil_div(pairs, B) + num_experts;
    if (*M * B > INT32_MAX) return RMOE_ERR_INVALID_ARGUMENT;
    if (!group_sizes || !group_offsets || !group_padded_offsets || !group_idx_for_bx || !bad_ids)
        return RMOE_ERR_INVALID_ARGUMENT;
    if (pairs > 0 && (!topk_ids || !order || !padded_row_of_pair || !compact_pos_of_pair))
        return RMOE_ERR_INVALID_ARGUMENT;
    if (capacity_blocks < *M) return RMOE_ERR_CAPACITY;
    if (!aligned4(topk_ids) || !aligned4(group_sizes) || !aligned4(group_offsets) ||
        !aligned4(group_padded_offsets) || !aligned4(group_idx_for_bx) || !aligned4(order) ||
        !aligned4(padded_row_of_pair) || !aligned4(compact_pos_of_pair) || !aligned4(bad_ids))
        return RMOE_ERR_MISALIGNED;
    return RMOE_OK;
}

}  // namespace

extern "C" {

int rmoe_build_contract_device(const int32_t *topk_ids, int64_t num_tokens, int32_t top_k,
                               int32_t num_experts, int32_t *group_sizes, int32_t *group_offsets,
                               int32_t *group_padded_offsets, int32_t *group_idx_for_bx,
                               int64_t capacity_blocks, int32_t *num_blocks_m, int32_t *order,
                               int32_t *padded_row_of_pair, int32_t *compact_pos_of_pair,
                               int32_t *bad_ids, void *workspace, size_t workspace_bytes,
                               void *stream) {
    int64_t M = 0;
    int st = check_contract_device(topk_ids, num_tokens, top_k, num_experts, group_sizes,
                                   group_offsets, group_padded_offsets, group_idx_for_bx,
                                   capacity_blocks, num_blocks_m, order, padded_row_of_pair,
                                   compact_pos_of_pair, bad_ids, &M);
    if (st != RMOE_OK) return st;
    const int64_t pairs = num_tokens * top_k;
    if (!workspace) return RMOE_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < rmoe_contract_workspace_bytes(pairs, num_experts)) return RMOE_ERR_CAPACITY;
    if (!aligned4(workspace)) return RMOE_ERR_MISALIGNED;
    *num_blocks_m = (int32_t)M;
    return to_status(rmoe::launch_contract(topk_ids, pairs, num_experts, (int32_t)M, group_sizes,
                                           group_offsets, group_padded_offsets, group_idx_for_bx,
                                           order, padded_row_of_pair, compact_pos_of_pair, bad_ids,
                                           static_cast<int32_t *>(workspace),
                                           static_cast<hipStream_t>(stream)));
}

size_t rmoe_contract_noalloc_max_words(void) { return (size_t)rmoe::kNoAllocScratchWords; }

int rmoe_build_contract_device_noalloc(const int32_t *topk_ids, int64_t num_tokens, int32_t top_k,
                                       int32_t num_experts, int32_t *group_sizes,
                                       int32_t *group_offsets, int32_t *group_padded_offsets,
                                       int32_t *group_idx_for_bx, int64_t capacity_blocks,
                                       int32_t *num_blocks_m, int32_t *order,
                                       int32_t *padded_row_of_pair, int32_t *compact_pos_of_pair,
                                       int32_t *bad_ids, void *stream) {
    int64_t M = 0;
    int st = check_contract_device(topk_ids, num_tokens, top_k, num_experts, group_sizes,
                                   group_offsets, group_padded_offsets, group_idx_for_bx,
                                   capacity_blocks, num_blocks_m, order, padded_row_of_pair,
                                   compact_pos_of_pair, bad_ids, &M);
    if (st != RMOE_OK) return st;
    const int64_t pairs = num_tokens * top_k;
    // the scratch this batch needs, against the static array (nothing is allocated)
    const size_t cap = (size_t)rmoe::kNoAllocScratchWords * sizeof(int32_t);
    if (rmoe_contract_workspace_bytes(pairs, num_experts) > cap) return RMOE_ERR_SCRATCH;
    int32_t *ws = nullptr;  // this device's copy of the static scratch
    if (rmoe::noalloc_scratch(&ws) != hipSuccess) return RMOE_ERR_LAUNCH;
    *num_blocks_m = (int32_t)M;
    return to_status(rmoe::launch_contract(topk_ids, pairs, num_experts, (int32_t)M, group_sizes,
                                           group_offsets, group_padded_offsets, group_idx_for_bx,
                                           order, padded_row_of_pair, compact_pos_of_pair, bad_ids,
                                           ws, static_cast<hipStream_t>(stream)));
}

// ---- router ----------------------------------------------------------------

int rmoe_router_f16(const void *x, const void *router_w, int64_t num_tokens, int64_t hidden,
                    int32_t num_experts, int32_t top_k, int32_t *topk_ids, float *topk_weights,
                    void *stream) {
    if (num_tokens < 0 || hidden <= 0 || num_experts < 1 || top_k < 0 || top_k > num_experts)
        return RMOE_ERR_INVALID_ARGUMENT;
    if (num_experts > 256 || top_k > 32 || hidden % 64 != 0) return RMOE_ERR_UNSUPPORTED_SHAPE;
    if (num_tokens == 0 || top_k == 0) return RMOE_OK;
    if (!x || !router_w || !topk_ids || !topk_weights) return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(router_w) || !aligned4(topk_ids) || !aligned4(topk_weights))
        return RMOE_ERR_MISALIGNED;
    return to_status(rmoe::launch_router(static_cast<const _Float16 *>(x),
                                         static_cast<const _Float16 *>(router_w), num_tokens, hidden,
                                         num_experts, top_k, topk_ids, topk_weights,
                                         static_cast<hipStream_t>(stream)));
}

// Sizes of the training router, forward and backward.
static int check_router_train(int64_t num_tokens, int64_t hidden, int32_t num_experts, int32_t top_k) {
    if (num_tokens < 0 || hidden <= 0 || num_experts < 1 || top_k < 1 || top_k > num_experts)
        return RMOE_ERR_INVALID_ARGUMENT;
    if (num_experts > 256 || top_k > 32 || hidden % 64 != 0 || hidden > (int64_t)1 << 20 ||
        num_tokens > INT32_MAX / top_k)
        return RMOE_ERR_UNSUPPORTED_SHAPE;
    return RMOE_OK;
}

size_t rmoe_router_train_scratch_bytes(int64_t num_tokens, int32_t num_experts) {
    if (num_tokens <= 0 || num_experts < 1 || num_experts > 256 || num_tokens > INT32_MAX) return 0;
    return (size_t)rmoe::router_train_parts(num_tokens) * (2u * (size_t)num_experts + 2u) * 4u;
}

int rmoe_router_train_f16(const void *x, const void *router_w, const uint8_t *token_mask, int64_t num_tokens,
                          int64_t hidden, int32_t num_experts, int32_t top_k, int32_t *topk_ids, float *topk_weights,
                          float *probs, float *lse, int32_t *counts, float *losses, void *scratch, void *stream) {
    const int st = check_router_train(num_tokens, hidden, num_experts, top_k);
    if (st != RMOE_OK) return st;
    if (!router_w || !counts || !losses ||
        (num_tokens > 0 && (!x || !topk_ids || !topk_weights || !probs || !lse || !scratch)))
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(router_w) || !aligned4(topk_ids) || !aligned4(topk_weights) || !aligned4(probs) ||
        !aligned4(lse) || !aligned4(counts) || !aligned4(losses) || (reinterpret_cast<uintptr_t>(scratch) & 7u))
        return RMOE_ERR_MISALIGNED;
    rmoe::RouterTrainArgs a{};
    a.x = static_cast<const _Float16 *>(x), a.w = static_cast<const _Float16 *>(router_w), a.mask = token_mask;
    a.T = num_tokens, a.H = hidden, a.E = num_experts, a.k = top_k;
    a.ids = topk_ids, a.vals = topk_weights, a.probs = probs, a.lse = lse, a.counts = counts, a.losses = losses;
    const int64_t parts = rmoe::router_train_parts(num_tokens);
    a.parts = static_cast<rmoe::RouterPart *>(scratch);
    a.tokens = a.parts + parts * num_experts;
    return to_status(rmoe::launch_router_train(a, static_cast<hipStream_t>(stream)));
}

size_t rmoe_router_backward_scratch_bytes(int64_t num_tokens, int64_t hidden, int32_t num_experts) {
    if (check_router_train(num_tokens, hidden, num_experts, 1) != RMOE_OK) return 0;
    return (size_t)rmoe::router_backward_scratch(num_tokens, hidden, num_experts);
}

int rmoe_router_backward_f16(const void *x, const void *router_w, const uint8_t *token_mask, const int32_t *topk_ids,
                             const float *probs, const float *lse, const int32_t *counts, const float *drw,
                             const int32_t *compact_pos_of_pair, const float *dlosses, const void *dx_add, void *dx,
                             float *drouter_w, void *scratch, int64_t num_tokens, int64_t hidden, int32_t num_experts,
                             int32_t top_k, void *stream) {
    const int st = check_router_train(num_tokens, hidden, num_experts, top_k);
    if (st != RMOE_OK) return st;
    if (!router_w || !counts || !drouter_w || !scratch ||
        (num_tokens > 0 && (!x || !topk_ids || !probs || !lse || !drw || !dx)))
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(router_w) || !aligned16(dx_add) || !aligned16(dx) || !aligned16(drouter_w) ||
        !aligned16(scratch) || !aligned4(topk_ids) || !aligned4(probs) || !aligned4(lse) || !aligned4(counts) ||
        !aligned4(drw) || !aligned4(compact_pos_of_pair) || !aligned4(dlosses))
        return RMOE_ERR_MISALIGNED;
    rmoe::RouterBackArgs a{};
    a.x = static_cast<const _Float16 *>(x), a.w = static_cast<const _Float16 *>(router_w), a.mask = token_mask;
    a.ids = topk_ids, a.probs = probs, a.lse = lse, a.counts = counts, a.drw = drw, a.cpos = compact_pos_of_pair;
    a.dlosses = dlosses, a.add = static_cast<const _Float16 *>(dx_add), a.dx = static_cast<_Float16 *>(dx);
    a.dw = drouter_w, a.scratch = static_cast<unsigned char *>(scratch);
    a.T = num_tokens, a.H = hidden, a.E = num_experts, a.k = top_k;
    return to_status(rmoe::launch_router_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- MXFP4 -----------------------------------------------------------------

namespace {

bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
int64_t mx_chunks(int64_t cols) { return ceil_div(cols, 256); }
bool bad_type(int32_t t) { return t != RMOE_TYPE_F16 && t != RMOE_TYPE_BF16 && t != RMOE_TYPE_F32; }
rmoe::MxType mx_type(int32_t t) {
    return t == RMOE_TYPE_F16 ? rmoe::MxType::f16 : t == RMOE_TYPE_BF16 ? rmoe::MxType::bf16 : rmoe::MxType::f32;
}

// Sizes of a quantisation: RMOE_OK with *empty set where there is nothing to do.
int check_mx_sizes(int32_t type, int64_t batch, int64_t rows, int64_t cols, bool *empty) {
    if (bad_type(type) || batch < 0 || rows < 0 || cols <= 0) return RMOE_ERR_INVALID_ARGUMENT;
    if (cols % 8 != 0) return RMOE_ERR_UNSUPPORTED_SHAPE;
    *empty = batch == 0 || rows == 0;
    int64_t n = 0, u = 0;
    if (__builtin_mul_overflow(batch, rows, &n) || __builtin_mul_overflow(n, mx_chunks(cols), &u) || u > INT32_MAX)
        return RMOE_ERR_UNSUPPORTED_SHAPE;
    return RMOE_OK;
}

// Streaming reads an expert's weights once per 64 rows of each of its blocks.
// Forward times of both families (one MI355X): E=8 (4096, 14336) streams 32%
// faster at 48 rows per expert and 4% at 64, tiles 24% faster at 96; E=2 (same
// sizes) streams 38% faster at 64 and tiles 6% faster at 96; E=64 (2048, 1408)
// streams 19% faster at 48 (25% under Zipf 1.2) and tiles 6% faster at 64 (13%
// slower under Zipf); E=128 (7168, 2048) streams 12% faster at 48 and tiles
// 28% faster at 64.
int pick_variant_mx(int32_t variant, int64_t pairs, int32_t num_experts) {
    if (variant == RMOE_VARIANT_STREAM || variant == RMOE_VARIANT_TILE) return variant;
    return pairs <= (num_experts <= 8 ? 64 : 48) * (int64_t)num_experts ? RMOE_VARIANT_STREAM : RMOE_VARIANT_TILE;
}

int mx_gate_up_impl(rmoe::MxArgs a, int32_t variant, int64_t pairs, void *stream) {
    if (a.M == 0) return RMOE_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (pick_variant_mx(variant, pairs, a.E) == RMOE_VARIANT_STREAM)
        return to_status(rmoe::launch_mx_stream_gate_up(a, pairs, s));
    return to_status(rmoe::launch_mx_tile_gate_up(a, s));
}

int mx_down_impl(rmoe::MxArgs a, int32_t variant, int64_t pairs, void *stream) {
    if (a.M == 0) return RMOE_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (pick_variant_mx(variant, pairs, a.E) == RMOE_VARIANT_STREAM)
        return to_status(rmoe::launch_mx_stream_down(a, pairs, s));
    return to_status(rmoe::launch_mx_tile_down(a, s));
}

const unsigned char *bytes(const void *p) { return static_cast<const unsigned char *>(p); }
unsigned char *bytes(void *p) { return static_cast<unsigned char *>(p); }

// The two stages' checked arguments.
int mx_gate_up_args(rmoe::MxArgs *a, const void *xc, const void *xs, const void *gc, const void *gsc, const void *uc,
                    const void *us, const int32_t *gs, const int32_t *gpo, const int32_t *gidx, void *hc, void *hs,
                    int64_t hidden, int64_t intermediate, int32_t E, int64_t Tp, int32_t M) {
    if (!xc || !xs || !gc || !gsc || !uc || !us || !gs || !gpo || (M > 0 && !gidx) || !hc || !hs)
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(xc) || !aligned16(gc) || !aligned16(uc) || !aligned16(hc) || !aligned16(xs) || !aligned16(gsc) ||
        !aligned16(us) || !aligned16(hs) || !aligned4(gs) || !aligned4(gpo) || !aligned4(gidx))
        return RMOE_ERR_MISALIGNED;
    a->x = bytes(xc), a->xs = bytes(xs);
    a->w0 = bytes(gc), a->w0s = bytes(gsc), a->w1 = bytes(uc), a->w1s = bytes(us);
    a->gs = gs, a->gpo = gpo, a->gidx = gidx;
    a->yc = bytes(hc), a->ys = bytes(hs);
    a->N = intermediate, a->Tp = Tp, a->kc = (int32_t)mx_chunks(hidden), a->E = E, a->M = M;
    return RMOE_OK;
}

int mx_down_args(rmoe::MxArgs *a, const void *hc, const void *hs, const void *dc, const void *ds, const float *rw,
                 const int32_t *gs, const int32_t *go, const int32_t *gpo, const int32_t *gidx, void *out,
                 int64_t hidden, int64_t intermediate, int32_t E, int64_t Tp, int64_t pairs, int32_t M) {
    if (!hc || !hs || !dc || !ds || !gs || !go || !gpo || (M > 0 && !gidx) || !out || (pairs > 0 && !rw))
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(hc) || !aligned16(hs) || !aligned16(dc) || !aligned16(ds) || !aligned16(out) || !aligned4(rw) ||
        !aligned4(gs) || !aligned4(go) || !aligned4(gpo) || !aligned4(gidx))
        return RMOE_ERR_MISALIGNED;
    a->x = bytes(hc), a->xs = bytes(hs), a->w0 = bytes(dc), a->w0s = bytes(ds), a->rw = rw;
    a->gs = gs, a->go = go, a->gpo = gpo, a->gidx = gidx;
    a->y = static_cast<_Float16 *>(out);
    a->N = hidden, a->Tp = Tp, a->kc = (int32_t)mx_chunks(intermediate), a->E = E, a->M = M;
    return RMOE_OK;
}

int check_mx_dims(int64_t hidden, int64_t intermediate, int32_t E, int64_t Tp, int64_t pairs, int32_t M,
                  int32_t variant) {
    const int st = check_dims(hidden, intermediate, E, Tp, M);
    if (st != RMOE_OK) return st;
    if (bad_variant(variant) || pairs < 0) return RMOE_ERR_INVALID_ARGUMENT;
    // a chunk's token scales start 8 Tp bytes after the chunk's before: they
    // travel 16 bytes at a time, which an odd Tp would misalign
    return Tp % 2 ? RMOE_ERR_UNSUPPORTED_SHAPE : RMOE_OK;
}

}  // namespace

extern "C" {

int64_t rmoe_mxfp4_chunks(int64_t cols) { return cols <= 0 ? 0 : mx_chunks(cols); }
int64_t rmoe_mxfp4_row_bytes(int64_t cols) { return cols <= 0 ? 0 : 128 * mx_chunks(cols); }
size_t rmoe_mxfp4_code_bytes(int64_t rows, int64_t cols) {
    return rows <= 0 || cols <= 0 ? 0 : (size_t)rows * 128u * (size_t)mx_chunks(cols);
}
size_t rmoe_mxfp4_scale_bytes(int64_t rows, int64_t cols) {
    return rows <= 0 || cols <= 0 ? 0 : (size_t)rows * 8u * (size_t)mx_chunks(cols);
}

int rmoe_quantize_mxfp4(const void *x, int32_t type, int64_t batch, int64_t rows, int64_t cols, void *codes,
                        void *scales, void *stream) {
    bool empty = false;
    const int st = check_mx_sizes(type, batch, rows, cols, &empty);
    if (st != RMOE_OK) return st;
    if (empty) return RMOE_OK;
    if (!x || !codes || !scales) return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(codes) || !aligned8(scales)) return RMOE_ERR_MISALIGNED;
    return to_status(rmoe::launch_quantize(x, mx_type(type), batch, rows, cols, bytes(codes), bytes(scales),
                                           static_cast<hipStream_t>(stream)));
}

int rmoe_dequantize_mxfp4(const void *codes, const void *scales, int32_t type, int64_t batch, int64_t rows,
                          int64_t cols, void *y, void *stream) {
    bool empty = false;
    const int st = check_mx_sizes(type, batch, rows, cols, &empty);
    if (st != RMOE_OK) return st;
    if (empty) return RMOE_OK;
    if (!codes || !scales || !y) return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(y) || !aligned16(codes) || !aligned8(scales)) return RMOE_ERR_MISALIGNED;
    return to_status(rmoe::launch_dequantize(bytes(codes), bytes(scales), mx_type(type), batch, rows, cols, y,
                                             static_cast<hipStream_t>(stream)));
}

int rmoe_pack_mxfp4_f16(const void *x, const float *topk_weights, const int32_t *prow, const int32_t *cpos,
                        int64_t num_tokens, int32_t top_k, int64_t hidden, void *codes, void *scales,
                        float *w_compact, int64_t total_padded_tokens, void *stream) {
    if (top_k < 0 || total_padded_tokens < 0) return RMOE_ERR_INVALID_ARGUMENT;
    bool empty = false;
    const int st = check_mx_sizes(RMOE_TYPE_F16, 1, num_tokens, hidden, &empty);
    if (st != RMOE_OK) return st;
    if (empty || top_k == 0) return RMOE_OK;
    if (!x || !topk_weights || !prow || !cpos || !codes || !scales || !w_compact) return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(codes) || !aligned8(scales) || !aligned4(topk_weights) || !aligned4(prow) ||
        !aligned4(cpos) || !aligned4(w_compact))
        return RMOE_ERR_MISALIGNED;
    return to_status(rmoe::launch_pack_mx(static_cast<const _Float16 *>(x), topk_weights, prow, cpos, num_tokens,
                                          top_k, hidden, total_padded_tokens, bytes(codes), bytes(scales), w_compact,
                                          static_cast<hipStream_t>(stream)));
}

size_t rmoe_mxfp4_workspace_bytes(int64_t total_padded_tokens, int64_t intermediate) {
    return rmoe_mxfp4_code_bytes(total_padded_tokens, intermediate) +
           rmoe_mxfp4_scale_bytes(total_padded_tokens, intermediate);
}

int rmoe_pick_variant_mxfp4(int32_t variant, int64_t num_pairs, int32_t num_experts) {
    if (bad_variant(variant) || num_pairs < 0 || num_experts < 1) return RMOE_ERR_INVALID_ARGUMENT;
    return pick_variant_mx(variant, num_pairs, num_experts);
}

int rmoe_gate_up_mxfp4(const void *xc, const void *xs, const void *gc, const void *gsc, const void *uc,
                       const void *us, const int32_t *gs, const int32_t *gpo, const int32_t *gidx, void *hc, void *hs,
                       int64_t hidden, int64_t intermediate, int32_t num_experts, int64_t total_padded_tokens,
                       int64_t total_valid_tokens, int32_t num_blocks_m, int32_t variant, void *stream) {
    int st = check_mx_dims(hidden, intermediate, num_experts, total_padded_tokens, total_valid_tokens, num_blocks_m,
                           variant);
    if (st != RMOE_OK) return st;
    rmoe::MxArgs a{};
    st = mx_gate_up_args(&a, xc, xs, gc, gsc, uc, us, gs, gpo, gidx, hc, hs, hidden, intermediate, num_experts,
                         total_padded_tokens, num_blocks_m);
    return st != RMOE_OK ? st : mx_gate_up_impl(a, variant, total_valid_tokens, stream);
}

int rmoe_down_mxfp4(const void *hc, const void *hs, const void *dc, const void *ds, const float *rw,
                    const int32_t *gs, const int32_t *go, const int32_t *gpo, const int32_t *gidx, void *out,
                    int64_t hidden, int64_t intermediate, int32_t num_experts, int64_t total_padded_tokens,
                    int64_t total_valid_tokens, int32_t num_blocks_m, int32_t variant, void *stream) {
    int st = check_mx_dims(hidden, intermediate, num_experts, total_padded_tokens, total_valid_tokens, num_blocks_m,
                           variant);
    if (st != RMOE_OK) return st;
    rmoe::MxArgs a{};
    st = mx_down_args(&a, hc, hs, dc, ds, rw, gs, go, gpo, gidx, out, hidden, intermediate, num_experts,
                      total_padded_tokens, total_valid_tokens, num_blocks_m);
    return st != RMOE_OK ? st : mx_down_impl(a, variant, total_valid_tokens, stream);
}

int rmoe_forward_mxfp4(const void *xc, const void *xs, const void *gc, const void *gsc, const void *uc,
                       const void *us, const void *dc, const void *ds, const float *rw, const int32_t *gs,
                       const int32_t *go, const int32_t *gpo, const int32_t *gidx, void *workspace, void *out,
                       int64_t hidden, int64_t intermediate, int32_t num_experts, int64_t total_padded_tokens,
                       int64_t total_valid_tokens, int32_t num_blocks_m, int32_t variant, void *stream) {
    int st = check_mx_dims(hidden, intermediate, num_experts, total_padded_tokens, total_valid_tokens, num_blocks_m,
                           variant);
    if (st != RMOE_OK) return st;
    if (!workspace) return RMOE_ERR_INVALID_ARGUMENT;
    // the codes' bytes are a multiple of 128, so the scales keep the workspace's alignment
    void *hs = bytes(workspace) + rmoe_mxfp4_code_bytes(total_padded_tokens, intermediate);
    rmoe::MxArgs gu{}, dn{};
    st = mx_gate_up_args(&gu, xc, xs, gc, gsc, uc, us, gs, gpo, gidx, workspace, hs, hidden, intermediate, num_experts,
                         total_padded_tokens, num_blocks_m);
    if (st != RMOE_OK) return st;
    st = mx_down_args(&dn, workspace, hs, dc, ds, rw, gs, go, gpo, gidx, out, hidden, intermediate, num_experts,
                      total_padded_tokens, total_valid_tokens, num_blocks_m);
    if (st != RMOE_OK) return st;
    st = mx_gate_up_impl(gu, variant, total_valid_tokens, stream);
    return st != RMOE_OK ? st : mx_down_impl(dn, variant, total_valid_tokens, stream);
}

}  // extern "C"

// ---- 8-bit integers --------------------------------------------------------

namespace {

// 127^2 K must not pass 2^31 - 1
constexpr int64_t kMaxI8Sum = INT32_MAX / (127 * 127) / 128 * 128;

// Sizes of a quantisation: RMOE_OK with *empty set where there is nothing to do.
int check_i8_sizes(int32_t type, int64_t rows, int64_t cols, bool *empty) {
    if (bad_type(type) || rows < 0 || cols <= 0) return RMOE_ERR_INVALID_ARGUMENT;
    if (cols % 8 != 0) return RMOE_ERR_UNSUPPORTED_SHAPE;
    int64_t n = 0;
    if (__builtin_mul_overflow(rows, cols, &n) || n > (int64_t)1 << 56) return RMOE_ERR_UNSUPPORTED_SHAPE;
    *empty = rows == 0;
    return RMOE_OK;
}

// Streaming reads an expert's weights once per 64 rows of each of its blocks,
// so its time jumps where groups pass 64 rows; the tiles leave CUs idle where
// they are few.  The borders go by the experts and the rows per expert alone,
// although shapes differ, and so weigh losses against each other.  Forward
// times, the tiled family's over the streaming one's (one MI355X, weights from
// HBM; above 1 streaming is faster).  Equal groups of 64, 80 and 128 rows:
//   E=1  (4096, 14336) 1.41 0.95 0.85, (2048, 8192) 1.42 1.05 1.00,
//        (1024, 4096) 1.25 1.04 1.10, (7168, 2048) 2.53 1.77 1.60
//   E=2  (4096, 14336) 1.21 0.74 0.69, (2048, 8192) 1.24 0.91 0.86,
//        (7168, 2048) 2.38 1.65 1.50
//   E=4  (4096, 14336) 1.23 0.72 0.61, (1024, 4096) 1.24 0.99 0.85,
//        (4096, 2048) 2.12 1.45 0.96
// Equal groups of 40, 56 and 64 rows; Zipf 1.2 of 40, 56 and 64 on average:
//   E=8  (4096, 14336) 1.09 1.03 1.05; 0.83 0.77 0.71
//        (2048, 5632) 1.26 1.18 1.18; 1.06 0.97 0.89
// Equal groups of 32, 40 and 64 rows; Zipf 1.2 of 32, 40 and 64:
//   E=16  (4096, 14336) 1.04 0.99 0.94; 0.90 0.82 0.86
//   E=32  (4096, 2048) 1.17 1.14 1.09; 1.24 1.22 0.94
//   E=64  (2048, 1408) 1.14 1.09 1.08; 1.18 1.12 1.05
//   E=128 (7168, 2048) 1.07 1.01 0.96; 1.03 0.96 0.81
// What a border costs at most there: one expert of 4096 x 14336 with 128 rows
// streams in 139 us (tiles 118); two of 7168 x 2048 with 80 rows take the tiles
// in 104 us (streaming 63); 8 of 4096 x 14336 with 56 skewed rows stream in
// 429 us (tiles 331).  A caller who knows its shape may name the family.
int pick_variant_i8(int32_t variant, int64_t pairs, int32_t num_experts) {
    if (variant == RMOE_VARIANT_STREAM || variant == RMOE_VARIANT_TILE) return variant;
    const int64_t rows = num_experts == 1   ? 128
                         : num_experts <= 4 ? 64
                         : num_experts <= 8 ? 56
                         : num_experts < 32 ? 32
                                            : 40;
    return pairs <= rows * num_experts ? RMOE_VARIANT_STREAM : RMOE_VARIANT_TILE;
}

int i8_gate_up_impl(const rmoe::I8Args &a, int32_t variant, int64_t pairs, void *stream) {
    if (a.M == 0) return RMOE_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int st = to_status(pick_variant_i8(variant, pairs, a.E) == RMOE_VARIANT_STREAM
                                 ? rmoe::launch_i8_stream_gate_up(a, pairs, s)
                                 : rmoe::launch_i8_tile_gate_up(a, s));
    return st != RMOE_OK ? st : to_status(rmoe::launch_quantize_hidden_i8(a, pairs, s));
}

int i8_down_impl(const rmoe::I8Args &a, int32_t variant, int64_t pairs, void *stream) {
    if (a.M == 0) return RMOE_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (pick_variant_i8(variant, pairs, a.E) == RMOE_VARIANT_STREAM)
        return to_status(rmoe::launch_i8_stream_down(a, pairs, s));
    return to_status(rmoe::launch_i8_tile_down(a, pairs, s));
}

int check_i8_dims(int64_t hidden, int64_t intermediate, int32_t E, int64_t Tp, int64_t pairs, int32_t M,
                  int32_t variant) {
    const int st = check_dims(hidden, intermediate, E, Tp, M);
    if (st != RMOE_OK) return st;
    if (bad_variant(variant) || pairs < 0) return RMOE_ERR_INVALID_ARGUMENT;
    return hidden > kMaxI8Sum || intermediate > kMaxI8Sum ? RMOE_ERR_UNSUPPORTED_SHAPE : RMOE_OK;
}

// The two stages' checked arguments.
int i8_gate_up_args(rmoe::I8Args *a, const void *xc, const float *xs, const void *gc, const float *gsc, const void *uc,
                    const float *us, const int32_t *gs, const int32_t *gpo, const int32_t *gidx, float *rows, void *hc,
                    float *hs, int64_t hidden, int64_t intermediate, int32_t E, int32_t M) {
    if (!xc || !xs || !gc || !gsc || !uc || !us || !gs || !gpo || (M > 0 && !gidx) || !rows || !hc || !hs)
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(xc) || !aligned16(gc) || !aligned16(uc) || !aligned16(gsc) || !aligned16(us) || !aligned16(rows) ||
        !aligned16(hc) || !aligned4(xs) || !aligned4(hs) || !aligned4(gs) || !aligned4(gpo) || !aligned4(gidx))
        return RMOE_ERR_MISALIGNED;
    a->x = bytes(xc), a->xs = xs, a->w0 = bytes(gc), a->w0s = gsc, a->w1 = bytes(uc), a->w1s = us;
    a->gs = gs, a->gpo = gpo, a->gidx = gidx;
    a->rows = rows, a->yc = bytes(hc), a->ys = hs;
    a->N = intermediate, a->K = hidden, a->E = E, a->M = M;
    return RMOE_OK;
}

int i8_down_args(rmoe::I8Args *a, const void *hc, const float *hs, const void *dc, const float *ds, const float *rw,
                 const int32_t *gs, const int32_t *go, const int32_t *gpo, const int32_t *gidx, void *out,
                 int64_t hidden, int64_t intermediate, int32_t E, int64_t pairs, int32_t M) {
    if (!hc || !hs || !dc || !ds || !gs || !go || !gpo || (M > 0 && !gidx) || !out || (pairs > 0 && !rw))
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(hc) || !aligned16(dc) || !aligned16(ds) || !aligned16(out) || !aligned4(hs) || !aligned4(rw) ||
        !aligned4(gs) || !aligned4(go) || !aligned4(gpo) || !aligned4(gidx))
        return RMOE_ERR_MISALIGNED;
    a->x = bytes(hc), a->xs = hs, a->w0 = bytes(dc), a->w0s = ds, a->rw = rw;
    a->gs = gs, a->go = go, a->gpo = gpo, a->gidx = gidx;
    a->y = static_cast<_Float16 *>(out);
    a->N = hidden, a->K = intermediate, a->E = E, a->M = M;
    return RMOE_OK;
}

}  // namespace

extern "C" {

int rmoe_quantize_int8(const void *x, int32_t type, int64_t rows, int64_t cols, void *codes, float *scales,
                       void *stream) {
    bool empty = false;
    const int st = check_i8_sizes(type, rows, cols, &empty);
    if (st != RMOE_OK) return st;
    if (empty) return RMOE_OK;
    if (!x || !codes || !scales) return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(codes) || !aligned4(scales)) return RMOE_ERR_MISALIGNED;
    return to_status(rmoe::launch_quantize_i8(x, mx_type(type), rows, cols, bytes(codes), scales,
                                              static_cast<hipStream_t>(stream)));
}

int rmoe_dequantize_int8(const void *codes, const float *scales, int32_t type, int64_t rows, int64_t cols, void *y,
                         void *stream) {
    bool empty = false;
    const int st = check_i8_sizes(type, rows, cols, &empty);
    if (st != RMOE_OK) return st;
    if (empty) return RMOE_OK;
    if (!codes || !scales || !y) return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(y) || !aligned16(codes) || !aligned4(scales)) return RMOE_ERR_MISALIGNED;
    return to_status(rmoe::launch_dequantize_i8(bytes(codes), scales, mx_type(type), rows, cols, y,
                                                static_cast<hipStream_t>(stream)));
}

int rmoe_pack_int8_f16(const void *x, const float *topk_weights, const int32_t *prow, const int32_t *cpos,
                       int64_t num_tokens, int32_t top_k, int64_t hidden, void *codes, float *scales, float *w_compact,
                       int64_t total_padded_tokens, void *stream) {
    if (top_k < 0 || total_padded_tokens < 0) return RMOE_ERR_INVALID_ARGUMENT;
    bool empty = false;
    const int st = check_i8_sizes(RMOE_TYPE_F16, num_tokens, hidden, &empty);
    if (st != RMOE_OK) return st;
    if (num_tokens > INT32_MAX) return RMOE_ERR_UNSUPPORTED_SHAPE;
    if (empty || top_k == 0) return RMOE_OK;
    if (!x || !topk_weights || !prow || !cpos || !codes || !scales || !w_compact) return RMOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(codes) || !aligned4(scales) || !aligned4(topk_weights) || !aligned4(prow) ||
        !aligned4(cpos) || !aligned4(w_compact))
        return RMOE_ERR_MISALIGNED;
    return to_status(rmoe::launch_pack_i8(static_cast<const _Float16 *>(x), topk_weights, prow, cpos, num_tokens,
                                          top_k, hidden, total_padded_tokens, bytes(codes), scales, w_compact,
                                          static_cast<hipStream_t>(stream)));
}

size_t rmoe_int8_workspace_bytes(int64_t total_padded_tokens, int64_t intermediate) {
    if (total_padded_tokens <= 0 || intermediate <= 0) return 0;
    return (size_t)total_padded_tokens * (5u * (size_t)intermediate + 4u);
}

int rmoe_pick_variant_int8(int32_t variant, int64_t num_pairs, int32_t num_experts) {
    if (bad_variant(variant) || num_pairs < 0 || num_experts < 1) return RMOE_ERR_INVALID_ARGUMENT;
    return pick_variant_i8(variant, num_pairs, num_experts);
}

int rmoe_gate_up_int8(const void *xc, const float *xs, const void *gc, const float *gsc, const void *uc,
                      const float *us, const int32_t *gs, const int32_t *gpo, const int32_t *gidx, float *rows,
                      void *hc, float *hs, int64_t hidden, int64_t intermediate, int32_t num_experts,
                      int64_t total_padded_tokens, int64_t total_valid_tokens, int32_t num_blocks_m, int32_t variant,
                      void *stream) {
    int st = check_i8_dims(hidden, intermediate, num_experts, total_padded_tokens, total_valid_tokens, num_blocks_m,
                           variant);
    if (st != RMOE_OK) return st;
    rmoe::I8Args a{};
    st = i8_gate_up_args(&a, xc, xs, gc, gsc, uc, us, gs, gpo, gidx, rows, hc, hs, hidden, intermediate, num_experts,
                         num_blocks_m);
    return st != RMOE_OK ? st : i8_gate_up_impl(a, variant, total_valid_tokens, stream);
}

int rmoe_down_int8(const void *hc, const float *hs, const void *dc, const float *ds, const float *rw,
                   const int32_t *gs, const int32_t *go, const int32_t *gpo, const int32_t *gidx, void *out,
                   int64_t hidden, int64_t intermediate, int32_t num_experts, int64_t total_padded_tokens,
                   int64_t total_valid_tokens, int32_t num_blocks_m, int32_t variant, void *stream) {
    int st = check_i8_dims(hidden, intermediate, num_experts, total_padded_tokens, total_valid_tokens, num_blocks_m,
                           variant);
    if (st != RMOE_OK) return st;
    rmoe::I8Args a{};
    st = i8_down_args(&a, hc, hs, dc, ds, rw, gs, go, gpo, gidx, out, hidden, intermediate, num_experts,
                      total_valid_tokens, num_blocks_m);
    return st != RMOE_OK ? st : i8_down_impl(a, variant, total_valid_tokens, stream);
}

int rmoe_forward_int8(const void *xc, const float *xs, const void *gc, const float *gsc, const void *uc,
                      const float *us, const void *dc, const float *ds, const float *rw, const int32_t *gs,
                      const int32_t *go, const int32_t *gpo, const int32_t *gidx, void *workspace, void *out,
                      int64_t hidden, int64_t intermediate, int32_t num_experts, int64_t total_padded_tokens,
                      int64_t total_valid_tokens, int32_t num_blocks_m, int32_t variant, void *stream) {
    int st = check_i8_dims(hidden, intermediate, num_experts, total_padded_tokens, total_valid_tokens, num_blocks_m,
                           variant);
    if (st != RMOE_OK) return st;
    if (!workspace) return RMOE_ERR_INVALID_ARGUMENT;
    // codes, rows in fp32, scales: rows of 128 bytes and more keep the alignment
    unsigned char *hc = bytes(workspace);
    const size_t n = (size_t)total_padded_tokens * (size_t)intermediate;
    float *rows = reinterpret_cast<float *>(hc + n), *hs = rows + n;
    rmoe::I8Args gu{}, dn{};
    st = i8_gate_up_args(&gu, xc, xs, gc, gsc, uc, us, gs, gpo, gidx, rows, hc, hs, hidden, intermediate, num_experts,
                         num_blocks_m);
    if (st != RMOE_OK) return st;
    st = i8_down_args(&dn, hc, hs, dc, ds, rw, gs, go, gpo, gidx, out, hidden, intermediate, num_experts,
                      total_valid_tokens, num_blocks_m);
    if (st != RMOE_OK) return st;
    // the rows' room is free again once they are quantised
    dn.part = reinterpret_cast<int32_t *>(rows);
    dn.Tp = total_padded_tokens;
    st = i8_gate_up_impl(gu, variant, total_valid_tokens, stream);
    return st != RMOE_OK ? st : i8_down_impl(dn, variant, total_valid_tokens, stream);
}

}  // extern "C"

// ---- training --------------------------------------------------------------

namespace {

const _Float16 *f16(const void *p) { return static_cast<const _Float16 *>(p); }
_Float16 *f16(void *p) { return static_cast<_Float16 *>(p); }

template <class... T>
bool any_null(T... p) {
    return (!p || ...);
}
template <class... T>
bool all16(T... p) {
    return (aligned16(p) && ...);
}
template <class... T>
bool all4(T... p) {
    return (aligned4(p) && ...);
}

constexpr int64_t kMaxGradTiles = (int64_t)1 << 23;  // their positions are ints

int check_train_dims(rmoe::TrainArgs *a, int64_t hidden, int64_t intermediate, int32_t E, int64_t Tp, int64_t pairs,
                     int32_t M) {
    const int st = check_dims(hidden, intermediate, E, Tp, M);
    if (st != RMOE_OK) return st;
    if (pairs < 0) return RMOE_ERR_INVALID_ARGUMENT;
    a->H = hidden, a->I = intermediate, a->E = E, a->Tp = Tp, a->pairs = pairs, a->M = M;
    return RMOE_OK;
}

// Checked arguments of each stage.
int down_backward_args(rmoe::TrainArgs *a, const void *dout, const void *down_w, const float *rw, const void *gate,
                       const void *up, const int32_t *gs, const int32_t *go, const int32_t *gpo, const int32_t *gidx,
                       void *dgate, void *dup, void *whidden, void *scratch, float *drw) {
    if (any_null(dout, down_w, gate, up, gs, go, gpo, dgate, dup, whidden) || (a->M > 0 && !gidx) ||
        (a->pairs > 0 && any_null(rw, scratch, drw)))
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!all16(dout, down_w, gate, up, dgate, dup, whidden) || !all4(rw, gs, go, gpo, gidx, scratch, drw))
        return RMOE_ERR_MISALIGNED;
    a->dy = f16(dout), a->wd = f16(down_w), a->rw = rw, a->g = f16(gate), a->u = f16(up);
    a->gs = gs, a->go = go, a->gpo = gpo, a->gidx = gidx;
    a->dg = f16(dgate), a->du = f16(dup), a->hw = f16(whidden);
    a->part = static_cast<float *>(scratch), a->drw = drw;
    return RMOE_OK;
}

int gate_up_backward_args(rmoe::TrainArgs *a, const void *dgate, const void *dup, const void *gate_w,
                          const void *up_w, const int32_t *gs, const int32_t *gpo, const int32_t *gidx, void *dx) {
    if (any_null(dgate, dup, gate_w, up_w, gs, gpo, dx) || (a->M > 0 && !gidx)) return RMOE_ERR_INVALID_ARGUMENT;
    if (!all16(dgate, dup, gate_w, up_w, dx) || !all4(gs, gpo, gidx)) return RMOE_ERR_MISALIGNED;
    // the kernel only reads dgate and dup
    a->dg = const_cast<_Float16 *>(f16(dgate)), a->du = const_cast<_Float16 *>(f16(dup));
    a->wg = f16(gate_w), a->wu = f16(up_w), a->gs = gs, a->gpo = gpo, a->gidx = gidx, a->dx = f16(dx);
    return RMOE_OK;
}

int weight_grad_args(rmoe::TrainArgs *a, const void *x, const void *dout, const void *dgate, const void *dup,
                     const void *whidden, const int32_t *gs, const int32_t *gpo, void *dgate_w, void *dup_w,
                     void *ddown_w) {
    if (rmoe::weight_grad_tiles(a->H, a->I, a->E) > kMaxGradTiles) return RMOE_ERR_UNSUPPORTED_SHAPE;
    if (any_null(x, dout, dgate, dup, whidden, gs, gpo, dgate_w, dup_w, ddown_w)) return RMOE_ERR_INVALID_ARGUMENT;
    if (!all16(x, dout, dgate, dup, whidden, dgate_w, dup_w, ddown_w) || !all4(gs, gpo)) return RMOE_ERR_MISALIGNED;
    a->x = f16(x), a->dy = f16(dout);
    a->dg = const_cast<_Float16 *>(f16(dgate)), a->du = const_cast<_Float16 *>(f16(dup));
    a->hw = const_cast<_Float16 *>(f16(whidden));
    a->gs = gs, a->gpo = gpo, a->dwg = f16(dgate_w), a->dwu = f16(dup_w), a->dwd = f16(ddown_w);
    return RMOE_OK;
}

}  // namespace

extern "C" {

int rmoe_gate_up_train_f16(const void *x, const void *gate_w, const void *up_w, const int32_t *gs,
                           const int32_t *gpo, const int32_t *gidx, void *gate, void *up, void *hidden_rows,
                           int64_t hidden, int64_t intermediate, int32_t num_experts, int64_t total_padded_tokens,
                           int64_t total_valid_tokens, int32_t num_blocks_m, void *stream) {
    const int st = check_dims(hidden, intermediate, num_experts, total_padded_tokens, num_blocks_m);
    if (st != RMOE_OK) return st;
    if (total_valid_tokens < 0 || any_null(x, gate_w, up_w, gs, gpo, gate, up, hidden_rows) ||
        (num_blocks_m > 0 && !gidx))
        return RMOE_ERR_INVALID_ARGUMENT;
    if (!all16(x, gate_w, up_w, gate, up, hidden_rows) || !all4(gs, gpo, gidx)) return RMOE_ERR_MISALIGNED;
    if (num_blocks_m == 0) return RMOE_OK;
    rmoe::TrainArgs a{};
    a.x = f16(x), a.wg = f16(gate_w), a.wu = f16(up_w);
    a.gs = gs, a.gpo = gpo, a.gidx = gidx;
    a.yg = f16(gate), a.yu = f16(up), a.yh = f16(hidden_rows);
    a.H = hidden, a.I = intermediate, a.E = num_experts, a.Tp = total_padded_tokens, a.M = num_blocks_m;
    return to_status(rmoe::launch_gate_up_train(a, static_cast<hipStream_t>(stream)));
}

size_t rmoe_backward_scratch_bytes(int64_t num_pairs, int64_t intermediate) {
    return num_pairs <= 0 || intermediate <= 0 ? 0 : (size_t)num_pairs * (size_t)ceil_div(intermediate, 128) * 4u;
}

int rmoe_down_backward_f16(const void *dout, const void *down_w, const float *rw, const void *gate, const void *up,
                           const int32_t *gs, const int32_t *go, const int32_t *gpo, const int32_t *gidx, void *dgate,
                           void *dup, void *whidden, void *scratch, float *drw, int64_t hidden, int64_t intermediate,
                           int32_t num_experts, int64_t total_padded_tokens, int64_t total_valid_tokens,
                           int32_t num_blocks_m, void *stream) {
    rmoe::TrainArgs a{};
    int st = check_train_dims(&a, hidden, intermediate, num_experts, total_padded_tokens, total_valid_tokens,
                              num_blocks_m);
    if (st != RMOE_OK) return st;
    st = down_backward_args(&a, dout, down_w, rw, gate, up, gs, go, gpo, gidx, dgate, dup, whidden, scratch, drw);
    if (st != RMOE_OK || num_blocks_m == 0) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    st = to_status(rmoe::launch_hidden_grad(a, s));
    return st != RMOE_OK ? st : to_status(rmoe::launch_drw(a, s));
}

int rmoe_gate_up_backward_f16(const void *dgate, const void *dup, const void *gate_w, const void *up_w,
                              const int32_t *gs, const int32_t *gpo, const int32_t *gidx, void *dx, int64_t hidden,
                              int64_t intermediate, int32_t num_experts, int64_t total_padded_tokens,
                              int64_t total_valid_tokens, int32_t num_blocks_m, void *stream) {
    rmoe::TrainArgs a{};
    int st = check_train_dims(&a, hidden, intermediate, num_experts, total_padded_tokens, total_valid_tokens,
                              num_blocks_m);
    if (st != RMOE_OK) return st;
    st = gate_up_backward_args(&a, dgate, dup, gate_w, up_w, gs, gpo, gidx, dx);
    if (st != RMOE_OK || num_blocks_m == 0) return st;
    return to_status(rmoe::launch_gate_up_backward(a, static_cast<hipStream_t>(stream)));
}

int rmoe_weight_grad_f16(const void *x, const void *dout, const void *dgate, const void *dup, const void *whidden,
                         const int32_t *gs, const int32_t *gpo, void *dgate_w, void *dup_w, void *ddown_w,
                         int64_t hidden, int64_t intermediate, int32_t num_experts, int64_t total_padded_tokens,
                         void *stream) {
    rmoe::TrainArgs a{};
    int st = check_train_dims(&a, hidden, intermediate, num_experts, total_padded_tokens, 0, 0);
    if (st != RMOE_OK) return st;
    st = weight_grad_args(&a, x, dout, dgate, dup, whidden, gs, gpo, dgate_w, dup_w, ddown_w);
    if (st != RMOE_OK) return st;
    return to_status(rmoe::launch_weight_grad(a, static_cast<hipStream_t>(stream)));
}

int rmoe_backward_f16(const void *x, const void *dout, const void *gate_w, const void *up_w, const void *down_w,
                      const float *rw, const void *gate, const void *up, const int32_t *gs, const int32_t *go,
                      const int32_t *gpo, const int32_t *gidx, void *dgate, void *dup, void *whidden, void *scratch,
                      void *dx, void *dgate_w, void *dup_w, void *ddown_w, float *drw, int64_t hidden,
                      int64_t intermediate, int32_t num_experts, int64_t total_padded_tokens,
                      int64_t total_valid_tokens, int32_t num_blocks_m, void *stream) {
    rmoe::TrainArgs a{};
    int st = check_train_dims(&a, hidden, intermediate, num_experts, total_padded_tokens, total_valid_tokens,
                              num_blocks_m);
    if (st != RMOE_OK) return st;
    st = down_backward_args(&a, dout, down_w, rw, gate, up, gs, go, gpo, gidx, dgate, dup, whidden, scratch, drw);
    if (st != RMOE_OK) return st;
    st = gate_up_backward_args(&a, dgate, dup, gate_w, up_w, gs, gpo, gidx, dx);
    if (st != RMOE_OK) return st;
    st = weight_grad_args(&a, x, dout, dgate, dup, whidden, gs, gpo, dgate_w, dup_w, ddown_w);
    if (st != RMOE_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (num_blocks_m == 0) return to_status(rmoe::launch_weight_grad(a, s));
    st = to_status(rmoe::launch_hidden_grad(a, s));
    return st != RMOE_OK ? st : to_status(rmoe::launch_grads(a, s));
}

}  // extern "C"
