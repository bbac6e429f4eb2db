// Host check of what the persistent workgroups of the MXFP4 and training
// kernels take (csrc/rmoe_sched.h, the same code the kernels run).
//   items:  stdin "items E NT grid", E group sizes, then a count of blocks
//           that the block table maps to another expert, and those blocks.
//           Every (live block, slice) exactly once, by an item of its expert
//           with its rows; remapped blocks by none.
//   tiles:  stdin "tiles E nh ni grid busy lead".  Every weight-gradient tile
//           of every matrix exactly once, whoever starts ahead.
// Prints "ok <items or tiles> <most of one workgroup>" or "FAIL <reason>".
#include <cstdio>
#include <cstring>
#include <vector>

#include "../mixture_experts_routed_grouped_amd/csrc/rmoe_sched.h"

using namespace rmoe;

static int items() {
    int E, NT, grid, n;
    if (std::scanf("%d %d %d", &E, &NT, &grid) != 3) return 2;
    std::vector<int32_t> gs(E), gpo(E + 1, 0);
    for (int e = 0; e < E; ++e)
        if (std::scanf("%d", &gs[e]) != 1) return 2;
    for (int e = 0; e < E; ++e) gpo[e + 1] = gpo[e] + (gs[e] / kItemRows + 1) * kItemRows;
    const int M = gpo[E] / kItemRows;
    std::vector<int32_t> gidx(M);
    std::vector<int> own(M);
    for (int e = 0; e < E; ++e)
        for (int bx = gpo[e] / kItemRows; bx < gpo[e + 1] / kItemRows; ++bx) gidx[bx] = own[bx] = e;
    if (std::scanf("%d", &n) != 1) return 2;
    for (int i = 0; i < n; ++i) {
        int bx;
        if (std::scanf("%d", &bx) != 1 || bx < 0 || bx >= M) return 2;
        gidx[bx] = (gidx[bx] + 1) % (E + 1);
    }
    std::vector<int> hits((size_t)M * NT, 0);
    long total = 0, most = 0;
    for (int w = 0; w < grid; ++w) {
        ItemWalk<const int32_t *> walk(gs.data(), gpo.data(), gidx.data(), E, NT, w, grid);
        TileItem it;
        long mine = 0;
        while (walk.next(it)) {
            ++mine;
            if (it.e < 0 || it.e >= E || it.nt < 0 || it.nt >= NT || (it.rows0 == 0 && it.rows1 == 0) ||
                it.bx * kItemRows != gpo[it.e] + it.off) {
                std::printf("FAIL item w=%d e=%d nt=%d bx=%d\n", w, it.e, it.nt, it.bx);
                return 1;
            }
            for (int b = 0; b < 2; ++b) {
                const int rows = b ? it.rows1 : it.rows0;
                if (rows == 0) continue;
                int want = gs[it.e] - it.off - b * kItemRows;
                want = want > kItemRows ? kItemRows : want;
                if (rows != want || it.bx + b >= M || own[it.bx + b] != it.e) {
                    std::printf("FAIL rows w=%d bx=%d rows=%d want=%d\n", w, it.bx + b, rows, want);
                    return 1;
                }
                ++hits[(size_t)(it.bx + b) * NT + it.nt];
            }
        }
        total += mine;
        most = mine > most ? mine : most;
    }
    for (int bx = 0; bx < M; ++bx)
        for (int nt = 0; nt < NT; ++nt) {
            const int e = own[bx], want = gidx[bx] == e && gs[e] > bx * kItemRows - gpo[e];
            if (hits[(size_t)bx * NT + nt] != want) {
                std::printf("FAIL coverage bx=%d nt=%d hits=%d want=%d\n", bx, nt, hits[(size_t)bx * NT + nt], want);
                return 1;
            }
        }
    std::printf("ok %ld %ld\n", total, most);
    return 0;
}

static int tiles() {
    int E, nh, ni, grid, busy, lead;
    if (std::scanf("%d %d %d %d %d %d", &E, &nh, &ni, &grid, &busy, &lead) != 6) return 2;
    const int per = nh * ni, total = 3 * E * per;
    std::vector<int> hits(total, 0);
    long most = 0, sum = 0;
    for (int w = 0; w < grid; ++w) {
        GradWalk walk(total, busy, lead, w, grid);
        long mine = 0;
        for (int item; (item = walk.next()) >= 0; ++mine) {
            if (item >= total) {
                std::printf("FAIL w=%d item=%d\n", w, item);
                return 1;
            }
            const GradTile t = grad_tile(item, nh, ni);
            const int nA = t.m < 2 ? nh : ni, nB = t.m < 2 ? ni : nh;
            if (t.e < 0 || t.e >= E || t.m < 0 || t.m > 2 || t.a < 0 || t.a >= nA || t.b < 0 || t.b >= nB) {
                std::printf("FAIL tile item=%d e=%d m=%d a=%d b=%d\n", item, t.e, t.m, t.a, t.b);
                return 1;
            }
            ++hits[((size_t)t.e * 3 + t.m) * per + (size_t)t.b * nA + t.a];
        }
        sum += mine;
        most = mine > most ? mine : most;
    }
    for (int i = 0; i < total; ++i)
        if (hits[i] != 1) {
            std::printf("FAIL tile %d taken %d times\n", i, hits[i]);
            return 1;
        }
    std::printf("ok %ld %ld\n", sum, most);
    return 0;
}

int main() {
    char what[16];
    if (std::scanf("%15s", what) != 1) return 2;
    return std::strcmp(what, "items") == 0 ? items() : tiles();
}
