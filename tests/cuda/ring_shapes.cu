// Host-only check of the rings that the layer norm's kernels are launched with:
// ring_holds takes what fit_ring makes for every row length, and refuses a ring
// whose chunks, slots, threads or sums are not the kernel's.
#include <algorithm>
#include <cstdio>
#include <cstring>

#include "internal.h"
#include "row_ring.cuh"

using namespace gemm;

int main() {
    int64_t fitted = 0, bad = 0;
    auto refuse = [&](bool held, const char* what, int64_t d) {
        if (held && bad++ < 20) std::printf("taken: %s, d = %lld\n", what, static_cast<long long>(d));
    };
    for (int64_t d = 17; d <= 8192; d += d < 600 ? 1 : 23)
        for (int64_t rows : {int64_t(305), int64_t(1301), int64_t(40000), int64_t(1) << 30})
            for (int es : {2, 4})
                for (int arrays : {1, 2, 3})
                    for (int mode = 0; mode < 3; ++mode) {   // pairs of aligned rows, dense runs, pairs of unaligned rows
                        if (mode == 0 && d % 8) continue;
                        RingShape r;
                        r.dense = mode == 1 ? 1 : 0;
                        const int64_t units = mode == 0 ? d / 8 : d;
                        if (mode == 0) {
                            r.per = kPair;
                            team_of(&r, units, {2, 1});
                        } else if (mode == 1 && d <= 512) {
                            r.per = rows_of_a_warp(d * es);
                            r.team = 32;
                            r.each = static_cast<int>((d + 31) / 32);
                        } else {
                            r.per = 2;
                            team_of(&r, d, {16, 14, 12, 10, 8});
                        }
                        const int64_t slot = arrays * ChunkRing::place(d * es, r.per, r.dense);
                        const int64_t out = mode == 0 ? 0 : 2 * ChunkRing::place(d * es, r.per, r.dense), sums = 4 * d;
                        if (!fit_ring(&r, rows, slot, out, 152)) continue;
                        ++fitted;
                        if (!ring_holds(r, r.per, units, slot, out, arrays == 1 && es == 2 ? 0 : sums) && bad++ < 20)
                            std::printf("refused: d = %lld, rows = %lld, mode %d\n", static_cast<long long>(d), static_cast<long long>(rows), mode);
                        RingShape x = r;
                        x.per = r.per == 1 ? 2 : 1;
                        refuse(ring_holds(x, r.per, units, slot, out, sums), "another number of rows", d);
                        // a ring sized for chunks of one row under a kernel that takes two
                        if (mode == 0) {
                            RingShape one = r;
                            one.per = 1;
                            if (fit_ring(&one, rows, arrays * ChunkRing::place(d * es, 1, false), 0, 152))
                                refuse(ring_holds(one, kPair, units, slot, 0, sums), "chunks of one row", d);
                        }
                        refuse(ring_holds(r, r.per, static_cast<int64_t>(r.each) * r.team + 1, slot, out, sums), "longer rows", d);
                        refuse(ring_holds(r, r.per, units, slot + 16, out, sums), "larger slots", d);
                        refuse(ring_holds(r, r.per, units, slot, out + 16, sums), "larger staging buffers", d);
                        refuse(ring_holds(r, r.per, units, slot, out, r.smem / r.teams + 4), "larger sums", d);
                    }
    std::printf("%lld rings, %lld wrong\n", static_cast<long long>(fitted), static_cast<long long>(bad));
    return bad || fitted < 1000 ? 1 : 0;
}
