// Host check of the matrix-product launches' schedule (csrc/schedule.h): every unit is visited once, by
// one pair, in increasing order; and no pair's work exceeds the shortest schedule's by more than a unit.
#include <cstdio>
#include <vector>

#include "schedule.h"

int main() {
    const int lengths[][2] = {{448, 64}, {64, 64}, {512, 64}, {20, 3}, {7, 5}, {64, 1}};
    for (int pairs : {1, 2, 3, 7, 76, 152}) {
        for (int n_long : {0, 1, 2, 75, 76, 77, 100, 152, 256, 300}) {
            for (int n_short : {0, 1, 5, 20, 75, 76, 144, 333, 2688}) {
                for (auto& len : lengths) {
                    const int n = n_long + n_short;
                    if (n == 0) continue;
                    const int width = pairs < n ? pairs : n;  // as the launch takes them
                    const forge::UnitPlan plan = forge::plan_units(n, n_long, width, len[0], len[1]);
                    std::vector<int> seen(n, 0);
                    long long total = 0, most = 0;
                    for (int p = 0; p < width; ++p) {
                        forge::UnitCursor cur;
                        long long mine = 0;
                        int last = -1;
                        for (int u = cur.next(plan, p, width); u >= 0; u = cur.next(plan, p, width)) {
                            if (u >= n || u <= last || seen[u]++) {
                                std::printf("pairs %d long %d short %d: unit %d\n", pairs, n_long, n_short, u);
                                return 1;
                            }
                            last = u;
                            mine += u < n_long ? len[0] : len[1];
                        }
                        total += mine;
                        if (mine > most) most = mine;
                    }
                    for (int u = 0; u < n; ++u)
                        if (!seen[u]) {
                            std::printf("pairs %d long %d short %d: unit %d is never visited\n", pairs, n_long, n_short, u);
                            return 1;
                        }
                    // an even share, and one unit: a long one, or where short ones even the rest out, two of those
                    const bool evened = n_long % width == 0 || n_short >= (width - n_long % width) * (len[0] / len[1]);
                    const long long allowed = (total + width - 1) / width + (evened ? 2 * len[1] : len[0]);
                    if (most > allowed) {
                        std::printf("pairs %d long %d short %d len %d/%d: %lld > %lld\n", pairs, n_long, n_short, len[0],
                                    len[1], most, allowed);
                        return 1;
                    }
                }
            }
        }
    }
    std::printf("ok\n");
    return 0;
}
