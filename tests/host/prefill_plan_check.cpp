// Host-side check of the prompt chunks' work plan: units on a line cut into ranges for clusters, with the
// gap that a unit change costs there (csrc/prefill.cuh, the arithmetic in csrc/full.cuh). Every tile
// belongs to one range, a unit is whole or leaves its pieces in the slots where the join looks for them, and
// no range is empty. Exits non-zero on the first failure.
#include <algorithm>
#include <cstdio>
#include <map>
#include <random>
#include <vector>

#include "prefill.cuh"

using namespace dsa;

#define CHECK(cond, ...)                     \
    do {                                     \
        if (!(cond)) {                       \
            std::printf("FAIL %s: ", #cond); \
            std::printf(__VA_ARGS__);        \
            std::printf("\n");               \
            return 1;                        \
        }                                    \
    } while (0)

int main() {
    std::mt19937_64 g(11);
    const int counts[] = {1, 2, 3, 5, 20, 64, 75, 76, 77, 300, 2000};
    const int tops[] = {1, 3, 8, 100, 2000, 16000};
    const int grids[] = {1, 2, 7, 74, 76};
    for (int trial = 0; trial < 4000; ++trial) {
        const int n = counts[g() % 11], top = tops[g() % 6], clusters = grids[g() % 5];
        std::vector<int64_t> tiles(n), start(n);
        int64_t all = 0;
        for (auto& t : tiles) all += t = 1 + static_cast<int64_t>(g() % top);
        const full::Line line = full::make_line(all, n, clusters, prefill::kGap);
        CHECK(line.ctas == std::min<int64_t>(all, clusters) && line.gap <= prefill::kGap && 4 * line.gap * clusters <= all, "trial %d", trial);
        std::vector<full::UnitPieces> pieces(n);
        std::vector<int> first(line.ctas, -1);
        int64_t at = 0;
        for (int u = 0; u < n; ++u) {
            start[u] = at + line.gap * u;
            at += tiles[u];
            int32_t c0, c1;
            pieces[u] = full::unit_pieces(line, u, start[u], start[u] + tiles[u], &c0, &c1);
            for (int c = c0; c < c1; ++c) {
                CHECK(c < line.ctas && first[c] < 0, "trial %d: range %d of %d", trial, c, line.ctas);
                first[c] = u;
            }
        }
        std::vector<int64_t> covered(n, 0);
        std::vector<int> whole(n, 0);
        std::map<int, int> slots;
        for (int c = 0; c < line.ctas; ++c) {
            const int64_t begin = full::range_begin(line, c), end = full::range_begin(line, c + 1);
            CHECK(begin < end && first[c] >= 0, "trial %d: range %d", trial, c);
            for (int u = first[c];; ++u) {
                CHECK(u < n, "trial %d: range %d runs past the last unit", trial, c);
                const int64_t e = start[u] + tiles[u], t0 = std::max(begin, start[u]) - start[u], t1 = std::min(end, e) - start[u];
                CHECK(t0 < t1 && t0 == covered[u], "trial %d: range %d unit %d", trial, c, u);
                covered[u] = t1;
                if (begin <= start[u] && e <= end) whole[u]++;
                else CHECK(slots.emplace(2 * c + (u == first[c] ? 0 : 1), u).second, "trial %d: a slot of range %d twice", trial, c);
                if (e + line.gap >= end) break;
            }
        }
        size_t found = 0;
        for (int u = 0; u < n; ++u) {
            CHECK(covered[u] == tiles[u] && (pieces[u].pieces < 2) == (whole[u] == 1), "trial %d: unit %d", trial, u);
            for (int i = 0; pieces[u].pieces > 1 && i < pieces[u].pieces; ++i, ++found) {
                const auto it = slots.find(i == 0 ? pieces[u].slot_lo : 2 * (pieces[u].c_lo + i));
                CHECK(it != slots.end() && it->second == u, "trial %d: unit %d piece %d", trial, u, i);
            }
        }
        CHECK(found == slots.size() && static_cast<int>(found) <= 2 * clusters, "trial %d: %zu of %zu slots", trial, found, slots.size());
    }
    // Units of a call at most, whatever its requests' rows are.
    for (int trial = 0; trial < 20000; ++trial) {
        const int64_t heads = 1 + g() % 300, n = 1 + g() % 40;
        int64_t rows = g() % 3, units = 0;
        for (int64_t s = 0; s < n; ++s) {
            const int64_t k = g() % 2 ? g() % 4 : g() % 300;
            rows += k;
            units += (k * heads + prefill::kPairs - 1) / prefill::kPairs;
        }
        CHECK(units <= prefill::max_units(n, std::max<int64_t>(rows, 1), heads), "trial %d", trial);
    }
    std::printf("prefill plan ok\n");
    return 0;
}
