// Host-side checks of the full-cache decode's work plan (csrc/full.cuh): walking every CTA's
// stretches as the kernel does, every tile of every unit is covered exactly once, a unit is
// either written whole by one CTA or leaves pieces in exactly the slots where the join looks
// for them, and every range has a first unit and at least one tile. Also the division by a
// divisor known on the host (csrc/common.cuh). Exits non-zero on the first failure.
#include <algorithm>
#include <cstdio>
#include <map>
#include <random>
#include <vector>

#include "full.cuh"

using namespace dsa::full;

#define CHECK(cond, ...)                                         \
    do {                                                         \
        if (!(cond)) {                                           \
            std::printf("FAIL %s: ", #cond);                     \
            std::printf(__VA_ARGS__);                            \
            std::printf("\n");                                   \
            return 1;                                            \
        }                                                        \
    } while (0)

int main() {
    std::mt19937_64 g(7);
    const int counts[] = {1, 1, 2, 3, 5, 20, 64, 150, 152, 153, 300};
    const int tops[] = {1, 130, 1000, 20000, 200000, 2000000};
    const int grids[] = {1, 2, 7, 148, 152};
    for (int trial = 0; trial < 3000; ++trial) {
        const int n = counts[g() % 11], top = tops[g() % 6], max_ctas = grids[g() % 5];
        std::vector<int32_t> lens;
        int64_t tiles = 0;
        for (int i = 0; i < n; ++i) {
            const int32_t len = g() % 3 == 0 ? 0 : static_cast<int32_t>(g() % (top + 1));
            if (len > 0) lens.push_back(len);
            tiles += (len + kTile - 1) / kTile;
        }
        const int live = static_cast<int>(lens.size());
        if (live == 0) continue;
        const Line line = make_line(tiles, live, max_ctas);
        CHECK(line.ctas >= 1 && line.ctas <= max_ctas && line.ctas <= tiles, "trial %d", trial);
        std::vector<int64_t> start(live);
        std::vector<UnitPieces> pieces(live);
        std::vector<int> first(line.ctas, -1);
        int64_t at = 0;
        for (int k = 0; k < live; ++k) {
            const int64_t t = (lens[k] + kTile - 1) / kTile;
            start[k] = at + line.gap * k;
            int32_t c0, c1;
            pieces[k] = unit_pieces(line, k, start[k], start[k] + t, &c0, &c1);
            for (int c = c0; c < c1; ++c) {
                CHECK(c < line.ctas && first[c] < 0, "trial %d: range %d of %d", trial, c, line.ctas);
                first[c] = k;
            }
            at += t;
        }
        std::vector<int64_t> covered(live, 0);
        std::vector<int> whole(live, 0);
        std::map<int, int> slots;
        for (int c = 0; c < line.ctas; ++c) {
            const int64_t begin = range_begin(line, c), end = range_begin(line, c + 1);
            CHECK(begin < end && first[c] >= 0, "trial %d: range %d", trial, c);
            bool is_first = true;
            for (int k = first[c];; ++k, is_first = false) {
                CHECK(k < live, "trial %d: range %d runs past the last unit", trial, c);
                const Segment s = segment(begin, end, line.gap, c, is_first, k, k, start[k], lens[k], lens[k]);
                // Stretches come in order, so covering [0, t1) so far means the next starts there.
                CHECK(s.t0 < s.t1 && s.t0 == covered[k], "trial %d: range %d unit %d: %d..%d after %lld", trial, c, k, s.t0, s.t1,
                      static_cast<long long>(covered[k]));
                covered[k] = s.t1;
                if (s.part < 0) whole[k]++;
                else CHECK(slots.emplace(s.part, k).second, "trial %d: slot %d twice", trial, s.part);
                if (s.last) break;
            }
        }
        size_t found = 0;
        for (int k = 0; k < live; ++k) {
            CHECK(covered[k] == (lens[k] + kTile - 1) / kTile, "trial %d: unit %d", trial, k);
            const UnitPieces& q = pieces[k];
            CHECK((q.pieces < 2) == (whole[k] == 1), "trial %d: unit %d: %d pieces", trial, k, q.pieces);
            for (int i = 0; q.pieces > 1 && i < q.pieces; ++i, ++found) {
                const auto it = slots.find(i == 0 ? q.slot_lo : 2 * (q.c_lo + i));
                CHECK(it != slots.end() && it->second == k, "trial %d: unit %d piece %d", trial, k, i);
            }
        }
        CHECK(found == slots.size(), "trial %d: %zu of %zu slots", trial, found, slots.size());
    }
    for (int trial = 0; trial < 200000; ++trial) {
        const uint32_t few[] = {1, 2, 3, 7, 16, 48, 64, 100, 127, 128, 0x7FFFFFFFu, 0x40000000u, 0x40000001u};
        const uint32_t d = trial < 13 ? few[trial] : 1u + static_cast<uint32_t>(g() >> (33 + g() % 31)) % 0x7FFFFFFFu;
        const dsa::FastDiv f = dsa::fast_div(d);
        const uint32_t q = 0xFFFFFFFFu / d;
        const uint32_t xs[] = {0, 1, d - 1, d, d + 1, q * d, q * d - 1, 0x7FFFFFFFu, 0x80000000u, 0xFFFFFFFFu, static_cast<uint32_t>(g())};
        for (uint32_t x : xs) CHECK(dsa::divide(x, f) == x / d, "%u / %u", x, d);
    }
    std::printf("full plan ok\n");
    return 0;
}
