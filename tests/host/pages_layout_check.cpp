// Host-side check of the page operators' workspace (csrc/pages.cuh): whatever two pool sizes take
// turns with it, no list entry of one call lies where a mark of another call is, every mark word and
// every entry has a place of its own inside the bytes asked for, and 16-byte pieces of marks stay
// together. Exits non-zero on the first failure.
#include <cstdio>
#include <vector>

#include "pages.cuh"

using namespace dsa::pages;

#define CHECK(cond, ...)                          \
    do {                                          \
        if (!(cond)) {                            \
            std::printf("FAIL %s: ", #cond);      \
            std::printf(__VA_ARGS__);             \
            std::printf("\n");                    \
            return 1;                             \
        }                                         \
    } while (0)

int main() {
    const int64_t sizes[] = {1, 33, 128, 1000, 16383, 16384, 16385, 40000, 100000, 1000000};
    const int64_t most = 1000000;
    // What each word of the largest workspace is for: 0 nothing, 1 marks, 2.. the lists.
    std::vector<char> use(layout(most).total / 4, 0);
    size_t before = 0;
    for (const int64_t n : sizes) {
        const Layout L = layout(n);
        CHECK(L.total % 256 == 0 && L.total >= before && L.marks >= sizeof(Head), "%lld pages", static_cast<long long>(n));
        before = L.total;
        for (uint32_t w = 0; w < mark_words(n); ++w) {
            const size_t at = L.marks / 4 + static_cast<size_t>(mark_at(w));
            CHECK(at < L.total / 4 && (use[at] == 0 || use[at] == 1), "mark word %u of %lld pages", w, static_cast<long long>(n));
            CHECK(mark_at(w) == mark_at(w & ~3u) + (w & 3) && mark_at(w & ~3u) % 4 == 0, "piece of word %u", w);
            use[at] = 1;
        }
        const size_t lists[] = {L.rank, L.src, L.dst};
        const int64_t entries = n > DSA_MAX_PLAN_SEQS ? n : DSA_MAX_PLAN_SEQS;  // by page, or by fork
        for (int l = 0; l < 3; ++l) {
            std::vector<char> taken(use.size(), 0);
            for (uint32_t i = 0; i < entries; ++i) {
                const size_t at = lists[l] / 4 + static_cast<size_t>(entry_at(i));
                CHECK(at < L.total / 4 && (use[at] == 0 || use[at] == 2 + l) && !taken[at], "entry %u of list %d, %lld pages", i, l,
                      static_cast<long long>(n));
                use[at] = static_cast<char>(2 + l);
                taken[at] = 1;
            }
        }
    }
    // A fork reads and writes its lists without entry_at.
    CHECK(entry_at(DSA_MAX_PLAN_SEQS - 1) == DSA_MAX_PLAN_SEQS - 1, "forks");
    std::printf("pages layout ok\n");
    return 0;
}
