// Host check of region.h: overlap() against sets of bytes, for regions of a few rows of equal
// and unequal strides, and at the ends of the address space.
#include <cstdio>
#include <cstdlib>
#include <set>

#include "region.h"

int main() {
    std::srand(1);
    const auto pick = [](int lo, int hi) { return lo + std::rand() % (hi - lo + 1); };
    int seen[2] = {0, 0};
    for (int n = 0; n < 200000; ++n) {
        tcq::Region r[2];
        std::set<long> bytes[2];
        const int same = pick(0, 2) == 0 ? pick(6, 20) : 0;
        for (int k = 0; k < 2; ++k) {
            const int rows = pick(0, 6), cols = pick(0, 6), size = 1;
            const int ld = same ? same : cols + pick(0, 16) + (cols == 0);
            const long at = 10000 + pick(-60, 60);
            r[k] = tcq::region("", reinterpret_cast<void *>(at), rows, ld, cols, size);
            for (int i = 0; i < rows; ++i)
                for (int c = 0; c < cols; ++c) bytes[k].insert(at + long(i) * ld + c);
        }
        bool want = false;
        for (long b : bytes[0]) want = want || bytes[1].count(b);
        ++seen[want];
        if (tcq::overlap(r[0], r[1]) != want || tcq::overlap(r[1], r[0]) != want) {
            std::printf("case %d: overlap is %d\n", n, want);
            return 1;
        }
    }
    // sizes whose products pass 64 bits
    const auto far = reinterpret_cast<void *>(~uintptr_t{0} - 100);
    const auto low = reinterpret_cast<void *>(uintptr_t{4096});
    const tcq::Region wide = tcq::region("", low, 1 << 23, INT64_MAX / 2, 1 << 21, 4);
    if (tcq::overlap(wide, tcq::region("", far, 1, 4, 4, 4))) return 1;
    if (!tcq::overlap(wide, tcq::region("", low, 1, 4, 4, 4))) return 1;
    if (seen[0] < 20000 || seen[1] < 20000) return 1;
    std::printf("regions ok\n");
    return 0;
}
