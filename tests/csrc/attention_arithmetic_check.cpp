// Host check of the paged attention's integer arithmetic (paged_attention.cuh):
// quotients by a product against the machine's, at every multiple's edges, and
// the division of tiles among groups: ranges that follow one another without a
// gap, and the group of every tile.  Run on the CPU, compiled by nvcc as CUDA
// source; prints the number of quotients and of tiles checked.
#include <cstdio>
#include <initializer_list>

#include "paged_attention.cuh"

int main() {
    long quotients = 0, tiles = 0;
    auto check = [&](int x, int d, const gdn::Division &by) {
        if (x < 0 || x >= 1 << 30) return true;
        ++quotients;
        if (by.of(x) == x / d) return true;
        std::printf("%d / %d: %d\n", x, d, by.of(x));
        return false;
    };
    auto divisor = [&](int d) {
        const gdn::Division by = gdn::Division::by(d);
        for (int k = 0; k < 64; ++k)
            for (long q : {(long)k, ((1L << 30) - 1) / d - k, (1L << 30) / d / 64 * k})
                for (int off = -1; off <= 1; ++off)
                    if (!check((int)(q * d + off), d, by)) return false;
        return check((1 << 30) - 1, d, by);
    };
    for (int d = 1; d <= 5000; ++d)
        if (!divisor(d)) return 1;
    for (int s = 13; s <= 20; ++s)
        for (int off = -3; off <= 3; ++off)
            if ((1 << s) + off <= 1 << 20 && !divisor((1 << s) + off)) return 1;

    for (int64_t total : {1L, 2L, 5L, 303L, 304L, 305L, 1216L, 1217L, 99991L})
        for (int most : {1, 2, 4, 152, 304, 1216}) {
            const int groups = (int)(total < most ? total : most);
            int64_t at = 0;
            for (int g = 0; g < most; ++g) {
                const int64_t begin = gdn::first_tile(total, groups, g), end = gdn::first_tile(total, groups, g + 1);
                if (begin != at || end < begin || (g < groups) != (end > begin)) return 1;
                for (int64_t t = begin; t < end; ++t, ++tiles)
                    if (gdn::group_of(total, groups, t) != g) return 1;
                at = end;
            }
            if (at != total) return 1;
        }
    std::printf("%ld %ld\n", quotients, tiles);
    return 0;
}
