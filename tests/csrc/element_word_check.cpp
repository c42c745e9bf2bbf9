// Host check of what the kernels' copies of single 16-bit elements read
// (element_word in block.cuh): for a tensor of `n` elements that starts at any
// place of a buffer, every element's read holds the element (or is left to a
// load by itself) and lies between the tensor's first and last byte.  Run on
// the CPU, compiled by nvcc as CUDA source; prints the number of reads checked.
#include <cstdio>

#include "block.cuh"

int main() {
    alignas(16) static uint16_t buffer[64];
    int checked = 0;
    for (int start = 0; start < 8; ++start)
        for (int n = 1; n <= 24; ++n) {
            const uint16_t *first = buffer + start, *end = first + n;
            for (const uint16_t *p = first; p < end; ++p, ++checked) {
                const auto w = gdn::element_word(p, gdn::odd(p), p == first);
                const auto *from = reinterpret_cast<const char *>(w.from);
                const auto *at = reinterpret_cast<const char *>(p);
                const bool word = reinterpret_cast<uintptr_t>(from) % 4 == 0;
                const bool inside = from >= reinterpret_cast<const char *>(first) &&
                                    from + w.bytes <= reinterpret_cast<const char *>(end);
                const bool holds = from <= at && from + w.bytes >= at + 2;
                const bool alone = w.bytes == 0 && p == first && gdn::odd(p);
                if (!word || !(alone || (inside && holds && (w.bytes == 2 || w.bytes == 4)))) {
                    std::printf("start %d, n %d, element %d: %d bytes at %d\n", start, n,
                                (int)(p - first), w.bytes,
                                (int)(from - reinterpret_cast<const char *>(first)));
                    return 1;
                }
            }
        }
    std::printf("%d\n", checked);
    return 0;
}
