// The chunk scans' offsets of float32 token rows near the longest sequence that the entry points take (T H d 4 bytes just
// below 4 GiB): rows of tokens before T lie where they belong, rows from T on lie past the buffer's end, where the
// hardware drops the store.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "layout.hpp"

int main() {
    long failures = 0, rows = 0, wraps = 0;
    for (int d : {64, 128})
        for (int H : {1, 2, 3, 5, 6, 7, 12, 16, 24, 31, 48, 100, 1000, 4096}) {
            const uint64_t HD = uint64_t(H) * d;
            const int limit = int(0xffffffffull / (HD * 4));  // longest T that is not refused
            for (int T = limit; T > limit - 17 && T > 0; --T)
                for (int h : {0, H / 2, H - 1})
                    for (int j0 = 0; j0 < d; j0 += 16) {
                        const uint32_t bytes = uint32_t(uint64_t(T) * HD - uint64_t(h) * d - j0) * 4u;
                        for (int t0 = (T / 16 - 2) * 16; t0 < (T / 256 + 1) * 256; t0 += 16) {
                            if (t0 < 0) continue;
                            const uint32_t shared = uint32_t(t0 < T ? t0 : T) * uint32_t(HD) * 4u;
                            for (int x = 0; x < 16; ++x)
                                for (int g = 0; g < 4; ++g) {
                                    const uint32_t lane = uint32_t(x * HD + 4 * g) * 4u;
                                    const uint32_t off = muir::whole_offset(lane, shared);
                                    const uint64_t want = uint64_t(lane) + shared;
                                    ++rows;
                                    wraps += want > 0xffffffffull;
                                    // Sixteen bytes, none of which may wrap to the buffer's start.
                                    const bool live = t0 + x < T;
                                    const bool good = live ? off == want && want + 16 <= bytes
                                                           : off >= bytes && uint64_t(off) + 16 <= 0x100000000ull;
                                    if (!good && failures++ < 5)
                                        printf("d=%d H=%d T=%d h=%d column %d token %d: offset %u of %u bytes\n", d, H, T, h, j0, t0 + x,
                                               off, bytes);
                                }
                        }
                    }
        }
    printf("%ld rows, %ld past 32 bits, %ld failures\n", rows, wraps, failures);
    return failures != 0 || wraps == 0;
}
