// Host check of the tokens whose pages the loading warps of attention over codes ask for ahead, at the end of the longest contexts, for every
// lane and box.  Prints "ok <places looked at> <places that a lane's own offset would have put past 32 bits>" or the first that is wrong.
#include <stdint.h>
#include <stdio.h>

#include "sv_attend_feed8.cuh"

using namespace sv;

int main() {
    long long seen = 0, past = 0;
    for (int64_t end = (int64_t)kMaxSlots - 2000; end <= kMaxSlots; ++end) {
        for (int64_t key0 : {(int64_t)0, (int64_t)1, end / 2, end - 700, end - 1}) {
            const int64_t tiles = (end - key0 + kTcKeys - 1) / kTcKeys;   // k0 .. k1 of a piece end here at most; one tile is asked for past them
            for (int64_t k = tiles - 3 < 0 ? 0 : tiles - 3; k <= tiles; ++k)
                for (int rows : {8, 16, 32})
                    for (int lane = 0; lane < 32; ++lane) {
                        const int64_t first = key0 + k * kTcKeys, own = first + lane * rows, at = first + box_offset(lane, rows);
                        if (at > INT32_MAX || (lane * rows < kTcKeys && at != own))
                            return printf("tile at %lld, lane %d, boxes of %d: %lld\n", (long long)first, lane, rows, (long long)at), 1;
                        past += own > INT32_MAX;
                        ++seen;
                    }
        }
    }
    printf("ok %lld %lld\n", seen, past);
    return 0;
}
