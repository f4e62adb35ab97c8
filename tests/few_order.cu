// Host check of the order in which the few-row attention kernel over codes issues its products: walks pieces of random lengths with the kernel's own rule
// and looks for scores that go to a buffer whose last tile has no weighted sum yet.  Prints "ok <cases> <tiles>" or the first that does.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>
#include <vector>

#include "sv_attend_few.cuh"

using namespace sv;

static std::mt19937_64 rng(1);

struct Order {
    uint32_t n = 0, weighed = 0, groups = 0, tiles[2] = {0, 0};
    std::vector<int> buffer;   // of tile i: 2 * group + place
    int last[4] = {-1, -1, -1, -1};   // the tile that a buffer holds
    int rests = 0, most_ahead = 0;

    // false: scores over ones that are still read.  `eager`: what comes next is always ready, so that sums are issued only when they are due.
    template <class Due>
    bool piece(int nk, bool eager, Due due) {
        if (nk == 1) rests ^= 1;
        const int first = nk == 1 ? rests ^ 1 : 0;
        for (int i = -1; i < nk; ++i) {   // -1: the piece itself
            const int gr = first ^ (i & 1);
            while (weighed < n && (due(n - weighed, groups, i < 0 ? -1 : gr) || !(eager || rng() % 2))) {
                ++weighed;
                groups >>= 1;
            }
            if (i < 0) continue;
            const int b = gr * 2 + (tiles[gr] & 1);
            if (last[b] >= (int)weighed) return false;
            last[b] = (int)n;
            groups |= (uint32_t)gr << (n - weighed);
            ++tiles[gr];
            ++n;
            most_ahead = std::max(most_ahead, (int)(n - weighed));
        }
        return true;
    }
};

int main() {
    const auto rule = [](uint32_t waiting, uint32_t groups, int next) { return sum_is_due(waiting, groups, next); };
    const auto three = [](uint32_t waiting, uint32_t, int) { return waiting == 3; };   // without a look at the groups
    Order bad;
    if (bad.piece(3, true, three) && bad.piece(1, true, three) && bad.piece(2, true, three)) {
        printf("three tiles of one group in a row were not met\n");
        return 1;
    }
    long long tiles = 0;
    const int cases = 20000;
    for (int c = 0; c < cases; ++c) {
        Order o;
        const bool eager = c % 2;
        std::vector<int> done;
        for (int p = 0; p < 40; ++p) {
            done.push_back(1 + (int)(rng() % (c % 3 == 0 ? 3 : c % 3 == 1 ? 2 : 9)));
            if (!o.piece(done.back(), eager, rule)) {
                printf("overwritten after pieces of");
                for (int nk : done) printf(" %d", nk);
                printf("\n");
                return 1;
            }
        }
        tiles += o.n;
        Order whole;   // a long piece keeps its lead of two tiles
        whole.piece(50, true, rule);
        if (whole.most_ahead != 3) {
            printf("a lead of %d\n", whole.most_ahead);
            return 1;
        }
    }
    printf("ok %d %lld\n", cases, tiles);
    return 0;
}
