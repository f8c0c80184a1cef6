// The counts of blocks before each round of sequences (hc_prompt_plan.h), for sequences that all overlap and have more
// blocks together than an int holds, and for ordinary ones: they never fall, and are right where they fit. Prints what
// went wrong; exits 0 if nothing did.
#include <algorithm>
#include <cstdio>
#include <vector>

#include "hc_prompt_plan.h"

namespace {

int look(const std::vector<int> &starts, int N, int rows, const char *what)
{
    const int S = (int)starts.size() - 1;
    int sum = 0, wrong = 0;
    long truth = 0;
    for (int r = 0; r * tshc::kRound < S; ++r) {
        long round = 0;
        for (int s = r * tshc::kRound; s < std::min(S, (r + 1) * tshc::kRound); ++s)
            round += std::max(tshc::blocks_of_rows(starts[s], starts[s + 1], N, rows), 0);
        truth += round;
        const int next = round <= INT_MAX ? tshc::add_blocks(sum, (int)round) : -1;
        if (next < sum || next != std::min<long>(truth, INT_MAX)) {
            std::printf("%s: round %d: %d blocks after %d, %ld in truth\n", what, r, next, sum, truth);
            ++wrong;
        }
        sum = next;
    }
    return wrong;
}

}  // namespace

int main()
{
    int wrong = 0;
    std::vector<int> overlap(65536), plain(1001);
    for (int N : {5000, 524304, 1 << 30, INT_MAX}) {
        for (int i = 0; i < 65536; ++i)
            overlap[i] = i % 2 ? N : 0;
        for (int rows : {8, 256})
            wrong += look(overlap, N, rows, "overlapping");
    }
    for (int i = 0; i <= 1000; ++i)
        plain[i] = i * 37 - i % 5;
    wrong += look(plain, 37000, 8, "plain");
    for (int bad : {-1, INT_MIN})
        wrong += tshc::blocks_of_rows(bad, 10, 100, 8) != -1;
    wrong += tshc::blocks_of_rows(5, 4, 100, 8) != -1 || tshc::blocks_of_rows(0, 101, 100, 8) != -1 || tshc::blocks_of_rows(3, 3, 100, 8) != 0;
    return wrong != 0;
}
