// The room for the segments' ends (hc_delta_plan.h): no call that a workspace is large enough for has more of them than
// it has places. Prints what went wrong; exits 0 if nothing did.
#include <cstdio>

#include "hc_delta_plan.h"

int main()
{
    int wrong = 0;
    for (int Hv : {1, 2, 3, 4, 8, 16, 32, 50, 51, 64, 1024})
        for (int S = 1; S < 60; ++S)
            for (int N = 1; N < 400000; N += N < 6000 ? 61 : 977) {
                const int seg = tshc::segment_chunks(N, S, Hv);
                const long most = tshc::most_segment_slots(N, S, Hv);
                if ((seg > 0 && tshc::segment_slots(N, S, seg) > most) || most > tshc::most_segment_slots(N + 61, S, Hv) ||
                    most > tshc::most_segment_slots(N, S + 1, Hv)) {
                    std::printf("N %d S %d Hv %d: segments of %d, %ld places\n", N, S, Hv, seg, most);
                    ++wrong;
                }
            }
    return wrong != 0;
}
