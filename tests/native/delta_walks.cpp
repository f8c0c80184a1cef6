// The walks of the gated delta rule's segments (hc_delta_plan.h): within a launch no walk reads or writes what another
// one writes, each reads what an earlier launch left, and each segment's outputs and the last state are made once.
// Prints what went wrong; exits 0 if nothing did.
#include <cstdio>
#include <set>
#include <string>
#include <vector>

#include "hc_delta_plan.h"

namespace {

int wrong = 0;

void expect(bool ok, const char *what, long last, long at)
{
    if (!ok) {
        std::printf("%s: segment %ld of %ld\n", what, at, last + 1);
        ++wrong;
    }
}

struct Access {
    std::string from, to;
    long at;
};

std::string place(tshc::Place p, long at, bool values)
{
    switch (p) {
    case tshc::kState: return "state";  // state_out may be state_in
    case tshc::kEnd: return (values ? "B" : "F") + std::to_string(at);
    case tshc::kEndBefore: return "B" + std::to_string(at - 1);
    default: return "";
    }
}

}  // namespace

int main()
{
    for (long last = 0; last < 9; ++last) {
        std::set<std::string> left = {"state"};  // what has been written before the launch
        std::vector<int> outputs(last + 1, 0);
        int states = 0;
        for (int again = 0; again < 2; ++again) {
            std::vector<Access> walks;
            for (long at = -1; at <= last + 1; ++at)
                for (int values = again; values < 2; ++values) {
                    const tshc::Walk w = tshc::walk_of(at, last, values, again);
                    expect(w.mine || (w.from == tshc::kNowhere && w.to == tshc::kNowhere && !w.outputs), "not a walk, but has a place", last, at);
                    if (!w.mine)
                        continue;
                    expect(at >= 0 && at <= last, "out of the sequence", last, at);
                    walks.push_back({place(w.from, at, values), place(w.to, at, values), at});
                    outputs[at] += w.outputs;
                    states += w.to == tshc::kState;
                }
            for (size_t i = 0; i < walks.size(); ++i) {
                expect(walks[i].from.empty() || left.count(walks[i].from), "reads what nothing has written", last, walks[i].at);
                for (size_t j = 0; j < walks.size(); ++j)
                    if (i != j && !walks[i].to.empty())
                        expect(walks[i].to != walks[j].from && walks[i].to != walks[j].to, "writes what another walk of the launch uses", last, walks[i].at);
            }
            for (const Access &w : walks)
                left.insert(w.to);
            if (!again)  // the joining kernel: B at <- F at (B at-1) + B at, from the second segment to the last but one
                for (long at = 1; at < last; ++at)
                    expect(left.count("F" + std::to_string(at)) && left.count("B" + std::to_string(at)), "joins what nothing has written", last, at);
        }
        for (long at = 0; at <= last; ++at)
            expect(outputs[at] == 1, "outputs not made once", last, at);
        expect(states == 1, "the last state not made once", last, last);
    }
    return wrong != 0;
}
