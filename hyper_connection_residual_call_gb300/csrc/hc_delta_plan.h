// hc_delta_plan.h -- how the gated delta rule over packed prompts (hc_delta_prompt.cu) is cut into chunks, and long
// sequences into segments. Host and device; no pointers, so that the plan can be looked through on a CPU.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>

namespace tshc {

constexpr int kChunk = 64;

// Chunks of a segment, where sequences are cut into segments that are walked side by side; 0: they are not.
// A segment after the first is walked for what it makes of a state, S -> F S + B (F from the identity and no
// values, B from a state of zeros), then the segments' states are known one after the other, and it is walked again,
// but for the first, for its outputs. So n segments take the time of two, with 2 n - 3 walks a head at once: n is what
// the SMs hold, a walk a SM, and at least three, of eight chunks at least. One sequence, without and with segments: 8192
// tokens of 32 heads of 128 (three segments) 571 and 471 us, of 8 heads 455 and 228; 65536 tokens of 4 heads 3290 and
// 672; 2048 tokens of 8 heads 125 and 113; but 1100 tokens of 4 heads 81 and 96, hence the 24 chunks. (Before the first
// and the joining kernel had their present form; by now the second of each pair are 394, 175, 536 and 101.)
// kSms is the GPU's, not asked of the device: the workspace's size follows from the plan and is known without one.
constexpr int kSms = 152, kLeastSegment = 8, kLeastCut = 24;
inline int segment_chunks(int N, int S, int Hv)
{
    const long walks = (long)S * Hv, chunks = ((long)N + kChunk - 1) / kChunk;
    const long n = walks > 0 ? (kSms / walks + 3) / 2 : 0;
    if (n < 3)
        return 0;
    const long each = std::max<long>((chunks + S * n - 1) / (S * n), kLeastSegment);
    return chunks > S * std::max<long>(2 * each, kLeastCut) ? (int)each : 0;
}

// Whether the last segments' part of the first kernel runs beside the first walks, which do not need it, on the SMs that
// these leave idle: where that is a quarter of them, and there is enough of it. 8192 tokens of 32 heads of 128, 96
// walks, 419 us without and 394 with, but 2048 tokens 130 and 134.
constexpr int kLeastApart = 40;               // chunks a sequence
inline bool apart(int N, int S, int Hv, int seg)
{
    const long chunks = ((long)N + kChunk - 1) / kChunk, n = (chunks + (long)S * seg - 1) / ((long)S * seg);
    return (long)S * Hv * (2 * n - 3) <= kSms * 3 / 4 && chunks >= (long)S * kLeastApart;
}

// The segments' ends lie by head, and within one by the sequence's first token / 64 / seg, plus the sequence, plus the
// segment: no two sequences' overlap.
__host__ __device__ inline long segment_slots(int N, int S, int seg) { return (long)N / kChunk / seg + S; }

// The most of them that any call of up to N tokens and S sequences has, so that a workspace for the largest call serves
// every smaller one: by s sequences, N / 64 / seg is at most N / 64 / kLeastSegment and at most their s n segments.
inline long most_segment_slots(int N, int S, int Hv)
{
    const long chunks = ((long)N + kChunk - 1) / kChunk;
    long most = 0;
    for (long s = 1; s <= S && chunks > s * kLeastCut; ++s) {
        const long n = (kSms / (s * Hv) + 3) / 2;
        if (n < 3)
            break;
        most = std::max(most, std::min((long)N / kChunk / kLeastSegment, s * n) + s);
    }
    return most;
}

// Where a segment's walk takes its state from and leaves it.
enum Place {
    kNowhere,
    kState,      // state_in, state_out
    kEnd,        // the segment's own end: B's, or F's where the walk has no values
    kEndBefore   // the joined end (B's place) of the segment before
};
struct Walk {
    bool mine = false, outputs = false;
    Place from = kNowhere, to = kNowhere;
};
// The walk of segment `at` of a sequence whose last segment is `last`: the first walks (`values`: with them, for B;
// without, for F) or, `again`, those for the outputs. Walks of one launch run in any order: what one of them writes
// none of the others reads.
__host__ __device__ inline Walk walk_of(long at, long last, bool values, bool again)
{
    Walk w;
    w.mine = at >= 0 && at <= last && (again ? at > 0 : at == 0 ? values : at < last);
    if (!w.mine)
        return w;
    w.from = at == 0 ? kState : again ? kEndBefore : kNowhere;
    // (again, only the last one's state is anyone's: the joined end, which the next segment's walk begins from, stays)
    w.to = at == last ? kState : again ? kNowhere : kEnd;
    w.outputs = again || at == 0;
    return w;
}

}  // namespace tshc
