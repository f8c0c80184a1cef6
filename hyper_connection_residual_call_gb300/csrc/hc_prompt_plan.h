// hc_prompt_plan.h -- the counts of blocks of the attention over packed prompts (hc_prompt_attn.cu). Host and device;
// no pointers, so that they can be looked through on a CPU.
#pragma once

#include <cuda_runtime.h>

#include <climits>

namespace tshc {

constexpr int kRound = 256;  // sequences whose blocks are taken in turn

// Blocks that are counted of a sequence, so that a round's fit an int. (A block has 32 KB of queries or more, and of
// results: more blocks than these are no GPU's.)
constexpr int kMostBlocks = INT_MAX / kRound;

// Blocks of `rows` tokens of a sequence that has the rows lo .. hi - 1 of N; -1 for one that is out of range.
__host__ __device__ inline int blocks_of_rows(int lo, int hi, int N, int rows)
{
    if (lo < 0 || hi < lo || hi > N)
        return -1;
    const unsigned n = ((unsigned)(hi - lo) + (unsigned)rows - 1) / (unsigned)rows;  // (32 bits: a planning warp waits for it)
    return n < (unsigned)kMostBlocks ? (int)n : kMostBlocks;
}

// Blocks up to a round's end: at most INT_MAX, for sequences that overlap, where starts descends, can have more
// (the grid has not).
__host__ __device__ inline int add_blocks(int before, int round)
{
    return round < INT_MAX - before ? before + round : INT_MAX;
}

}  // namespace tshc
