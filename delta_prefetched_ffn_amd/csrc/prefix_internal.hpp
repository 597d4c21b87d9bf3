// Internal declarations of the attention over shared first pages: what the host side (np_prefix.hip) passes to the gfx950
// kernels of k_prefix.hip.
#pragma once

#include "kv_internal.hpp"

namespace np {

// Shared runs of pages that one call works out once each, at most; further ones are read by each sequence.
constexpr int kMaxRuns = 32;
constexpr int kRunWaves = 4;       // waves of a workgroup
constexpr uint8_t kNoRun = 255;

// A run of tokens [t0, t1) (whole pages) that the sequences [s0, s1) of the batch share.
struct PrefixRun {
    int32_t t0, t1;
    int32_t item0;      // its first work item: (row tile, split)
    int32_t part0;      // its first partial row (of one kv head)
    uint16_t splits;
    uint8_t s0, s1;
};

struct PrefixArgs {
    KvView kv;
    const void* q;
    void* out;
    float* lse;                            // [rows][heads] or nullptr
    int64_t q_row, q_head, o_row, o_head;  // strides in elements
    float* part;                           // partial rows: [row][64 slabs + 2]
    float scale2;                          // softmax scale * log2(e)
    int32_t window, sinks, layer;
    int32_t n, n_runs;
    int32_t leaf_item, leaf_part;          // the sequences' own items and partial rows start here
    int32_t leaf_cap;                      // rows of their largest tile
    int32_t even;                          // the new tokens of every sequence, or 0: they differ
    int32_t rows;
    PrefixRun run[kMaxRuns];
    // The batch, in an order in which sequences that share a run are neighbours.
    int32_t before[kMaxBatch];             // tokens before the new ones
    int32_t cum[kMaxBatch + 1];            // new tokens of the sequences in front
    int32_t row0[kMaxBatch];               // first row in the caller's tensors
    int32_t item0[kMaxBatch + 1];          // first work item of its own tokens, from leaf_item
    uint16_t seq[kMaxBatch], splits[kMaxBatch];
    uint8_t deepest[kMaxBatch];            // the last run that it is part of (its own tokens start behind), or kNoRun
};
static_assert(sizeof(PrefixArgs) <= 4096, "kernel arguments are limited to 4 KiB");

// Row tiles of 16 that a workgroup takes over a run (or over a sequence's own tokens, where it has more than 16 rows), and the
// waves that a SIMD then holds. A wave issues an instruction about every 11 clocks, a SIMD takes a vector one every 4: more
// waves of fewer rows are ahead of few of many (also at 128 values a head, where three waves leave 2 registers to be spilled). Measured in bf16 at head_dim 128 and 8 kv heads, two tiles at
// three waves against four tiles at two: 32 sequences behind 8,011 tokens 24.8 us for 29, 8 sequences of 31 rows x 4 behind
// 8,000 tokens 58 for 66; only very long runs of many rows go the other way (two of 30 Ki tokens at most for 540 rows each, 205 for 181).
constexpr int run_tiles(int dtype, int slabs) { return slabs <= 2 ? 2 : 1; }
constexpr int run_eu(int dtype, int slabs) { return slabs == 1 ? 4 : slabs == 4 ? 2 : 3; }

hipError_t launch_prefix(const PrefixArgs& a, int dtype, hipStream_t s);
hipError_t prefix_prepare();  // lets the current device's kernels use the LDS they ask for

}  // namespace np
