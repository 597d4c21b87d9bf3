// Internal declarations of the rotary positions: what the host side (np_rope.hip) passes to the gfx950 kernels of
// k_rope.hip.
#pragma once

#include "kv_internal.hpp"

namespace np {

// A rotation as the kernels see it.
struct RopeView {
    const uint64_t* turns;  // [rot / 2]: what a pair turns by per position, in 2^-64 of a full turn
    float amplitude;
    float eps;
    int32_t hd, rot;        // head dimension, its first values that turn
    int32_t layout;         // np_rope_layout
};

// One tensor [rows][heads][hd] with its result and the weights of its norm (nullptr: none).
struct RopeTensor {
    const void* in;
    void* out;
    const float* weight;
    int64_t in_row, in_head, out_row, out_head;  // strides in elements
    int32_t heads;
};

struct RopeArgs {
    RopeView rope;
    RopeTensor x[2];             // queries, keys (no heads: none)
    const int32_t* positions;    // [rows], or nullptr: first + row
    int32_t first;
    int64_t rows;
    int32_t per;                 // head groups that a wave takes (rope_groups() in a row)
};

// The current batch without what attention alone needs.
struct RopeBatch {
    int32_t n;
    int32_t seq[kMaxBatch], before[kMaxBatch], fresh[kMaxBatch], row0[kMaxBatch];
    int32_t item0[kMaxBatch + 1];  // item = one touched page of one sequence
};

struct RopeAppendArgs {
    KvView kv;
    RopeView rope;
    RopeTensor q;       // its rows are the current tokens'
    const void* kx[2];  // K, V
    const float* k_weight;
    int64_t row_stride[2], head_stride[2];
    int32_t layer;
    int32_t rows;
    int32_t per;        // as above, for q
    int32_t heads;      // of K that a workgroup takes
    RopeBatch b;
};
static_assert(sizeof(RopeAppendArgs) <= 4096, "kernel arguments are limited to 4 KiB");

// Lanes that hold one head: 16 values each, a power of two.
constexpr int rope_lanes(int hd) { return hd <= 16 ? 1 : hd <= 32 ? 2 : hd <= 64 ? 4 : hd <= 128 ? 8 : 16; }
// The same on the way into the cache, whose blocks hold whole slabs of 64 values.
constexpr int append_lanes(int hd, int slabs) { return rope_lanes(hd) > slabs * 4 ? rope_lanes(hd) : slabs * 4; }
// Threads of a workgroup there: 16 values each of a page's tokens, up to four tokens' where 512 do not reach.
constexpr int kAppendWg = 512;
constexpr int append_threads(int page_shift, int hd, int slabs) {
    return (append_lanes(hd, slabs) << page_shift) < kAppendWg ? append_lanes(hd, slabs) << page_shift : kAppendWg;
}
// Groups of heads in a row (one wave's worth each).
constexpr int rope_groups(int hd, int heads) { return (heads + 64 / rope_lanes(hd) - 1) / (64 / rope_lanes(hd)); }

// Workgroups of a call.
inline int64_t append_grid(const RopeAppendArgs& a) {
    const int groups = rope_groups(a.kv.hd, a.q.heads), waves = append_threads(a.kv.page_shift, a.kv.hd, a.kv.slabs) / 64;
    const int64_t rows = (int64_t)a.rows * ((groups + a.per - 1) / a.per);
    return (int64_t)a.b.item0[a.b.n] * (a.kv.n_kv + (a.kv.n_kv + a.heads - 1) / a.heads) + (rows + waves - 1) / waves;
}

hipError_t launch_rope(const RopeArgs& a, int dtype, hipStream_t s);
hipError_t launch_rope_append(const RopeAppendArgs& a, int dtype, hipStream_t s);

}  // namespace np
