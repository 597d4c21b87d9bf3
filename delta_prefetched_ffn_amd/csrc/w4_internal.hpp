// Internal declarations of the products with 4-bit weights: what the host side (np_w4.hip) passes to the gfx950 kernels
// of k_w4.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace np {

// The weight tile: 16 outputs x 128 inputs = 1024 bytes, in the lane order of the 16x16x32 matrix instructions: lane
// 16 g + o holds output o's inputs 32 s + 8 g + j, dword s, nibble 2 j (j < 4) or 2 j - 7.
constexpr int kW4Outs = 16;
constexpr int kW4Ins = 128;
constexpr int kW4TileBytes = kW4Outs * kW4Ins / 2;

struct W4View {
    const uint8_t* tiles;   // [out tiles][chunks][1024]
    // [out tiles][chunks * per_chunk][16] groups of scale_words dwords: the scale as fp32, and the zero point in the low 4 bits of the last
    // dword. A 16-bit scale leaves those bits of its fp32 value free, so one dword holds both; an fp32 scale takes two.
    const uint32_t* scales;
    int32_t n_out, n_in;
    int32_t out_tiles, chunks;
    int32_t per_chunk;      // groups of a chunk: 1, 2 or 4
    int32_t scale_words;
};

struct W4Args {
    W4View w;
    const void* x;
    void* y;
    int64_t rows, x_row, y_row;  // strides in elements
    int32_t y_dtype;
    int32_t accumulate;
};

struct W4PackArgs {
    const uint8_t* codes;   // [n_out][n_in / 2]
    const void* scales;     // [n_out][groups]
    const uint8_t* zeros;   // the same shape, or nullptr
    uint8_t* tiles;
    uint32_t* scales_out;
    int32_t n_out, n_in, out_tiles, chunks, per_chunk;
    int32_t group, groups;  // inputs of a group, groups of a row, as given
    int32_t scale_dtype;
};

hipError_t launch_w4_pack(const W4PackArgs& a, hipStream_t s);
hipError_t launch_w4(const W4Args& a, int x_dtype, hipStream_t s);
hipError_t w4_prepare();  // lets the current device's kernels use the LDS they ask for

}  // namespace np
