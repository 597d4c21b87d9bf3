// Internal declarations of the 8-bit key/value cache: what the host library passes to the gfx950
// kernels of k_kv.hip (append, page table, page copies) and k_attn.hip (attention).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace np {

// Limits (also documented in include/np.h).
constexpr int kMaxHeadDim = 256;
constexpr int kMaxPageTokens = 128;
constexpr int kMaxBatch = 128;        // sequences of one np_kv_extend
constexpr int kMaxSeqTokens = 1 << 28;

// The code tile: 16 tokens x 64 values = 1024 bytes, laid out in the lane order of the 16x16x32
// matrix instructions so that a wave reads a tile as 64 consecutive 16-byte chunks, each lane's
// chunk being exactly its operand (np.h gives the byte order).
constexpr int kTileTokens = 16;
constexpr int kTileDims = 64;
constexpr int kTileBytes = kTileTokens * kTileDims;

// One cache as the kernels see it (by value in every launch's arguments).
struct KvView {
    uint8_t* codes;        // [layers][pages][kv heads][2][page_tokens / 16][slabs][1024]
    int8_t* exps;          // [layers][pages][kv heads][2]
    const int32_t* table;  // [max_seqs][max_pages] page of each sequence position, -1: dropped
    int64_t page_bytes;    // codes of one page of one layer
    int64_t layer_bytes;   // codes of one layer
    int32_t n_pages, max_pages;
    int32_t page_shift;    // log2(page_tokens)
    int32_t n_heads, n_kv, hd, slabs;  // slabs: 64-value columns of a head (ceil(hd / 64))
};

// The sequences of the current np_kv_extend, by value. row0 is a sequence's first row in the
// caller's tensors; item0 the first work item of the sequence in this launch (items of all
// sequences are numbered through, item0[n] is their count).
struct KvBatch {
    int32_t n;
    int32_t seq[kMaxBatch];
    int32_t before[kMaxBatch];  // tokens before the new ones
    int32_t fresh[kMaxBatch];   // new tokens
    int32_t row0[kMaxBatch];
    int32_t item0[kMaxBatch + 1];
    // Attention only: pieces of the key axis per row tile, and the sequence's first partial result
    // (in units of one item of every kv head; sequences with one piece have none).
    int32_t splits[kMaxBatch];
    int32_t part0[kMaxBatch];
};

struct AppendArgs {
    KvView kv;
    const void* x[2];       // K, V
    int64_t row_stride[2];  // elements
    int64_t head_stride[2];
    int32_t layer;
    KvBatch b;  // item = one touched page of one sequence
};

struct AttnArgs {
    KvView kv;
    const void* q;
    void* out;
    float* lse;  // [rows][heads] or nullptr
    int64_t q_row, q_head, o_row, o_head;  // strides in elements
    float scale2;        // softmax scale * log2(e)
    int32_t window;      // 0: none
    int32_t sinks;
    int32_t layer;
    int32_t row_cap;     // rows of the largest tile in this launch (LDS is sized for it)
    float* part;         // [partial][kv head][row_cap][64 slabs + 2] partial results
    uint32_t* arrived;   // [partial][kv head] splits done (at the tile's first partial), 0 between launches
    KvBatch b;  // item = one (row tile, split) of one sequence
};
static_assert(sizeof(AttnArgs) <= 4096 && sizeof(AppendArgs) <= 4096, "kernel arguments are limited to 4 KiB");

// Attention over few rows: how many partial results (workgroups that share a row tile with others)
// one launch may have, and how many rows these may have together; the waves of a workgroup.
constexpr int kAttnWaves = 8;
constexpr int kRowTile = 16;
constexpr int kPieceTokens = 32;
constexpr int kMaxPartials = 8192;
constexpr int kMaxPartialRows = 32768;

// Page table entries to write: table[at[k]] = page[k], k < n.
constexpr int kTableEntries = 480;
struct TableArgs {
    int32_t* table;
    int32_t n;
    int32_t at[kTableEntries], page[kTableEntries];
};

constexpr int kCopyPairs = 448;
struct CopyArgs {
    uint8_t* codes;
    int8_t* exps;
    int64_t page_bytes, layer_bytes;
    int32_t exps_page;   // exponent bytes of one page of one layer
    int64_t exps_layer;
    int32_t n, layers;
    int32_t src[kCopyPairs], dst[kCopyPairs];
};

enum KvDtype { kF32 = 0, kBF16 = 1, kF16 = 2 };

hipError_t launch_kv_append(const AppendArgs& a, int dtype, hipStream_t s);
hipError_t launch_kv_table(const TableArgs& a, hipStream_t s);
hipError_t launch_kv_copy(const CopyArgs& a, hipStream_t s);
// part set: few rows a sequence (items are row tiles of kRowTile rows, split); part nullptr: many
// rows (items are attn_tile_rows() rows each; 0: there is no such kernel).
hipError_t launch_attn(const AttnArgs& a, int dtype, hipStream_t s);
int attn_tile_rows(int dtype, int slabs);
// Lets the attention kernels of the current device use the LDS they ask for (above 64 KiB).
hipError_t attn_prepare();

}  // namespace np
