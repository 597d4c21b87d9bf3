// The 8-bit key/value cache for gfx950: taking up new tokens (quantisation), the page table and
// page copies. The cache's format is in include/np.h.
//
// Quantisation of one block (the tokens of one page, one head, K or V), with x the new tokens and
// c the codes the block already holds at exponent e0:
//     e = max(e0 if any, smallest e with max |x| <= 448 * 2^e),  code(x) = rne_e4m3(x * 2^-e),
//     c' = rne_e4m3(c * 2^(e0 - e)) where e > e0, else c.
// The scale is a power of two, so x * 2^-e and c * 2^(e0 - e) are exact and a value is rounded
// once; codes that are rescaled lose bits only where they become subnormal.
#include "kv_device.hpp"

namespace np {
namespace {

// Smallest e in [-120, 120] with a <= 448 * 2^e: a = m * 2^(x - 127), 448 = 1.75 * 2^8.
__device__ inline int exp_for(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(-120, min(120, e));
}

__device__ inline float block_max(float x, int threads, int use) {
    __shared__ float s[2][4];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x = fmaxf(x, __shfl_xor(x, d));
    if ((threadIdx.x & 63) == 0) s[use][threadIdx.x >> 6] = x;
    __syncthreads();
    for (int w = 0; w < threads >> 6; ++w) x = fmaxf(x, s[use][w]);
    return x;
}

// One workgroup per (touched page, kv head, K or V): the block's new values are read once and stay
// in registers between the maximum and the rounding. A thread holds CPT chunks of 16 codes: for K
// 16 values of one token, for V four tokens of four values (np.h), so that every store is one
// aligned 16-byte chunk of the tile. Chunks with old and new tokens (V, where the sequence did not
// end on a multiple of four) are merged in registers. Bound by memory: 4,097 tokens x 32 heads of bf16
// 28.5 us (3.5 TB/s; a large copy reaches 4.85), five prompts of fp32 31.7 us (4.25 TB/s). With pages
// first in the grid instead of heads 28.9 and 33.1 us; saturating every value 29.4 and 33.3 us. One token:
// 8.1 us a call, of which the kernel is 5: page, row, maximum over the block, store.
template <typename T, int CPT>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a) {
    const KvView& kv = a.kv;
    const int item = blockIdx.x / kv.n_kv, h = blockIdx.x - item * kv.n_kv, side = blockIdx.y;
    const int b = find_item(a.b, item);
    const int pt = 1 << kv.page_shift;
    const int before = a.b.before[b], fresh = a.b.fresh[b];
    const int index = (before >> kv.page_shift) + (item - a.b.item0[b]);
    const int t0 = index << kv.page_shift;
    const int lo = max(0, before - t0), hi = min(pt, before + fresh - t0);  // new tokens of the page
    const int page = page_of(kv, a.b.seq[b], index);
    if (page < 0) return;
    const T* const x = static_cast<const T*>(a.x[side]) + (int64_t)h * a.head_stride[side] +
                       (int64_t)(a.b.row0[b] + t0 - before) * a.row_stride[side];
    const int64_t rs = a.row_stride[side];
    int8_t* const ep = kv.exps + (((int64_t)a.layer * kv.n_pages + page) * kv.n_kv + h) * 2 + side;
    u32x4* const block = reinterpret_cast<u32x4*>(kv.codes + a.layer * kv.layer_bytes + page * kv.page_bytes +
                                                  (int64_t)(h * 2 + side) * (pt * kv.slabs * kTileDims));
    const int chunks = pt * kv.slabs * 4, nt = blockDim.x;
    const int e0 = lo > 0 ? *ep : -128;

    float v[CPT][16];
    u32x4 old[CPT];
    float top = 0.0f;
#pragma unroll
    for (int u = 0; u < CPT; ++u) {
        const int c = threadIdx.x + u * nt;
#pragma unroll
        for (int k = 0; k < 16; ++k) v[u][k] = 0.0f;
        if (c >= chunks) continue;
        if (lo > 0) old[u] = block[c];
        // chunk c: 64 per tile, tiles ordered (token group, slab)
        const int tile = c >> 6, grp = tile / kv.slabs, slab = tile - grp * kv.slabs, in = c & 63;
        if (side == 0) {
            const int t = grp * 16 + (in & 15), d = slab * 64 + (in >> 4) * 16;
            if (t >= lo && t < hi) {
                if (d < kv.hd) load_row<8>(v[u], x + t * rs + d);
                if (d + 8 < kv.hd) load_row<8>(v[u] + 8, x + t * rs + d + 8);
            }
        } else {
            const int t = grp * 16 + (in >> 4) * 4, d = slab * 64 + (in & 15) * 4;
            if (d < kv.hd) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (t + k >= lo && t + k < hi) load_row<4>(v[u] + 4 * k, x + (t + k) * rs + d);
            }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(v[u][k]));  // ignores NaN
    }
    top = block_max(top, nt, 0);
    const bool infinite = top == __builtin_inff();
    if (infinite) {  // infinities do not set the scale, and saturate
        top = 0.0f;
#pragma unroll
        for (int u = 0; u < CPT; ++u)
#pragma unroll
            for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(v[u][k]) < __builtin_inff() ? fabsf(v[u][k]) : 0.0f);
        top = block_max(top, nt, 1);
    }
    const int e = max(exp_for(top), e0);
    const bool grown = lo > 0 && e > e0;
    const float down = pow2i(max(-126, e0 - e)), unit = pow2i(-e);
#pragma unroll
    for (int u = 0; u < CPT; ++u)
#pragma unroll
        for (int k = 0; k < 16; ++k) v[u][k] *= unit;
    if (infinite) {
#pragma unroll
        for (int u = 0; u < CPT; ++u)
#pragma unroll
            for (int k = 0; k < 16; ++k) v[u][k] = sat448(v[u][k]);
    }

#pragma unroll
    for (int u = 0; u < CPT; ++u) {
        const int c = threadIdx.x + u * nt;
        if (c >= chunks) continue;
        const int tile = c >> 6, grp = tile / kv.slabs, in = c & 63;
        u32x4 w = old[u];
        if (side == 0) {
            const int t = grp * 16 + (in & 15);
            if (t >= hi || (t < lo && !grown)) continue;
            if (t >= lo) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = to_e4m3(v[u][4 * k], v[u][4 * k + 1], v[u][4 * k + 2], v[u][4 * k + 3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = rescale_e4m3(w[k], down);
            }
        } else {
            const int t = grp * 16 + (in >> 4) * 4;
            if (t >= hi || (t + 4 <= lo && !grown)) continue;
            // bytes of the word: tokens t .. t + 3 of one value
            uint32_t fresh_m = 0, old_m = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (t + k >= lo && t + k < hi) fresh_m |= 0xffu << (8 * k);
                if (t + k < lo) old_m |= 0xffu << (8 * k);
            }
            if (fresh_m != ~0u && lo == 0) w = block[c];  // tokens past the new ones keep what they hold
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t n = to_e4m3(v[u][k], v[u][4 + k], v[u][8 + k], v[u][12 + k]);
                uint32_t r = (w[k] & ~fresh_m) | (n & fresh_m);
                if (grown && old_m) r = (r & ~old_m) | (rescale_e4m3(w[k], down) & old_m);
                w[k] = r;
            }
        }
        block[c] = w;
    }
    if (threadIdx.x == 0 && e != e0) *ep = (int8_t)e;
}

template <typename T>
hipError_t append_as(const AppendArgs& a, hipStream_t s) {
    const int chunks = (1 << a.kv.page_shift) * a.kv.slabs * 4;  // 64 .. 2048, a multiple of 64
    const int nt = chunks < 256 ? chunks : 256;
    const int per = (chunks + nt - 1) / nt;
    const dim3 grid((unsigned)a.b.item0[a.b.n] * a.kv.n_kv, 2);  // heads first: neighbours read neighbouring parts of the same rows
    if (per <= 1) k_kv_append<T, 1><<<grid, nt, 0, s>>>(a);
    else if (per <= 2) k_kv_append<T, 2><<<grid, nt, 0, s>>>(a);
    else if (per <= 4) k_kv_append<T, 4><<<grid, nt, 0, s>>>(a);
    else k_kv_append<T, 8><<<grid, nt, 0, s>>>(a);
    return hipGetLastError();
}

__global__ __launch_bounds__(kTableEntries) void k_kv_table(TableArgs a) {
    const int k = threadIdx.x;
    if (k < a.n) a.table[a.at[k]] = a.page[k];
}

// Page copies, every layer at once: blockIdx.z = pair, blockIdx.y = layer, blockIdx.x = piece of
// the page. Each thread moves kCopyU 16-byte chunks, all loads issued before the stores. 217 copies of
// 512 KiB pages from 31 sources 28 us (4.1 TB/s written), about 1,000 of 64 KiB 31 us (4.2 TB/s read and
// written; a large copy reaches 4.85).
constexpr int kCopyU = 4;
__global__ __launch_bounds__(256) void k_kv_copy(CopyArgs a) {
    const int64_t src = a.src[blockIdx.z], dst = a.dst[blockIdx.z], layer = blockIdx.y;
    const u32x4* const s = reinterpret_cast<const u32x4*>(a.codes + layer * a.layer_bytes + src * a.page_bytes);
    u32x4* const d = reinterpret_cast<u32x4*>(a.codes + layer * a.layer_bytes + dst * a.page_bytes);
    const int64_t chunks = a.page_bytes / 16, c0 = (int64_t)blockIdx.x * 256 * kCopyU + threadIdx.x;
    u32x4 v[kCopyU];
#pragma unroll
    for (int u = 0; u < kCopyU; ++u)
        if (c0 + u * 256 < chunks) v[u] = s[c0 + u * 256];
#pragma unroll
    for (int u = 0; u < kCopyU; ++u)
        if (c0 + u * 256 < chunks) d[c0 + u * 256] = v[u];
    if (blockIdx.x == 0)
        for (int k = threadIdx.x; k < a.exps_page; k += 256)
            a.exps[layer * a.exps_layer + dst * a.exps_page + k] = a.exps[layer * a.exps_layer + src * a.exps_page + k];
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, int dtype, hipStream_t s) {
    if (dtype == kF32) return append_as<float>(a, s);
    if (dtype == kBF16) return append_as<__bf16>(a, s);
    return append_as<_Float16>(a, s);
}

hipError_t launch_kv_table(const TableArgs& a, hipStream_t s) {
    k_kv_table<<<1, kTableEntries, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv_copy(const CopyArgs& a, hipStream_t s) {
    const int64_t per = 256 * kCopyU * 16;
    k_kv_copy<<<dim3((unsigned)((a.page_bytes + per - 1) / per), a.layers, a.n), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace np
