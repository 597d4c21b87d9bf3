// The 8-bit key/value cache for gfx950: taking up new tokens (quantisation), the page table and
// page copies. The cache's format is in include/np.h.
//
// Quantisation of one block (the tokens of one page, one head, K or V), with x the new tokens and
// c the codes the block already holds at exponent e0:
//     e = max(e0 if any, smallest e with max |x| <= 448 * 2^e),  code(x) = rne_e4m3(x * 2^-e),
//     c' = rne_e4m3(c * 2^(e0 - e)) where e > e0, else c.
// The scale is a power of two, so x * 2^-e and c * 2^(e0 - e) are exact and a value is rounded
// once; codes that are rescaled lose bits only where they become subnormal.
#include "kv_quant.hpp"

namespace np {
namespace {

// One workgroup per (touched page, kv head, K or V): the block's new values are read once and stay
// in registers between the maximum and the rounding (quantise_block). Bound by memory: 4,097 tokens x 32 heads of bf16
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
    const auto load_k = [&](float* v, int t, int d) {
        load_row<8>(v, x + t * rs + d);
        if (d + 8 < kv.hd) load_row<8>(v + 8, x + t * rs + d + 8);
    };
    const auto load_v = [&](float* v, int t, int d) { load_row<4>(v, x + t * rs + d); };
    quantise_block<CPT>(kv, a.layer, page, h, side, lo, hi, load_k, load_v);
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
