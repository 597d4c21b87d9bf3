// Quantisation of one block of the 8-bit key/value cache by one workgroup: the rule is in k_kv.hip.
#pragma once

#include "kv_device.hpp"

namespace np {

// Smallest e in [-120, 120] with a <= 448 * 2^e: a = m * 2^(x - 127), 448 = 1.75 * 2^8.
__device__ inline int exp_for(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(-120, min(120, e));
}

// The maximum over the workgroup (at most 512 threads); `use` numbers the calls of one kernel.
__device__ inline float block_max(float x, int threads, int use) {
    __shared__ float s[2][8];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x = fmaxf(x, __shfl_xor(x, d));
    if ((threadIdx.x & 63) == 0) s[use][threadIdx.x >> 6] = x;
    __syncthreads();
    for (int w = 0; w < threads >> 6; ++w) x = fmaxf(x, s[use][w]);
    return x;
}

// The block's exponent, from its new values v and the one it has (e0; -128: none), by which it then scales v.
template <int CPT>
__device__ inline int scale_block(float (&v)[CPT][16], int e0, int nt) {
    float top = 0.0f;
#pragma unroll
    for (int u = 0; u < CPT; ++u)
#pragma unroll
        for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(v[u][k]));  // ignores NaN
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
    const float unit = pow2i(-e);
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
    return e;
}

// Stores the new tokens [lo, hi) of block (layer, page, head h, side: 0 K, 1 V). A thread holds CPT chunks of 16
// codes: for K 16 values of one token, for V four tokens of four values (np.h), so that every store is one
// aligned 16-byte chunk of the tile. Chunks with old and new tokens (V, where the sequence did not end on a
// multiple of four) are merged in registers. load_k(v, t, d) gives K's values d .. d + 15 of token t, load_v(v, t, d)
// V's values d .. d + 3 of token t, as fp32 (those past the head dimension left as they are: 0).
template <int CPT, typename LoadK, typename LoadV>
__device__ inline void quantise_block(const KvView& kv, int layer, int page, int h, int side, int lo, int hi, LoadK load_k, LoadV load_v) {
    const int pt = 1 << kv.page_shift;
    int8_t* const ep = kv.exps + (((int64_t)layer * kv.n_pages + page) * kv.n_kv + h) * 2 + side;
    u32x4* const block = reinterpret_cast<u32x4*>(kv.codes + layer * kv.layer_bytes + page * kv.page_bytes +
                                                  (int64_t)(h * 2 + side) * (pt * kv.slabs * kTileDims));
    const int chunks = pt * kv.slabs * 4, nt = blockDim.x;
    const int e0 = lo > 0 ? *ep : -128;

    float v[CPT][16];
    u32x4 old[CPT];
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
            if (t >= lo && t < hi && d < kv.hd) load_k(v[u], t, d);
        } else {
            const int t = grp * 16 + (in >> 4) * 4, d = slab * 64 + (in & 15) * 4;
            if (d < kv.hd) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (t + k >= lo && t + k < hi) load_v(v[u] + 4 * k, t + k, d);
            }
        }
    }
    const int e = scale_block(v, e0, nt);
    const bool grown = lo > 0 && e > e0;
    const float down = pow2i(max(-126, e0 - e));

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

}  // namespace np
