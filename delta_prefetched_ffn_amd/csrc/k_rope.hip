// Rotary positions for gfx950, with the norms of queries and keys in the same pass, and the same on the way into the
// 8-bit key/value cache (semantics: include/np.h).
//
// For a head x of `hd` values at position p, with w the norm's weights (none: x as it is):
//     y = x * w / sqrt(mean(x^2) + eps),   (y_a, y_b) -> A (y_a cos t - y_b sin t, y_a sin t + y_b cos t)
// for pair i = (a, b) of the first `rot` values, t = 2 pi p F_i. F_i, a fraction of a turn, is held to the nearest 2^-64, so p F_i
// mod 1 is the low half of an integer product, off by |p| 2^-65 (2^-34 at the farthest positions), where a float product p F_i
// loses the angle of far ones. What is left is an eighth of a turn at most, whose sine and cosine come from their power series in
// fp32 (off by 4.5e-8 at most, of which their rounding to fp32 is 3.0e-8).
//
// Bound by memory where there are many rows: 4,099 rows of 40 heads of 128 in fp16, 64 values of each turned, 17.2 us (4.9 TB/s, a large
// copy's rate), one row of 64 heads 4.6 us in the trace, of which an empty launch is 3.4.
#include "kv_quant.hpp"
#include "rope_internal.hpp"

namespace np {
namespace {

// 2 pi / 2^32, and what fp32 leaves out of it.
constexpr float kTurn = 1.46291807926715968e-9f, kTurnRest = (float)(1.46291807926715968105e-9 - (double)kTurn);
// cos and sin of the angle of pair i at position p, times the amplitude.
__device__ inline f32x2 turn_of(uint64_t f, int p) {
    const uint32_t lo = (uint32_t)f, hi = (uint32_t)(f >> 32), u = (uint32_t)p;
    // (f * p) mod 2^64, p sign-extended: its upper word t, and the lower one
    const uint64_t prod = (uint64_t)lo * u;
    const uint32_t t = (uint32_t)(prod >> 32) + hi * u - (p < 0 ? lo : 0u), below = (uint32_t)prod;
    // t = q quarters + r, r in [-1/8, 1/8) turns
    const uint32_t q = (t + 0x20000000u) >> 30;
    // x + e = (r + below / 2^32) 2 pi / 2^32, |x| <= pi / 4: the upper bits of r are exact in fp32, and so is what the product with
    // them leaves out.
    const int32_t r = (int32_t)(t - (q << 30)), r0 = r & ~255;
    const float u0 = (float)r0, x = u0 * kTurn;
    const float rest = __builtin_fmaf((float)below, 0x1p-32f, (float)(r - r0));
    const float e = __builtin_fmaf(rest, kTurn, __builtin_fmaf(u0, kTurnRest, __builtin_fmaf(u0, kTurn, -x)));
    const float z = __builtin_fmaf(x, x, 2.0f * x * e);
    // Taylor series: what is left out is below 2^-28 of the sine and 2^-32 of the cosine, whose 1 - z / 2 keeps what its rounding leaves out.
    float s = __builtin_fmaf(z, 2.75573192e-6f, -1.98412698e-4f);
    s = __builtin_fmaf(z, s, 8.33333333e-3f);
    s = __builtin_fmaf(z, s, -1.66666667e-1f);
    s = x + __builtin_fmaf(z * x, s, e);
    float c = __builtin_fmaf(z, -2.75573192e-7f, 2.48015873e-5f);
    c = __builtin_fmaf(z, c, -1.38888889e-3f);
    c = __builtin_fmaf(z, c, 4.16666667e-2f);
    const float h = __builtin_fmaf(z, -0.5f, 1.0f);
    c = h + __builtin_fmaf(z * z, c, __builtin_fmaf(z, -0.5f, 1.0f - h));
    // a quarter turn on: (c, s) -> (-s, c)
    const float a = q & 1 ? s : c, b = q & 1 ? c : s;
    return f32x2{(q + 1) & 2 ? -a : a, q & 2 ? -b : b};
}

// How a lane's 16 values lie in its head. Aligned: chunks of 8 values u and u + rot / 16 of the half layout, whose
// values pair with each other (rot a multiple of 16). Pairs: 16 values in a row, pairs of neighbours. Far: 16 values
// in a row of a half layout whose halves are no whole chunks: the other of a pair lies in another lane.
enum { kAligned, kPairs, kFarPairs };

// One lane's share of the heads at one position. Lanes of one head are neighbours, rope_lanes() of them.
template <int MODE>
struct Turner {
    int d[2];          // first value of the lane's chunks
    bool has[2];
    f32x2 cs[8];       // cos, sin of the lane's pairs (kAligned, kPairs)
    int lane, lanes;   // within the head

    __device__ void place(const RopeView& r, int in_head, int of_head) {
        lane = in_head;
        lanes = of_head;
        int c[2] = {2 * lane, 2 * lane + 1};
        if constexpr (MODE == kAligned) {
            const int half = r.rot / 16;
            if (lane < half) {
                c[0] = lane;
                c[1] = lane + half;
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            d[k] = 8 * c[k];
            has[k] = d[k] < r.hd;
        }
    }
    __device__ static f32x2 pair(const RopeView& r, int i, int p) {
        if (i >= r.rot / 2) return f32x2{1.0f, 0.0f};
        const f32x2 cs = turn_of(r.turns[i], p);
        return f32x2{cs[0] * r.amplitude, cs[1] * r.amplitude};
    }
    __device__ void at(const RopeView& r, int p) {
        if constexpr (MODE == kAligned) {
#pragma unroll
            for (int k = 0; k < 8; ++k) cs[k] = pair(r, lane < r.rot / 16 ? 8 * lane + k : r.hd, p);
        } else if constexpr (MODE == kPairs) {
#pragma unroll
            for (int k = 0; k < 8; ++k) cs[k] = pair(r, 8 * lane + k, p);
        }
    }
    template <typename T>
    __device__ void load(float* x, const T* head, bool real) const {
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (real && has[k]) load_row<8>(x + 8 * k, head + d[k]);
    }
    // x = x * weight / sqrt(mean(x^2) + eps). Every lane of the wave takes part in the sum; w nullptr: x stays.
    __device__ void norm(const RopeView& r, float* x, const float* w) const {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s = __builtin_fmaf(x[k], x[k], s);
        for (int m = 1; m < lanes; m <<= 1) s += __shfl_xor(s, m);
        if (!w) return;
        const float f = 1.0f / sqrtf(s / (float)r.hd + r.eps);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!has[k]) continue;
            float v[8];
            __builtin_memcpy(v, __builtin_assume_aligned(w + d[k], 16), sizeof v);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[8 * k + j] = x[8 * k + j] * f * v[j];
        }
    }
    // lds (kFarPairs only): 16 * lanes floats of this head.
    __device__ void turn(const RopeView& r, float* x, float* lds, int p) const {
        if constexpr (MODE == kAligned) {
            if (lane < r.rot / 16) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float a = x[k], b = x[8 + k];
                    x[k] = a * cs[k][0] - b * cs[k][1];
                    x[8 + k] = a * cs[k][1] + b * cs[k][0];
                }
            }
        } else if constexpr (MODE == kPairs) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (8 * lane + k >= r.rot / 2) continue;
                const float a = x[2 * k], b = x[2 * k + 1];
                x[2 * k] = a * cs[k][0] - b * cs[k][1];
                x[2 * k + 1] = a * cs[k][1] + b * cs[k][0];
            }
        } else {
            // The lanes of a head are in one wave: its LDS operations are in order.
#pragma unroll
            for (int k = 0; k < 16; ++k) lds[16 * lane + k] = x[k];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            const int half = r.rot / 2;
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {
                const int e = 16 * lane + k;
                if (e >= r.rot) break;
                const f32x2 t = pair(r, e < half ? e : e - half, p);
                const float other = lds[e < half ? e + half : e - half];
                const float mine = lds[e];
                const float y = e < half ? mine * t[0] - other * t[1] : other * t[1] + mine * t[0];
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = j == k ? y : x[j];
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    }
    template <typename T>
    __device__ void store(const float* x, T* head) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!has[k]) continue;
            T y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = (T)x[8 * k + j];
            __builtin_memcpy(__builtin_assume_aligned(head + d[k], 16), y, sizeof y);
        }
    }
};

constexpr int kWg = 256;

// Heads [g0, g1) * (64 / lanes) of one row, queries first, by one wave.
template <typename T, int MODE>
__device__ inline void turn_heads(const RopeView& r, const RopeTensor* x, int n_tensors, int lanes, int64_t row, int p, int g0, int g1, float* lds) {
    const int own = threadIdx.x & 63, at_once = 64 / lanes, slot = own / lanes;
    Turner<MODE> t;
    t.place(r, own - slot * lanes, lanes);
    t.at(r, p);
    const bool norms = x[0].weight || (n_tensors > 1 && x[1].weight);
    const int all = x[0].heads + (n_tensors > 1 ? x[1].heads : 0);
    for (int g = g0; g < g1; ++g) {
        int h = g * at_once + slot;
        const bool real = h < all, second = n_tensors > 1 && h >= x[0].heads;
        const RopeTensor& y = x[second ? 1 : 0];
        if (second) h -= x[0].heads;
        float v[16];
        t.load(v, static_cast<const T*>(y.in) + row * y.in_row + h * y.in_head, real);
        if (norms) t.norm(r, v, real ? y.weight : nullptr);
        t.turn(r, v, lds + slot * lanes * 16, p);
        if (real) t.store(v, static_cast<T*>(y.out) + row * y.out_row + h * y.out_head);
    }
}

// Queries and keys of many rows. A wave takes `per` groups of heads of one row, so that the angles are worked out once
// for them; `per` is 1 where there are few rows.
template <typename T, int MODE>
__global__ __launch_bounds__(kWg) void k_rope(RopeArgs a) {
    __shared__ float s_x[MODE == kFarPairs ? kWg * 16 : 1];
    const int at = threadIdx.x >> 6, lanes = rope_lanes(a.rope.hd);
    const int at_once = 64 / lanes, groups = (a.x[0].heads + a.x[1].heads + at_once - 1) / at_once;
    const int shares = (groups + a.per - 1) / a.per;
    const int64_t item = (int64_t)blockIdx.x * (kWg / 64) + at;
    const int64_t row = item / shares;
    if (row >= a.rows) return;
    const int g0 = (int)(item - row * shares) * a.per, g1 = min(g0 + a.per, groups);
    const int p = a.positions ? a.positions[row] : a.first + (int)row;
    turn_heads<T, MODE>(a.rope, a.x, 2, lanes, row, p, g0, g1, s_x + (MODE == kFarPairs ? at * 64 * 16 : 0));
}

// The sequence of a row.
__device__ inline int find_row(const RopeBatch& b, int row) {
    if (b.n == 1) return 0;
    int c = 0;
    const int lane = threadIdx.x & 63;
    for (int i0 = 0; i0 < b.n; i0 += 64) {
        const int i = i0 + lane;
        c += __popcll(__ballot(i < b.n && b.row0[min(i, b.n - 1)] + b.fresh[min(i, b.n - 1)] <= row));
    }
    return __builtin_amdgcn_readfirstlane(c);
}

// K of one page, every `step`th head from h0 on, one block of the cache after the other: a thread holds 16 values of each of CPT new tokens
// from their load to their codes, and a token's angles for all the heads: 4,097 tokens x 32 heads of 128 in bf16 with their queries
// and values 58 us with 8 heads a workgroup (2.9 TB/s). Measured when it was 55, before the angles' last bits cost it 2: 59 with 4
// heads, 63 with 2, 68 with 1; 81 when K went through LDS as fp32, which took the room of other workgroups. Eight waves a SIMD, for
// which the angles spill some 14 registers, beat six (58 us), and loading the next head during this one, at five, was worse still (66).
template <typename T, int CPT, int MODE>
__device__ inline void append_k(const RopeAppendArgs& a, int page, int h0, int step, int t0, int lo, int hi, const T* x, float* lds) {
    const KvView& kv = a.kv;
    const int pt = 1 << kv.page_shift, nt = blockDim.x, wave = threadIdx.x >> 6, own = threadIdx.x & 63;
    const int lanes = append_lanes(kv.hd, kv.slabs), at_once = 64 / lanes, slot = own / lanes;
    Turner<MODE> t[CPT];
#pragma unroll
    for (int u = 0; u < CPT; ++u) {
        t[u].place(a.rope, own - slot * lanes, lanes);
        t[u].at(a.rope, t0 + lo + (u * (nt >> 6) + wave) * at_once + slot);
    }
    for (int h = h0; h < kv.n_kv; h += step) {
        int8_t* const ep = kv.exps + (((int64_t)a.layer * kv.n_pages + page) * kv.n_kv + h) * 2;
        uint8_t* const block = kv.codes + a.layer * kv.layer_bytes + page * kv.page_bytes + (int64_t)(h * 2) * (pt * kv.slabs * kTileDims);
        const int e0 = lo > 0 ? *ep : -128;
        float v[CPT][16];
#pragma unroll
        for (int u = 0; u < CPT; ++u) {
            const int tok = lo + (u * (nt >> 6) + wave) * at_once + slot;
            t[u].load(v[u], x + h * a.head_stride[0] + tok * a.row_stride[0], tok < hi);
        }
#pragma unroll
        for (int u = 0; u < CPT; ++u) {
            if (a.k_weight) t[u].norm(a.rope, v[u], a.k_weight);
            t[u].turn(a.rope, v[u], lds + (wave * 64 + slot * lanes) * 16, t0 + lo + (u * (nt >> 6) + wave) * at_once + slot);
        }
        if (h > h0) __syncthreads();  // the last head's maximum has been read
        const int e = scale_block(v, e0, nt);
#pragma unroll
        for (int u = 0; u < CPT; ++u) {
            const int tok = lo + (u * (nt >> 6) + wave) * at_once + slot;
            if (tok >= hi) continue;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int d = t[u].d[k];
                if (d >= kv.slabs * kTileDims) continue;
                const float* const y = v[u] + 8 * k;
                // Chunk of 16 values: 64 of them to a tile, tiles ordered (16 tokens, 64 values).
                const int at = (((tok >> 4) * kv.slabs + (d >> 6)) * 64 + ((d >> 4) & 3) * 16 + (tok & 15)) * 16 + (d & 8);
                *reinterpret_cast<u32x2*>(block + at) = u32x2{to_e4m3(y[0], y[1], y[2], y[3]), to_e4m3(y[4], y[5], y[6], y[7])};
            }
        }
        if (lo > 0 && e > e0) {  // the tokens before keep their values
            const float down = pow2i(max(-126, e0 - e));
            for (int c = threadIdx.x; c < pt * kv.slabs * 4; c += nt) {
                if ((c >> 6) / kv.slabs * 16 + (c & 15) >= lo) continue;
                u32x4 w = reinterpret_cast<const u32x4*>(block)[c];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = rescale_e4m3(w[k], down);
                reinterpret_cast<u32x4*>(block)[c] = w;
            }
        }
        if (threadIdx.x == 0 && e != e0) *ep = (int8_t)e;
    }
}

// A step's queries, keys and values in one launch: first the workgroups for K (a touched page and a.heads of its heads each), then
// V's (a block of the cache each, as k_kv_append takes them), then the queries'.
template <typename T, int CPT, int MODE>
__global__ __launch_bounds__(kAppendWg, CPT == 1 ? 8 : CPT == 2 ? 4 : 2) void k_rope_append(RopeAppendArgs a) {
    extern __shared__ __attribute__((aligned(128))) float s_mem[];  // kFarPairs: 16 a lane
    const KvView& kv = a.kv;
    const int items = a.b.item0[a.b.n], shares = (kv.n_kv + a.heads - 1) / a.heads;
    int at = blockIdx.x;
    if (at >= items * (shares + kv.n_kv)) {
        at -= items * (shares + kv.n_kv);
        const int wave = threadIdx.x >> 6, lanes = rope_lanes(kv.hd);
        const int at_once = 64 / lanes, groups = (a.q.heads + at_once - 1) / at_once, q_shares = (groups + a.per - 1) / a.per;
        const int64_t item = (int64_t)at * (blockDim.x >> 6) + wave;
        const int64_t row = item / q_shares;
        if (row >= a.rows) return;
        const int g0 = (int)(item - row * q_shares) * a.per, g1 = min(g0 + a.per, groups);
        const int b = find_row(a.b, (int)row);
        turn_heads<T, MODE>(a.rope, &a.q, 1, lanes, row, a.b.before[b] + ((int)row - a.b.row0[b]), g0, g1, s_mem + wave * 64 * 16);
        return;
    }
    const int side = at >= items * shares ? 1 : 0;
    if (side) at -= items * shares;
    const int of = side ? kv.n_kv : shares, item = at / of, share = at - item * of;
    const int b = find_item(a.b, item);
    const int before = a.b.before[b], fresh = a.b.fresh[b];
    const int index = (before >> kv.page_shift) + (item - a.b.item0[b]);
    const int t0 = index << kv.page_shift;
    const int lo = max(0, before - t0), hi = min(1 << kv.page_shift, before + fresh - t0);  // new tokens of the page
    const int page = page_of(kv, a.b.seq[b], index);
    if (page < 0) return;
    const T* const x = static_cast<const T*>(a.kx[side]) + (int64_t)(a.b.row0[b] + t0 - before) * a.row_stride[side];
    if (side == 0) {
        append_k<T, CPT, MODE>(a, page, share, shares, t0, lo, hi, x, s_mem);
        return;
    }
    const auto load_v = [&](float* v, int t, int d) { load_row<4>(v, x + share * a.head_stride[1] + t * a.row_stride[1] + d); };
    quantise_block<CPT>(kv, a.layer, page, share, 1, lo, hi, load_v, load_v);
}

int mode_of(const RopeView& r) { return r.layout == 1 ? kPairs : r.rot % 16 == 0 ? kAligned : kFarPairs; }

template <typename T, int MODE>
hipError_t rope_as(const RopeArgs& a, hipStream_t s) {
    const int groups = rope_groups(a.rope.hd, a.x[0].heads + a.x[1].heads);
    const int64_t items = a.rows * ((groups + a.per - 1) / a.per);
    k_rope<T, MODE><<<(unsigned)((items + kWg / 64 - 1) / (kWg / 64)), kWg, 0, s>>>(a);
    return hipGetLastError();
}
template <typename T>
hipError_t rope_any(const RopeArgs& a, hipStream_t s) {
    const int m = mode_of(a.rope);
    return m == kAligned ? rope_as<T, kAligned>(a, s) : m == kPairs ? rope_as<T, kPairs>(a, s) : rope_as<T, kFarPairs>(a, s);
}

template <typename T, int CPT, int MODE>
hipError_t append_as(const RopeAppendArgs& a, int nt, hipStream_t s) {
    k_rope_append<T, CPT, MODE><<<(unsigned)append_grid(a), nt, MODE == kFarPairs ? nt * 16 * sizeof(float) : 0, s>>>(a);
    return hipGetLastError();
}
template <typename T, int MODE>
hipError_t append_mode(const RopeAppendArgs& a, hipStream_t s) {
    const int threads = (1 << a.kv.page_shift) * append_lanes(a.kv.hd, a.kv.slabs);  // 64 .. 2048, a multiple of 64
    const int nt = append_threads(a.kv.page_shift, a.kv.hd, a.kv.slabs);
    if (threads <= nt) return append_as<T, 1, MODE>(a, nt, s);
    if (threads <= 2 * nt) return append_as<T, 2, MODE>(a, nt, s);
    return append_as<T, 4, MODE>(a, nt, s);
}
template <typename T>
hipError_t append_any(const RopeAppendArgs& a, hipStream_t s) {
    const int m = mode_of(a.rope);
    return m == kAligned ? append_mode<T, kAligned>(a, s) : m == kPairs ? append_mode<T, kPairs>(a, s) : append_mode<T, kFarPairs>(a, s);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int dtype, hipStream_t s) {
    if (dtype == kF32) return rope_any<float>(a, s);
    if (dtype == kBF16) return rope_any<__bf16>(a, s);
    return rope_any<_Float16>(a, s);
}

hipError_t launch_rope_append(const RopeAppendArgs& a, int dtype, hipStream_t s) {
    if (dtype == kF32) return append_any<float>(a, s);
    if (dtype == kBF16) return append_any<__bf16>(a, s);
    return append_any<_Float16>(a, s);
}

}  // namespace np
