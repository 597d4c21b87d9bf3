// Attention over the 8-bit key/value cache for sequences that share their first pages, for gfx950 (semantics: include/np.h;
// the products and what stays in registers: k_attn.hip).
//
// A softmax's sums join: over disjoint token sets A and B, with their maxima m, sums l and weighted values o,
//     m = max(mA, mB),  l = lA 2^(mA - m) + lB 2^(mB - m),  o likewise.
// So the rows of all sequences that share a run of pages are one tile after another over that run, whose keys and values are
// read (and widened) once per tile instead of once per sequence, and each sequence's rows run over its own tokens behind.
// Every (row tile, split) leaves its rows' m, l and o; a second launch joins them, run by run and split by split.
#include <algorithm>
#include <atomic>

#include "attn_device.hpp"
#include "prefix_internal.hpp"

namespace np {
namespace {

constexpr int kRows = kRowTile;
constexpr int kPiece = kPieceTokens;
constexpr int W = kRunWaves;
constexpr int kMaxTileRows = 4 * kRows;  // as many as a wave has lanes

// The pieces of 32 tokens of [t0, t1) that rows at positions pos_lo and up see: the first tokens', then the window's.
struct Pieces {
    int t0, n_sink, first, total;
    __device__ int operator[](int u) const { return t0 + kPiece * (u < n_sink ? u : first + (u - n_sink)); }
};
__device__ inline Pieces pieces_of(int t0, int t1, int pos_lo, int window, int sinks) {
    const int lo = window ? max(0, pos_lo - window + 1) : 0;
    const int all = max(0, (t1 - t0 + kPiece - 1) / kPiece);
    Pieces p;
    p.t0 = t0;
    p.n_sink = min(all, max(0, (min(sinks, lo) - t0 + kPiece - 1) / kPiece));
    p.first = min(all, max(p.n_sink, max(0, lo - t0) / kPiece));
    p.total = p.n_sink + all - p.first;
    return p;
}

// One tile of rows over one split of a token range.
struct Work {
    int seq;             // a sequence whose page list has the range
    int h;               // kv head
    int t0, t1;          // tokens; every row's position is at least t1 - 1, or the row's own causal limit counts
    int pos_lo, pos_hi;  // of the tile's rows
    int rows;            // of the tile
    int split, splits;
    float* part;         // the tile's first partial row
};

__device__ inline bool group_seen(const PrefixArgs& a, const Work& w, int t) {
    return t < w.t1 && t <= w.pos_hi && (!a.window || w.pos_lo - (t + 15) < a.window || t < a.sinks);
}

// What a wave takes of it: every W-th piece of the split.
struct Share {
    Pieces pc;
    int first, count;
    __device__ int operator[](int n) const { return pc[first + n * W]; }
};
__device__ inline Share share_of(const PrefixArgs& a, const Work& w, int wave) {
    Share s;
    s.pc = pieces_of(w.t0, w.t1, w.pos_lo, a.window, a.sinks);
    const int each = s.pc.total / w.splits, more = s.pc.total - each * w.splits;
    const int u0 = w.split * each + min(w.split, more), u1 = u0 + each + (w.split < more ? 1 : 0);
    s.first = u0 + wave;
    s.count = u1 > s.first ? (u1 - s.first + W - 1) / W : 0;
    return s;
}
// Page of group i % 2 of piece n0 + i / 2, i the lane; -1 where it is not held or nobody sees it.
__device__ inline int page_ahead(const PrefixArgs& a, const Work& w, const Share& s, int n0, int lane) {
    const int n = n0 + (lane >> 1), t = n < s.count ? s[n] + 16 * (lane & 1) : w.t1;
    return group_seen(a, w, t) ? page_of(a.kv, w.seq, t >> a.kv.page_shift) : -1;
}

// R row tiles of 16 over the range, by the workgroup's waves: each takes every W-th piece of the split, with K asked for a
// piece ahead and V behind the scores' products, and widened once for all R. s_pos: the rows' positions; s_mem: their q as operands; s_bad: per row, a bit
// per value that meets a NaN (0 before). Ends with the rows' partial results in memory.
template <typename T, int NS, int R>
__device__ inline void attend_rows(const PrefixArgs& a, const Work& w, const Share& share, int ahead_page, const int* s_pos, uint32_t* s_bad, float* s_mem) {
    typedef AttnKind<T> Kd;
    typedef typename Kd::Q Q;
    typedef typename Kd::P P;
    typedef typename Vec8<Q>::t Q8;
    typedef typename Vec8<P>::t P8;
    const KvView& kv = a.kv;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const Q8* const s_q = reinterpret_cast<const Q8*>(s_mem);  // [R][NS][2][kQ][64 lanes]
    const uint8_t* const codes = kv.codes + a.layer * kv.layer_bytes;
    const int8_t* const exps = kv.exps + (int64_t)a.layer * kv.n_pages * kv.n_kv * 2;
    const int side_bytes = (1 << kv.page_shift) * kv.slabs * kTileDims;

    // Lane i, of group i % 2 of piece (n & ~31) + i / 2: its K codes' address (page 0 where it is not held or nobody sees it: its
    // tokens are hidden below), its K factor and V exponent; a bit per group of whether it is held.
    const int count = share.count;
    uint64_t ahead_at = 0, ahead_held = 0;
    float ahead_kf = 0.0f;
    int ahead_ev = 0;
    const auto fetch = [&](int n0) __attribute__((always_inline)) {
        const int n = n0 + (lane >> 1), t = n < count ? share[n] + 16 * (lane & 1) : 0, page = max(ahead_page, 0);
        const int e = *reinterpret_cast<const uint16_t*>(exps + ((int64_t)page * kv.n_kv + w.h) * 2);
        ahead_at = reinterpret_cast<uint64_t>(codes + page * kv.page_bytes + (int64_t)2 * w.h * side_bytes +
                                              (int64_t)((t & ((1 << kv.page_shift) - 1)) >> 4) * (kv.slabs * kTileBytes));
        ahead_held = __ballot(ahead_page >= 0);
        ahead_kf = fmaxf(a.scale2 * pow2i(max(-126, (int)(int8_t)e)), 1.2e-38f);  // never 0: a hidden score is -inf, and stays it times this
        ahead_ev = max(-126, (int)(int8_t)(e >> 8));
    };
    fetch(0);

    f32x4 o[R][NS][4];
    float m[R], l[R];
    uint32_t seen = 0;  // a bit per row tile
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -__builtin_inff();
        l[r] = 0.0f;
#pragma unroll
        for (int c = 0; c < NS; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[r][c][i] = f32x4{0, 0, 0, 0};
    }
    int unit = kNoUnit, top = kNoUnit;  // o is in units of 2^unit

    u32x4 k[2][NS], v[2][NS];
    uint64_t at[2];
    int lane16 = lane * 16;
    const auto locate = [&](int n) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int from = (n & 31) * 2 + g;
            at[g] = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(ahead_at >> 32), from) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)ahead_at, from);
        }
    };
    typedef const __attribute__((address_space(1))) uint8_t code;
    typedef const __attribute__((address_space(1))) u32x4 chunk;
    const auto load_k = [&] {
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int c = 0; c < NS; ++c) k[g][c] = *reinterpret_cast<chunk*>(reinterpret_cast<code*>(at[g]) + c * kTileBytes + lane16);
    };
    const auto load_v = [&] {
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int c = 0; c < NS; ++c) v[g][c] = *reinterpret_cast<chunk*>(reinterpret_cast<code*>(at[g] + side_bytes) + c * kTileBytes + lane16);
    };
    if (count) {
        locate(0);
        load_k();
    }
    for (int n = 0; n < count; ++n) {
        const int tok = share[n];
        bool held[2];
        float kf[2];
        int ev[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int from = (n & 31) * 2 + g;
            held[g] = (ahead_held >> from & 1) != 0;
            kf[g] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ahead_kf), from));
            ev[g] = __builtin_amdgcn_readlane(ahead_ev, from);
        }
        f32x4 acc[R][2];  // raw scores of tokens tok + 16 g + 4 quad + j
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][0] = acc[r][1] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < NS; ++c)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const Q8 k0 = widen<Q>(k[0][c][2 * f], k[0][c][2 * f + 1], 1.0f, 1.0f), k1 = widen<Q>(k[1][c][2 * f], k[1][c][2 * f + 1], 1.0f, 1.0f);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int t = 0; t < Kd::kQ; ++t) {
                        const Q8 q = s_q[(((r * NS + c) * 2 + f) * Kd::kQ + t) * 64 + lane];
                        acc[r][0] = mfma(k0, q, acc[r][0]);
                        acc[r][1] = mfma(k1, q, acc[r][1]);
                    }
            }
        // Operands come from LDS a few products ahead.
        constexpr int kMfma = 0x8, kDsRead = 0x100, kReads = NS * 2 * R * Kd::kQ, kAhead = kReads < 4 ? kReads : 4;
        __builtin_amdgcn_sched_group_barrier(kDsRead, kAhead, 0);
#pragma unroll
        for (int i = 0; i < kReads - kAhead; ++i) {
            __builtin_amdgcn_sched_group_barrier(kMfma, 2, 0);
            __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(kMfma, 2 * kAhead, 0);
        __builtin_amdgcn_sched_barrier(0);
        load_v();
        const bool last = n + 1 >= count;
        if (!last) {
            if ((n & 31) == 31) {
                ahead_page = page_ahead(a, w, share, n + 1, lane);
                fetch(n + 1);
                asm volatile("" : "+v"(ahead_kf), "+v"(ahead_ev));  // waited for here, in this branch
            }
            locate(n + 1);
        } else {
            // The same number of loads in every turn; these read one line of the pool's start.
            at[0] = at[1] = reinterpret_cast<uint64_t>(codes);
            lane16 = 0;
        }
        load_k();

        // A piece that every row of the tile sees whole needs no comparisons.
        const bool whole = held[0] && held[1] && tok + kPiece <= w.t1 && tok + kPiece - 1 <= w.pos_lo &&
                           (!a.window || tok > w.pos_hi - a.window || tok + kPiece <= a.sinks);
        P8 pv[R][Kd::kP];
        uint32_t vis = ~0u;  // 8 bits a row tile
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!whole) {
                const int mine = here(lane), pos = s_pos[r * kRows + (mine & 15)], t0 = tok + 4 * (mine >> 4);
                uint32_t see = 0;
#pragma unroll
                for (int k8 = 0; k8 < 8; ++k8) {
                    const int t = t0 + 16 * (k8 >> 2) + (k8 & 3);
                    const bool ok = t <= pos && t < w.t1 && held[k8 >> 2] && (!a.window || pos - t < a.window || t < a.sinks);
                    see |= ok ? 1u << k8 : 0u;
                    if (!ok) acc[r][k8 >> 2][k8 & 3] = -__builtin_inff();
                }
                vis = (vis & ~(0xffu << (8 * r))) | see << (8 * r);
            }
            float mx = -__builtin_inff();
#pragma unroll
            for (int g = 0; g < 2; ++g) mx = fmaxf(mx, fmaxf(fmaxf(acc[r][g][0], acc[r][g][1]), fmaxf(acc[r][g][2], acc[r][g][3])) * kf[g]);
            if (__any(mx > m[r] + kLazy)) {
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                const float m1 = fmaxf(m[r], mx);
                const float f = m1 == m[r] ? 1.0f : __builtin_amdgcn_exp2f(m[r] - m1);
                m[r] = m1;
                l[r] *= f;
#pragma unroll
                for (int c = 0; c < NS; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[r][c][i] *= f;
            }
            const float m0 = (m[r] == -__builtin_inff() ? 0.0f : m[r]) - Kd::kLift;  // 0: a row that has seen nothing finite
            float p[8];  // 0 for hidden tokens
#pragma unroll
            for (int k8 = 0; k8 < 8; ++k8) {
                p[k8] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[r][k8 >> 2][k8 & 3], kf[k8 >> 2], -m0));
                l[r] += p[k8];
            }
            split<P, Kd::kP>(pv[r], p);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) seen |= vis >> (8 * r) & 0xff ? 1u << r : 0u;

        // Tokens that no row of the tile sees (often bytes never written) are cleared. What is NaN besides leaves the product, where 0
        // times it would be NaN for rows that do not see it, and goes to those that do: a second product says whether a row
        // sees a token whose value is NaN.
        if (!whole) {
            uint32_t bad = 0;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint32_t some = 0;
                const int t0 = tok + 16 * g + 4 * (here(lane) >> 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = t0 + j;
                    if (held[g] && t < w.t1 && t <= w.pos_hi && (!a.window || w.pos_lo - t < a.window || t < a.sinks)) some |= 0xffu << (8 * j);
                }
#pragma unroll
                for (int c = 0; c < NS; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[g][c][i] &= some;
                        bad |= nan_bytes(v[g][c][i]);
                    }
            }
            if (__any(bad != 0)) {
#pragma unroll
                for (int c = 0; c < NS; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t n0 = nan_bytes(v[0][c][i]) >> 7, n1 = nan_bytes(v[1][c][i]) >> 7;
                        if (!__any((n0 | n1) != 0)) continue;
                        const P8 odd = widen<P>(n0 * 0x38u, n1 * 0x38u, 1.0f, 1.0f);  // 0x38: 1
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            P8 sees;
#pragma unroll
                            for (int k8 = 0; k8 < 8; ++k8) sees[k8] = (P)(vis >> (8 * r + k8) & 1 ? 1.0f : 0.0f);
                            const f32x4 x = mfma(odd, sees, f32x4{0, 0, 0, 0});
                            const int mine = here(lane);
                            uint32_t note = 0;  // value 64 c + 16 quad + 4 j + i
#pragma unroll
                            for (int j = 0; j < 4; ++j) note |= x[j] > 0.0f ? 1u << (4 * j + i) : 0u;
                            if (note) atomicOr(&s_bad[(r * kRows + (mine & 15)) * (2 * NS) + 2 * c + (mine >> 5)], note << (mine & 16));
                            __builtin_amdgcn_sched_barrier(0);  // this path must not cost registers
                        }
                        v[0][c][i] &= ~(n0 * 255u);
                        v[1][c][i] &= ~(n1 * 255u);
                    }
            }
        }
        // O += V^T P^T. Both groups at once, or one at a time where their V scales lie too far apart for one unit.
        const auto fit_unit = [&](int ea, int eb) {
            const int lo_e = min(ea, eb), hi_e = max(ea, eb);
            top = max(top, hi_e);
            const int to = max(min(hi_e, lo_e + kFar), top - kDrop);
            if (to != unit && (hi_e > unit + kNear || lo_e < unit - kFar)) {
                float f = pow2i(max(-126, unit - to));
                asm volatile("" : "+v"(f));  // a branch, not a product with 1 in every turn
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int c = 0; c < NS; ++c)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[r][c][i] *= f;
                unit = to;
            }
        };
        // Exponents of groups that are not held are page 0's: they must not move the unit.
        const int e0 = held[0] ? ev[0] : held[1] ? ev[1] : unit, e1 = held[1] ? ev[1] : e0;
        const bool near = e0 - e1 <= kNear + kFar && e1 - e0 <= kNear + kFar;
        for (int pass = 0; pass < (near ? 1 : 2); ++pass) {
            // One group at a time: the other one's codes, times 2^-126, are nothing beside the sums.
            const int ea = near || pass == 0 ? e0 : e1, eb = near || pass == 1 ? e1 : e0;
            fit_unit(ea, eb);
            const float f0 = pow2i(near || pass == 0 ? max(-126, e0 - unit) : -126), f1 = pow2i(near || pass == 1 ? max(-126, e1 - unit) : -126);
#pragma unroll
            for (int c = 0; c < NS; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const P8 vv = widen<P>(v[0][c][i], v[1][c][i], f0, f1);
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int t = 0; t < Kd::kP; ++t) o[r][c][i] = mfma(vv, pv[r][t], o[r][c][i]);
                }
        }
    }

    // Join the waves, 16 rows at a time: rows' maximum, sum and O in true units.
    constexpr int D = NS * 64, DS = D + 4, PS = D + 2;
    float* const s_m = s_mem;             // [W][16]
    float* const s_l = s_m + W * kRows;   // [W][16]
    float* const s_o = s_l + W * kRows;   // [W][16][DS]
    const float back = __builtin_amdgcn_ldexpf(1.0f, unit - Kd::kLift);
    const int D4 = kv.hd / 4;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float ll = l[r], mm = m[r];
        ll += __shfl_xor(ll, 16);
        ll += __shfl_xor(ll, 32);
        ll *= 1.0f / (1 << Kd::kLift);
        const bool any = (__ballot(seen >> r & 1) >> col & 0x0001000100010001ull) != 0;
        // Every score this wave saw is -inf: beside finite scores they weigh 0; alone, 0 / 0.
        if (any && mm == -__builtin_inff()) mm = -__FLT_MAX__;
        __syncthreads();  // the q tile, or the rows before, are done with
        float* const dst = s_o + (wave * kRows + col) * DS + quad * 16;
#pragma unroll
        for (int c = 0; c < NS; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f32x4*>(dst + c * 64 + 4 * j) = f32x4{o[r][c][0][j], o[r][c][1][j], o[r][c][2][j], o[r][c][3][j]} * back;
        if (quad == 0) {
            s_m[wave * kRows + col] = mm;
            s_l[wave * kRows + col] = ll;
        }
        __syncthreads();
        const int n_out = min(kRows, w.rows - r * kRows) * D4;
        for (int i = threadIdx.x; i < n_out; i += 64 * W) {
            const int row = i / D4, d = (i - row * D4) * 4;
            float top_m = s_m[row], sum = 0.0f;
#pragma unroll
            for (int x = 1; x < W; ++x) top_m = fmaxf(top_m, s_m[x * kRows + row]);
            f32x4 y = {0, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < W; ++x) join(y, sum, top_m, s_m[x * kRows + row], s_l[x * kRows + row], *reinterpret_cast<const f32x4*>(s_o + (x * kRows + row) * DS + d));
            const uint32_t odd = s_bad[(r * kRows + row) * (2 * NS) + (d >> 5)] >> (d & 31);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (odd >> j & 1) y[j] = __builtin_nanf("");
            float* const p = w.part + (int64_t)(r * kRows + row) * PS;
            *reinterpret_cast<f32x2*>(p + 2 + d) = f32x2{y[0], y[1]};
            *reinterpret_cast<f32x2*>(p + 4 + d) = f32x2{y[2], y[3]};
            if (d == 0) *reinterpret_cast<f32x2*>(p) = f32x2{top_m, sum};
        }
    }
}

// The sequence (in the batch's order) that new token t belongs to.
__device__ inline int sequence_of(const PrefixArgs& a, const int* cum, int t, int lo, int hi) {
    if (a.even) return t / a.even;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <typename T, int NS>
constexpr int kTiles = run_tiles(sizeof(T) == 4 ? kF32 : kBF16, NS);

// Bound by vector issue: vector instructions take 0.71 of a SIMD's time, the matrix products among them keep their units busy for 0.37 of
// it, and a wave waits for its turn to issue for 0.36 of its time, for data and barriers for 0.23. 90 sequences of 3 new tokens behind two prompts of up to 30 Ki tokens, 32 over 8 heads of 128 in
// bf16, 205 us with the join's 10 (634 TFLOP/s). Few rows are latency: 32 sequences behind one prompt of 8,011 tokens 24.8 us, of
// which the join takes 6.6.
//
// Workgroups of a kv head's items are 8 apart where 8 divides the heads, so a head's tiles over one run share a die's cache.
template <typename T, int NS>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(run_eu(sizeof(T) == 4 ? kF32 : kBF16, NS)))) void k_prefix(PrefixArgs a) {
    typedef AttnKind<T> Kd;
    typedef typename Kd::Q Q;
    typedef typename Vec8<Q>::t Q8;
    constexpr int R = kTiles<T, NS>, D = NS * 64;
    const KvView& kv = a.kv;
    const int item = blockIdx.x / kv.n_kv, h = blockIdx.x - item * kv.n_kv;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int group = kv.n_heads / kv.n_kv;
    __shared__ int s_cum[kMaxBatch + 1];
    __shared__ int s_pos[kMaxTileRows];
    __shared__ int64_t s_row[kMaxTileRows];  // where the row's q begins
    __shared__ uint32_t s_bad[R * kRows * 2 * NS];
    extern __shared__ __attribute__((aligned(128))) float s_mem[];

    Work w;
    w.h = h;
    int first, rows_all, tile, wide, s0, s1;  // first new token (in the batch's order) and rows of the tile's range of rows
    if (item < a.leaf_item) {
        const int k = __popcll(__ballot(lane < a.n_runs && (lane + 1 < a.n_runs ? a.run[min(lane + 1, kMaxRuns - 1)].item0 : a.leaf_item) <= item));
        const PrefixRun run = a.run[__builtin_amdgcn_readfirstlane(k)];
        s0 = run.s0;
        s1 = run.s1;
        w.t0 = run.t0;
        w.t1 = run.t1;
        w.splits = run.splits;
        tile = (item - run.item0) / w.splits;
        w.split = item - run.item0 - tile * w.splits;
        first = a.cum[s0];
        rows_all = (a.cum[s1] - first) * group;
        wide = R;
        const int cap = min(R * kRows, rows_all);
        w.part = a.part + ((int64_t)(run.part0 + (tile * w.splits + w.split) * cap) * kv.n_kv + h * cap) * (D + 2);
    } else {
        const int own = item - a.leaf_item;
        int c = 0;
        for (int i0 = 0; i0 < a.n; i0 += 64) {
            const int i = i0 + lane;
            c += __popcll(__ballot(i < a.n && a.item0[min(i, a.n - 1) + 1] <= own));
        }
        s0 = __builtin_amdgcn_readfirstlane(c);
        s1 = s0 + 1;
        w.t0 = a.deepest[s0] == kNoRun ? 0 : a.run[a.deepest[s0]].t1;
        w.splits = a.splits[s0];
        tile = (own - a.item0[s0]) / w.splits;
        w.split = own - a.item0[s0] - tile * w.splits;
        first = a.cum[s0];
        rows_all = (a.cum[s1] - first) * group;
        wide = rows_all <= kRows ? 1 : R;
        w.t1 = a.before[s0] + (a.cum[s1] - first);
        w.part = a.part + ((int64_t)(a.leaf_part + own * a.leaf_cap) * kv.n_kv + h * a.leaf_cap) * (D + 2);
    }
    w.seq = a.seq[s0];
    const int r0 = tile * wide * kRows;
    w.rows = min(wide * kRows, rows_all - r0);
    if (!a.even && s1 - s0 > 1) {
        for (int i = threadIdx.x; i <= a.n; i += 64 * W) s_cum[i] = a.cum[i];
        __syncthreads();
    }
    for (int i = threadIdx.x; i < R * kRows * 2 * NS; i += 64 * W) s_bad[i] = 0;
    if ((int)threadIdx.x < kMaxTileRows) {
        const int row = r0 + min((int)threadIdx.x, w.rows - 1), t = first + row / group, g = row - row / group * group;
        const int s = s1 - s0 == 1 ? s0 : sequence_of(a, s_cum, t, s0, s1);
        const int tq = t - a.cum[s];
        s_pos[threadIdx.x] = a.before[s] + tq;
        s_row[threadIdx.x] = (int64_t)(a.row0[s] + tq) * a.q_row + (int64_t)(h * group + g) * a.q_head;
    }
    __syncthreads();
    {
        int lo = s_pos[lane], hi = lo;  // 64 rows: every one of the tile, the last repeated
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            lo = min(lo, __shfl_xor(lo, d));
            hi = max(hi, __shfl_xor(hi, d));
        }
        w.pos_lo = __builtin_amdgcn_readfirstlane(lo);
        w.pos_hi = __builtin_amdgcn_readfirstlane(hi);
    }
    w.t1 = min(w.t1, w.pos_hi + 1);
    const Share share = share_of(a, w, wave);
    const int pages = page_ahead(a, w, share, 0, lane);  // on its way beside q
    Q8* const s_q = reinterpret_cast<Q8*>(s_mem);
    for (int cf = wave; cf < 2 * NS * wide; cf += W) {
        const int r = cf / (2 * NS), d = (cf >> 1) % NS * 64 + quad * 16 + (cf & 1) * 8, row = r * kRows + col;
        const T* const q = static_cast<const T*>(a.q) + s_row[row] + d;
        u32x4 raw[sizeof(T) / 2];
#pragma unroll
        for (int x = 0; x < (int)sizeof(T) / 2; ++x) {
            raw[x] = u32x4{0, 0, 0, 0};
            if (row < w.rows && d < kv.hd) raw[x] = reinterpret_cast<const u32x4*>(q)[x];
        }
        if constexpr (sizeof(T) == 2) {
            s_q[cf * 64 + lane] = __builtin_bit_cast(Q8, raw[0]);
        } else {
            float x[8];
            __builtin_memcpy(x, raw, sizeof x);
            Q8 t[Kd::kQ];
            split<Q, Kd::kQ>(t, x);
#pragma unroll
            for (int n = 0; n < Kd::kQ; ++n) s_q[(cf * Kd::kQ + n) * 64 + lane] = t[n];
        }
    }
    __syncthreads();
    if (R == 1 || wide == 1) attend_rows<T, NS, 1>(a, w, share, pages, s_pos, s_bad, s_mem);
    else attend_rows<T, NS, R>(a, w, share, pages, s_pos, s_bad, s_mem);
}

// Joins a row's partial results: a thread per four values of a (new token, head).
template <typename T, int NS>
__global__ __launch_bounds__(256) void k_prefix_join(PrefixArgs a) {
    constexpr int R = kTiles<T, NS>, PS = NS * 64 + 2;
    const KvView& kv = a.kv;
    __shared__ int s_cum[kMaxBatch + 1];
    if (!a.even) {
        for (int i = threadIdx.x; i <= a.n; i += 256) s_cum[i] = a.cum[i];
        __syncthreads();
    }
    const int D4 = kv.hd / 4, group = kv.n_heads / kv.n_kv;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, unit = at / D4;
    if (unit >= (int64_t)a.rows * kv.n_heads) return;
    const int d = (int)(at - unit * D4) * 4, t = (int)(unit / kv.n_heads), head = (int)(unit - (int64_t)t * kv.n_heads), h = head / group, g = head - h * group;
    const int s = sequence_of(a, s_cum, t, 0, a.n);
    const int tq = t - a.cum[s];
    float mm = -__builtin_inff(), ll = 0.0f;
    f32x4 x = {0, 0, 0, 0};
    // `splits` partial rows, `step` rows apart.
    const auto take = [&](int64_t row, int64_t step, int splits) {
        const float* const p = a.part + row * PS;
        constexpr int U = 8;  // in flight
        for (int s0 = 0; s0 < splits; s0 += U) {
            f32x2 ml[U], xa[U], xb[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float* const q = p + min(s0 + i, splits - 1) * step * PS;
                ml[i] = *reinterpret_cast<const f32x2*>(q);
                xa[i] = *reinterpret_cast<const f32x2*>(q + 2 + d);
                xb[i] = *reinterpret_cast<const f32x2*>(q + 4 + d);
            }
            float m1 = mm;
#pragma unroll
            for (int i = 0; i < U; ++i) m1 = fmaxf(m1, ml[i][0]);
            if (m1 != mm) {
                const float f = __builtin_amdgcn_exp2f(mm - m1);
                x *= f;
                ll *= f;
                mm = m1;
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (s0 + i < splits) join(x, ll, mm, ml[i][0], ml[i][1], f32x4{xa[i][0], xa[i][1], xb[i][0], xb[i][1]});
        }
    };
    for (int k = 0; k < a.n_runs; ++k) {
        const PrefixRun run = a.run[k];
        if (s < run.s0 || s >= run.s1) continue;
        const int first = a.cum[run.s0], cap = min(R * kRows, (a.cum[run.s1] - first) * group);
        const int row = (t - first) * group + g, tile = row / (R * kRows);
        take((int64_t)(run.part0 + tile * run.splits * cap) * kv.n_kv + h * cap + (row - tile * R * kRows), (int64_t)cap * kv.n_kv, run.splits);
    }
    {
        const int rows = (a.cum[s + 1] - a.cum[s]) * group, wide = rows <= kRows ? kRows : R * kRows;
        const int row = tq * group + g, tile = row / wide, splits = a.splits[s];
        take((int64_t)(a.leaf_part + (a.item0[s] + tile * splits) * a.leaf_cap) * kv.n_kv + h * a.leaf_cap + (row - tile * wide), (int64_t)a.leaf_cap * kv.n_kv, splits);
    }
    const bool none = mm == -__builtin_inff() && ll == 0.0f;  // no visible token: 0
    const float inv = none ? 0.0f : 1.0f / ll;
    T y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = (T)(x[j] * inv);
    const int64_t row = a.row0[s] + tq;
    __builtin_memcpy(__builtin_assume_aligned(static_cast<T*>(a.out) + row * a.o_row + (int64_t)head * a.o_head + d, 4 * sizeof(T)), y, sizeof y);
    if (a.lse && d == 0) a.lse[row * kv.n_heads + head] = none ? -__builtin_inff() : ll == 0.0f ? __builtin_nanf("") : (mm + __builtin_amdgcn_logf(ll)) * 0.69314718055994531f;
}

// LDS: q of a tile as operands, then the waves' results of 16 rows.
template <typename T, int NS>
constexpr int kLds = std::max(kTiles<T, NS> * NS * 2 * AttnKind<T>::kQ * 1024, W * kRows * (2 + NS * 64 + 4) * 4);

template <typename T, int NS>
hipError_t prefix_as(const PrefixArgs& a, hipStream_t s) {
    k_prefix<T, NS><<<(unsigned)(a.leaf_item + a.item0[a.n]) * a.kv.n_kv, 64 * W, kLds<T, NS>, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t threads = (int64_t)a.rows * a.kv.n_heads * (a.kv.hd / 4);
    k_prefix_join<T, NS><<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(a);
    return hipGetLastError();
}
template <typename T>
hipError_t prefix_any(const PrefixArgs& a, hipStream_t s) {
    switch (a.kv.slabs) {
        case 1: return prefix_as<T, 1>(a, s);
        case 2: return prefix_as<T, 2>(a, s);
        case 3: return prefix_as<T, 3>(a, s);
        default: return prefix_as<T, 4>(a, s);
    }
}

template <typename T>
hipError_t prepare_all() {
    const auto allow = [](const void* f, int bytes) { return hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, bytes); };
    for (hipError_t e : {allow(reinterpret_cast<const void*>(k_prefix<T, 1>), kLds<T, 1>), allow(reinterpret_cast<const void*>(k_prefix<T, 2>), kLds<T, 2>),
                         allow(reinterpret_cast<const void*>(k_prefix<T, 3>), kLds<T, 3>), allow(reinterpret_cast<const void*>(k_prefix<T, 4>), kLds<T, 4>)})
        if (e != hipSuccess) return e;
    return hipSuccess;
}

}  // namespace

hipError_t launch_prefix(const PrefixArgs& a, int dtype, hipStream_t s) {
    if (dtype == kF32) return prefix_any<float>(a, s);
    if (dtype == kBF16) return prefix_any<__bf16>(a, s);
    return prefix_any<_Float16>(a, s);
}

hipError_t prefix_prepare() {
    static std::atomic<uint64_t> done{0};  // a bit per device
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
    for (hipError_t x : {prepare_all<float>(), prepare_all<__bf16>(), prepare_all<_Float16>()})
        if (x != hipSuccess) e = x;
    if (e == hipSuccess && dev < 64) done.fetch_or(1ull << dev);
    return e;
}

}  // namespace np
